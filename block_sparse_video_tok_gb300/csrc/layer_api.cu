// layer_api.cu -- the extern "C" entry points declared in include/vsa_layer.h: argument checks and
// the stream-ordered launches of each operator.
#include <climits>
#include <cmath>
#include <mutex>

#include "layer_internal.cuh"

namespace {

constexpr int MAX_DEVICES = 64;
static __device__ uint32_t g_error_word[2] = {0, 0};  // the word; what the last read took out of it
std::mutex g_word_mutex, g_read_mutex;
uint32_t* g_word_addr[MAX_DEVICES] = {nullptr};

// Reads and clears in one step: a bit that another stream raises meanwhile is read now or stays.
__global__ void take_error_word_kernel(uint32_t* word) { word[1] = atomicExch(word, 0u); }

vsa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? VSA_OK : vsa::record_cuda_failure(e); }

vsa_status check_device() {
  int dev = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return vsa::record_cuda_failure(e);
  return major == 10 && minor == 3 ? VSA_OK : VSA_ERR_UNSUPPORTED;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool present(const vsa_heads* x) { return x && x->data; }

// A tensor of `batch` x x->heads x `tokens` heads of `dim` elements of `size` bytes: 16-byte
// aligned data and strides; strides of dimensions of length 1 do not matter (and become 0).
// An output must not have overlapping elements: its strides, sorted, step past one another.
vsa_status view_of(const vsa_heads* x, int batch, int tokens, int dim, int size, bool output,
                   vsa::HeadsView* v) {
  if (!present(x) || x->heads < 1) return VSA_ERR_INVALID_ARG;
  v->data = x->data;
  v->heads = x->heads;
  v->batch = batch > 1 ? x->batch_stride : 0;
  v->head = x->heads > 1 ? x->head_stride : 0;
  v->token = tokens > 1 ? x->token_stride : 0;
  if (!aligned(x->data, 16)) return VSA_ERR_INVALID_ARG;
  const int64_t st[3] = {v->batch, v->head, v->token};
  const int64_t n[3] = {batch, x->heads, tokens};
  for (int i = 0; i < 3; ++i) {
    if (st[i] < 0 || st[i] > LLONG_MAX / 4 / n[i] / size || st[i] * size % 16 != 0) return VSA_ERR_INVALID_ARG;
  }
  if (output) {
    int o[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (st[o[j]] > st[o[j + 1]]) {
          const int t = o[j];
          o[j] = o[j + 1];
          o[j + 1] = t;
        }
    int64_t extent = dim;
    for (int i = 0; i < 3; ++i) {
      if (n[o[i]] == 1) continue;
      if (st[o[i]] < extent) return VSA_ERR_INVALID_ARG;
      extent = st[o[i]] * (n[o[i]] - 1) + extent;
    }
  }
  return VSA_OK;
}

int dtype_size(int dtype) { return dtype == VSA_F32 ? 4 : 2; }

// ------------------------------------------------------------------------------ norm_rope

vsa_status check_norm_rope(const vsa_norm_rope* op) {
  if (!op || op->batch < 1 || op->tokens < 1 || op->rows < 1) return VSA_ERR_INVALID_ARG;
  if (op->head_dim < 8 || op->head_dim > 256 || op->head_dim % 8 != 0) return VSA_ERR_UNSUPPORTED;
  if (op->dtype != VSA_BF16 && op->dtype != VSA_F16 && op->dtype != VSA_F32) return VSA_ERR_UNSUPPORTED;
  if (op->weight_dtype != VSA_F32 && op->weight_dtype != op->dtype) return VSA_ERR_UNSUPPORTED;
  if (op->rot < 0 || op->rot > op->head_dim) return VSA_ERR_INVALID_ARG;
  if (op->rot % (op->halves ? 16 : 8) != 0) return VSA_ERR_UNSUPPORTED;
  if (!std::isfinite(op->eps) || op->eps < 0.f) return VSA_ERR_INVALID_ARG;
  if (op->rot > 0) {
    if (!op->cosines || !op->sines || !aligned(op->cosines, 16) || !aligned(op->sines, 16)) return VSA_ERR_INVALID_ARG;
    if (op->table_batch_stride < 0 || op->table_batch_stride % 4 != 0) return VSA_ERR_INVALID_ARG;
  }
  if (!aligned(op->q_weight, 16) || !aligned(op->k_weight, 16) || !aligned(op->order, 4) || !aligned(op->inverse, 4))
    return VSA_ERR_INVALID_ARG;
  if (!op->order && (op->rows != op->tokens || op->inverse)) return VSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(op->batch) * op->tokens > INT_MAX ||
      static_cast<int64_t>(op->batch) * op->rows > INT_MAX)
    return VSA_ERR_UNSUPPORTED;
  return VSA_OK;
}

void fill_norm_rope(const vsa_norm_rope* op, vsa::NormRopeArgs* a) {
  a->weight[0] = op->q_weight;
  a->weight[1] = op->k_weight;
  a->cosines = op->cosines;
  a->sines = op->sines;
  a->table_batch = op->table_batch_stride;
  a->order = op->order;
  a->inverse = op->inverse;
  a->batch = op->batch;
  a->tokens = op->tokens;
  a->rows = op->rows;
  a->head_dim = op->head_dim;
  a->rot = op->rot;
  a->dtype = op->dtype;
  a->weight_dtype = op->weight_dtype;
  a->halves = op->halves != 0;
  a->eps = op->eps;
}

// ------------------------------------------------------------------------------ cross attention

vsa_status check_cross(const vsa_cross* op) {
  if (!op || op->batch < 1 || op->heads < 1 || op->kv_heads < 1 || op->q_tokens < 1 || op->kv_tokens < 1)
    return VSA_ERR_INVALID_ARG;
  if (op->heads % op->kv_heads != 0 || !std::isfinite(op->sm_scale)) return VSA_ERR_INVALID_ARG;
  if (op->head_dim != vsa::HEAD_DIM) return VSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(op->batch) * op->heads > 65535) return VSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(op->batch) * op->heads * op->q_tokens > INT_MAX / 2 ||
      static_cast<int64_t>(op->batch) * op->kv_heads * op->kv_tokens > INT_MAX / 2)
    return VSA_ERR_UNSUPPORTED;
  if (!aligned(op->kv_len, 4)) return VSA_ERR_INVALID_ARG;
  return VSA_OK;
}

// A cross-attention operand: heads and tokens must not be broadcast (a tile spans several).
vsa_status cross_view(const vsa_heads* x, int batch, int tokens, bool output, vsa::HeadsView* v) {
  const vsa_status st = view_of(x, batch, tokens, vsa::HEAD_DIM, 2, output, v);
  if (st != VSA_OK) return st;
  return (x->heads > 1 && v->head == 0) || (tokens > 1 && v->token == 0) ? VSA_ERR_INVALID_ARG : VSA_OK;
}

vsa_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return VSA_OK;
  return workspace && aligned(workspace, 256) && bytes >= need ? VSA_OK : VSA_ERR_WORKSPACE;
}

void fill_cross(const vsa_cross* op, vsa::CrossArgs* a) {
  a->kv_len = op->kv_len;
  a->batch = op->batch;
  a->heads = op->heads;
  a->kv_heads = op->kv_heads;
  a->q_tokens = op->q_tokens;
  a->kv_tokens = op->kv_tokens;
  a->sm_scale = op->sm_scale;
  a->wait_ns = vsa::wait_limit_ns();
}

}  // namespace

namespace vsa {

vsa_status layer_error_word(uint32_t** word) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda_failure(e);
  if (dev < 0 || dev >= MAX_DEVICES) return VSA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_word_mutex);
  if (!g_word_addr[dev]) {
    void* addr = nullptr;
    e = cudaGetSymbolAddress(&addr, g_error_word);
    if (e != cudaSuccess || !addr) return record_cuda_failure(e);
    g_word_addr[dev] = static_cast<uint32_t*>(addr);
  }
  *word = g_word_addr[dev];
  return VSA_OK;
}

}  // namespace vsa

extern "C" {

vsa_status vsa_norm_rope_fwd(const vsa_norm_rope* op, const vsa_heads* q, const vsa_heads* k,
                             const vsa_heads* v, const vsa_heads* q_out, const vsa_heads* k_out,
                             const vsa_heads* v_out, void* stream) {
  vsa_status st = check_norm_rope(op);
  if (st != VSA_OK) return st;
  vsa::NormRopeArgs a{};
  fill_norm_rope(op, &a);
  const vsa_heads* in[3] = {q, k, v};
  const vsa_heads* out[3] = {q_out, k_out, v_out};
  const int size = dtype_size(op->dtype);
  bool any = false;
  for (int i = 0; i < 3; ++i) {
    if (!present(in[i]) && !present(out[i])) continue;
    any = true;
    if ((st = view_of(in[i], op->batch, op->tokens, op->head_dim, size, false, &a.in[i])) != VSA_OK) return st;
    if ((st = view_of(out[i], op->batch, op->rows, op->head_dim, size, true, &a.out[i])) != VSA_OK) return st;
    if (a.in[i].heads != a.out[i].heads) return VSA_ERR_INVALID_ARG;
  }
  if (!any) return VSA_ERR_INVALID_ARG;
  if ((st = check_device()) != VSA_OK || (st = vsa::layer_error_word(&a.err)) != VSA_OK) return st;
  return cuda_status(vsa::launch_norm_rope_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t vsa_norm_rope_bwd_workspace_bytes(const vsa_norm_rope* op) {
  return check_norm_rope(op) == VSA_OK ? vsa::norm_rope_bwd_workspace(op->head_dim) : 0;
}

vsa_status vsa_norm_rope_bwd(const vsa_norm_rope* op, const vsa_heads* dq_out,
                             const vsa_heads* dk_out, const vsa_heads* dv_out, const vsa_heads* q,
                             const vsa_heads* k, const vsa_heads* dq, const vsa_heads* dk,
                             const vsa_heads* dv, void* dq_weight, void* dk_weight,
                             void* workspace, size_t workspace_bytes, void* stream) {
  vsa_status st = check_norm_rope(op);
  if (st != VSA_OK) return st;
  vsa::NormRopeArgs a{};
  fill_norm_rope(op, &a);
  const vsa_heads* dy[3] = {dq_out, dk_out, dv_out};
  const vsa_heads* dx[3] = {dq, dk, dv};
  const vsa_heads* x[2] = {q, k};
  void* dw[2] = {dq_weight, dk_weight};
  const int size = dtype_size(op->dtype);
  bool any = false;
  for (int i = 0; i < 3; ++i) {
    if (!present(dy[i]) && !present(dx[i]) && (i == 2 || (!present(x[i]) && !dw[i]))) continue;
    any = true;
    if ((st = view_of(dy[i], op->batch, op->rows, op->head_dim, size, false, &a.in[i])) != VSA_OK) return st;
    if ((st = view_of(dx[i], op->batch, op->tokens, op->head_dim, size, true, &a.out[i])) != VSA_OK) return st;
    if (a.in[i].heads != a.out[i].heads) return VSA_ERR_INVALID_ARG;
    if (i == 2) continue;
    if ((st = view_of(x[i], op->batch, op->tokens, op->head_dim, size, false, &a.x[i])) != VSA_OK) return st;
    if (a.x[i].heads != a.in[i].heads || !aligned(dw[i], 4)) return VSA_ERR_INVALID_ARG;
    a.dweight[i] = dw[i];
  }
  if (!any) return VSA_ERR_INVALID_ARG;
  const size_t need = a.dweight[0] || a.dweight[1] ? vsa::norm_rope_bwd_workspace(op->head_dim) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != VSA_OK) return st;
  a.partial = static_cast<float*>(workspace);
  if ((st = check_device()) != VSA_OK || (st = vsa::layer_error_word(&a.err)) != VSA_OK) return st;
  return cuda_status(vsa::launch_norm_rope_bwd(a, static_cast<cudaStream_t>(stream)));
}

size_t vsa_cross_fwd_workspace_bytes(const vsa_cross* op) {
  return check_cross(op) == VSA_OK ? vsa::cross_fwd_workspace(op->batch, op->heads, op->kv_heads,
                                                              op->q_tokens, op->kv_tokens)
                                   : 0;
}

size_t vsa_cross_bwd_workspace_bytes(const vsa_cross* op) {
  return check_cross(op) == VSA_OK ? vsa::cross_bwd_workspace(op->batch, op->heads, op->kv_heads,
                                                              op->q_tokens, op->kv_tokens)
                                   : 0;
}

vsa_status vsa_cross_fwd(const vsa_cross* op, const vsa_heads* q, const vsa_heads* k,
                         const vsa_heads* v, const vsa_heads* o, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  vsa_status st = check_cross(op);
  if (st != VSA_OK) return st;
  vsa::CrossArgs a{};
  fill_cross(op, &a);
  const int B = op->batch, Sq = op->q_tokens, Sk = op->kv_tokens;
  if ((st = cross_view(q, B, Sq, false, &a.q)) != VSA_OK) return st;
  if ((st = cross_view(k, B, Sk, false, &a.k)) != VSA_OK) return st;
  if ((st = cross_view(v, B, Sk, false, &a.v)) != VSA_OK) return st;
  if ((st = cross_view(o, B, Sq, true, &a.o)) != VSA_OK) return st;
  if (a.q.heads != op->heads || a.o.heads != op->heads || a.k.heads != op->kv_heads || a.v.heads != op->kv_heads)
    return VSA_ERR_INVALID_ARG;
  if (!lse || !aligned(lse, 4)) return VSA_ERR_INVALID_ARG;
  a.lse = lse;
  if ((st = check_workspace(workspace, workspace_bytes, vsa_cross_fwd_workspace_bytes(op))) != VSA_OK) return st;
  a.workspace = static_cast<uint8_t*>(workspace);
  if ((st = check_device()) != VSA_OK || (st = vsa::layer_error_word(&a.err)) != VSA_OK) return st;
  return cuda_status(vsa::launch_cross_fwd(a, static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_cross_bwd(const vsa_cross* op, const vsa_heads* dout, const vsa_heads* q,
                         const vsa_heads* k, const vsa_heads* v, const vsa_heads* o,
                         const float* lse, const vsa_heads* dq, const vsa_heads* dk,
                         const vsa_heads* dv, void* workspace, size_t workspace_bytes,
                         void* stream) {
  vsa_status st = check_cross(op);
  if (st != VSA_OK) return st;
  vsa::CrossArgs a{};
  fill_cross(op, &a);
  const int B = op->batch, Sq = op->q_tokens, Sk = op->kv_tokens;
  struct {
    const vsa_heads* x;
    int tokens, heads;
    bool output;
    vsa::HeadsView* view;
  } t[] = {{dout, Sq, op->heads, false, &a.dout}, {q, Sq, op->heads, false, &a.q},
           {k, Sk, op->kv_heads, false, &a.k},    {v, Sk, op->kv_heads, false, &a.v},
           {o, Sq, op->heads, false, &a.o},       {dq, Sq, op->heads, true, &a.dq},
           {dk, Sk, op->kv_heads, true, &a.dk},   {dv, Sk, op->kv_heads, true, &a.dv}};
  for (auto& x : t) {
    if ((st = cross_view(x.x, B, x.tokens, x.output, x.view)) != VSA_OK) return st;
    if (x.view->heads != x.heads) return VSA_ERR_INVALID_ARG;
  }
  if (!lse || !aligned(lse, 4)) return VSA_ERR_INVALID_ARG;
  a.lse = const_cast<float*>(lse);
  if ((st = check_workspace(workspace, workspace_bytes, vsa_cross_bwd_workspace_bytes(op))) != VSA_OK) return st;
  a.workspace = static_cast<uint8_t*>(workspace);
  if ((st = check_device()) != VSA_OK || (st = vsa::layer_error_word(&a.err)) != VSA_OK) return st;
  return cuda_status(vsa::launch_cross_bwd(a, static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_layer_device_error(uint32_t* bits, void* stream) {
  if (!bits) return VSA_ERR_INVALID_ARG;
  uint32_t* word = nullptr;
  const vsa_status st = vsa::layer_error_word(&word);
  if (st != VSA_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_read_mutex);  // readers share word[1]
  void* args[] = {&word};
  cudaError_t e = cudaLaunchKernel(take_error_word_kernel, dim3(1), dim3(1), args, 0, s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(bits, word + 1, sizeof(uint32_t), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return cuda_status(e);
}

}  // extern "C"
