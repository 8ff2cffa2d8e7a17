// block_api.cu -- the extern "C" entry points declared in include/vsa_block.h: argument checks and
// the stream-ordered launches of each operator.
#include <atomic>
#include <climits>
#include <cmath>

#include "block_internal.cuh"

namespace {

constexpr int64_t MAX_TOKENS = 1 << 30;
constexpr int MAX_FEATURES = 1 << 24;
constexpr int64_t MAX_ELEMENTS = 1ll << 44;  // tiles are counted in 32 bits

vsa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? VSA_OK : vsa::record_cuda_failure(e); }

// The current device's capability, looked up once for each.
vsa_status check_device() {
  static std::atomic<uint64_t> known{0};
  int dev = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (e == cudaSuccess && (known.load(std::memory_order_relaxed) & bit) != 0) return VSA_OK;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return vsa::record_cuda_failure(e);
  if (major != 10 || minor != 3) return VSA_ERR_UNSUPPORTED;
  known.fetch_or(bit, std::memory_order_relaxed);
  return VSA_OK;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int size_of(int dtype) { return dtype == VSA_F32 ? 4 : 2; }

// A stride of n > 1 entries of `size` bytes.
bool stride_ok(int64_t stride, int64_t n, int size) {
  return stride >= 0 && stride <= LLONG_MAX / 4 / n / size && stride * size % 16 == 0;
}

vsa_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return VSA_OK;
  return workspace && aligned(workspace, 256) && bytes >= need ? VSA_OK : VSA_ERR_WORKSPACE;
}

// ------------------------------------------------------------------------------ gate_norm

bool is_dtype(int d) { return d == VSA_BF16 || d == VSA_F16 || d == VSA_F32; }

bool mod_ok(const vsa_modulation& m, const vsa_gate_norm* op) {
  if (!m.data) return true;
  const int size = size_of(op->mod_dtype);
  return aligned(m.data, 16) && (op->batch == 1 || stride_ok(m.batch_stride, op->batch, size)) &&
         (op->groups == 1 || stride_ok(m.group_stride, op->groups, size));
}

vsa_status check_gate_norm(const vsa_gate_norm* op) {
  if (!op || op->batch < 1 || op->tokens < 1 || op->groups < 1) return VSA_ERR_INVALID_ARG;
  if (op->channels < 8 || op->channels > 8192 || op->channels % 8 != 0) return VSA_ERR_UNSUPPORTED;
  if (op->kind != VSA_LAYER_NORM && op->kind != VSA_RMS_NORM) return VSA_ERR_UNSUPPORTED;
  if (!is_dtype(op->dtype) || !is_dtype(op->branch_dtype) || !is_dtype(op->mod_dtype) || !is_dtype(op->weight_dtype))
    return VSA_ERR_UNSUPPORTED;
  if (op->branch_dtype != op->dtype && op->dtype != VSA_F32) return VSA_ERR_UNSUPPORTED;
  if ((op->mod_dtype != VSA_F32 && op->mod_dtype != op->branch_dtype) ||
      (op->weight_dtype != VSA_F32 && op->weight_dtype != op->branch_dtype))
    return VSA_ERR_UNSUPPORTED;
  if (!std::isfinite(op->eps) || op->eps < 0.f || !std::isfinite(op->post_eps) || op->post_eps < 0.f)
    return VSA_ERR_INVALID_ARG;
  if (op->tokens % op->groups != 0) return VSA_ERR_INVALID_ARG;
  if (op->groups > 1 && !op->gate.data && !op->scale.data && !op->shift.data) return VSA_ERR_INVALID_ARG;
  if (!mod_ok(op->gate, op) || !mod_ok(op->scale, op) || !mod_ok(op->shift, op)) return VSA_ERR_INVALID_ARG;
  if (!aligned(op->post_weight, 16) || !aligned(op->weight, 16) || !aligned(op->bias, 16)) return VSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(op->batch) * op->tokens > MAX_TOKENS) return VSA_ERR_UNSUPPORTED;
  return VSA_OK;
}

vsa_status tokens_view(const vsa_tokens* x, const vsa_gate_norm* op, int dtype, bool output, vsa::TokensView* v) {
  if (!x || !x->data || !aligned(x->data, 16)) return VSA_ERR_INVALID_ARG;
  v->data = x->data;
  v->batch = op->batch > 1 ? x->batch_stride : 0;
  v->token = op->tokens > 1 ? x->token_stride : 0;
  const int size = size_of(dtype);
  if ((op->batch > 1 && !stride_ok(v->batch, op->batch, size)) ||
      (op->tokens > 1 && !stride_ok(v->token, op->tokens, size)))
    return VSA_ERR_INVALID_ARG;
  if (!output) return VSA_OK;
  // Entries of the smaller stride, then of the larger, step past one another.
  const bool token_first = op->batch == 1 || (op->tokens > 1 && v->token <= v->batch);
  const int64_t s0 = token_first ? v->token : v->batch, n0 = token_first ? op->tokens : op->batch;
  const int64_t s1 = token_first ? v->batch : v->token, n1 = token_first ? op->batch : op->tokens;
  int64_t extent = op->channels;
  if (n0 > 1) {
    if (s0 < extent) return VSA_ERR_INVALID_ARG;
    extent += s0 * (n0 - 1);
  }
  return n1 > 1 && s1 < extent ? VSA_ERR_INVALID_ARG : VSA_OK;
}

void fill_gate_norm(const vsa_gate_norm* op, vsa::GateNormArgs* a) {
  a->batch = op->batch;
  a->tokens = op->tokens;
  a->channels = op->channels;
  a->groups = op->groups;
  a->kind = op->kind;
  a->dtype = op->dtype;
  a->branch_dtype = op->branch_dtype;
  a->mod_dtype = op->mod_dtype;
  a->weight_dtype = op->weight_dtype;
  a->eps = op->eps;
  a->post_eps = op->post_eps;
  const vsa_modulation* from[3] = {&op->gate, &op->scale, &op->shift};
  vsa::ModView* to[3] = {&a->gate, &a->scale, &a->shift};
  for (int i = 0; i < 3; ++i) {
    to[i]->data = from[i]->data;
    to[i]->batch = op->batch > 1 ? from[i]->batch_stride : 0;
    to[i]->group = op->groups > 1 ? from[i]->group_stride : 0;
  }
  a->post_weight = op->post_weight;
  a->weight = op->weight;
  a->bias = op->bias;
}

// ------------------------------------------------------------------------------ linear

bool is_act(int act) { return act >= VSA_ACT_NONE && act <= VSA_SILU; }

bool matrix_ok(const vsa_matrix* x, int rows, int columns) {
  return x && x->data && aligned(x->data, 16) &&
         (rows == 1 || (stride_ok(x->row_stride, rows, 2) && x->row_stride >= columns));
}

vsa::MatrixView matrix_view(const vsa_matrix* x, int rows, int columns) {
  return {x->data, rows == 1 ? columns : x->row_stride};
}

bool present(const vsa_matrix* x) { return x && x->data; }

vsa_status check_linear(const vsa_linear* op) {
  if (!op || op->rows < 1) return VSA_ERR_INVALID_ARG;
  if (op->in_features < 8 || op->in_features % 8 != 0 || op->in_features > MAX_FEATURES ||
      op->out_features < 8 || op->out_features % 8 != 0 || op->out_features > MAX_FEATURES || op->rows > MAX_TOKENS)
    return VSA_ERR_UNSUPPORTED;
  const int64_t m = op->rows, k = op->in_features, n = op->out_features;
  if (m * k > MAX_ELEMENTS || m * n > MAX_ELEMENTS || n * k > MAX_ELEMENTS) return VSA_ERR_UNSUPPORTED;
  if (op->dtype != VSA_BF16 && op->dtype != VSA_F16) return VSA_ERR_UNSUPPORTED;
  if (op->bias_dtype != VSA_F32 && op->bias_dtype != op->dtype) return VSA_ERR_UNSUPPORTED;
  if (!is_act(op->act)) return VSA_ERR_UNSUPPORTED;
  if (!matrix_ok(&op->weight, op->out_features, op->in_features) || !aligned(op->bias, 16)) return VSA_ERR_INVALID_ARG;
  return VSA_OK;
}

void fill_linear(const vsa_linear* op, void* workspace, vsa::LinearArgs* a) {
  a->rows = op->rows;
  a->in = op->in_features;
  a->out_features = op->out_features;
  a->dtype = op->dtype;
  a->bias_dtype = op->bias_dtype;
  a->act = op->act;
  a->weight = matrix_view(&op->weight, op->out_features, op->in_features);
  a->bias = op->bias;
  a->workspace = static_cast<uint8_t*>(workspace);
  a->wait_ns = vsa::wait_limit_ns();
}

}  // namespace

extern "C" {

vsa_status vsa_gate_norm_fwd(const vsa_gate_norm* op, const vsa_tokens* x, const vsa_tokens* y,
                             const vsa_tokens* x_out, const vsa_tokens* h, void* stream) {
  vsa_status st = check_gate_norm(op);
  if (st != VSA_OK) return st;
  vsa::GateNormArgs a{};
  fill_gate_norm(op, &a);
  const bool branch = y && y->data;
  if (branch != (x_out && x_out->data)) return VSA_ERR_INVALID_ARG;
  if (!branch && (op->gate.data || op->post_weight)) return VSA_ERR_INVALID_ARG;
  if ((st = tokens_view(x, op, op->dtype, false, &a.x)) != VSA_OK) return st;
  if ((st = tokens_view(h, op, op->branch_dtype, true, &a.h)) != VSA_OK) return st;
  if (branch) {
    if ((st = tokens_view(y, op, op->branch_dtype, false, &a.y)) != VSA_OK) return st;
    if ((st = tokens_view(x_out, op, op->dtype, true, &a.x_out)) != VSA_OK) return st;
  }
  if ((st = check_device()) != VSA_OK) return st;
  return cuda_status(vsa::launch_gate_norm_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t vsa_gate_norm_bwd_workspace_bytes(const vsa_gate_norm* op) {
  if (check_gate_norm(op) != VSA_OK) return 0;
  vsa::GateNormArgs a{};
  fill_gate_norm(op, &a);
  // (Only which gradients there are counts.)
  a.dgate = const_cast<void*>(op->gate.data);
  a.dscale = const_cast<void*>(op->scale.data);
  a.dshift = const_cast<void*>(op->shift.data);
  a.dpost = const_cast<void*>(op->post_weight);
  a.dweight = const_cast<void*>(op->weight);
  a.dbias = const_cast<void*>(op->bias);
  return vsa::gate_norm_bwd_workspace(a);
}

vsa_status vsa_gate_norm_bwd(const vsa_gate_norm* op, const vsa_tokens* dh,
                             const vsa_tokens* dx_out, const vsa_tokens* x_out,
                             const vsa_tokens* y, const vsa_tokens* dx, const vsa_tokens* dy,
                             const vsa_gate_norm_grads* grads, void* workspace,
                             size_t workspace_bytes, void* stream) {
  vsa_status st = check_gate_norm(op);
  if (st != VSA_OK) return st;
  vsa::GateNormArgs a{};
  fill_gate_norm(op, &a);
  const bool branch = y && y->data;
  if (branch != (dy && dy->data)) return VSA_ERR_INVALID_ARG;
  if (!branch && (op->gate.data || op->post_weight)) return VSA_ERR_INVALID_ARG;
  if ((st = tokens_view(dh, op, op->branch_dtype, false, &a.dh)) != VSA_OK) return st;
  if ((st = tokens_view(x_out, op, op->dtype, false, &a.x_out)) != VSA_OK) return st;
  if ((st = tokens_view(dx, op, op->dtype, true, &a.dx)) != VSA_OK) return st;
  if (dx_out && dx_out->data && (st = tokens_view(dx_out, op, op->dtype, false, &a.dx_out)) != VSA_OK) return st;
  if (branch) {
    if ((st = tokens_view(y, op, op->branch_dtype, false, &a.y)) != VSA_OK) return st;
    if ((st = tokens_view(dy, op, op->branch_dtype, true, &a.dy)) != VSA_OK) return st;
  }
  if (grads) {
    struct {
      void* grad;
      const void* of;
      void** to;
    } g[] = {{grads->gate, op->gate.data, &a.dgate},          {grads->scale, op->scale.data, &a.dscale},
             {grads->shift, op->shift.data, &a.dshift},       {grads->post_weight, op->post_weight, &a.dpost},
             {grads->weight, op->weight, &a.dweight},         {grads->bias, op->bias, &a.dbias}};
    for (auto& x : g) {
      if (!x.grad) continue;
      if (!x.of || !aligned(x.grad, 16)) return VSA_ERR_INVALID_ARG;
      *x.to = x.grad;
    }
    if ((st = check_workspace(workspace, workspace_bytes, vsa::gate_norm_bwd_workspace(a))) != VSA_OK) return st;
    a.workspace = static_cast<float*>(workspace);
  }
  if ((st = check_device()) != VSA_OK) return st;
  return cuda_status(vsa::launch_gate_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

size_t vsa_linear_fwd_workspace_bytes(const vsa_linear* op) {
  return check_linear(op) == VSA_OK ? vsa::linear_fwd_workspace(op->rows, op->in_features, op->out_features) : 0;
}

size_t vsa_linear_bwd_workspace_bytes(const vsa_linear* op) {
  return check_linear(op) == VSA_OK
             ? vsa::linear_bwd_workspace(op->rows, op->in_features, op->out_features, op->act)
             : 0;
}

vsa_status vsa_linear_fwd(const vsa_linear* op, const vsa_matrix* x, const vsa_matrix* residual,
                          const vsa_matrix* out, const vsa_matrix* pre, void* workspace,
                          size_t workspace_bytes, void* stream) {
  vsa_status st = check_linear(op);
  if (st != VSA_OK) return st;
  const int m = op->rows, k = op->in_features, n = op->out_features;
  if (!matrix_ok(x, m, k) || !matrix_ok(out, m, n) || (present(residual) && !matrix_ok(residual, m, n)) ||
      (present(pre) && !matrix_ok(pre, m, n)))
    return VSA_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes, vsa_linear_fwd_workspace_bytes(op))) != VSA_OK) return st;
  vsa::LinearArgs a{};
  fill_linear(op, workspace, &a);
  a.x = matrix_view(x, m, k);
  a.out = matrix_view(out, m, n);
  if (present(residual)) a.residual = matrix_view(residual, m, n);
  if (present(pre)) a.pre = matrix_view(pre, m, n);
  if ((st = check_device()) != VSA_OK || (st = vsa::layer_error_word(&a.err)) != VSA_OK) return st;
  return cuda_status(vsa::launch_linear_fwd(a, static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_linear_bwd(const vsa_linear* op, int32_t x_act, const vsa_matrix* dout,
                          const vsa_matrix* x, const vsa_matrix* pre, const vsa_matrix* x_pre,
                          const vsa_matrix* dx, const vsa_matrix* dweight, void* dbias,
                          void* workspace, size_t workspace_bytes, void* stream) {
  vsa_status st = check_linear(op);
  if (st != VSA_OK) return st;
  const int m = op->rows, k = op->in_features, n = op->out_features;
  if (!is_act(x_act)) return VSA_ERR_UNSUPPORTED;
  if (present(pre) != (op->act != VSA_ACT_NONE) || present(x_pre) != (x_act != VSA_ACT_NONE)) return VSA_ERR_INVALID_ARG;
  if (!present(dx) && !present(dweight) && !dbias) return VSA_ERR_INVALID_ARG;
  if (!matrix_ok(dout, m, n) || (present(pre) && !matrix_ok(pre, m, n)) ||
      (present(dweight) && (!matrix_ok(x, m, k) || !matrix_ok(dweight, n, k))) ||
      (present(dx) && !matrix_ok(dx, m, k)) || (present(x_pre) && !matrix_ok(x_pre, m, k)) || !aligned(dbias, 16))
    return VSA_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes, vsa_linear_bwd_workspace_bytes(op))) != VSA_OK) return st;
  vsa::LinearArgs a{};
  fill_linear(op, workspace, &a);
  a.dout = matrix_view(dout, m, n);
  a.x_act = x_act;
  if (present(dweight)) {
    a.x = matrix_view(x, m, k);
    a.dweight = matrix_view(dweight, n, k);
  }
  if (present(pre)) a.pre = matrix_view(pre, m, n);
  if (present(dx)) a.dx = matrix_view(dx, m, k);
  if (present(dx) && present(x_pre)) a.x_pre = matrix_view(x_pre, m, k);
  a.dbias = dbias;
  if ((st = check_device()) != VSA_OK || (st = vsa::layer_error_word(&a.err)) != VSA_OK) return st;
  return cuda_status(vsa::launch_linear_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
