// linear.cu -- out = act(x W^T + bias) + residual and its gradients: which kernels a call takes.
//
// Forward: one product with its epilogue (linear_rows.cu up to 8 to 24 rows, gemm_small.cu for small products,
// gemm.cu).  Backward: dz = dout act'(pre) and the columns' sums in a pass of their own, then dx = dz W and
// dweight = dz^T x.  The pass is left out where there is neither an activation nor a bias; and a chain of two
// products does not pay for it twice, as the second's dx goes on through the activation in its
// epilogue (x_act).
// dz is rounded to 16 bits there, as the tensor cores' operands are: dx and dweight are 0.00235 of their norm off in
// bf16 (0.00029 in fp16) where the rounding of the results alone is 0.00166 (0.00021).  A second operand with
// what the rounding lost would take both products twice as long.  dbias adds up dz before it is rounded.
#include "act.cuh"
#include "gemm.cuh"
#include "vec8.cuh"

namespace vsa {

namespace {

// Columns of 8 to a thread, 32 threads of a warp side by side, ROWS warps down the rows, AHEAD rows of a thread in
// flight (32760 x 6144 with gelu_tanh: 188 us, 95 % of the copy rate; 4 in flight 204, 1 214; sums alone 60, 84,
// 63).
constexpr int ROWS = 8, AHEAD = 2;

// dz = dout act'(pre) (not written without an activation) and the sums of its columns over `chunk`
// rows, to partial [blockIdx.y][n] fp32 (unless null).  Bound by HBM: one read of each input, one write.
template <typename E>
__global__ void __launch_bounds__(32 * ROWS) slope_kernel(MatrixView dout, MatrixView pre, E* dz, float* partial, int m, int n,
                                                          int chunk, int act) {
  __shared__ float sums[ROWS][257];
  grid_dependency_wait();
  const int c = (blockIdx.x * 32 + threadIdx.x) * 8, r1 = min(m, (static_cast<int>(blockIdx.y) + 1) * chunk);
  float sum[8] = {};
  if (c < n) {
    for (int r0 = blockIdx.y * chunk + threadIdx.y; r0 < r1; r0 += AHEAD * ROWS) {
      Raw<E> rg[AHEAD], rz[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int r = r0 + i * ROWS;
        rg[i].zero();
        rz[i].zero();
        if (r >= r1) continue;
        rg[i].load(static_cast<const E*>(dout.data) + r * dout.stride + c);
        if (act) rz[i].load(static_cast<const E*>(pre.data) + r * pre.stride + c);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int r = r0 + i * ROWS;
        float g[8];
        rg[i].widen(g);
        if (r >= r1) continue;
        if (act) {
          float z[8];
          rz[i].widen(z);
          slope8(act, z, g);
          store8(dz + static_cast<int64_t>(r) * n + c, g);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) sum[x] += g[x];
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[threadIdx.y][threadIdx.x * 8 + i] = sum[i];
  __syncthreads();
  const int t = threadIdx.y * 32 + threadIdx.x, to = blockIdx.x * 256 + t;
  if (to >= n) return;
  float s = 0.f;
#pragma unroll
  for (int y = 0; y < ROWS; ++y) s += sums[y][t];
  partial[static_cast<int64_t>(blockIdx.y) * n + to] = s;
}

// dbias: the chunks' sums, 32 columns a block, 32 strided chunks each, joined in their order.
template <typename E>
__global__ void __launch_bounds__(1024) dbias_kernel(const float* partial, int parts, int n, void* dbias, bool f32) {
  __shared__ float sums[32][33];
  grid_dependency_wait();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < n)
    for (int i = threadIdx.y; i < parts; i += 32) s += partial[static_cast<int64_t>(i) * n + c];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= n) return;
  s = 0.f;
#pragma unroll
  for (int y = 0; y < 32; ++y) s += sums[y][threadIdx.x];
  if (f32) static_cast<float*>(dbias)[c] = s;
  else narrow(s, static_cast<E*>(dbias) + c);
}

// Rows of a block: about four blocks to an SM, 32 rows at least.
int chunk_rows(int rows, int n) {
  const int64_t columns = (n + 255) / 256, blocks = (4 * device_sm_count() + columns - 1) / columns;
  const int64_t chunk = (rows + blocks - 1) / blocks;
  return static_cast<int>(chunk < 32 ? 32 : (chunk + ROWS - 1) / ROWS * ROWS);
}

struct Layout {
  int chunk, parts;
  size_t partial, gemm, total;  // dz is at 0
};
Layout layout_of(int rows, int in, int out, int act) {
  Layout l;
  l.chunk = chunk_rows(rows, out);
  l.parts = (rows + l.chunk - 1) / l.chunk;
  l.partial = act ? align_up(static_cast<size_t>(rows) * out * 2, 256) : 0;
  l.gemm = align_up(l.partial + static_cast<size_t>(l.parts) * out * sizeof(float), 256);
  const size_t dx = gemm_workspace(rows, in, out), dw = gemm_workspace(out, in, rows);
  l.total = l.gemm + (dx > dw ? dx : dw);
  return l;
}

template <typename E>
cudaError_t slopes(const LinearArgs& a, const Layout& l, cudaStream_t stream) {
  const int n = a.out_features;
  float* partial = a.dbias ? reinterpret_cast<float*>(a.workspace + l.partial) : nullptr;
  cudaError_t e = launch_dependent(slope_kernel<E>, dim3((n + 255) / 256, l.parts), dim3(32, ROWS), 0, stream, a.dout, a.pre,
                                   reinterpret_cast<E*>(a.workspace), partial, a.rows, n, l.chunk, a.act);
  if (e != cudaSuccess || !a.dbias) return e;
  return launch_dependent(dbias_kernel<E>, dim3((n + 31) / 32), dim3(32, 32), 0, stream, partial, l.parts, n, a.dbias,
                          a.bias_dtype == VSA_F32);
}

}  // namespace

size_t linear_fwd_workspace(int rows, int in, int out) {
  return use_linear_rows(rows, in, out) ? 0 : gemm_workspace(rows, out, in);
}
size_t linear_bwd_workspace(int rows, int in, int out, int act) { return layout_of(rows, in, out, act).total; }

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t stream) {
  if (use_linear_rows(a.rows, a.in, a.out_features)) return launch_linear_rows(a, stream);
  GemmArgs g{};
  g.a = a.x;
  g.b = a.weight;
  g.out = a.out;
  g.pre = a.pre;
  g.aux = a.residual;
  g.bias = a.bias;
  g.bias_f32 = a.bias_dtype == VSA_F32;
  g.m = a.rows, g.n = a.out_features, g.k = a.in;
  g.act = a.act;
  g.dtype = a.dtype;
  g.workspace = a.workspace;
  g.err = a.err;
  g.wait_ns = a.wait_ns;
  return launch_gemm(GEMM_FWD, g, stream);
}

cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t stream) {
  const Layout l = layout_of(a.rows, a.in, a.out_features, a.act);
  cudaError_t e = cudaSuccess;
  if (a.act || a.dbias)
    e = a.dtype == VSA_F16 ? slopes<__half>(a, l, stream) : slopes<__nv_bfloat16>(a, l, stream);
  if (e != cudaSuccess) return e;
  GemmArgs g{};
  g.a = a.act ? MatrixView{a.workspace, a.out_features} : a.dout;  // dz
  g.dtype = a.dtype;
  g.workspace = a.workspace + l.gemm;
  g.err = a.err;
  g.wait_ns = a.wait_ns;
  GemmArgs w = g;
  if (a.dx.data) {
    g.b = a.weight;
    g.out = a.dx;
    g.aux = a.x_pre;
    g.act = a.x_act;
    g.m = a.rows, g.n = a.in, g.k = a.out_features;
  }
  if (a.dweight.data) {
    w.b = a.x;
    w.out = a.dweight;
    w.m = a.out_features, w.n = a.in, w.k = a.rows;
  }
  if (a.dx.data && a.dweight.data && use_gemm_small_pair(g, w)) return launch_gemm_small_pair(GEMM_DX, g, GEMM_DW, w, stream);
  if (a.dx.data && (e = launch_gemm(GEMM_DX, g, stream)) != cudaSuccess) return e;
  return a.dweight.data ? launch_gemm(GEMM_DW, w, stream) : cudaSuccess;
}

}  // namespace vsa
