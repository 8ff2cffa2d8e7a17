// linear.cu -- out = act(x W^T + bias) + residual and its gradients.
#include "act.cuh"
#include "vec8.cuh"

namespace vsa {

namespace {

constexpr int T = 64, KT = 16;  // tile of the result, step of the sum

// C[i][j] = sum_k A(i, k) B(j, k), element (i, k) of A at a[i * ai + k * ak], and what follows it.
template <typename E>
struct Product {
  const E *a, *b;
  int64_t ai, ak, bj, bk;
  int m, n, k;
  const void* bias;
  bool bias_f32;
  int act;                 // out = act(z) + residual
  MatrixView residual, pre, out;
  MatrixView slope;        // out *= act'(slope)
  int slope_act;
};

template <typename E>
__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ Product<E> p) {
  __shared__ float sa[KT][T + 1], sb[KT][T + 1];
  grid_dependency_wait();
  const int i0 = blockIdx.y * T, j0 = blockIdx.x * T, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += KT) {
    for (int x = threadIdx.x; x < T * KT; x += 256) {
      const int r = p.ak == 1 ? x / KT : x % T, k = p.ak == 1 ? x % KT : x / T;
      sa[k][r] = i0 + r < p.m && k0 + k < p.k ? widen16(p.a[(i0 + r) * p.ai + (k0 + k) * p.ak]) : 0.f;
      const int s = p.bk == 1 ? x / KT : x % T, l = p.bk == 1 ? x % KT : x / T;
      sb[l][s] = j0 + s < p.n && k0 + l < p.k ? widen16(p.b[(j0 + s) * p.bj + (k0 + l) * p.bk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = i0 + ty * 4 + i, c = j0 + tx * 4 + j;
      if (r >= p.m || c >= p.n) continue;
      float z = acc[i][j];
      if (p.bias) z += p.bias_f32 ? static_cast<const float*>(p.bias)[c] : widen16(static_cast<const E*>(p.bias)[c]);
      if (p.pre.data) narrow(z, static_cast<E*>(p.pre.data) + r * p.pre.stride + c);
      z = act_value(z, p.act);
      if (p.residual.data) z += widen16(static_cast<const E*>(p.residual.data)[r * p.residual.stride + c]);
      if (p.slope.data) z *= act_slope(widen16(static_cast<const E*>(p.slope.data)[r * p.slope.stride + c]), p.slope_act);
      narrow(z, static_cast<E*>(p.out.data) + r * p.out.stride + c);
    }
}

// dz = dout act'(pre) (not written without an activation) and the sums of its columns over `chunk`
// rows, to partial [blockIdx.y][n] fp32.
template <typename E>
__global__ void __launch_bounds__(256) slope_kernel(MatrixView dout, MatrixView pre, E* dz, float* partial, int m, int n,
                                                    int chunk, int act) {
  grid_dependency_wait();
  const int c = blockIdx.x * 256 + threadIdx.x, r1 = min(m, (static_cast<int>(blockIdx.y) + 1) * chunk);
  if (c >= n) return;
  float sum = 0.f;
  for (int r = blockIdx.y * chunk; r < r1; ++r) {
    float g = widen16(static_cast<const E*>(dout.data)[r * dout.stride + c]);
    if (act) {
      g *= act_slope(widen16(static_cast<const E*>(pre.data)[r * pre.stride + c]), act);
      narrow(g, dz + static_cast<int64_t>(r) * n + c);
    }
    sum += g;
  }
  if (partial) partial[static_cast<int64_t>(blockIdx.y) * n + c] = sum;
}

template <typename E>
__global__ void __launch_bounds__(256) dbias_kernel(const float* partial, int parts, int n, void* dbias, bool f32) {
  grid_dependency_wait();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  float sum = 0.f;
  for (int i = 0; i < parts; ++i) sum += partial[static_cast<int64_t>(i) * n + c];
  if (f32) static_cast<float*>(dbias)[c] = sum;
  else narrow(sum, static_cast<E*>(dbias) + c);
}

int chunk_rows(int rows) { return rows / 256 > 16 ? rows / 256 : 16; }
size_t dz_bytes(int rows, int n, int act) {
  return act ? align_up(static_cast<size_t>(rows) * n * 2, 256) : 0;
}

template <typename E>
cudaError_t multiply(const Product<E>& p, cudaStream_t stream) {
  return launch_dependent(product_kernel<E>, dim3((p.n + T - 1) / T, (p.m + T - 1) / T), dim3(256), 0, stream, p);
}

template <typename E>
cudaError_t forward(const LinearArgs& a, cudaStream_t stream) {
  Product<E> p{};
  p.a = static_cast<const E*>(a.x.data), p.ai = a.x.stride, p.ak = 1;
  p.b = static_cast<const E*>(a.weight.data), p.bj = a.weight.stride, p.bk = 1;
  p.m = a.rows, p.n = a.out_features, p.k = a.in;
  p.bias = a.bias, p.bias_f32 = a.bias_dtype == VSA_F32, p.act = a.act;
  p.residual = a.residual, p.pre = a.pre, p.out = a.out;
  return multiply(p, stream);
}

template <typename E>
cudaError_t backward(const LinearArgs& a, cudaStream_t stream) {
  const int m = a.rows, n = a.out_features, chunk = chunk_rows(m), parts = (m + chunk - 1) / chunk;
  E* dz = reinterpret_cast<E*>(a.workspace);
  float* partial = reinterpret_cast<float*>(a.workspace + dz_bytes(m, n, a.act));
  cudaError_t e = cudaSuccess;
  if (a.act || a.dbias) {
    e = launch_dependent(slope_kernel<E>, dim3((n + 255) / 256, parts), dim3(256), 0, stream, a.dout, a.pre, dz,
                         a.dbias ? partial : nullptr, m, n, chunk, a.act);
    if (e == cudaSuccess && a.dbias)
      e = launch_dependent(dbias_kernel<E>, dim3((n + 255) / 256), dim3(256), 0, stream, partial, parts, n, a.dbias,
                           a.bias_dtype == VSA_F32);
    if (e != cudaSuccess) return e;
  }
  const E* g = a.act ? dz : static_cast<const E*>(a.dout.data);
  const int64_t gs = a.act ? n : a.dout.stride;
  if (a.dx.data) {
    Product<E> p{};
    p.a = g, p.ai = gs, p.ak = 1;
    p.b = static_cast<const E*>(a.weight.data), p.bj = 1, p.bk = a.weight.stride;
    p.m = m, p.n = a.in, p.k = n;
    p.out = a.dx;
    p.slope = a.x_pre, p.slope_act = a.x_act;
    if ((e = multiply(p, stream)) != cudaSuccess) return e;
  }
  if (a.dweight.data) {
    Product<E> p{};
    p.a = g, p.ai = 1, p.ak = gs;
    p.b = static_cast<const E*>(a.x.data), p.bj = 1, p.bk = a.x.stride;
    p.m = n, p.n = a.in, p.k = m;
    p.out = a.dweight;
    e = multiply(p, stream);
  }
  return e;
}

}  // namespace

size_t linear_fwd_workspace(int, int, int) { return 0; }
size_t linear_bwd_workspace(int rows, int, int out, int act) {
  const int chunk = chunk_rows(rows);
  return align_up(dz_bytes(rows, out, act) + static_cast<size_t>((rows + chunk - 1) / chunk) * out * sizeof(float), 256);
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t stream) {
  return a.dtype == VSA_F16 ? forward<__half>(a, stream) : forward<__nv_bfloat16>(a, stream);
}
cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t stream) {
  return a.dtype == VSA_F16 ? backward<__half>(a, stream) : backward<__nv_bfloat16>(a, stream);
}

}  // namespace vsa
