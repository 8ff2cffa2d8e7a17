// cross_bwd.cu -- attention to an encoder's states of another length, backward: dQ with one warp
// per query row (which also leaves Delta = rowsum(O dO)), then dK and dV with one warp per key.
#include "layer_internal.cuh"

namespace vsa {

namespace {

__device__ __forceinline__ float4 load4(const HeadsView& x, int b, int h, int t, int lane) {
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(x.data) +
                                                  b * x.batch + h * x.head + t * x.token + lane * 4);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

__device__ __forceinline__ void store4(const HeadsView& x, int b, int h, int t, int lane, float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(x.data) + b * x.batch + h * x.head +
                            t * x.token + lane * 4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

__device__ __forceinline__ float warp_dot(float4 x, float4 y) {
  float v = x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float4 fma4(float s, float4 x, float4 y) {
  return make_float4(fmaf(s, x.x, y.x), fmaf(s, x.y, y.y), fmaf(s, x.z, y.z), fmaf(s, x.w, y.w));
}

__device__ __forceinline__ float4 scale4(float s, float4 x) { return make_float4(s * x.x, s * x.y, s * x.z, s * x.w); }

__global__ void __launch_bounds__(256) cross_dq_kernel(const CrossArgs a) {
  grid_dependency_wait();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(a.batch) * a.heads * a.q_tokens) return;
  const int i = static_cast<int>(w % a.q_tokens), bh = static_cast<int>(w / a.q_tokens);
  const int b = bh / a.heads, h = bh % a.heads, kh = h / (a.heads / a.kv_heads);
  const int n = visible_keys(a.kv_len, b, a.kv_tokens, a.err);
  const float c = a.sm_scale * LOG2E_F;
  const float4 q = load4(a.q, b, h, i, lane), g = load4(a.dout, b, h, i, lane);
  const float delta = warp_dot(g, load4(a.o, b, h, i, lane));
  const float lse = a.lse[w] == -INFINITY ? 0.f : a.lse[w];
  float4 dq = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < n; ++j) {
    const float4 k = load4(a.k, b, kh, j, lane);
    const float p = exp2f(warp_dot(q, k) * c - lse);
    dq = fma4(p * (warp_dot(g, load4(a.v, b, kh, j, lane)) - delta), k, dq);
  }
  store4(a.dq, b, h, i, lane, scale4(a.sm_scale, dq));
  if (lane == 0) reinterpret_cast<float*>(a.workspace)[w] = delta;
}

__global__ void __launch_bounds__(256) cross_dkv_kernel(const CrossArgs a) {
  grid_dependency_wait();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(a.batch) * a.kv_heads * a.kv_tokens) return;
  const int j = static_cast<int>(w % a.kv_tokens), bh = static_cast<int>(w / a.kv_tokens);
  const int b = bh / a.kv_heads, kh = bh % a.kv_heads, share = a.heads / a.kv_heads;
  const float c = a.sm_scale * LOG2E_F;
  float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
  const bool visible = j < visible_keys(a.kv_len, b, a.kv_tokens, a.err);
  if (visible) {
    const float4 k = load4(a.k, b, kh, j, lane), v = load4(a.v, b, kh, j, lane);
    for (int h = kh * share; h < (kh + 1) * share; ++h)
      for (int i = 0; i < a.q_tokens; ++i) {
        const int64_t row = (static_cast<int64_t>(b) * a.heads + h) * a.q_tokens + i;
        const float4 q = load4(a.q, b, h, i, lane), g = load4(a.dout, b, h, i, lane);
        const float lse = a.lse[row] == -INFINITY ? 0.f : a.lse[row];
        const float p = exp2f(warp_dot(q, k) * c - lse);
        dv = fma4(p, g, dv);
        dk = fma4(p * (warp_dot(g, v) - reinterpret_cast<const float*>(a.workspace)[row]), q, dk);
      }
  }
  store4(a.dk, b, kh, j, lane, visible ? scale4(a.sm_scale, dk) : dk);  // +0 where hidden
  store4(a.dv, b, kh, j, lane, dv);
}

}  // namespace

size_t cross_bwd_workspace(int batch, int heads, int, int q_tokens, int) {
  return align_up(static_cast<size_t>(batch) * heads * q_tokens * sizeof(float), 256);
}

cudaError_t launch_cross_bwd(const CrossArgs& a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.batch) * a.heads * a.q_tokens;
  const int64_t keys = static_cast<int64_t>(a.batch) * a.kv_heads * a.kv_tokens;
  cudaError_t e = launch_dependent(cross_dq_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(cross_dkv_kernel, dim3(static_cast<unsigned>((keys + 7) / 8)), dim3(256), 0, stream, a);
}

}  // namespace vsa
