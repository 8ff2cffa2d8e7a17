// cross_fwd.cu -- attention to an encoder's states of another length, forward: one warp per query
// row, one pass over the row's visible keys with the running maximum and sum of the softmax.
#include "layer_internal.cuh"

namespace vsa {

namespace {

__device__ __forceinline__ float4 load4(const void* base, int64_t at) {
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + at);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(256) cross_fwd_kernel(const CrossArgs a) {
  grid_dependency_wait();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(a.batch) * a.heads * a.q_tokens) return;
  const int i = static_cast<int>(w % a.q_tokens), bh = static_cast<int>(w / a.q_tokens);
  const int b = bh / a.heads, h = bh % a.heads, kh = h / (a.heads / a.kv_heads);
  const int n = visible_keys(a.kv_len, b, a.kv_tokens, a.err);
  const float c = a.sm_scale * LOG2E_F;
  const float4 q = load4(a.q.data, b * a.q.batch + h * a.q.head + i * a.q.token + lane * 4);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < n; ++j) {
    const float4 k = load4(a.k.data, b * a.k.batch + kh * a.k.head + j * a.k.token + lane * 4);
    const float4 v = load4(a.v.data, b * a.v.batch + kh * a.v.head + j * a.v.token + lane * 4);
    const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * c;
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ref), p = exp2f(s - ref);
    m = mn;
    l = l * f + p;
    o.x = o.x * f + p * v.x, o.y = o.y * f + p * v.y, o.z = o.z * f + p * v.z, o.w = o.w * f + p * v.w;
  }
  const float inv = l == 0.f ? 1.f : 1.f / l;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o.data) + b * a.o.batch + h * a.o.head + i * a.o.token + lane * 4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (lane == 0) a.lse[w] = m + log2f(l);
}

}  // namespace

size_t cross_fwd_workspace(int, int, int, int, int) { return 0; }

cudaError_t launch_cross_fwd(const CrossArgs& a, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(a.batch) * a.heads * a.q_tokens;
  return launch_dependent(cross_fwd_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0, stream, a);
}

}  // namespace vsa
