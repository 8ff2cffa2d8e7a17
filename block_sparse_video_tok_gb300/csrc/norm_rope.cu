// norm_rope.cu -- the RMS norm of every query and key head with the position rotation, in the
// pass that moves q, k and v between token order and attention rows, and its backward.
//
// Forward, per row r (token t = order[r]) and head x of q or k:
//   n = x rsqrt(mean(x^2) + eps),  y = R_t (n w);   v: y = x.
// Backward, per token t (row r = order[t]): u = R_t^T dy,
//   dw += u n,  dx = rsqrt(..) (u w - n mean(u w n));   v: dx = dy.
//
// Both are bound by HBM: one read and one write of every activation, next to which the table
// (4 rot bytes a token, read once for all heads) is small.  A head is held by LPR neighbouring
// lanes, 8 elements (16 bytes of bf16) each, so the mean is a shuffle reduction and no element
// passes through shared memory; a group of LPR lanes keeps one token's table values in registers
// and walks the heads, UNROLL loads in flight per lane.  Head sizes that are no power of two
// leave the last lanes of a group idle.  When the tokens alone do not fill the GPU (single tokens
// above all), the heads are spread over the grid's second dimension.
#include "layer_internal.cuh"

namespace vsa {

namespace {

// Heads in flight per group of lanes, and what the backward's registers leave room for: 6 heads and
// four CTAs of 128 threads per SM.  (12 heads of 128, bf16: forward of 131040 tokens 388 us, 99 % of
// the measured copy rate, with 4 heads 394; backward of 2 x 32760 266 us, 90 %, with 4 heads 287,
// with 8 heads 340.  One number for all sizes is a compromise: heads come in sixes, 8 as 6 + 2.  2 x
// 32760 tokens, as many heads of k and v as of q, us with 6, 4 and 8 in flight:
//   heads of         forward            backward
//   8 x 128, bf16    152, 140, 139      214, 198, 205
//   16 x 128, bf16   273, 273, 269      369, 381, 405
//   24 x 128, bf16   403, 407, 401      517, 564, 591
//   8 x 256, bf16    296, 273, 273      442, 386, 405
//   8 x 64, fp32     138, 137, 136      204, 181, 237
//   12 x 128, fp32   397, 399, 397      579, 525, 750.)
constexpr int THREADS = 128, BWD_CTAS = 4;
constexpr int UNROLL = 6;
constexpr unsigned FULL = 0xffffffffu;

// 8 elements as loaded (16 or 32 bytes), widened where they are used: a lane keeps several heads'
// worth in flight.
template <typename T>
struct Raw {
  uint4 u[sizeof(T) / 2];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
  }
  __device__ __forceinline__ void widen(float* v) const;
};
template <>
__device__ __forceinline__ void Raw<float>::widen(float* v) const {
  v[0] = __uint_as_float(u[0].x), v[1] = __uint_as_float(u[0].y), v[2] = __uint_as_float(u[0].z);
  v[3] = __uint_as_float(u[0].w), v[4] = __uint_as_float(u[1].x), v[5] = __uint_as_float(u[1].y);
  v[6] = __uint_as_float(u[1].z), v[7] = __uint_as_float(u[1].w);
}
template <>
__device__ __forceinline__ void Raw<__nv_bfloat16>::widen(float* v) const {
  const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void Raw<__half>::widen(float* v) const {
  const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  Raw<T> r;
  r.load(p);
  r.widen(v);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

struct Params {
  NormRopeArgs a;
  float inv_dim;
  int chunk;  // heads per block of the grid's second dimension
};

// order[i] if it is -1 or in [0, n), else -1 with the error bit raised; i itself without an order.
__device__ __forceinline__ int mapped(const int32_t* order, int i, int n, uint32_t* err) {
  if (!order) return i;
  const int t = order[i];
  if (t >= -1 && t < n) return t;
  atomicOr(err, VSA_DEVERR_ORDER);
  return -1;
}

// Entries of an order of n entries in [-1, m) that the other direction's order does not name back.  The
// grid's threads take one entry after another when their activations are done: values kept for it
// beside them cost up to 9 of 394 us in spilled registers.
__device__ __forceinline__ void check_inverse(const NormRopeArgs& a, int n, int m) {
  if (!a.inverse || blockIdx.y > 0) return;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * THREADS) {
    const int t = a.order[i];
    if (t >= 0 && t < m && a.inverse[t] != i) atomicOr(a.err, VSA_DEVERR_ORDER);
  }
}

// One lane's share of a token's rotation: the angles of its 8 elements and, with HALVES, the lane
// that holds the other element of each pair.  Lanes past `rot` get the identity.
template <int LPR, bool HALVES>
struct Rotation {
  float c[8], s[8];  // HALVES: per element, s negative for a pair's first; else 4 pairs used
  int partner;

  __device__ __forceinline__ void load(const NormRopeArgs& a, int b, int t, int lane, bool on) {
    const int half = a.rot >> 1, e = (lane & (LPR - 1)) * 8;
    partner = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    if (e >= a.rot) return;
    if (HALVES) {
      partner = e < half ? lane + half / 8 : lane - half / 8;
      if (!on) return;
      const int64_t at = b * a.table_batch + static_cast<int64_t>(t) * half + (e < half ? e : e - half);
      load8(a.cosines + at, c);
      load8(a.sines + at, s);
      if (e < half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
      }
    } else if (on) {
      const int64_t at = b * a.table_batch + static_cast<int64_t>(t) * half + e / 2;
      const float4 cc = *reinterpret_cast<const float4*>(a.cosines + at);
      const float4 ss = *reinterpret_cast<const float4*>(a.sines + at);
      c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
      s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
    }
  }

  // v = R v, or R^T v with INVERSE.  The whole warp takes part.
  template <bool INVERSE>
  __device__ __forceinline__ void turn(float* v) const {
    if (HALVES) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = __shfl_sync(FULL, v[i], partner);
        v[i] = fmaf(INVERSE ? -w : w, s[i], v[i] * c[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1], z = INVERSE ? -s[i] : s[i];
        v[2 * i] = fmaf(-b, z, a * c[i]);
        v[2 * i + 1] = fmaf(a, z, b * c[i]);
      }
    }
  }
};

template <typename W>
__device__ __forceinline__ void load_weight(const void* w, int e, bool on, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 1.f;
  if (w && on) load8(static_cast<const W*>(w) + e, v);
}

template <typename T, typename W, int LPR, bool HALVES>
__global__ void __launch_bounds__(THREADS) norm_rope_fwd_kernel(const Params p) {
  grid_dependency_wait();
  const NormRopeArgs& a = p.a;
  const int lane = threadIdx.x & 31, e = (lane & (LPR - 1)) * 8;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (THREADS / LPR) + threadIdx.x / LPR;
  const bool active = n < static_cast<int64_t>(a.batch) * a.rows && e < a.head_dim;
  const int b = active ? static_cast<int>(n / a.rows) : 0;
  const int row = active ? static_cast<int>(n - static_cast<int64_t>(b) * a.rows) : 0;
  const int t = active ? mapped(a.order, row, a.tokens, a.err) : -1;
  const bool has = t >= 0;
  Rotation<LPR, HALVES> rot;
  rot.load(a, b, t, lane, has);
  float w[2][8];
  load_weight<W>(a.weight[0], e, has, w[0]);
  load_weight<W>(a.weight[1], e, has, w[1]);
  const int lo = blockIdx.y * p.chunk, hi = lo + p.chunk;
  int first = 0;
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int h0 = max(lo - first, 0), h1 = min(hi - first, a.in[x].heads);
    first += a.in[x].heads;
    const T* src = static_cast<const T*>(a.in[x].data) + b * a.in[x].batch + t * a.in[x].token + e;
    T* dst = static_cast<T*>(a.out[x].data) + b * a.out[x].batch + row * a.out[x].token + e;
    for (int h = h0; h < h1; h += UNROLL) {
      Raw<T> raw[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        raw[u].zero();
        if (has && h + u < h1) raw[u].load(src + (h + u) * a.in[x].head);
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        T* to = dst + (h + u) * a.out[x].head;
        if (x == 2) {
          if (active && h + u < h1) raw[u].store(to);
          continue;
        }
        float v[8], ss = 0.f;
        raw[u].widen(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
        const float r = rsqrtf(fmaf(group_sum<LPR>(ss), p.inv_dim, a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = has ? v[i] * r * w[x & 1][i] : 0.f;
        rot.template turn<false>(v);
        if (active && h + u < h1) store8(to, v);
      }
    }
  }
  check_inverse(a, a.rows, a.tokens);
}

template <typename T, typename W, int LPR, bool HALVES>
__global__ void __launch_bounds__(THREADS, BWD_CTAS) norm_rope_bwd_kernel(const Params p) {
  __shared__ float sums[THREADS / LPR][LPR * 8];
  grid_dependency_wait();
  const NormRopeArgs& a = p.a;
  const int lane = threadIdx.x & 31, group = threadIdx.x / LPR, e = (lane & (LPR - 1)) * 8;
  float w[2][8], dw[2][8];
  load_weight<W>(a.weight[0], e, e < a.head_dim, w[0]);
  load_weight<W>(a.weight[1], e, e < a.head_dim, w[1]);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  const int lo = blockIdx.y * p.chunk, hi = lo + p.chunk;
  const int64_t total = static_cast<int64_t>(a.batch) * a.tokens;
  // The trip count is the same for every group of a CTA, so that whole warps meet the shuffles.
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * (THREADS / LPR); base < total;
       base += static_cast<int64_t>(gridDim.x) * (THREADS / LPR)) {
    const int64_t n = base + group;
    const bool active = n < total && e < a.head_dim;
    const int b = active ? static_cast<int>(n / a.tokens) : 0;
    const int t = active ? static_cast<int>(n - static_cast<int64_t>(b) * a.tokens) : 0;
    const int row = active ? mapped(a.order, t, a.rows, a.err) : -1;
    const bool has = row >= 0;
    Rotation<LPR, HALVES> rot;
    rot.load(a, b, t, lane, has);
    int first = 0;
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const int h0 = max(lo - first, 0), h1 = min(hi - first, a.in[x].heads);
      first += a.in[x].heads;
      const T* dy = static_cast<const T*>(a.in[x].data) + b * a.in[x].batch + row * a.in[x].token + e;
      T* dx = static_cast<T*>(a.out[x].data) + b * a.out[x].batch + t * a.out[x].token + e;
      const T* src = static_cast<const T*>(a.x[x & 1].data) + b * a.x[x & 1].batch +
                     t * a.x[x & 1].token + e;
      for (int h = h0; h < h1; h += UNROLL) {
        Raw<T> ry[UNROLL], rx[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
          ry[k].zero();
          rx[k].zero();
          if (has && h + k < h1) {
            ry[k].load(dy + (h + k) * a.in[x].head);
            if (x < 2) rx[k].load(src + (h + k) * a.x[x & 1].head);
          }
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
          T* to = dx + (h + k) * a.out[x].head;
          if (x == 2) {
            if (active && h + k < h1) ry[k].store(to);
            continue;
          }
          float u[8], v[8], ss = 0.f, sg = 0.f;
          ry[k].widen(u);
          rx[k].widen(v);
          rot.template turn<true>(u);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(v[i], v[i], ss);
            sg = fmaf(u[i] * w[x & 1][i], v[i], sg);
          }
          // Lanes without a row hold zeros, but the root is infinite there when eps is 0.
          const float root = rsqrtf(fmaf(group_sum<LPR>(ss), p.inv_dim, a.eps)), r = has ? root : 0.f;
          const float m = group_sum<LPR>(sg) * p.inv_dim * r;  // mean(u w n)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float n = v[i] * r;
            dw[x & 1][i] = fmaf(u[i], n, dw[x & 1][i]);
            u[i] = r * fmaf(-n, m, u[i] * w[x & 1][i]);
          }
          if (active && h + k < h1) store8(to, u);
        }
      }
    }
  }
  check_inverse(a, a.tokens, a.rows);
  if (!a.dweight[0] && !a.dweight[1]) return;
  // The groups' sums, added in group order.
  float* part = a.partial + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * a.head_dim;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[group][e + i] = dw[x][i];
    __syncthreads();
    for (int d = threadIdx.x; d < a.head_dim; d += THREADS) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < THREADS / LPR; ++g) s += sums[g][d];
      part[x * a.head_dim + d] = s;
    }
  }
}

// dw[x][d] = sum of the CTAs' partial sums: 32 columns a block, 32 strided rows each, joined in
// row order.
template <typename W>
__global__ void __launch_bounds__(1024) norm_rope_dweight_kernel(const float* partial, int parts,
                                                                 int dim, W* dq, W* dk) {
  __shared__ float sums[32][33];
  grid_dependency_wait();
  const int d = blockIdx.x * 32 + threadIdx.x;
  W* out = blockIdx.y == 0 ? dq : dk;
  float s = 0.f;
  if (d < dim)
    for (int i = threadIdx.y; i < parts; i += 32)
      s += partial[(static_cast<int64_t>(i) * 2 + blockIdx.y) * dim + d];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && d < dim && out) {
    float t = 0.f;
#pragma unroll
    for (int y = 0; y < 32; ++y) t += sums[y][threadIdx.x];
    out[d] = static_cast<W>(t);
  }
}

int lanes_per_head(int head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }

// Blocks of the grid's second dimension: one unless the tokens leave SMs without a block (8 tokens
// of 12 heads: forward 3.0 us, heads not spread 5.5; 256 of 48: 4.5 and 12.0, backward 8.4 and 17.1).
int head_chunks(int64_t blocks, int heads) {
  const int64_t want = 2LL * device_sm_count();
  if (blocks >= want || heads < 2) return 1;
  const int64_t c = (want + blocks - 1) / blocks;
  return static_cast<int>(c < heads ? c : heads);
}

// CTAs of the backward: as many as are resident, each leaving one partial sum of dw.  head_chunks
// keeps within it too: x blocks < 2 SMs become x ceil(2 SMs / x) < x + 2 SMs < 4 SMs.
int max_ctas() { return BWD_CTAS * device_sm_count(); }
static_assert(BWD_CTAS >= 4, "head_chunks");

struct BwdGrid {
  int x, y, chunk;
};
BwdGrid bwd_grid(int batch, int tokens, int head_dim, int heads) {
  const int64_t per = THREADS / lanes_per_head(head_dim);
  const int64_t blocks = (static_cast<int64_t>(batch) * tokens + per - 1) / per;
  const int64_t most = max_ctas();
  BwdGrid g;
  g.x = static_cast<int>(blocks < most ? blocks : most);
  const int c = head_chunks(blocks, heads);
  g.chunk = (heads + c - 1) / c;
  g.y = (heads + g.chunk - 1) / g.chunk;
  return g;
}

template <typename T, typename W, int LPR, bool HALVES>
cudaError_t launch(const NormRopeArgs& a, bool forward, cudaStream_t stream) {
  Params p;
  p.a = a;
  p.inv_dim = 1.f / static_cast<float>(a.head_dim);
  const int heads = a.in[0].heads + a.in[1].heads + a.in[2].heads;
  if (forward) {
    const int64_t per = THREADS / LPR;
    const int64_t blocks = (static_cast<int64_t>(a.batch) * a.rows + per - 1) / per;
    const int c = head_chunks(blocks, heads);
    p.chunk = (heads + c - 1) / c;
    const dim3 grid(static_cast<unsigned>(blocks), (heads + p.chunk - 1) / p.chunk);
    return launch_dependent(norm_rope_fwd_kernel<T, W, LPR, HALVES>, grid, dim3(THREADS), 0, stream, p);
  }
  const BwdGrid g = bwd_grid(a.batch, a.tokens, a.head_dim, heads);
  p.chunk = g.chunk;
  cudaError_t e = launch_dependent(norm_rope_bwd_kernel<T, W, LPR, HALVES>, dim3(g.x, g.y),
                                   dim3(THREADS), 0, stream, p);
  if (e != cudaSuccess || (!a.dweight[0] && !a.dweight[1])) return e;
  return launch_dependent(norm_rope_dweight_kernel<W>, dim3((a.head_dim + 31) / 32, 2), dim3(32, 32),
                          0, stream, a.partial, g.x * g.y, a.head_dim, static_cast<W*>(a.dweight[0]),
                          static_cast<W*>(a.dweight[1]));
}

template <typename T, typename W>
cudaError_t launch_shape(const NormRopeArgs& a, bool forward, cudaStream_t stream) {
  switch (lanes_per_head(a.head_dim)) {
    case 8:
      return a.halves ? launch<T, W, 8, true>(a, forward, stream) : launch<T, W, 8, false>(a, forward, stream);
    case 16:
      return a.halves ? launch<T, W, 16, true>(a, forward, stream) : launch<T, W, 16, false>(a, forward, stream);
    default:
      return a.halves ? launch<T, W, 32, true>(a, forward, stream) : launch<T, W, 32, false>(a, forward, stream);
  }
}

cudaError_t launch_typed(const NormRopeArgs& a, bool forward, cudaStream_t stream) {
  const bool wide = a.weight_dtype == VSA_F32;
  if (a.dtype == VSA_F32) return launch_shape<float, float>(a, forward, stream);
  if (a.dtype == VSA_F16)
    return wide ? launch_shape<__half, float>(a, forward, stream) : launch_shape<__half, __half>(a, forward, stream);
  return wide ? launch_shape<__nv_bfloat16, float>(a, forward, stream)
              : launch_shape<__nv_bfloat16, __nv_bfloat16>(a, forward, stream);
}

}  // namespace

size_t norm_rope_bwd_workspace(int head_dim) {
  return static_cast<size_t>(max_ctas()) * 2 * head_dim * sizeof(float);
}

cudaError_t launch_norm_rope_fwd(const NormRopeArgs& a, cudaStream_t stream) { return launch_typed(a, true, stream); }
cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, cudaStream_t stream) { return launch_typed(a, false, stream); }

}  // namespace vsa
