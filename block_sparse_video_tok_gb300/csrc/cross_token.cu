// cross_token.cu -- cross attention forward for one or two query rows per key head (single tokens in
// serving).
//
// Bound by the read of K and V, 512 bytes a key: each key is loaded once for all its rows, and the
// arithmetic (about 20 instructions a row and two keys) stays on the CUDA cores, where fp32
// products need no tile of 128 rows.  Half a warp holds a key's 128 columns, 8 a lane (16 bytes
// of K and V each), with its own online softmax and O; KEYS keys per half-warp are in flight.  The
// halves' results are joined in shared memory in a fixed order.  Where the (batch, key head) pairs
// are fewer than the SMs, the keys are split over CTAs and a second kernel joins the parts: 2 key
// heads of 32768 keys take 12 us, in one part each 338.  Short calls are bound by latency (8 x 12
// heads of 512 keys: 7.6 us), long ones by instructions and HBM (64 x
// 8 heads of 2048 keys: 102 us, 5.3 TB/s).
#include "cross_common.cuh"

namespace vsa {

namespace {

constexpr int THREADS = 256, HALVES = THREADS / 16, KEYS = 4;

struct Params {
  CrossArgs a;
  int share, rows;  // query heads of a key head; rows = share * q_tokens
  int splits;
  float* part_o;    // [batch * kv_heads][split][rows][128]
  float2* part_ml;  // [batch * kv_heads][split][rows]
};

__device__ __forceinline__ void widen8(uint4 u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <int ROWS>
__global__ void __launch_bounds__(THREADS, 2) cross_token_kernel(const __grid_constant__ Params p) {
  __shared__ float sh_o[HALVES][ROWS][HEAD_DIM];
  __shared__ float2 sh_ml[HALVES][ROWS];
  grid_dependency_wait();
  const int bk = blockIdx.x, b = bk / p.a.kv_heads, kh = bk - b * p.a.kv_heads, split = blockIdx.y;
  const int half = threadIdx.x >> 4, e = (threadIdx.x & 15) * 8;
  const int n = visible_keys(p.a.kv_len, b, p.a.kv_tokens, p.a.err);
  const int per = (n + p.splits - 1) / p.splits, k0 = min(split * per, n), k1 = min(k0 + per, n);
  const float c1 = p.a.sm_scale * LOG2E_F;

  float q[ROWS][8], o[ROWS][8], m[ROWS], l[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int h = kh * p.share + r / p.a.q_tokens, t = r % p.a.q_tokens;
    m[r] = -INFINITY;
    l[r] = 0.f;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (r < p.rows)
      u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.q.data) + b * p.a.q.batch +
                                          h * p.a.q.head + t * p.a.q.token + e);
    widen8(u, q[r]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[r][i] *= c1;
      o[r][i] = 0.f;
    }
  }
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.a.k.data) + b * p.a.k.batch + kh * p.a.k.head + e;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.a.v.data) + b * p.a.v.batch + kh * p.a.v.head + e;
  // The trip count is the same for both halves of a warp, which meet in the shuffles.
  for (int base = k0 + (half & ~1); base < k1; base += HALVES * KEYS) {
    uint4 kr[KEYS], vr[KEYS];
    bool there[KEYS];
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
      const int key = base + (half & 1) + u * HALVES;
      there[u] = key < k1;
      kr[u] = vr[u] = make_uint4(0u, 0u, 0u, 0u);
      if (there[u]) {
        kr[u] = *reinterpret_cast<const uint4*>(k + key * p.a.k.token);
        vr[u] = *reinterpret_cast<const uint4*>(v + key * p.a.v.token);
      }
    }
    float s[KEYS][ROWS];
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
      float x[8];
      widen8(kr[u], x);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) d = fmaf(q[r][i], x[i], d);
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
        s[u][r] = there[u] ? d : -INFINITY;
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float mn = m[r];
#pragma unroll
      for (int u = 0; u < KEYS; ++u) mn = fmaxf(mn, s[u][r]);
      const float ref = mn == -INFINITY ? 0.f : mn, f = ex2(m[r] - ref);
      m[r] = mn;
      l[r] *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[r][i] *= f;
#pragma unroll
      for (int u = 0; u < KEYS; ++u) {
        s[u][r] = ex2(s[u][r] - ref);
        l[r] += s[u][r];
      }
    }
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
      float x[8];
      widen8(vr[u], x);
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[r][i] = fmaf(s[u][r], x[i], o[r][i]);
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sh_o[half][r][e + i] = o[r][i];
    if (e == 0) sh_ml[half][r] = make_float2(m[r], l[r]);
  }
  __syncthreads();
  for (int x = threadIdx.x; x < p.rows * HEAD_DIM; x += THREADS) {
    const int r = x / HEAD_DIM, d = x - r * HEAD_DIM;
    float mm = -INFINITY, ll = 0.f, oo = 0.f;
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      const float2 ml = sh_ml[h][r];
      if (ml.y == 0.f) continue;  // no key (NaN is kept)
      float f, w;
      join(mm, ll, ml.x, ml.y, &f, &w);
      oo = oo * f + sh_o[h][r][d] * w;
    }
    if (p.splits > 1) {
      const int64_t at = (static_cast<int64_t>(bk) * p.splits + split) * p.rows + r;
      p.part_o[at * HEAD_DIM + d] = oo;
      if (d == 0) p.part_ml[at] = make_float2(mm, ll);
    } else {
      const int h = kh * p.share + r / p.a.q_tokens, t = r % p.a.q_tokens;
      static_cast<__nv_bfloat16*>(p.a.o.data)[b * p.a.o.batch + h * p.a.o.head + t * p.a.o.token + d] =
          __float2bfloat16_rn(ll == 0.f ? 0.f : oo / ll);
      if (d == 0) p.a.lse[(static_cast<int64_t>(b) * p.a.heads + h) * p.a.q_tokens + t] = mm + log2f(ll);
    }
  }
}

// Joins the parts of one row: four groups of 128 threads take every fourth part, one column each,
// and are joined in group order.
__global__ void __launch_bounds__(512) cross_token_join_kernel(const __grid_constant__ Params p) {
  __shared__ float sh_o[4][HEAD_DIM];
  __shared__ float2 sh_ml[4];
  grid_dependency_wait();
  const int bk = blockIdx.x, r = blockIdx.y, g = threadIdx.x / HEAD_DIM, d = threadIdx.x % HEAD_DIM;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int s0 = g; s0 < p.splits; s0 += 16) {  // four parts' loads at a time
    float2 ml[4];
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = s0 + 4 * i;
      const int64_t at = (static_cast<int64_t>(bk) * p.splits + s) * p.rows + r;
      ml[i] = s < p.splits ? p.part_ml[at] : make_float2(-INFINITY, 0.f);
      x[i] = s < p.splits ? p.part_o[at * HEAD_DIM + d] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ml[i].y == 0.f) continue;
      float f, w;
      join(m, l, ml[i].x, ml[i].y, &f, &w);
      o = o * f + x[i] * w;
    }
  }
  sh_o[g][d] = o;
  if (d == 0) sh_ml[g] = make_float2(m, l);
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (sh_ml[i].y == 0.f) continue;
    float f, w;
    join(m, l, sh_ml[i].x, sh_ml[i].y, &f, &w);
    o = o * f + sh_o[i][d] * w;
  }
  const int b = bk / p.a.kv_heads, kh = bk - b * p.a.kv_heads;
  const int h = kh * p.share + r / p.a.q_tokens, t = r % p.a.q_tokens;
  static_cast<__nv_bfloat16*>(p.a.o.data)[b * p.a.o.batch + h * p.a.o.head + t * p.a.o.token + d] =
      __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
  if (d == 0) p.a.lse[(static_cast<int64_t>(b) * p.a.heads + h) * p.a.q_tokens + t] = m + log2f(l);
}

// Query rows of a key head that this kernel takes; more go to the kernel of 128-row tiles, whose
// time does not depend on them.  (8 x 12 key heads of 512 keys: 1, 2, 4 rows 7.7, 9.1, 14.0 us here,
// 10.5 there; 64 x 8 key heads of 2048 keys: 103, 102, 142 us here, 98 there; 2 of 32768 keys: 12.6
// us here for one row, 24 there.)
constexpr int MAX_ROWS = 2;

// Parts of the keys: one while a CTA has few keys or the pairs fill the SMs; else two CTAs per SM
// with at least 256 keys each.  (96 pairs of 512 keys: 7.5 us in one part, 7.8 in two.)
int token_splits(int64_t pairs, int kv_tokens) {
  int64_t s = 2LL * device_sm_count() / pairs;
  if (s > kv_tokens / 256) s = kv_tokens / 256;
  if (kv_tokens < 1024) s = 1;
  return s < 2 ? 1 : static_cast<int>(s);
}

}  // namespace

bool use_cross_token(int heads, int kv_heads, int q_tokens) {
  return static_cast<int64_t>(heads / kv_heads) * q_tokens <= MAX_ROWS;
}

size_t cross_token_workspace(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens) {
  const int64_t pairs = static_cast<int64_t>(batch) * kv_heads;
  const int s = token_splits(pairs, kv_tokens);
  if (s == 1) return 0;
  const size_t rows = static_cast<size_t>(pairs) * s * (heads / kv_heads) * q_tokens;
  return align_up(rows * (HEAD_DIM * sizeof(float) + sizeof(float2)), 256);
}

cudaError_t launch_cross_token(const CrossArgs& a, cudaStream_t stream) {
  const int pairs = a.batch * a.kv_heads;
  Params p{};
  p.a = a;
  p.share = a.heads / a.kv_heads;
  p.rows = p.share * a.q_tokens;
  p.splits = token_splits(pairs, a.kv_tokens);
  p.part_o = reinterpret_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(pairs) * p.splits * p.rows * HEAD_DIM);
  const dim3 grid(pairs, p.splits);
  cudaError_t e;
  if (p.rows == 1)
    e = launch_dependent(cross_token_kernel<1>, grid, dim3(THREADS), 0, stream, p);
  else
    e = launch_dependent(cross_token_kernel<MAX_ROWS>, grid, dim3(THREADS), 0, stream, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_dependent(cross_token_join_kernel, dim3(pairs, p.rows), dim3(512), 0, stream, p);
}

}  // namespace vsa
