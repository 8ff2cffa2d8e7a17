// gate_norm.cu -- the end of one branch and the start of the next in one pass, and its backward.
//
// Forward, per token:  u = y (or its RMS norm times post_weight),  x' = x + gate u,
//   n = (x' - mean) / sqrt(var + eps)  (RMS: x' / sqrt(mean(x'^2) + eps)),
//   h = n a + c  with  a = weight (1 + scale),  c = bias (1 + scale) + shift.
// Backward, per token, with g = dh a:
//   dx = dx_out + r (g - mean(g) - n mean(g n))  (RMS: without mean(g)),
//   du = gate dx,  dy = du  (post norm: r_y (q - n_y mean(q n_y)),  q = du post_weight).
// Every parameter's gradient follows from three sums over the tokens of a modulation row,
//   S1 = sum dh,  S2 = sum dh n,  S3 = sum dx n_y   (n_y = y without a post norm):
//   dshift = S1, dscale = weight S2 + bias S1, dgate = post_weight S3, and over all rows
//   dbias = sum (1 + scale) S1, dweight = sum (1 + scale) S2, dpost_weight = sum gate S3.
//
// Both passes are bound by HBM: each activation is read and written once.  A token is held by `wpr`
// warps, 8 NV elements to a lane, so that a lane's share of the parameters (a, c, gate) and of the
// three sums stays in registers while it walks the tokens of a unit: a part of one modulation
// row's tokens.  The means are shuffles and one exchange of the warps' sums in shared memory per
// round; the variance takes a round of its own, around the mean, so that tokens far from zero keep
// their precision.  The next tokens' loads are issued before the rounds.
//
// Measured, one GB300: forward of 131040 x 1536 bf16 with gate, scale and shift 246 us, 96 % of the copy
// rate.  Backward of 2 x 32760 x 1536 202 us, 88 %: its warps' instructions take 58 % of the issue slots, and
// a token's round of sums is a chain of shuffles and a barrier that 4 x 3 warps an SM do not quite
// hide.  What made it fast, from 514 us: one round of sums a token instead of two, 9 instructions of
// exchange instead of some 40, inputs through shared memory instead of registers, and packed pairs of fp32
// (247, then 227); two vectors to a lane, so that half as many warps take part in a round (213); the
// copies asked for before the round instead of after it (202).  Tried without gain: two tokens a round (289
// where one took 227), five or six tokens ahead (267, 279 where four took 251), 80 registers and a fourth
// CTA (332).
#include <type_traits>

#include "block_internal.cuh"
#include "cross_common.cuh"
#include "vec8.cuh"

namespace vsa {

namespace {

constexpr int MAX_WPR = 16;   // warps of a token
constexpr int CTA_WARPS = 8;  // warps of a CTA that holds several tokens
constexpr int FWD_ROWS = 2;   // tokens in flight per group of warps

// Registers of a thread with NV vectors: the CTAs of an SM follow from them.  Backward, two vectors: 168 where a
// CTA's threads leave room for them; more than 6144 channels do not, and there 128 spill (8192 channels run at
// a third of the copy rate).
constexpr int fwd_regs(int nv) { return nv == 1 ? 80 : 112; }
constexpr int BWD_REGS_1 = 96, BWD_REGS_2 = 168, BWD_REGS_4 = 255;

// 8 parameters of either type, or `fallback`.  In two steps, so that both modulations' loads of the backward are
// under way before the first is used (a modulation of every token, above: 139 us, one after the other 160).  The
// forward has no registers for that (16384 tokens of 1024 channels: 27 us instead of 24.5).
struct Param8 {
  Raw<float> r;

  __device__ __forceinline__ void load(const void* p, int64_t at, int dtype) {
    r.zero();
    if (!p) return;
    if (dtype == VSA_F32) r.load(static_cast<const float*>(p) + at);
    else r.u[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  }
  __device__ __forceinline__ void widen(const void* p, int dtype, float fallback, float* v) const {
    if (!p) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fallback;
    } else if (dtype == VSA_F32) {
      r.widen(v);
    } else if (dtype == VSA_BF16) {
      Raw<__nv_bfloat16>{r.u[0]}.widen(v);
    } else {
      Raw<__half>{r.u[0]}.widen(v);
    }
  }
};
__device__ __forceinline__ void load_param(const void* p, int64_t at, int dtype, float fallback, float* v) {
  Param8 x;
  x.load(p, at, dtype);
  x.widen(p, dtype, fallback, v);
}

__device__ __forceinline__ float param(const void* p, int64_t at, int dtype, float fallback) {
  if (!p) return fallback;
  if (dtype == VSA_F32) return static_cast<const float*>(p)[at];
  if (dtype == VSA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
  return __half2float(static_cast<const __half*>(p)[at]);
}

__device__ __forceinline__ void store_param(void* p, int64_t at, int dtype, float v) {
  if (!p) return;
  if (dtype == VSA_F32) static_cast<float*>(p)[at] = v;
  else if (dtype == VSA_BF16) static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[at] = __float2half_rn(v);
}

__device__ __forceinline__ void store_params(void* p, int64_t at, int dtype, const float* v) {
  if (!p) return;
  if (dtype == VSA_F32) store8(static_cast<float*>(p) + at, v);
  else if (dtype == VSA_BF16) store8(static_cast<__nv_bfloat16*>(p) + at, v);
  else store8(static_cast<__half*>(p) + at, v);
}

struct Params {
  GateNormArgs a;
  int wpr, per_cta;  // warps of a token, teams of a CTA
  int len;           // tokens of a modulation row
  int parts, chunk;  // units of a modulation row, tokens of a unit
  int share;         // NARROW, backward: a unit is a CTA's; tokens of each of its teams
  int units;
  float dim, inv_dim;  // channels
};

// sum / channels: the product with the rounded 1 / channels, corrected once, so that a constant token is its
// own mean, here and in the backward (a token of 15000s of 1000 channels is 0.001 off without it, 0.7 of the
// deviation that eps leaves).
__device__ __forceinline__ float mean_of(const Params& p, float sum) {
  const float m = sum * p.inv_dim;
  return fmaf(fmaf(-m, p.dim, sum), p.inv_dim, m);
}

// Lanes that hold a token of few channels: a part of a warp.
constexpr int NARROW_CHANNELS = 128;
__host__ __device__ constexpr int narrow_lanes(int channels) { return channels <= 64 ? 8 : 16; }

// The warps (NARROW: lanes) that hold a token together: sums over all of its elements, the same for every
// lane.
template <bool NARROW>
struct Team {
  float (*buf)[4][MAX_WPR];  // [2]: warps' sums of this round and of the one before
  int wpr, warp, lane, bar, width;
  uint32_t round;

  __device__ __forceinline__ Team(float (*b)[4][MAX_WPR], const Params& p) {
    buf = b;
    wpr = p.wpr;
    const int w = threadIdx.x >> 5;
    warp = w % wpr;
    lane = threadIdx.x & 31;
    bar = 1 + w / wpr;
    width = NARROW ? narrow_lanes(p.a.channels) : 32;
    round = 0;
  }

  // v[i] = its sum, for N = 1, 2 or 4 values at once: the lanes halve the values among them while
  // they add (4 values: 6 exchanges, where one by one take 20), and the same lanes then add the warps'.
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
    static_assert(N == 1 || N == 2 || N == 4, "values are halved");
    if (NARROW) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 4; o > 0; o /= 2) v[i] += __shfl_xor_sync(FULL, v[i], o);
        const float other = __shfl_xor_sync(FULL, v[i], 8);
        if (width == 16) v[i] += other;
      }
      return;
    }
    constexpr int LANES = 32 / N;  // that add one value
    float k[N];
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = v[i];
#pragma unroll
    for (int n = N / 2, o = 16; n > 0; n /= 2, o /= 2) {
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = upper ? k[i] : k[i + n], keep = upper ? k[i + n] : k[i];
        k[i] = keep + __shfl_xor_sync(FULL, give, o);
      }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o /= 2) k[0] += __shfl_xor_sync(FULL, k[0], o);
    if (wpr > 1) {
      // Two buffers: a warp that writes round k + 2 has passed the barrier of round k + 1, which every
      // warp reaches after its reads of round k.
      float (*b)[MAX_WPR] = buf[round & 1u];
      ++round;
      const int value = lane / LANES, w = lane % LANES;
      if (w == 0) b[value][warp] = k[0];
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(wpr * 32) : "memory");
      k[0] = w < wpr ? b[value][w & (MAX_WPR - 1)] : 0.f;
      if (LANES < MAX_WPR && w + LANES < wpr) k[0] += b[value][(w + LANES) & (MAX_WPR - 1)];
#pragma unroll
      for (int o = (LANES < MAX_WPR ? LANES : MAX_WPR) / 2; o > 0; o /= 2) k[0] += __shfl_xor_sync(FULL, k[0], o);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(FULL, k[0], i * LANES);
  }
};

// A unit: tokens [t0, t1) of batch entry b, of the modulation row bg = b * groups + g.
struct Unit {
  int b, bg, g, t0, t1;
};
__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  Unit x;
  x.bg = u / p.parts;
  x.b = x.bg / p.a.groups;
  x.g = x.bg - x.b * p.a.groups;
  const int first = (u - x.bg * p.parts) * p.chunk;
  x.t0 = x.g * p.len + min(first, p.len);
  x.t1 = x.g * p.len + min(first + p.chunk, p.len);
  return x;
}

__device__ __forceinline__ uint64_t pair(const float* v, int i) { return f2_pack(v[2 * i], v[2 * i + 1]); }
__device__ __forceinline__ float halves(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}

template <typename T>
__device__ __forceinline__ T* at(const TokensView& v, int b, int t) {
  return static_cast<T*>(v.data) + b * v.batch + t * v.token;
}

// NARROW: a warp has the tokens of several units, and every lane of it takes part in each round of sums.
template <typename TX, typename TY, int NV, bool NARROW>
__global__ void __maxnreg__(fwd_regs(NV)) gate_norm_fwd_kernel(const __grid_constant__ Params p) {
  constexpr int R = NV == 1 ? FWD_ROWS : 1;
  // A unit's first tokens before its parameters (a modulation of each of 16384 tokens of 1536 channels: 110 us,
  // after them 120); an fp32 stream has no registers for that (777 tokens of 1024: 5.1 us, after them 4.7).
  constexpr bool EARLY = sizeof(TX) == 2;
  __shared__ float sums[CTA_WARPS][2][4][MAX_WPR];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int group = (threadIdx.x >> 5) / p.wpr;
  Team<NARROW> team(sums[group], p);
  const int e0 = (team.warp * 32 + (team.lane & (team.width - 1))) * 8, step = p.wpr * 256;  // vectors e0, e0 + step, ..
  const bool branch = a.y.data != nullptr, post = a.post_weight != nullptr, layer = a.kind == VSA_LAYER_NORM;

  for (int u0 = blockIdx.x * p.per_cta + (NARROW ? group * (32 / team.width) : group); u0 < p.units;
       u0 += gridDim.x * p.per_cta) {
    const int u = NARROW ? u0 + team.lane / team.width : u0;
    Unit unit = unit_of(p, NARROW ? min(u, p.units - 1) : u);
    if (NARROW && u >= p.units) unit.t1 = unit.t0;
    Raw<TX> rx[R][NV];
    Raw<TY> ry[R][NV];
    auto load = [&](int t) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int e = e0 + k * step;
          rx[r][k].zero();
          ry[r][k].zero();
          if (t + r < unit.t1 && e < a.channels) {
            rx[r][k].load(at<const TX>(a.x, unit.b, t + r) + e);
            if (branch) ry[r][k].load(at<const TY>(a.y, unit.b, t + r) + e);
          }
        }
    };
    if (EARLY) load(unit.t0);
    float ca[NV][8], cc[NV][8], cg[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = e0 + k * step;
      if (e >= a.channels) continue;
      float w[8], s[8], t[8];
      load_param(a.weight, e, a.weight_dtype, 1.f, ca[k]);
      load_param(a.bias, e, a.weight_dtype, 0.f, cc[k]);
      load_param(a.scale.data, unit.b * a.scale.batch + unit.g * a.scale.group + e, a.mod_dtype, 0.f, s);
      load_param(a.shift.data, unit.b * a.shift.batch + unit.g * a.shift.group + e, a.mod_dtype, 0.f, t);
      load_param(a.gate.data, unit.b * a.gate.batch + unit.g * a.gate.group + e, a.mod_dtype, 1.f, cg[k]);
      load_param(a.post_weight, e, a.weight_dtype, 1.f, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ca[k][i] *= 1.f + s[i];
        cc[k][i] = fmaf(cc[k][i], 1.f + s[i], t[i]);
        cg[k][i] *= w[i];
      }
    }
    if (!EARLY) load(unit.t0);
    for (int t = unit.t0, i = 0; NARROW ? i < p.chunk : t < unit.t1; t += R, i += R) {
      float v[R][NV][8], s[R];
      float inv[R];
#pragma unroll
      for (int r = 0; r < R; ++r) inv[r] = 1.f;
      if (post) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s[r] = 0.f;
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            ry[r][k].widen(v[r][k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[r] = fmaf(v[r][k][i], v[r][k][i], s[r]);
          }
        }
        team.sum(s);
#pragma unroll
        for (int r = 0; r < R; ++r) inv[r] = rsqrtf(fmaf(s[r], p.inv_dim, a.post_eps));
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int e = e0 + k * step;
          rx[r][k].widen(v[r][k]);
          if (e >= a.channels) continue;
          if (branch) {
            float y[8];
            ry[r][k].widen(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][k][i] = fmaf(y[i] * inv[r], cg[k][i], v[r][k][i]);
            if (t + r < unit.t1) store8(at<TX>(a.x_out, unit.b, t + r) + e, v[r][k]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) s[r] += v[r][k][i];
        }
      }
      load(t + R);
      if (layer) {
        team.sum(s);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float mean = mean_of(p, s[r]);
#pragma unroll
          for (int k = 0; k < NV; ++k)
            if (e0 + k * step < a.channels) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[r][k][i] -= mean;
            }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[r] = fmaf(v[r][k][i], v[r][k][i], s[r]);
      }
      team.sum(s);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = rsqrtf(fmaf(s[r], p.inv_dim, a.eps));
        if (t + r >= unit.t1) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int e = e0 + k * step;
          if (e >= a.channels) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[r][k][i] = fmaf(v[r][k][i] * f, ca[k][i], cc[k][i]);
          store8(at<TY>(a.h, unit.b, t + r) + e, v[r][k]);
        }
      }
    }
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's own 8 NV elements of `slots` tokens of one tensor in shared memory, written by asynchronous
// copies and read by the lane that asked for them.
template <typename T, int NV>
struct Ring {
  static constexpr int PIECES = NV * static_cast<int>(sizeof(T) / 2);  // 16 bytes each, a CTA's side by side
  const T* from;  // null: absent, the ring holds zeros
  int64_t stride;
  int span, left;  // elements from one vector to the next; vectors of this lane
  uint32_t at, step;

  __device__ __forceinline__ static uint32_t bytes(int slots, int threads) { return slots * PIECES * threads * 16u; }
  __device__ __forceinline__ Ring(uint32_t base, int slots, int vector_step, int vectors) {
    at = base + threadIdx.x * 16u;
    step = blockDim.x * 16u;
    span = vector_step;
    left = vectors;
    for (int i = 0; i < slots * PIECES; ++i)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + i * step), "r"(0) : "memory");
  }
  __device__ __forceinline__ void open(const TokensView& v, int b, int e0) {
    from = v.data ? static_cast<const T*>(v.data) + b * v.batch + e0 : nullptr;
    stride = v.token;
  }
  __device__ __forceinline__ void load(int slot, int t) const {
    if (!from) return;
    const T* p = from + t * stride;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (k < left) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
          copy16(at + ((slot * NV + k) * (sizeof(T) / 2) + i) * step, p + k * span + i * (16 / sizeof(T)));
      }
  }
  __device__ __forceinline__ void get(int slot, int k, float* v) const {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.u[i].x), "=r"(r.u[i].y), "=r"(r.u[i].z), "=r"(r.u[i].w)
                   : "r"(at + ((slot * NV + k) * static_cast<uint32_t>(sizeof(T) / 2) + i) * step)
                   : "memory");
    r.widen(v);
  }
};

// The same without a ring: read where it is used.
template <typename T, int NV>
struct NoRing {
  const T* from;
  int64_t stride;
  int span, left;

  __device__ __forceinline__ static uint32_t bytes(int, int) { return 0u; }
  __device__ __forceinline__ NoRing(uint32_t, int, int vector_step, int vectors) {
    span = vector_step;
    left = vectors;
  }
  __device__ __forceinline__ void open(const TokensView& v, int b, int e0) {
    from = v.data ? static_cast<const T*>(v.data) + b * v.batch + e0 : nullptr;
    stride = v.token;
  }
  __device__ __forceinline__ void load(int, int) const {}
  __device__ __forceinline__ void get(int t, int k, float* v) const {
    Raw<T> r;
    r.zero();
    if (from && k < left) r.load(from + t * stride + k * span);
    r.widen(v);
  }
};

// Tokens of the backward's rings, and their bytes: x', dx_out, dh and y.  Two are the fewest; four fit
// where a token's lane has 16 bytes of each.  fp32 beyond 4096 channels leaves no room for dx_out's.
template <typename TX, int NV>
constexpr int slots_of() { return NV == 1 && sizeof(TX) == 2 ? 4 : 2; }
template <typename TX, typename TY, int NV>
constexpr bool o_direct() { return NV > 1 && sizeof(TX) == 4 && sizeof(TY) == 4; }
template <typename TX, typename TY, int NV>
constexpr int ring_bytes(int threads) {
  return slots_of<TX, NV>() * ((o_direct<TX, TY, NV>() ? 1 : 2) * Ring<TX, NV>::PIECES + 2 * Ring<TY, NV>::PIECES) * 16 * threads;
}
constexpr int SPARE_BYTES = 32;  // of a lane, NARROW: one of the three sums at a time
constexpr int SM_SMEM = 228 * 1024, CTA_SMEM = 227 * 1024, STATIC_SMEM = CTA_WARPS * 2 * 4 * MAX_WPR * 4 + 1024;

// One round of sums a token: those of the token itself around its mean, and the mean of the next one.
// A post norm takes a second round.  The inputs come SLOTS - 1 tokens ahead through shared memory: in
// registers beside the three sums there is room for one.  SUMS: the unit's S1, S2, S3 go to the workspace,
// or, where it is the whole of a modulation row, to the row's gradients (a modulation of each of 16384
// tokens of 1536 channels: 139 us, through the workspace 361; both ways in one kernel cost the others 4 %).
// NARROW: a unit is a CTA's and shared out to its many teams, whose sums are added before they leave (65520 x 64:
// 19 us, a unit to a team 46; with more channels 1 to 2 % slower).
enum Sums { NO_SUMS, WORKSPACE, FINISH };
template <typename TX, typename TY, int NV, int REGS, bool NARROW, Sums SUMS>
__global__ void __maxnreg__(REGS) gate_norm_bwd_kernel(const __grid_constant__ Params p) {
  constexpr int SLOTS = slots_of<TX, NV>();
  constexpr bool DIRECT = o_direct<TX, TY, NV>();
  extern __shared__ uint4 room[];
  __shared__ float sums[CTA_WARPS][2][4][MAX_WPR];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int group = (threadIdx.x >> 5) / p.wpr;
  Team<NARROW> team(sums[group], p);
  const int e0 = (team.warp * 32 + (team.lane & (team.width - 1))) * 8, step = p.wpr * 256;
  const bool branch = a.y.data != nullptr, post = a.post_weight != nullptr, layer = a.kind == VSA_LAYER_NORM;
  const int vectors = a.channels > e0 ? (a.channels - e0 + step - 1) / step : 0;
  uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(room));
  Ring<TX, NV> x(base, SLOTS, step, vectors);
  base += Ring<TX, NV>::bytes(SLOTS, blockDim.x);
  using Other = typename std::conditional<DIRECT, NoRing<TX, NV>, Ring<TX, NV>>::type;
  Other o(base, SLOTS, step, vectors);
  base += Other::bytes(SLOTS, blockDim.x);
  Ring<TY, NV> h(base, SLOTS, step, vectors);
  base += Ring<TY, NV>::bytes(SLOTS, blockDim.x);
  Ring<TY, NV> y(base, SLOTS, step, vectors);

  const int mine = group * (32 / team.width) + team.lane / team.width;  // NARROW: team of the CTA
  for (int u = NARROW ? blockIdx.x : blockIdx.x * p.per_cta + group; u < p.units; u += gridDim.x * (NARROW ? 1 : p.per_cta)) {
    Unit unit = unit_of(p, u);
    if (NARROW) {
      unit.t0 = min(unit.t0 + mine * p.share, unit.t1);
      unit.t1 = min(unit.t0 + p.share, unit.t1);
    }
    x.open(a.x_out, unit.b, e0);
    o.open(a.dx_out, unit.b, e0);
    h.open(a.dh, unit.b, e0);
    y.open(a.y, unit.b, e0);
    // Copies go in groups: group i has token i's dh, dx_out and y, and x' of token i + 1.
    if (unit.t0 < unit.t1) x.load(0, unit.t0);
    auto ahead = [&](int t) {  // t0 + i: slot i % SLOTS
      const int slot = (t - unit.t0) & (SLOTS - 1);
      if (t < unit.t1) {
        h.load(slot, t);
        o.load(slot, t);
        y.load(slot, t);
      }
      if (t + 1 < unit.t1) x.load((slot + 1) & (SLOTS - 1), t + 1);
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < SLOTS - 1; ++i) ahead(unit.t0 + i);
    uint64_t ca[NV][4], cg[NV][4], acc[SUMS ? NV : 1][3][4];  // pairs; cg: gate, times post_weight
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = e0 + k * step;
#pragma unroll
      for (int j = 0; SUMS && j < 3; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[SUMS ? k : 0][j][i] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) ca[k][i] = cg[k][i] = 0;
      if (k >= vectors) continue;
      Param8 scale, gate;
      scale.load(a.scale.data, unit.b * a.scale.batch + unit.g * a.scale.group + e, a.mod_dtype);
      gate.load(a.gate.data, unit.b * a.gate.batch + unit.g * a.gate.group + e, a.mod_dtype);
      float w[8], s[8];
      load_param(a.weight, e, a.weight_dtype, 1.f, w);
      scale.widen(a.scale.data, a.mod_dtype, 0.f, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) ca[k][i] = f2_pack(w[2 * i] * (1.f + s[2 * i]), w[2 * i + 1] * (1.f + s[2 * i + 1]));
      gate.widen(a.gate.data, a.mod_dtype, 1.f, w);
      load_param(a.post_weight, e, a.weight_dtype, 1.f, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) cg[k][i] = f2_pack(w[2 * i] * s[2 * i], w[2 * i + 1] * s[2 * i + 1]);
    }
    TX* pdx = static_cast<TX*>(a.dx.data) + unit.b * a.dx.batch + unit.t0 * a.dx.token + e0;
    TY* pdy = static_cast<TY*>(a.dy.data) + unit.b * a.dy.batch + unit.t0 * a.dy.token + e0;
    auto total = [&](int slot) {
      uint64_t s = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float v[8];
        x.get(slot, k, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) s = f2_add(s, pair(v, i));
      }
      return halves(s);
    };
    float sum = 0.f;  // of x' of the token at hand
    if (layer) {
      copy_wait<SLOTS - 2>();
      float s[1] = {total(0)};
      team.sum(s);
      sum = s[0];
    }
    for (int t = unit.t0, i = 0; NARROW ? i < p.share : t < unit.t1; ++t, ++i) {
      const bool here = !NARROW || t < unit.t1;
      const int slot = (t - unit.t0) & (SLOTS - 1);
      copy_wait<SLOTS - 2>();
      // Taken here and for layer norms alone, the corrected mean costs nothing; where the sum is made, its
      // registers spill (2 x 32760 x 1536: 212 us instead of 202; four vectors to a lane gained by it, 2 x 32760 x
      // 8192 1548 and 1338).
      float mean = 0.f;
      if (layer) mean = mean_of(p, sum);
      uint64_t v[NV][4], s2[3] = {0, 0, 0};
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float w[8], g[8];
        x.get(slot, k, w);
        h.get(slot, k, g);
        const float off = k < vectors ? -mean : 0.f;
        const uint64_t off2 = f2_pack(off, off);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[k][i] = f2_add(pair(w, i), off2);
          const uint64_t ga = f2_mul(pair(g, i), ca[k][i]);
          s2[0] = f2_fma(v[k][i], v[k][i], s2[0]);
          s2[1] = f2_fma(ga, v[k][i], s2[1]);
          s2[2] = f2_add(ga, s2[2]);
        }
      }
      // v^2, g v, g of this token; x' of the next
      float s[4] = {halves(s2[0]), halves(s2[1]), halves(s2[2]), 0.f};
      if (layer) s[3] = total((slot + 1) & (SLOTS - 1));
      ahead(t + SLOTS - 1);  // into the slots of token t - 1, and of x' of token t
      team.sum(s);
      const float f = rsqrtf(fmaf(s[0], p.inv_dim, a.eps));
      const float m1 = layer ? -s[2] * p.inv_dim : 0.f, m2 = -s[1] * f * p.inv_dim;
      const uint64_t f2 = f2_pack(f, f), m12 = f2_pack(m1, m1), m22 = f2_pack(m2, m2);
      sum = s[3];
      uint64_t z2[2] = {0, 0};  // post norm: q y, y^2
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float g[8], d[8], w[8];
        h.get(slot, k, g);
        o.get(DIRECT ? t : slot, k, d);
        y.get(slot, k, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t n = f2_mul(v[k][i], f2), gi = pair(g, i), yi = pair(w, i);
          const uint64_t dx = f2_fma(f2, f2_fma(n, m22, f2_fma(gi, ca[k][i], m12)), pair(d, i));
          if (SUMS && here) {
            acc[SUMS ? k : 0][0][i] = f2_add(acc[SUMS ? k : 0][0][i], gi);
            acc[SUMS ? k : 0][1][i] = f2_fma(gi, n, acc[SUMS ? k : 0][1][i]);
          }
          v[k][i] = dx;
          const uint64_t q = f2_mul(dx, cg[k][i]);
          if (post) {
            z2[0] = f2_fma(q, yi, z2[0]);
            z2[1] = f2_fma(yi, yi, z2[1]);
          } else if (SUMS && here) {
            acc[SUMS ? k : 0][2][i] = f2_fma(dx, yi, acc[SUMS ? k : 0][2][i]);
          }
          f2_unpack(dx, d[2 * i], d[2 * i + 1]);
          f2_unpack(q, g[2 * i], g[2 * i + 1]);
        }
        if (k < vectors && here) {
          store8(pdx + k * step, d);
          if (branch && !post) store8(pdy + k * step, g);
        }
      }
      if (post) {
        float z[2] = {halves(z2[0]), halves(z2[1])};
        team.sum(z);
        const float fy = rsqrtf(fmaf(z[1], p.inv_dim, a.post_eps)), m = -z[0] * fy * p.inv_dim;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float w[8];
          y.get(slot, k, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t ny = f2_mul(pair(w, i), f2_pack(fy, fy));
            if (SUMS && here) acc[SUMS ? k : 0][2][i] = f2_fma(v[k][i], ny, acc[SUMS ? k : 0][2][i]);
            f2_unpack(f2_mul(f2_fma(ny, f2_pack(m, m), f2_mul(v[k][i], cg[k][i])), f2_pack(fy, fy)), w[2 * i], w[2 * i + 1]);
          }
          if (k < vectors && here) store8(pdy + k * step, w);
        }
      }
      pdx += a.dx.token;
      pdy += a.dy.token;
    }
    if (SUMS) {
      if (!NARROW) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if (k >= vectors) continue;
          if (SUMS == FINISH) {  // as finish_row
            const int e = e0 + k * step;
            const int64_t to = static_cast<int64_t>(unit.bg) * a.channels + e;
            float v[8], s[8], c[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(acc[SUMS ? k : 0][0][i], s[2 * i], s[2 * i + 1]);
            store_params(a.dshift, to, a.mod_dtype, s);
            load_param(a.bias, e, a.weight_dtype, 0.f, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] *= c[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(acc[SUMS ? k : 0][1][i], v[2 * i], v[2 * i + 1]);
            load_param(a.weight, e, a.weight_dtype, 1.f, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = fmaf(c[i], v[i], s[i]);
            store_params(a.dscale, to, a.mod_dtype, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(acc[SUMS ? k : 0][2][i], v[2 * i], v[2 * i + 1]);
            load_param(a.post_weight, e, a.weight_dtype, 1.f, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= c[i];
            store_params(a.dgate, to, a.mod_dtype, v);
            continue;
          }
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(acc[SUMS ? k : 0][j][i], w[2 * i], w[2 * i + 1]);
            store8(a.workspace + (static_cast<int64_t>(u) * 3 + j) * a.channels + e0 + k * step, w);
          }
        }
      } else {
        // The teams' sums, added in their order.
        float* to = a.workspace + static_cast<int64_t>(u) * 3 * a.channels;
        float* spare = reinterpret_cast<float*>(room) + ring_bytes<TX, TY, NV>(blockDim.x) / 4;
#pragma unroll
        for (int j = 0; j < 3; ++j, to += a.channels) {
          float w[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f2_unpack(acc[0][j][i], w[2 * i], w[2 * i + 1]);
          if (vectors) store8(spare + mine * a.channels + e0, w);
          __syncthreads();
          for (int c = threadIdx.x; c < a.channels; c += blockDim.x) {
            float sum = 0.f;
            for (int m = 0; m < p.per_cta; ++m) sum += spare[m * a.channels + c];
            to[c] = sum;
          }
          __syncthreads();
        }
      }
    }
  }
}

// What a modulation row's sums s give its gradients at column c; and its share of the weights' gradients.
__device__ __forceinline__ void finish_row(const GateNormArgs& a, int bg, int c, float* s) {
  const int b = bg / a.groups, g = bg - b * a.groups;
  const float w = param(a.weight, c, a.weight_dtype, 1.f), bias = param(a.bias, c, a.weight_dtype, 0.f);
  const int64_t to = static_cast<int64_t>(bg) * a.channels + c;
  store_param(a.dshift, to, a.mod_dtype, s[0]);
  store_param(a.dscale, to, a.mod_dtype, fmaf(w, s[1], bias * s[0]));
  store_param(a.dgate, to, a.mod_dtype, param(a.post_weight, c, a.weight_dtype, 1.f) * s[2]);
  const float one = 1.f + param(a.scale.data, b * a.scale.batch + g * a.scale.group + c, a.mod_dtype, 0.f);
  s[0] *= one;
  s[1] *= one;
  s[2] *= param(a.gate.data, b * a.gate.batch + g * a.gate.group + c, a.mod_dtype, 1.f);
}
__device__ __forceinline__ void finish_weights(const GateNormArgs& a, int c, const float* s) {
  store_param(a.dbias, c, a.weight_dtype, s[0]);
  store_param(a.dweight, c, a.weight_dtype, s[1]);
  store_param(a.dpost, c, a.weight_dtype, s[2]);
}

// The units' sums of a modulation row, joined in unit order: 32 columns a block, Y strided units
// each, joined in their order.  Writes the row's gradients and, for the weights' gradients, its
// share of them: the result itself if there is one row, else to `share` [row][3][channels].
template <int Y>
__global__ void __launch_bounds__(32 * Y) gate_norm_sums_kernel(const __grid_constant__ Params p, float* share) {
  __shared__ float sums[3][Y][33];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int c = blockIdx.x * 32 + threadIdx.x, bg = blockIdx.y;
  float s[3] = {0.f, 0.f, 0.f};
  if (c < a.channels) {
#pragma unroll 4
    for (int i = threadIdx.y; i < p.parts; i += Y) {
      const float* from = a.workspace + (static_cast<int64_t>(bg) * p.parts + i) * 3 * a.channels + c;
#pragma unroll
      for (int j = 0; j < 3; ++j) s[j] += from[static_cast<int64_t>(j) * a.channels];
    }
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) sums[j][threadIdx.y][threadIdx.x] = s[j];
  __syncthreads();
  if (threadIdx.y != 0 || c >= a.channels) return;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    s[j] = 0.f;
#pragma unroll
    for (int y = 0; y < Y; ++y) s[j] += sums[j][y][threadIdx.x];
  }
  finish_row(a, bg, c, s);
  if (a.batch * a.groups == 1) {
    finish_weights(a, c, s);
  } else if (share) {
    float* to = share + static_cast<int64_t>(bg) * 3 * a.channels + c;
#pragma unroll
    for (int j = 0; j < 3; ++j) to[static_cast<int64_t>(j) * a.channels] = s[j];
  }
}

// Both in one launch, of few rows: a block has X columns of all rows, the units of a row are strided over its
// equal part of the block's 1024 / X slots.  X: as many as make up to 256 blocks (8 columns are a sector of
// each unit's sums; 2 x 1000 tokens of 8192 channels 75 us with 8, 60 with 32, 68 in two launches).  Taken
// where the weights' gradients are wanted (a backward of 64 x 128 tokens of 1536 37 us, in two launches 42;
// 2 x 13 frames of 157 tokens of 1000 18.2 and 17.6, called 59 and 62), and without them where a row to a
// block makes more than ten blocks to an SM (64 x 128 of 1536 36 and 39, but 26 rows of 1000 17.4 and 15.4).
template <int X>
__global__ void __launch_bounds__(1024) gate_norm_join_kernel(const __grid_constant__ Params p) {
  constexpr int SLOTS = 1024 / X;
  __shared__ float sums[3][SLOTS][X];
  __shared__ float shares[3][SLOTS][X];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int rows = a.batch * a.groups, each = SLOTS / rows;  // slots of a row
  const int x = threadIdx.x, y = threadIdx.y, c = blockIdx.x * X + x, bg = y / each;
  float s[3] = {0.f, 0.f, 0.f};
  if (bg < rows && c < a.channels) {
#pragma unroll 4
    for (int i = y - bg * each; i < p.parts; i += each) {
      const float* from = a.workspace + (static_cast<int64_t>(bg) * p.parts + i) * 3 * a.channels + c;
#pragma unroll
      for (int j = 0; j < 3; ++j) s[j] += from[static_cast<int64_t>(j) * a.channels];
    }
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) sums[j][y][x] = s[j];
  __syncthreads();
  if (y < rows && c < a.channels) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      s[j] = 0.f;
      for (int i = 0; i < each; ++i) s[j] += sums[j][y * each + i][x];
    }
    finish_row(a, y, c, s);
#pragma unroll
    for (int j = 0; j < 3; ++j) shares[j][y][x] = s[j];
  }
  __syncthreads();
  if (y != 0 || c >= a.channels) return;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    s[j] = 0.f;
    for (int i = 0; i < rows; ++i) s[j] += shares[j][i][x];
  }
  finish_weights(a, c, s);
}

// The same for many rows of few units: a thread has a column of few_rows rows, as many as let all threads run
// at once, and leaves one share for them.  (A row of 32 columns to a block as above, one unit each: 4082 rows
// of 1000 channels took 600 us.  16 rows a thread, whatever their number: 150 rows of 40 tokens of 1536 55 us,
// now 27; 600 of 16 65, now 46.)
constexpr int FEW_UNITS = 8, FEW_ROWS = 16;  // at most
__global__ void __launch_bounds__(256) gate_norm_few_kernel(const __grid_constant__ Params p, float* share, int few_rows) {
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int c = blockIdx.y * 256 + threadIdx.x, rows = a.batch * a.groups;
  if (c >= a.channels) return;
  float total[3] = {0.f, 0.f, 0.f};
  const int first = blockIdx.x * few_rows;
  for (int bg = first; bg < rows && bg < first + few_rows; ++bg) {
    float s[3] = {0.f, 0.f, 0.f};
    for (int i = 0; i < p.parts; ++i) {
      const float* from = a.workspace + (static_cast<int64_t>(bg) * p.parts + i) * 3 * a.channels + c;
#pragma unroll
      for (int j = 0; j < 3; ++j) s[j] += from[static_cast<int64_t>(j) * a.channels];
    }
    finish_row(a, bg, c, s);
#pragma unroll
    for (int j = 0; j < 3; ++j) total[j] += s[j];
  }
  if (!share) return;
  float* to = share + static_cast<int64_t>(blockIdx.x) * 3 * a.channels + c;
#pragma unroll
  for (int j = 0; j < 3; ++j) to[static_cast<int64_t>(j) * a.channels] = total[j];
}

// dbias, dweight, dpost_weight: the sums of the shares, likewise.
__global__ void __launch_bounds__(1024) gate_norm_weights_kernel(const __grid_constant__ Params p, const float* share, int shares) {
  __shared__ float sums[32][33];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y;
  float s = 0.f;
  if (c < a.channels) {
#pragma unroll 4
    for (int i = threadIdx.y; i < shares; i += 32) s += share[(static_cast<int64_t>(i) * 3 + j) * a.channels + c];
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= a.channels) return;
  s = 0.f;
#pragma unroll
  for (int y = 0; y < 32; ++y) s += sums[y][threadIdx.x];
  store_param(j == 0 ? a.dbias : j == 1 ? a.dweight : a.dpost, c, a.weight_dtype, s);
}

// Vectors of a lane.  Forward: as few as 16 warps allow.  Backward: two where they fill four fifths of the lanes
// (2 x 32760 tokens of 512 channels 75 us, one vector 80; 1024: 138 and 148; 768, three quarters: 121 and
// 113); from 2056 to 4096 channels one, as two leave an SM 8 or 10 warps (2304: 321 and 338; 4096: 568 and 611);
// beyond, two and four.
int fwd_vectors(int channels) { return channels <= 256 * MAX_WPR ? 1 : 2; }
int bwd_vectors(int channels) {
  if ((channels + 511) / 512 * 32 * BWD_REGS_2 > 65536) return 4;
  if (channels > 256 * MAX_WPR) return 2;
  const int full = (channels + 511) / 512 * 512;
  return channels > 2048 || channels * 5 < full * 4 ? 1 : 2;
}
int bwd_regs(int channels) {
  const int nv = bwd_vectors(channels);
  return nv == 1 ? BWD_REGS_1 : nv == 2 ? BWD_REGS_2 : BWD_REGS_4;
}

// Units: parts of every modulation row.  The grid takes them in waves of `slots`, each as long as a
// unit's tokens and what a unit costs besides (`extra` tokens); the least of up to four waves.
constexpr int FWD_EXTRA = 2, BWD_EXTRA = 4;
struct Plan {
  int wpr, warps, per_cta;  // warps of a token, of a CTA; teams of a CTA
  int ctas, parts, chunk, share, units;
};
Plan plan_of(int batch, int tokens, int channels, int groups, bool forward, int lane_bytes, bool narrowed) {
  const int extra = forward ? FWD_EXTRA : BWD_EXTRA;
  Plan q{};
  const int nv = forward ? fwd_vectors(channels) : bwd_vectors(channels);
  q.wpr = (channels + 256 * nv - 1) / (256 * nv);
  const int64_t rows = static_cast<int64_t>(batch) * groups;
  const int len = tokens / groups;
  // Teams of a CTA: as many on an SM as its registers and shared memory hold, in at most 4 CTAs (a CTA
  // takes 16 of an SM's 64 barriers); where a unit is a CTA's, no more than a modulation row's tokens.
  const int warp_regs = (forward ? fwd_regs(nv) : bwd_regs(channels)) * 32;
  const int narrow = narrowed ? 32 / narrow_lanes(channels) : 1;  // teams of a warp
  const bool shared = !forward && narrow > 1;                                        // a unit is a CTA's
  int teams = 0, sm_ctas = 0;
  for (int n = 1; n == 1 || (n * q.wpr <= CTA_WARPS && (!shared || n * narrow <= len)); ++n) {
    int ctas = 65536 / (warp_regs * q.wpr * n);
    ctas = ctas < 4 ? ctas : 4;
    const int bytes = lane_bytes + (shared ? SPARE_BYTES : 0);
    const int room = SM_SMEM / (bytes * 32 * q.wpr * n + STATIC_SMEM);
    ctas = ctas < room ? ctas : room;
    if (ctas * n > teams) {
      teams = ctas * n;
      sm_ctas = ctas;
      q.warps = n * q.wpr;
      q.per_cta = n * narrow;
    }
  }
  // Units that run at once.
  const int64_t slots = static_cast<int64_t>(device_sm_count()) * (shared ? sm_ctas : teams * narrow);
  int64_t best = INT64_MAX;
  for (int w = 1; w <= 4; ++w) {
    int64_t parts = w * slots / rows;
    if (parts < 1) parts = 1;
    if (parts > len) parts = len;
    if (channels <= NARROW_CHANNELS && !narrowed) parts = 1;
    const int64_t chunk = (len + parts - 1) / parts;
    parts = (len + chunk - 1) / chunk;
    const int64_t share = shared ? (chunk + q.per_cta - 1) / q.per_cta : chunk;
    const int64_t waves = (rows * parts + slots - 1) / slots, cost = waves * (share + extra);
    if (cost < best) {
      best = cost;
      q.parts = static_cast<int>(parts);
      q.chunk = static_cast<int>(chunk);
      q.share = static_cast<int>(share);
    }
  }
  q.units = static_cast<int>(rows * q.parts);
  const int64_t per = shared ? 1 : q.per_cta, need = (q.units + per - 1) / per, grid = slots / per;
  q.ctas = static_cast<int>(need < grid ? need : grid);
  return q;
}

// How the units' sums are joined: by rows (gate_norm_few_kernel) or a row to a block, and the shares of the
// weights' gradients that leaves.
bool few_units(int64_t rows, int parts) { return rows > 64 && parts <= FEW_UNITS; }
int few_rows(int64_t rows, int channels) {
  const int64_t at_once = 2048LL * device_sm_count(), fill = (rows * channels + at_once - 1) / at_once;
  return static_cast<int>(fill < 1 ? 1 : fill < FEW_ROWS ? fill : FEW_ROWS);
}
int64_t shares_of(int64_t rows, int channels, bool few) {
  const int each = few ? few_rows(rows, channels) : 1;
  return (rows + each - 1) / each;
}
bool wants_sums(const GateNormArgs& a) {
  return a.dgate || a.dscale || a.dshift || a.dpost || a.dweight || a.dbias;
}

bool wants_weights(const GateNormArgs& a) { return a.dpost || a.dweight || a.dbias; }

Params params_of(const GateNormArgs& a, const Plan& q) {
  Params p;
  p.a = a;
  p.wpr = q.wpr;
  p.per_cta = q.per_cta;
  p.len = a.tokens / a.groups;
  p.parts = q.parts;
  p.chunk = q.chunk;
  p.units = q.units;
  p.share = q.share;
  p.dim = static_cast<float>(a.channels);
  p.inv_dim = 1.f / p.dim;
  return p;
}

template <typename TX, typename TY, int NV, bool NARROW>
cudaError_t launch_fwd(const GateNormArgs& a, cudaStream_t stream) {
  const Plan q = plan_of(a.batch, a.tokens, a.channels, a.groups, true, 0, NARROW);
  return launch_dependent(gate_norm_fwd_kernel<TX, TY, NV, NARROW>, dim3(q.ctas), dim3(q.warps * 32), 0, stream,
                          params_of(a, q));
}

template <typename TX, typename TY, int NV, int REGS, bool NARROW, Sums SUMS>
cudaError_t launch_main(const Params& p, const Plan& q, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = ensure_smem_limit(gate_norm_bwd_kernel<TX, TY, NV, REGS, NARROW, SUMS>, CTA_SMEM - STATIC_SMEM, smem_set);
  if (e != cudaSuccess) return e;
  const int threads = q.warps * 32;
  return launch_dependent(gate_norm_bwd_kernel<TX, TY, NV, REGS, NARROW, SUMS>, dim3(q.ctas), dim3(threads),
                          ring_bytes<TX, TY, NV>(threads) + (NARROW ? SPARE_BYTES * threads : 0), stream, p);
}

template <int X>
cudaError_t launch_join(const Params& p, cudaStream_t stream) {
  return launch_dependent(gate_norm_join_kernel<X>, dim3((p.a.channels + X - 1) / X), dim3(X, 1024 / X), 0, stream, p);
}

// Whether the units' sums become their rows' gradients at once, without the workspace.
bool finishes(const Plan& q, bool narrow, bool weights) { return !narrow && q.parts == 1 && !weights; }

// Bytes of the units' sums and of the weights' shares (these also where no weight's gradient is wanted, so that one
// size serves every choice of gradients but the one that needs none).
size_t workspace_of(const GateNormArgs& a, const Plan& q, bool narrow) {
  if (!wants_sums(a) || finishes(q, narrow, wants_weights(a))) return 0;
  const int64_t rows = static_cast<int64_t>(a.batch) * a.groups;
  const int64_t shares = shares_of(rows, a.channels, few_units(rows, q.parts));
  return align_up(static_cast<size_t>(q.units + shares) * 3 * a.channels * sizeof(float), 256);
}

// The backward's launches, or, with `bytes`, the workspace that they need.
template <typename TX, typename TY, int NV, int REGS, bool NARROW>
cudaError_t launch_bwd(const GateNormArgs& a, size_t* bytes, cudaStream_t stream) {
  const Plan q = plan_of(a.batch, a.tokens, a.channels, a.groups, false, ring_bytes<TX, TY, NV>(1), NARROW);
  if (bytes) {
    *bytes = workspace_of(a, q, NARROW);
    return cudaSuccess;
  }
  const Params p = params_of(a, q);
  const bool weights = wants_weights(a);
  if (!wants_sums(a)) return launch_main<TX, TY, NV, REGS, NARROW, NO_SUMS>(p, q, stream);
  if constexpr (!NARROW)
    if (finishes(q, NARROW, weights)) return launch_main<TX, TY, NV, REGS, NARROW, FINISH>(p, q, stream);
  cudaError_t e = launch_main<TX, TY, NV, REGS, NARROW, WORKSPACE>(p, q, stream);
  if (e != cudaSuccess) return e;
  const int rows = a.batch * a.groups, columns = (a.channels + 31) / 32;
  float* share = rows > 1 && weights
                     ? a.workspace + static_cast<int64_t>(q.units) * 3 * a.channels
                     : nullptr;
  if (share || static_cast<int64_t>(rows) * columns > 10 * device_sm_count()) {
    const int x = a.channels <= 8 * 256 ? 8 : a.channels <= 16 * 256 ? 16 : 32;
    if (rows <= 1024 / x)
      return x == 8 ? launch_join<8>(p, stream) : x == 16 ? launch_join<16>(p, stream) : launch_join<32>(p, stream);
  }
  const bool few = few_units(rows, q.parts);
  const int shares = static_cast<int>(shares_of(rows, a.channels, few));
  if (few)  // (more than 65535 rows are of one unit each)
    e = launch_dependent(gate_norm_few_kernel, dim3(shares, (a.channels + 255) / 256), dim3(256), 0, stream, p, share,
                         few_rows(rows, a.channels));
  else if (q.parts > 64)
    e = launch_dependent(gate_norm_sums_kernel<32>, dim3(columns, rows), dim3(32, 32), 0, stream, p, share);
  else
    e = launch_dependent(gate_norm_sums_kernel<8>, dim3(columns, rows), dim3(32, 8), 0, stream, p, share);
  if (e != cudaSuccess || !share) return e;
  return launch_dependent(gate_norm_weights_kernel, dim3(columns, 3), dim3(32, 32), 0, stream, p,
                          static_cast<const float*>(share), shares);
}

// Up to 128 channels, rows too short for the teams of a CTA: the backward has a warp to a token and a unit to a row
// (128 channels, 20000 rows of one token 140 us, now 35; 5000 of 4 33 and 17; 2500 of 8 19.5 either way).
bool short_rows(const GateNormArgs& a) { return a.tokens / a.groups < 8; }

template <typename TX, typename TY>
cudaError_t launch_width_fwd(const GateNormArgs& a, cudaStream_t stream) {
  if (a.channels <= NARROW_CHANNELS) return launch_fwd<TX, TY, 1, true>(a, stream);
  return fwd_vectors(a.channels) == 1 ? launch_fwd<TX, TY, 1, false>(a, stream) : launch_fwd<TX, TY, 2, false>(a, stream);
}
template <typename TX, typename TY>
cudaError_t launch_width_bwd(const GateNormArgs& a, size_t* bytes, cudaStream_t stream) {
  if (a.channels <= NARROW_CHANNELS && !short_rows(a)) return launch_bwd<TX, TY, 1, BWD_REGS_1, true>(a, bytes, stream);
  switch (bwd_regs(a.channels)) {
    case BWD_REGS_1: return launch_bwd<TX, TY, 1, BWD_REGS_1, false>(a, bytes, stream);
    case BWD_REGS_2: return launch_bwd<TX, TY, 2, BWD_REGS_2, false>(a, bytes, stream);
    default: return launch_bwd<TX, TY, 4, BWD_REGS_4, false>(a, bytes, stream);
  }
}

cudaError_t bwd_typed(const GateNormArgs& a, size_t* bytes, cudaStream_t stream) {
  if (a.dtype == VSA_BF16) return launch_width_bwd<__nv_bfloat16, __nv_bfloat16>(a, bytes, stream);
  if (a.dtype == VSA_F16) return launch_width_bwd<__half, __half>(a, bytes, stream);
  if (a.branch_dtype == VSA_BF16) return launch_width_bwd<float, __nv_bfloat16>(a, bytes, stream);
  if (a.branch_dtype == VSA_F16) return launch_width_bwd<float, __half>(a, bytes, stream);
  return launch_width_bwd<float, float>(a, bytes, stream);
}

}  // namespace

size_t gate_norm_bwd_workspace(const GateNormArgs& a) {
  size_t bytes = 0;
  bwd_typed(a, &bytes, nullptr);
  return bytes;
}

cudaError_t launch_gate_norm_fwd(const GateNormArgs& a, cudaStream_t stream) {
  if (a.dtype == VSA_BF16) return launch_width_fwd<__nv_bfloat16, __nv_bfloat16>(a, stream);
  if (a.dtype == VSA_F16) return launch_width_fwd<__half, __half>(a, stream);
  if (a.branch_dtype == VSA_BF16) return launch_width_fwd<float, __nv_bfloat16>(a, stream);
  if (a.branch_dtype == VSA_F16) return launch_width_fwd<float, __half>(a, stream);
  return launch_width_fwd<float, float>(a, stream);
}
cudaError_t launch_gate_norm_bwd(const GateNormArgs& a, cudaStream_t stream) { return bwd_typed(a, nullptr, stream); }

}  // namespace vsa
