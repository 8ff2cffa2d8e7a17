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
#include "block_internal.cuh"
#include "vec8.cuh"

namespace vsa {

namespace {

constexpr int MAX_WPR = 16;   // warps of a token
constexpr int CTA_WARPS = 8;  // warps of a CTA that holds several tokens
constexpr int FWD_ROWS = 2;   // tokens in flight per group of warps

// Registers of a thread with NV vectors: the CTAs of an SM follow from them.
constexpr int fwd_regs(int nv) { return nv == 1 ? 80 : 112; }
constexpr int bwd_regs(int nv) { return nv == 1 ? 112 : 128; }

// 8 parameters of either type, or `fallback`.
__device__ __forceinline__ void load_param(const void* p, int64_t at, int dtype, float fallback, float* v) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fallback;
  } else if (dtype == VSA_F32) {
    load8(static_cast<const float*>(p) + at, v);
  } else if (dtype == VSA_BF16) {
    load8(static_cast<const __nv_bfloat16*>(p) + at, v);
  } else {
    load8(static_cast<const __half*>(p) + at, v);
  }
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

struct Params {
  GateNormArgs a;
  int wpr, per_cta;  // warps of a token, groups of them in a CTA
  int len;           // tokens of a modulation row
  int parts, chunk;  // units of a modulation row, tokens of a unit
  int units;
  float inv_dim;
};

// The warps that hold a token together: sums over all of its elements, the same for every lane.
struct Team {
  float (*buf)[4][MAX_WPR];  // [2]: warps' sums of this round and of the one before
  int wpr, warp, lane, bar, span;
  uint32_t round;

  __device__ __forceinline__ Team(float (*b)[4][MAX_WPR], const Params& p) {
    buf = b;
    wpr = p.wpr;
    const int w = threadIdx.x >> 5;
    warp = w % wpr;
    lane = threadIdx.x & 31;
    bar = 1 + w / wpr;
    span = 1;
    while (span < wpr) span *= 2;
    round = 0;
  }

  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
    static_assert(N <= 4, "room for the warps' sums");
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(FULL, v[i], o);
    if (wpr == 1) return;
    // Two buffers: a warp that writes round k + 2 has passed the barrier of round k + 1, which every
    // warp reaches after its reads of round k.
    float (*b)[MAX_WPR] = buf[round & 1u];
    ++round;
    if (lane < N) {
      float mine = v[0];
#pragma unroll
      for (int i = 1; i < N; ++i) mine = lane == i ? v[i] : mine;
      b[lane][warp] = mine;
    }
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(wpr * 32) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < wpr ? b[i][lane & (MAX_WPR - 1)] : 0.f;
    for (int o = span / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(FULL, v[i], o);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(FULL, v[i], 0);
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

template <typename T>
__device__ __forceinline__ T* at(const TokensView& v, int b, int t) {
  return static_cast<T*>(v.data) + b * v.batch + t * v.token;
}

template <typename TX, typename TY, int NV>
__global__ void __maxnreg__(fwd_regs(NV)) gate_norm_fwd_kernel(const __grid_constant__ Params p) {
  constexpr int R = NV == 1 ? FWD_ROWS : 1;
  __shared__ float sums[CTA_WARPS][2][4][MAX_WPR];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int group = (threadIdx.x >> 5) / p.wpr;
  Team team(sums[group], p);
  const int e0 = (team.warp * 32 + team.lane) * 8, step = p.wpr * 256;  // vectors e0, e0 + step, ..
  const bool branch = a.y.data != nullptr, post = a.post_weight != nullptr, layer = a.kind == VSA_LAYER_NORM;

  for (int u = blockIdx.x * p.per_cta + group; u < p.units; u += gridDim.x * p.per_cta) {
    const Unit unit = unit_of(p, u);
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
    load(unit.t0);
    for (int t = unit.t0; t < unit.t1; t += R) {
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
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int k = 0; k < NV; ++k)
            if (e0 + k * step < a.channels) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[r][k][i] = fmaf(-s[r], p.inv_dim, v[r][k][i]);
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

// SUMS: the unit's S1, S2, S3 go to the workspace.
template <typename TX, typename TY, int NV, bool SUMS>
__global__ void __maxnreg__(bwd_regs(NV)) gate_norm_bwd_kernel(const __grid_constant__ Params p) {
  __shared__ float sums[CTA_WARPS][2][4][MAX_WPR];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int group = (threadIdx.x >> 5) / p.wpr;
  Team team(sums[group], p);
  const int e0 = (team.warp * 32 + team.lane) * 8, step = p.wpr * 256;
  const bool branch = a.y.data != nullptr, post = a.post_weight != nullptr, layer = a.kind == VSA_LAYER_NORM;

  for (int u = blockIdx.x * p.per_cta + group; u < p.units; u += gridDim.x * p.per_cta) {
    const Unit unit = unit_of(p, u);
    float ca[NV][8], cg[NV][8], cp[NV][8], acc[SUMS ? NV : 1][3][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = e0 + k * step;
#pragma unroll
      for (int j = 0; SUMS && j < 3; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[SUMS ? k : 0][j][i] = 0.f;
      if (e >= a.channels) continue;
      float s[8];
      load_param(a.weight, e, a.weight_dtype, 1.f, ca[k]);
      load_param(a.scale.data, unit.b * a.scale.batch + unit.g * a.scale.group + e, a.mod_dtype, 0.f, s);
      load_param(a.gate.data, unit.b * a.gate.batch + unit.g * a.gate.group + e, a.mod_dtype, 1.f, cg[k]);
      if (post) load_param(a.post_weight, e, a.weight_dtype, 1.f, cp[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ca[k][i] *= 1.f + s[i];
    }
    Raw<TX> rx[NV], ro[NV];
    Raw<TY> rh[NV], ry[NV];
    auto load = [&](int t) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int e = e0 + k * step;
        rx[k].zero();
        ro[k].zero();
        rh[k].zero();
        ry[k].zero();
        if (t < unit.t1 && e < a.channels) {
          rx[k].load(at<const TX>(a.x_out, unit.b, t) + e);
          rh[k].load(at<const TY>(a.dh, unit.b, t) + e);
          if (a.dx_out.data) ro[k].load(at<const TX>(a.dx_out, unit.b, t) + e);
          if (branch) ry[k].load(at<const TY>(a.y, unit.b, t) + e);
        }
      }
    };
    load(unit.t0);
    for (int t = unit.t0; t < unit.t1; ++t) {
      float v[NV][8], g[NV][8], o[NV][8];
      Raw<TY> y[NV];
      float q = 0.f;  // sum of y^2
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        rx[k].widen(v[k]);
        rh[k].widen(g[k]);
        ro[k].widen(o[k]);
        y[k] = ry[k];
        if (post) {
          float z[8];
          y[k].widen(z);
#pragma unroll
          for (int i = 0; i < 8; ++i) q = fmaf(z[i], z[i], q);
        }
      }
      load(t + 1);
      if (layer) {
        float s[2] = {0.f, q};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] += v[k][i];
        team.sum(s);
        q = s[1];
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (e0 + k * step < a.channels) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = fmaf(-s[0], p.inv_dim, v[k][i]);
          }
      }
      float s[4] = {0.f, 0.f, 0.f, q};  // v^2, g v, g, y^2
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (e0 + k * step < a.channels) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float ga = g[k][i] * ca[k][i];
            s[0] = fmaf(v[k][i], v[k][i], s[0]);
            s[1] = fmaf(ga, v[k][i], s[1]);
            s[2] += ga;
          }
        }
      team.sum(s);
      if (!layer) q = s[3];
      const float f = rsqrtf(fmaf(s[0], p.inv_dim, a.eps));
      const float m1 = layer ? s[2] * p.inv_dim : 0.f, m2 = s[1] * f * p.inv_dim;
      const float fy = post ? rsqrtf(fmaf(q, p.inv_dim, a.post_eps)) : 1.f;
      float z[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int e = e0 + k * step;
        if (e >= a.channels) continue;
        float ny[8];
        if (branch) y[k].widen(ny);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = v[k][i] * f;
          const float dx = fmaf(f, fmaf(g[k][i], ca[k][i], -m1) - n * m2, o[k][i]);
          if (SUMS) {
            acc[SUMS ? k : 0][0][i] += g[k][i];
            acc[SUMS ? k : 0][1][i] = fmaf(g[k][i], n, acc[SUMS ? k : 0][1][i]);
          }
          o[k][i] = dx;
          if (branch) {
            ny[i] *= fy;
            if (SUMS) acc[SUMS ? k : 0][2][i] = fmaf(dx, ny[i], acc[SUMS ? k : 0][2][i]);
            g[k][i] = dx * cg[k][i];
            if (post) {
              g[k][i] *= cp[k][i];
              z[0] = fmaf(g[k][i], ny[i], z[0]);
            }
          }
        }
        store8(at<TX>(a.dx, unit.b, t) + e, o[k]);
        if (branch && !post) store8(at<TY>(a.dy, unit.b, t) + e, g[k]);
      }
      if (post) {
        team.sum(z);
        const float m = z[0] * p.inv_dim;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int e = e0 + k * step;
          if (e >= a.channels) continue;
          float ny[8];
          y[k].widen(ny);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[k][i] = fy * fmaf(-ny[i] * fy, m, g[k][i]);
          store8(at<TY>(a.dy, unit.b, t) + e, g[k]);
        }
      }
    }
    if (SUMS) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int e = e0 + k * step;
        if (e >= a.channels) continue;
#pragma unroll
        for (int j = 0; j < 3; ++j)
          store8(a.workspace + (static_cast<int64_t>(u) * 3 + j) * a.channels + e, acc[SUMS ? k : 0][j]);
      }
    }
  }
}

// The units' sums of a modulation row, joined in unit order: 32 columns a block, 32 strided units
// each, joined in their order.  Writes the row's gradients and, for the weights' gradients, its
// share of them: the result itself if there is one row, else to `share` [row][3][channels].
__global__ void __launch_bounds__(1024) gate_norm_sums_kernel(const __grid_constant__ Params p, float* share) {
  __shared__ float sums[3][32][33];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int c = blockIdx.x * 32 + threadIdx.x;
  const int rows = a.batch * a.groups;
  for (int bg = blockIdx.y; bg < rows; bg += gridDim.y) {
    float s[3] = {0.f, 0.f, 0.f};
    if (c < a.channels)
      for (int i = threadIdx.y; i < p.parts; i += 32) {
        const float* from = a.workspace + (static_cast<int64_t>(bg) * p.parts + i) * 3 * a.channels + c;
#pragma unroll
        for (int j = 0; j < 3; ++j) s[j] += from[static_cast<int64_t>(j) * a.channels];
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j) sums[j][threadIdx.y][threadIdx.x] = s[j];
    __syncthreads();
    if (threadIdx.y != 0 || c >= a.channels) continue;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      s[j] = 0.f;
#pragma unroll
      for (int y = 0; y < 32; ++y) s[j] += sums[j][y][threadIdx.x];
    }
    const int b = bg / a.groups, g = bg - b * a.groups;
    const float w = param(a.weight, c, a.weight_dtype, 1.f), bias = param(a.bias, c, a.weight_dtype, 0.f);
    const float post = param(a.post_weight, c, a.weight_dtype, 1.f);
    const int64_t to = static_cast<int64_t>(bg) * a.channels + c;
    store_param(a.dshift, to, a.mod_dtype, s[0]);
    store_param(a.dscale, to, a.mod_dtype, fmaf(w, s[1], bias * s[0]));
    store_param(a.dgate, to, a.mod_dtype, post * s[2]);
    const float one = 1.f + param(a.scale.data, b * a.scale.batch + g * a.scale.group + c, a.mod_dtype, 0.f);
    const float gate = param(a.gate.data, b * a.gate.batch + g * a.gate.group + c, a.mod_dtype, 1.f);
    if (rows == 1) {
      store_param(a.dbias, c, a.weight_dtype, one * s[0]);
      store_param(a.dweight, c, a.weight_dtype, one * s[1]);
      store_param(a.dpost, c, a.weight_dtype, gate * s[2]);
    } else if (share) {
      float* at = share + static_cast<int64_t>(bg) * 3 * a.channels + c;
      at[0] = one * s[0];
      at[a.channels] = one * s[1];
      at[2 * static_cast<int64_t>(a.channels)] = gate * s[2];
    }
  }
}

// dbias, dweight, dpost_weight: the modulation rows' shares, likewise.
__global__ void __launch_bounds__(1024) gate_norm_weights_kernel(const __grid_constant__ Params p, const float* share) {
  __shared__ float sums[32][33];
  grid_dependency_wait();
  const GateNormArgs& a = p.a;
  const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y, rows = a.batch * a.groups;
  float s = 0.f;
  if (c < a.channels)
    for (int i = threadIdx.y; i < rows; i += 32) s += share[(static_cast<int64_t>(i) * 3 + j) * a.channels + c];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= a.channels) return;
  s = 0.f;
#pragma unroll
  for (int y = 0; y < 32; ++y) s += sums[y][threadIdx.x];
  store_param(j == 0 ? a.dbias : j == 1 ? a.dweight : a.dpost, c, a.weight_dtype, s);
}

int vectors(int channels) { return channels <= 256 * MAX_WPR ? 1 : 2; }

// Units: parts of every modulation row.  The grid takes them in waves of `slots`, each as long as a
// unit's tokens and what a unit costs besides (`extra` tokens); the least of up to four waves.
constexpr int FWD_EXTRA = 2, BWD_EXTRA = 4;
struct Plan {
  int wpr, per_cta, ctas, parts, chunk, units;
};
Plan plan_of(int batch, int tokens, int channels, int groups, bool forward) {
  const int extra = forward ? FWD_EXTRA : BWD_EXTRA;
  Plan q{};
  const int nv = vectors(channels);
  q.wpr = (channels + 256 * nv - 1) / (256 * nv);
  q.per_cta = q.wpr < CTA_WARPS ? CTA_WARPS / q.wpr : 1;
  const int regs = (forward ? fwd_regs(nv) : bwd_regs(nv)) * 32 * q.wpr * q.per_cta;
  const int per_sm = 65536 / regs;
  const int64_t slots = static_cast<int64_t>(device_sm_count()) * per_sm * q.per_cta;
  const int64_t rows = static_cast<int64_t>(batch) * groups;
  const int len = tokens / groups;
  int64_t best = INT64_MAX;
  for (int w = 1; w <= 4; ++w) {
    int64_t parts = w * slots / rows;
    if (parts < 1) parts = 1;
    if (parts > len) parts = len;
    const int64_t chunk = (len + parts - 1) / parts;
    parts = (len + chunk - 1) / chunk;
    const int64_t waves = (rows * parts + slots - 1) / slots, cost = waves * (chunk + extra);
    if (cost < best) {
      best = cost;
      q.parts = static_cast<int>(parts);
      q.chunk = static_cast<int>(chunk);
    }
  }
  q.units = static_cast<int>(rows * q.parts);
  const int64_t need = (q.units + q.per_cta - 1) / q.per_cta, most = slots / q.per_cta;
  q.ctas = static_cast<int>(need < most ? need : most);
  return q;
}

bool wants_sums(const GateNormArgs& a) {
  return a.dgate || a.dscale || a.dshift || a.dpost || a.dweight || a.dbias;
}

template <typename TX, typename TY, int NV>
cudaError_t launch(const GateNormArgs& a, bool forward, cudaStream_t stream) {
  const Plan q = plan_of(a.batch, a.tokens, a.channels, a.groups, forward);
  Params p;
  p.a = a;
  p.wpr = q.wpr;
  p.per_cta = q.per_cta;
  p.len = a.tokens / a.groups;
  p.parts = q.parts;
  p.chunk = q.chunk;
  p.units = q.units;
  p.inv_dim = 1.f / static_cast<float>(a.channels);
  const dim3 grid(q.ctas), block(q.wpr * q.per_cta * 32);
  if (forward) return launch_dependent(gate_norm_fwd_kernel<TX, TY, NV>, grid, block, 0, stream, p);
  if (!wants_sums(a)) return launch_dependent(gate_norm_bwd_kernel<TX, TY, NV, false>, grid, block, 0, stream, p);
  cudaError_t e = launch_dependent(gate_norm_bwd_kernel<TX, TY, NV, true>, grid, block, 0, stream, p);
  if (e != cudaSuccess) return e;
  const int rows = a.batch * a.groups, columns = (a.channels + 31) / 32;
  float* share = rows > 1 && (a.dpost || a.dweight || a.dbias)
                     ? a.workspace + static_cast<int64_t>(q.units) * 3 * a.channels
                     : nullptr;
  e = launch_dependent(gate_norm_sums_kernel, dim3(columns, rows < 65535 ? rows : 65535), dim3(32, 32), 0, stream, p, share);
  if (e != cudaSuccess || !share) return e;
  return launch_dependent(gate_norm_weights_kernel, dim3(columns, 3), dim3(32, 32), 0, stream, p,
                          static_cast<const float*>(share));
}

template <typename TX, typename TY>
cudaError_t launch_width(const GateNormArgs& a, bool forward, cudaStream_t stream) {
  switch (vectors(a.channels)) {
    case 1: return launch<TX, TY, 1>(a, forward, stream);
    default: return launch<TX, TY, 2>(a, forward, stream);
  }
}

cudaError_t launch_typed(const GateNormArgs& a, bool forward, cudaStream_t stream) {
  if (a.dtype == VSA_BF16) return launch_width<__nv_bfloat16, __nv_bfloat16>(a, forward, stream);
  if (a.dtype == VSA_F16) return launch_width<__half, __half>(a, forward, stream);
  if (a.branch_dtype == VSA_BF16) return launch_width<float, __nv_bfloat16>(a, forward, stream);
  if (a.branch_dtype == VSA_F16) return launch_width<float, __half>(a, forward, stream);
  return launch_width<float, float>(a, forward, stream);
}

}  // namespace

size_t gate_norm_bwd_workspace(int batch, int tokens, int channels, int groups) {
  const Plan q = plan_of(batch, tokens, channels, groups, false);
  const size_t rows = static_cast<size_t>(batch) * groups;
  return align_up((q.units + rows) * 3 * channels * sizeof(float), 256);
}

cudaError_t launch_gate_norm_fwd(const GateNormArgs& a, cudaStream_t stream) { return launch_typed(a, true, stream); }
cudaError_t launch_gate_norm_bwd(const GateNormArgs& a, cudaStream_t stream) { return launch_typed(a, false, stream); }

}  // namespace vsa
