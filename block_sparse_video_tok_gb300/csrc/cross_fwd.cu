// cross_fwd.cu -- attention to an encoder's states of another length, forward:
//   O = softmax(q k^T sm_scale) v,  lse = max(s) + log2(sum 2^(s - max)),  s = q k^T sm_scale log2e.
//
// Work unit: two 128-row query tiles of one (batch, key head) -- see QTiles -- against a range of
// kv tiles of 128 keys.  One persistent CTA per SM; softmax group g (4 warps, one row per thread)
// owns tile g: its own S and O accumulators in TMEM, its own online softmax.  Per kv tile
//   S_g = Q_g K^T            128 x 128 x 128 UMMAs, operands in shared memory
//   m, P = 2^(s - m), l      in registers; m moves only when a row's maximum outgrows it by
//                            RESCALE (then O_g is scaled first), so P stays below 2^RESCALE
//   O_g += P V               P in TMEM as bf16 pairs over S_g's columns, V MN-major
// and the issuing warp alternates  PV_0(j) S_0(j+1) PV_1(j) S_1(j+1) ...: while one group is in
// its softmax the tensor pipe works for the other.  The groups share every K and V tile.
//
// P is rounded to bf16 because kind::f16 takes one type for both operands and V is the caller's
// bf16; l adds up the unrounded values.  The rounding is of the size of O's own (2^-9 relative,
// independent per key).
//
// The last kv tile multiplies only ceil16(keys left) columns; its other columns are masked in
// registers, and rows of V past the last key, which may hold anything, are zeroed in shared
// memory before P (0 there) meets them.
//
// When there are fewer units than SMs the keys are split: each part leaves its unnormalised O
// and (m, l) in the workspace, and cross_combine_kernel joins them in part order.
//
// Roles (384 threads): warps 0-3 and 4-7 softmax groups; warp 8 TMEM owner and TMA producer of Q
// and K; warp 9 UMMA issuer; warp 10 TMA producer of V.
// Shared memory: a Q tile per group, 2 K and 2 V tiles, and 4 KB per softmax warp through which O
// leaves in whole 128-byte lines.  A Q tile is free as soon as its unit's last S has been
// computed, a softmax and a P V before the next unit needs it, and its successor has been
// prefetched into L2 by then.  TMEM: O x2 [0, 256), S x2 [256, 512).
#include "cross_common.cuh"

namespace vsa {

namespace {

constexpr int NUM_THREADS = 384;  // warps are allocated in fours: the twelfth has no role
constexpr int TMA_WARP = 8, MMA_WARP = 9, V_WARP = 10;
constexpr int KV_STAGES = 2;
constexpr float RESCALE = 8.0f;  // log2 units

constexpr uint32_t SM_Q = 0;
constexpr uint32_t SM_K = 2 * TILE_BYTES;
constexpr uint32_t SM_V = SM_K + KV_STAGES * TILE_BYTES;
constexpr uint32_t SM_OUT = SM_V + KV_STAGES * TILE_BYTES;  // 8 warps x 32 rows x 128 bytes
constexpr uint32_t SM_BAR = SM_OUT + TILE_BYTES;

enum Bar : uint32_t {
  Q_FULL0 = 0,  // per group
  Q_EMPTY0 = Q_FULL0 + 2,
  K_FULL0 = Q_EMPTY0 + 2,
  K_EMPTY0 = K_FULL0 + KV_STAGES,
  V_FULL0 = K_EMPTY0 + KV_STAGES,
  V_EMPTY0 = V_FULL0 + KV_STAGES,
  S_FULL0 = V_EMPTY0 + KV_STAGES,  // per group: S_g of the next kv tile is in TMEM
  P_READY0 = S_FULL0 + 2,          // per group: P_g is in TMEM
  O_FULL0 = P_READY0 + 2,          // per group: O_g holds the unit's last product
  O_EMPTY0 = O_FULL0 + 2,          // per group: O_g has been read
  V_TAIL = O_EMPTY0 + 2,
  DRAIN,
  NUM_BARS
};
constexpr uint32_t SM_TMEM_SLOT = SM_BAR + NUM_BARS * 8;
constexpr uint32_t SM_ABORT = SM_TMEM_SLOT + 4;
constexpr uint32_t SMEM_BYTES = SM_ABORT + 4 + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

constexpr uint32_t TM_O = 0, TM_S = 256;  // O_g at TM_O + 128 g, S_g at TM_S + 128 g
constexpr uint32_t IDESC_S0 = idesc_f16_f32acc(128, 0, false, false, true);  // N is added
constexpr uint32_t IDESC_PV = idesc_f16_f32acc(128, 128, false, true, true);

struct Params {
  CrossArgs a;
  QTiles t;
  int pairs;   // units along the tiles of one (batch, key head)
  int splits;  // parts of the keys
  int total;   // units * splits
  float* part_o;    // [split][batch * kv_heads * tiles][128 columns][128 rows]
  float2* part_ml;  // [split][batch * kv_heads * tiles][128 rows]
};

struct Unit {
  int b, kh, tile0, split;
  int t0, t1;   // kv tiles
  int keys;     // visible keys
  bool second;  // group 1 has a tile
  __device__ __forceinline__ int count() const { return t1 - t0; }
  // Keys of kv tile j of this unit's range that are visible (128 but for the last).
  __device__ __forceinline__ int keys_of(int j) const { return min(TILE, keys - (t0 + j) * TILE); }
};

__device__ __forceinline__ Unit decode(const Params& p, int w) {
  Unit u;
  const int x = w % p.pairs;
  w /= p.pairs;
  u.kh = w % p.a.kv_heads;
  w /= p.a.kv_heads;
  u.b = w % p.a.batch;
  u.split = w / p.a.batch;
  u.tile0 = 2 * x;
  u.second = 2 * x + 1 < p.t.tiles;
  u.keys = visible_keys(p.a.kv_len, u.b, p.a.kv_tokens, p.a.err);
  const int n = (u.keys + TILE - 1) / TILE, per = (n + p.splits - 1) / p.splits;
  u.t0 = min(u.split * per, n);
  u.t1 = min(u.t0 + per, n);
  return u;
}

// First head and token of tile `tile` of the unit's (batch, key head).
__device__ __forceinline__ void tile_origin(const Params& p, const Unit& u, int tile, int* head,
                                            int* token) {
  const int g = tile / p.t.blocks;
  *head = u.kh * p.t.share + g * p.t.pack;
  *token = (tile - g * p.t.blocks) * p.t.box;
}

__device__ __forceinline__ int ceil16(int n) { return (n + 15) & ~15; }

// Maximum (or minimum) of 128 raw scores: four chains of 3-input instructions.
template <bool MIN>
__device__ __forceinline__ float extremum(const uint32_t* sv) {
  constexpr float sign = MIN ? -1.f : 1.f;
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    m[k] = fmaxf(sign * __uint_as_float(sv[2 * k]), sign * __uint_as_float(sv[2 * k + 1]));
#pragma unroll
  for (int u = 8; u < TILE; u += 2)
    m[(u >> 1) & 3] = max3(m[(u >> 1) & 3], sign * __uint_as_float(sv[u]), sign * __uint_as_float(sv[u + 1]));
  return sign * max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + SM_ABORT);
  const uint32_t* tmem_slot = reinterpret_cast<const uint32_t*>(gbase + SM_TMEM_SLOT);
  auto bar = [&](uint32_t b) { return base + SM_BAR + 8u * b; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.a.wait_ns;

  if (threadIdx.x == 0) {
    *abort = 0;
    for (uint32_t b = 0; b < NUM_BARS; ++b) {
      const bool four = (b >= P_READY0 && b < O_FULL0) || (b >= O_EMPTY0 && b < V_TAIL);
      mbar_init(bar(b), four ? 4 : 1);
    }
    fence_barrier_init();
  }
  if (warp == TMA_WARP) {
    tmem_alloc(base + SM_TMEM_SLOT, 512);
    tmem_relinquish();
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  grid_dependency_wait();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tile_rows_bytes = static_cast<uint32_t>(p.t.box * p.t.pack) * 256u;

  if (warp == TMA_WARP) {
    // ------------------------------------------------------------------ TMA producer: Q, K
    uint32_t qn[2] = {0, 0}, kn = 0;  // tiles loaded
    bool ok = true;
    const int halves = p.t.box * p.t.pack == TILE ? 1 : 2;  // copies of a Q tile
    auto load_k = [&](const Unit& u, int j) {
      const uint32_t s = kn % KV_STAGES;
      if (!mbar_wait_warp(bar(K_EMPTY0 + s), ((kn / KV_STAGES) & 1u) ^ 1u, abort, limit)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(K_FULL0 + s), TILE_BYTES);
        tma_load_5d(base + SM_K + s * TILE_BYTES, &tm_k, bar(K_FULL0 + s), 0, (u.t0 + j) * TILE, u.kh, 0,
                    p.a.k.batch ? u.b : 0);
      }
      __syncwarp();
      ++kn;
      return true;
    };
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0) continue;
      ok = load_k(u, 0);
      for (int g = 0; g < (u.second ? 2 : 1) && ok; ++g) {
        ok = mbar_wait_warp(bar(Q_EMPTY0 + g), (qn[g] & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        int head, token;
        tile_origin(p, u, u.tile0 + g, &head, &token);
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(Q_FULL0 + g), tile_rows_bytes);
          for (int h = 0; h < halves; ++h)
            tma_load_5d(base + SM_Q + g * TILE_BYTES + h * (TILE_BYTES / 2), &tm_q, bar(Q_FULL0 + g), 0, token, head, h,
                        p.a.q.batch ? u.b : 0);
        }
        __syncwarp();
        ++qn[g];
      }
      if (ok && lane == 0 && w + gridDim.x < p.total) {
        const Unit nu = decode(p, w + gridDim.x);
        for (int g = 0; g < (nu.count() == 0 ? 0 : nu.second ? 2 : 1); ++g) {
          int head, token;
          tile_origin(p, nu, nu.tile0 + g, &head, &token);
          for (int h = 0; h < halves; ++h) tma_prefetch_5d(&tm_q, 0, token, head, h, p.a.q.batch ? nu.b : 0);
        }
      }
      __syncwarp();
      for (int j = 1; j < u.count() && ok; ++j) ok = load_k(u, j);
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.a.err);
      // Let the copies already issued land before the CTA's shared memory goes away.
      volatile int never = 0;
      for (int g = 0; g < 2; ++g)
        if (qn[g] > 0) mbar_wait_bounded(bar(Q_FULL0 + g), (qn[g] - 1) & 1u, &never, DRAIN_LIMIT_NS);
      for (uint32_t i = kn > KV_STAGES ? kn - KV_STAGES : 0; i < kn; ++i)
        mbar_wait_bounded(bar(K_FULL0 + i % KV_STAGES), (i / KV_STAGES) & 1u, &never, DRAIN_LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == V_WARP) {
    // ------------------------------------------------------------------ TMA producer: V
    uint32_t vn = 0, tails = 0, tails_seen = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      for (int j = 0; j < u.count() && ok; ++j) {
        const uint32_t s = vn % KV_STAGES, tile = base + SM_V + s * TILE_BYTES;
        ok = mbar_wait_warp(bar(V_EMPTY0 + s), ((vn / KV_STAGES) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        // Past kv_tokens the copy itself fills with zeros; rows between the last visible key and
        // there are zeroed here, before the tile is handed on.
        const int n = u.keys_of(j);
        const bool patch = n < TILE && u.keys < p.a.kv_tokens;
        const uint32_t full = patch ? bar(V_TAIL) : bar(V_FULL0 + s);
        if (lane == 0) {
          mbar_arrive_expect_tx(full, TILE_BYTES);
          tma_load_5d(tile, &tm_v, full, 0, (u.t0 + j) * TILE, u.kh, 0, p.a.v.batch ? u.b : 0);
        }
        __syncwarp();
        if (patch) {
          ++tails;
          ok = mbar_wait_warp(full, (tails - 1) & 1u, abort, limit);
          if (!ok) break;
          tails_seen = tails;
          zero_rows(tile, n, ceil16(n), lane);
          if (lane == 0) mbar_arrive(bar(V_FULL0 + s));
        }
        ++vn;
      }
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.a.err);
      volatile int never = 0;
      if (tails > tails_seen) mbar_wait_bounded(bar(V_TAIL), (tails - 1) & 1u, &never, DRAIN_LIMIT_NS);
      for (uint32_t i = vn > KV_STAGES ? vn - KV_STAGES : 0; i < vn; ++i)
        mbar_wait_bounded(bar(V_FULL0 + i % KV_STAGES), (i / KV_STAGES) & 1u, &never, DRAIN_LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------------ UMMA issuer
    // The whole warp runs this role in lockstep; one elected lane issues.
    uint32_t kn = 0, vn = 0;                               // K and V tiles consumed
    uint32_t qn[2] = {0, 0}, pn[2] = {0, 0}, on[2] = {0, 0};  // per group: Q tiles, kv tiles, units
    bool ok = true, issued = false;
    const uint64_t q_desc = sdesc_sw128(base + SM_Q, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(base + SM_K, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(base + SM_V, TILE_BYTES / 2, 1024);
    // S_g = Q_g K^T over `keys` columns (rounded up to 16), K in stage kn; `last`: of the unit.
    auto issue_s = [&](int g, int keys, bool last) {
      const uint64_t qa = sdesc_advance(q_desc, g * TILE_BYTES);
      const uint64_t kd = sdesc_advance(k_desc, (kn % KV_STAGES) * TILE_BYTES);
      const uint32_t ts = tmem + TM_S + g * 128u;
      const uint32_t idesc = IDESC_S0 | (static_cast<uint32_t>(ceil16(keys) >> 3) << 17);
      umma_ss_elect<false>(ts, qa, kd, idesc);
#pragma unroll
      for (int kk = 1; kk < 8; ++kk) {
        const uint32_t off = (kk >> 2) * (TILE_BYTES / 2) + (kk & 3) * 32u;
        umma_ss_elect<true>(ts, sdesc_advance(qa, off), sdesc_advance(kd, off), idesc);
      }
      umma_commit_elect(bar(S_FULL0 + g));
      if (last) umma_commit_elect(bar(Q_EMPTY0 + g));
      issued = true;
    };
    auto issue_pv = [&](int g, bool fresh, int keys) {
      const uint64_t vd = sdesc_advance(v_desc, (vn % KV_STAGES) * TILE_BYTES);
      const uint32_t to = tmem + TM_O + g * 128u, pa = tmem + TM_S + g * 128u;
      if (fresh)
        umma_ts_elect<false>(to, pa, vd, IDESC_PV);
      else
        umma_ts_elect<true>(to, pa, vd, IDESC_PV);
      if (keys > TILE - 16) {
#pragma unroll
        for (int kk = 1; kk < 8; ++kk) umma_ts_elect<true>(to, pa + kk * 8u, sdesc_advance(vd, kk * 2048u), IDESC_PV);
      } else {
#pragma unroll 1
        for (int kk = 1; kk * 16 < keys; ++kk)
          umma_ts_elect<true>(to, pa + kk * 8u, sdesc_advance(vd, kk * 2048u), IDESC_PV);
      }
    };
    // The next unit with keys, from w on (total: none).
    auto next_unit = [&](int w, Unit* u) {
      for (; w < p.total; w += gridDim.x) {
        *u = decode(p, w);
        if (u->count() > 0) break;
      }
      return w;
    };
    Unit u{};
    int w = next_unit(blockIdx.x, &u);
    // S of unit x's first kv tile for one group (group 0 first).
    auto first_s = [&](const Unit& x, int g) {
      if (!mbar_wait_warp(bar(Q_FULL0 + g), qn[g] & 1u, abort, limit)) return false;
      if (g == 0 && !mbar_wait_warp(bar(K_FULL0 + kn % KV_STAGES), (kn / KV_STAGES) & 1u, abort, limit)) return false;
      tc_fence_after_sync();
      issue_s(g, x.keys_of(0), x.count() == 1);
      ++qn[g];
      return true;
    };
    if (w < p.total) {
      ok = first_s(u, 0) && (!u.second || first_s(u, 1));
      if (ok) {
        umma_commit_elect(bar(K_EMPTY0 + kn % KV_STAGES));
        ++kn;
      }
    }
    while (ok && w < p.total) {
      Unit nu{};
      const int nw = next_unit(w + gridDim.x, &nu);
      const int groups = u.second ? 2 : 1, n = u.count();
      for (int j = 0; j < n && ok; ++j) {
        const int keys = u.keys_of(j);
        for (int g = 0; g < groups; ++g) {
          ok = mbar_wait_warp(bar(P_READY0 + g), pn[g] & 1u, abort, limit) &&
               (g != 0 || mbar_wait_warp(bar(V_FULL0 + vn % KV_STAGES), (vn / KV_STAGES) & 1u, abort, limit)) &&
               (j != 0 || mbar_wait_warp(bar(O_EMPTY0 + g), (on[g] & 1u) ^ 1u, abort, limit));
          if (!ok) break;
          tc_fence_after_sync();
          issue_pv(g, j == 0, keys);
          ++pn[g];
          if (j + 1 < n) {
            if (g == 0 && !(ok = mbar_wait_warp(bar(K_FULL0 + kn % KV_STAGES), (kn / KV_STAGES) & 1u, abort, limit)))
              break;
            tc_fence_after_sync();
            issue_s(g, u.keys_of(j + 1), j + 2 == n);
          } else {
            umma_commit_elect(bar(O_FULL0 + g));
            ++on[g];
            // The next unit's first S of this group, while the softmax reads O_g.
            if (nw < p.total && (g == 0 || nu.second) && !(ok = first_s(nu, g))) break;
          }
        }
        if (!ok) break;
        // A unit without a second tile followed by one with: its first S is still to come.
        if (j + 1 == n && groups == 1 && nw < p.total && nu.second && !(ok = first_s(nu, 1))) break;
        umma_commit_elect(bar(V_EMPTY0 + vn % KV_STAGES));
        ++vn;
        if (j + 1 < n || nw < p.total) {
          umma_commit_elect(bar(K_EMPTY0 + kn % KV_STAGES));
          ++kn;
        }
      }
      u = nu;
      w = nw;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    if (issued) {
      // Every UMMA has completed before TMEM is released.
      umma_commit_elect(bar(DRAIN));
      volatile int never = 0;
      if (lane == 0) mbar_wait_bounded(bar(DRAIN), 0, &never, DRAIN_LIMIT_NS);
      __syncwarp();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax groups
    const int quarter = warp & 3, g = warp >> 2;
    const int r = quarter * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + TM_S + g * 128u, t_o = tmem + lane_off + TM_O + g * 128u;
    float c1 = p.a.sm_scale * LOG2E_F;
    if (c1 == 0.f) c1 = 1e-30f;  // keeps 0 * -inf out of the mask; finite scores still give s = 0
    const uint32_t pad = c1 > 0.f ? 0xff800000u : 0x7f800000u;  // scales to -inf
    const uint32_t stage = base + SM_OUT + warp * 4096u;  // this warp's 32 rows x 64 columns
    uint32_t sn = 0, on = 0;                              // kv tiles and units of this group
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (g == 1 && !u.second) continue;
      int head, token;
      tile_origin(p, u, u.tile0 + g, &head, &token);
      const int rh = r / p.t.box;
      head += rh;
      token += r - rh * p.t.box;
      const bool valid = rh < p.t.pack && token < p.a.q_tokens;
      const int64_t row = (static_cast<int64_t>(u.b) * p.a.heads + head) * p.a.q_tokens + token;
      const int64_t ptile =
          ((static_cast<int64_t>(u.split) * p.a.batch + u.b) * p.a.kv_heads + u.kh) * p.t.tiles + u.tile0 + g;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.a.o.data) + u.b * p.a.o.batch + head * p.a.o.head +
                            token * p.a.o.token;
      if (u.count() == 0) {
        if (!valid) continue;
        if (p.splits > 1) {
          p.part_ml[ptile * TILE + r] = make_float2(-INFINITY, 0.f);
          continue;
        }
        for (int c = 0; c < 16; ++c) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0u, 0u, 0u, 0u);
        p.a.lse[row] = -INFINITY;
        continue;
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < u.count(); ++j) {
        ok = warp_wait(bar(S_FULL0 + g), sn & 1u, abort, limit, lane);
        if (!ok) break;
        ++sn;
        tc_fence_after_sync();
        uint32_t sv[TILE];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(t_s + c * 32u, sv + c * 32);
        tmem_wait_ld();
        const int n = u.keys_of(j);
        if (n < TILE) {
#pragma unroll
          for (int i = 0; i < TILE; ++i)
            if (i >= n) sv[i] = pad;
        }
        const float mb = c1 * (c1 > 0.f ? extremum<false>(sv) : extremum<true>(sv));
        const bool need = mb > m + RESCALE;
        if (__any_sync(0xffffffffu, need)) {
          const float f = need ? ex2(m - mb) : 1.f;  // m = -inf: 0, nothing accumulated yet
          l *= f;
          if (need) m = mb;
          // S_g of this tile was issued after PV_g of the last one, so O_g is complete.
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t ov[16];
              tmem_ld_32x32b_x16(t_o + c * 16u, ov);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f);
              tmem_st_32x32b_x16(t_o + c * 16u, ov);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const uint64_t c2 = f2_pack(c1, c1), o2 = f2_pack(off, off);
        uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[c * 32 + 2 * i]), __uint_as_float(sv[c * 32 + 2 * i + 1])),
                             c2, o2),
                      a0, a1);
            const float p0 = ex2(a0), p1 = ex2(a1);
            acc[i & 1] = f2_add(acc[i & 1], f2_pack(p0, p1));
            pk[i] = pack_bf162(p0, p1);
          }
          tmem_st_32x32b_x16(t_s + c * 16u, pk);
        }
        float s0, s1;
        f2_unpack(f2_add(acc[0], acc[1]), s0, s1);
        l += s0 + s1;
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(P_READY0 + g));
      }
      if (!ok) break;
      ok = warp_wait(bar(O_FULL0 + g), on & 1u, abort, limit, lane);
      if (!ok) break;
      tc_fence_after_sync();
      if (p.splits > 1) {
        if (valid) p.part_ml[ptile * TILE + r] = make_float2(m, l);
        float* po = p.part_o + ptile * TILE * TILE + r;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t ov[32];
          tmem_ld_32x32b_x32(t_o + c * 32u, ov);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int i = 0; i < 32; ++i) po[(c * 32 + i) * TILE] = __uint_as_float(ov[i]);
          }
        }
      } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const uint64_t inv2 = f2_pack(inv, inv);
        const unsigned rows = __ballot_sync(0xffffffffu, valid);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // column halves of 64, through the warp's staging rows
          uint32_t ov[64];
          tmem_ld_32x32b_x32(t_o + h * 64u, ov);
          tmem_ld_32x32b_x32(t_o + h * 64u + 32u, ov + 32);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t pk[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float a0, a1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(ov[8 * i + 2 * x]), __uint_as_float(ov[8 * i + 2 * x + 1])), inv2),
                        a0, a1);
              pk[x] = pack_bf162(a0, a1);
            }
            st_shared16(stage + swizzled(lane, i), pk[0], pk[1], pk[2], pk[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // four rows of 128 bytes at a time
            const int rr = i * 4 + (lane >> 3);
            const uint64_t to = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(orow), rr);
            const uint4 x = ld_shared16(stage + swizzled(rr, lane & 7));
            if ((rows >> rr) & 1u) reinterpret_cast<uint4*>(to)[h * 8 + (lane & 7)] = x;
          }
          __syncwarp();
        }
        if (valid) p.a.lse[row] = m + log2f(l);
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(O_EMPTY0 + g));
      ++on;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == TMA_WARP) tmem_dealloc(tmem, 512);
}

// Joins the parts of the keys: per row, M = max m, w = 2^(m - M), O = sum w O / sum w l.  A warp
// handles 32 rows x 8 columns of a tile; a part without a visible key (l = 0) is not read.
__global__ void __launch_bounds__(128) cross_combine_kernel(const __grid_constant__ Params p) {
  grid_dependency_wait();
  const int tile = blockIdx.x, lane = threadIdx.x & 31;
  const int r = (threadIdx.x >> 5) * 32 + lane, c0 = blockIdx.y * 8;
  const int tiles = p.a.batch * p.a.kv_heads * p.t.tiles;
  const int x = tile % p.t.tiles, bk = tile / p.t.tiles, b = bk / p.a.kv_heads, kh = bk % p.a.kv_heads;
  const int rh = r / p.t.box;
  const int head = kh * p.t.share + x / p.t.blocks * p.t.pack + rh;
  const int token = x % p.t.blocks * p.t.box + r - rh * p.t.box;
  if (rh >= p.t.pack || token >= p.a.q_tokens) return;
  float mm = -INFINITY, l = 0.f, o[8] = {};
  for (int s = 0; s < p.splits; ++s) {
    const int64_t at = static_cast<int64_t>(s) * tiles + tile;
    const float2 ml = p.part_ml[at * TILE + r];
    if (ml.y == 0.f) continue;  // NaN is kept
    const float mn = fmaxf(mm, ml.x), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(mm - ref), w = ex2(ml.x - ref);
    mm = mn;
    l = l * f + ml.y * w;
    const float* po = p.part_o + (at * TILE + c0) * TILE + r;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * f + po[i * TILE] * w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.o.data) + b * p.a.o.batch + head * p.a.o.head +
                            token * p.a.o.token + c0) =
      make_uint4(pack_bf162(o[0] * inv, o[1] * inv), pack_bf162(o[2] * inv, o[3] * inv),
                 pack_bf162(o[4] * inv, o[5] * inv), pack_bf162(o[6] * inv, o[7] * inv));
  if (c0 == 0)
    p.a.lse[(static_cast<int64_t>(b) * p.a.heads + head) * p.a.q_tokens + token] = mm + log2f(l);
}

struct Plan {
  QTiles t;
  int pairs, splits;
  size_t ml_off, total;  // workspace
};

// Parts of the keys: one when the units fill the SMs; else as many as keep every SM busy with
// one, each of at least two kv tiles.
Plan plan_of(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens) {
  Plan p{};
  p.t = q_tiles(heads, kv_heads, q_tokens);
  p.pairs = (p.t.tiles + 1) / 2;
  const int64_t units = static_cast<int64_t>(batch) * kv_heads * p.pairs;
  const int64_t kv_tiles = (kv_tokens + TILE - 1) / TILE;
  int64_t s = device_sm_count() / units;
  if (s > kv_tiles / 2) s = kv_tiles / 2;
  p.splits = s < 1 ? 1 : static_cast<int>(s);
  if (p.splits > 1) {
    const size_t rows = static_cast<size_t>(p.splits) * batch * kv_heads * p.t.tiles * TILE;
    p.ml_off = rows * TILE * sizeof(float);
    p.total = align_up(p.ml_off + rows * sizeof(float2), 256);
  }
  return p;
}

}  // namespace

size_t cross_fwd_workspace(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens) {
  return plan_of(batch, heads, kv_heads, q_tokens, kv_tokens).total;
}

cudaError_t launch_cross_fwd(const CrossArgs& a, cudaStream_t stream) {
  const Plan plan = plan_of(a.batch, a.heads, a.kv_heads, a.q_tokens, a.kv_tokens);
  Params p{};
  p.a = a;
  p.t = plan.t;
  p.pairs = plan.pairs;
  p.splits = plan.splits;
  p.total = a.batch * a.kv_heads * plan.pairs * plan.splits;
  p.part_o = reinterpret_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(a.workspace + plan.ml_off);
  CUtensorMap tq, tk, tv;
  cudaError_t e;
  if ((e = make_tmap_heads(&tq, a.q, a.q_tokens, a.batch, p.t.box, p.t.pack)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&tk, a.k, a.kv_tokens, a.batch, TILE, 1)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&tv, a.v, a.kv_tokens, a.batch, TILE, 1)) != cudaSuccess) return e;
  static std::atomic<uint64_t> smem_set{0};
  if ((e = ensure_smem_limit(cross_fwd_kernel, static_cast<int>(SMEM_BYTES), smem_set)) != cudaSuccess) return e;
  const int sms = device_sm_count();
  e = launch_dependent(cross_fwd_kernel, dim3(p.total < sms ? p.total : sms), dim3(NUM_THREADS), SMEM_BYTES, stream,
                       tq, tk, tv, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_dependent(cross_combine_kernel, dim3(a.batch * a.kv_heads * p.t.tiles, 16), dim3(128), 0, stream, p);
}

}  // namespace vsa
