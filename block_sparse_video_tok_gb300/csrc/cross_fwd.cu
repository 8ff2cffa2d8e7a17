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
// bf16; l adds up the unrounded values.  The rounding is of the size of O's own (2^-8 relative at
// most, independent per key).
//
// The last kv tile multiplies only as many columns as have keys (S in steps of 16, P V of 64);
// scores past the last key are overwritten with -inf, and rows of V past it, which may hold
// anything, are zeroed in shared memory before P (0 there) meets them.
//
// When there are fewer units than SMs the keys are split: each part leaves its unnormalised O
// and (m, l) in the workspace, and cross_combine_kernel joins them in part order (2 x 8 heads, 64
// queries on 8191 keys: 19 to 22 us, without parts 89).
//
// Roles (512 threads): warp 0 TMEM owner and TMA producer of Q and K; warp 1 UMMA issuer; warp 2 TMA
// producer of V; warp 3 idle; warps 4-7 and 8-11 softmax groups; warps 12-15 output (one row of
// the tile per thread: O / l, rounded, written), so that a group goes on to its next unit's scores
// while its last O leaves.
// Shared memory: a Q tile per group, 2 K and 2 V tiles, and 4 KB per output warp through which O
// leaves in whole 128-byte lines.  A Q tile is free as soon as its unit's last S has been
// computed, a softmax and a P V before the next unit needs it.  TMEM: O x2 [0, 256), S x2 [256, 512).
//
// Measured: 131040 queries on 512 keys, 12 heads: 277 us in short bursts (1.49 PFLOP/s, 78 % of the
// measured burst peak), 306 to 317 us in a long run under the power cap (1.30 to 1.35, 76 to 79 % of
// the sustained peak).  What bounds it: of the 1630 cycles that a kv tile of a group takes, its two products fill
// 1036 of the tensor core, its exponentials 512 of the special function units.  The rest is no
// single role's: with half of the softmax left out the same run takes 263 us, without the output's
// stores 265, without exponentials 277.  Tried without gain: P handed over in halves, registers
// moved between the roles, K and V multicast to pairs of CTAs, a third K tile in place of the
// output's staging (287), two softmax warps for each 32 rows (323), an issuing warp for each group
// (336: their products alternate instruction by instruction).
#include "cross_common.cuh"

namespace vsa {

namespace {

constexpr int NUM_THREADS = 512;
constexpr int TMA_WARP = 0, MMA_WARP = 1, V_WARP = 2, SOFTMAX_WARP = 4, OUT_WARP = 12;
constexpr int KV_STAGES = 2;
constexpr float RESCALE = 8.0f;  // log2 units (0: 305 us where 278 are taken now, 131040 x 512, 12 heads)

constexpr uint32_t SM_Q = 0;
constexpr uint32_t SM_K = 2 * TILE_BYTES;
constexpr uint32_t SM_V = SM_K + KV_STAGES * TILE_BYTES;
constexpr uint32_t SM_OUT = SM_V + KV_STAGES * TILE_BYTES;  // 4 warps x 32 rows x 128 bytes
constexpr uint32_t SM_ML = SM_OUT + TILE_BYTES / 2;         // [group][128 rows] (m, l)
constexpr uint32_t SM_BAR = SM_ML + 2 * TILE * 8;

enum Bar : uint32_t {
  Q_FULL0 = 0,  // per group
  Q_EMPTY0 = Q_FULL0 + 2,
  K_FULL0 = Q_EMPTY0 + 2,
  V_FULL0 = K_FULL0 + KV_STAGES,
  // The issuer's step x: the products with V tile x - 1, then those with K tile x.  Completed
  // steps x = 0, 2, .. and x = 1, 3, .. arrive here, so K tile x + 2 may follow step x, and V tile
  // x + 1.
  STEP0 = V_FULL0 + KV_STAGES,
  S_FULL0 = STEP0 + 2,     // per group: S_g of the next kv tile is in TMEM
  P_READY0 = S_FULL0 + 2,  // per group: P_g is in TMEM
  O_FULL0 = P_READY0 + 2,  // per group: O_g holds the unit's last product
  O_EMPTY0 = O_FULL0 + 2,  // per group: O_g and (m, l) have been read
  ML_READY0 = O_EMPTY0 + 2,  // per group: the unit's (m, l) are in shared memory
  V_TAIL = ML_READY0 + 2,
  DRAIN,
  NUM_BARS
};
constexpr uint32_t SM_TMEM_SLOT = SM_BAR + NUM_BARS * 8;
constexpr uint32_t SM_ABORT = SM_TMEM_SLOT + 4;
constexpr uint32_t SMEM_BYTES = SM_ABORT + 4 + 1024;  // + alignment slack
static_assert(KV_STAGES == 2, "two step barriers");
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
  Divisor by_pairs, by_kv_heads, by_batch, by_splits, by_blocks;
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
  int q = p.by_pairs.quotient(w);
  u.tile0 = 2 * (w - q * p.pairs);
  w = q;
  q = p.by_kv_heads.quotient(w);
  u.kh = w - q * p.a.kv_heads;
  u.split = p.by_batch.quotient(q);
  u.b = q - u.split * p.a.batch;
  u.second = u.tile0 + 1 < p.t.tiles;
  u.keys = uniform(visible_keys(p.a.kv_len, u.b, p.a.kv_tokens, p.a.err));
  const int n = (u.keys + TILE - 1) / TILE, per = p.by_splits.quotient(n + p.splits - 1);
  u.t0 = min(u.split * per, n);
  u.t1 = min(u.t0 + per, n);
  return u;
}

// First head and token of tile `tile` of the unit's (batch, key head).
__device__ __forceinline__ void tile_origin(const Params& p, const Unit& u, int tile, int* head,
                                            int* token) {
  const int g = p.by_blocks.quotient(tile);
  *head = u.kh * p.t.share + g * p.t.pack;
  *token = (tile - g * p.t.blocks) * p.t.box;
}

__device__ __forceinline__ int ceil16(int n) { return (n + 15) & ~15; }
__device__ __forceinline__ int ceil64(int n) { return (n + 63) & ~63; }

// max(m, x) over 32 raw scores: two chains of 3-input instructions.
__device__ __forceinline__ float max32(const uint32_t* x, float m) {
  float a = m, b = __uint_as_float(x[0]);
#pragma unroll
  for (int i = 0; i < 30; i += 4) {
    a = max3(a, __uint_as_float(x[i + 1]), __uint_as_float(x[i + 2]));
    b = max3(b, __uint_as_float(x[i + 3]), __uint_as_float(x[(i + 4) & 31]));
  }
  return fmaxf(a, b);
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + SM_ABORT);
  auto bar = [&](uint32_t b) { return base + SM_BAR + 8u * b; };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
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
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they start at 0
  const uint32_t tile_rows_bytes = static_cast<uint32_t>(p.t.box * p.t.pack) * 256u;

  if (warp >= SOFTMAX_WARP && warp < OUT_WARP) {
    // ------------------------------------------------------------------ softmax groups
    const int quarter = warp & 3, g = (warp - SOFTMAX_WARP) >> 2;
    const int r = quarter * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + TM_S + g * 128u, t_o = tmem + lane_off + TM_O + g * 128u;
    // S carries the sign of the scale.  Scale 0: the least positive value, 2^-149, keeps 0 * -inf
    // out of the mask, and the largest finite scores give |s| < 2^-21.
    const float c1 = p.a.sm_scale == 0.f ? __uint_as_float(1u) : fabsf(p.a.sm_scale) * LOG2E_F;
    float2* ml = reinterpret_cast<float2*>(gbase + SM_ML) + g * TILE + r;
    uint32_t sn = 0, on = 0;  // kv tiles and units of this group
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0 || (g == 1 && !u.second)) continue;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < u.count(); ++j) {
        ok = warp_wait(bar(S_FULL0 + g), sn & 1u, abort, limit);
        if (!ok) break;
        ++sn;
        tc_fence_after_sync();
        // Two passes over S in chunks of 32 columns, each chunk's load in flight while the one
        // before is worked on.  The loops stay rolled: unrolled over the 128 columns they took 524
        // us where they now take 400 (131040 x 512, 12 heads), waiting for instructions.
        const int n = u.keys_of(j), cols = ceil64(n);
        if (n < cols) {
#pragma unroll 1
          for (int c = n; c < cols; ++c) tmem_st_32x32b_x1(t_s + c, 0xff800000u);
          tmem_wait_st();
        }
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(t_s, v[0]);
        float mb = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < cols; c += 64) {
          tmem_wait_ld_regs(v[0]);
          tmem_ld_32x32b_x32(t_s + c + 32u, v[1]);
          mb = max32(v[0], mb);
          tmem_wait_ld_regs(v[1]);
          tmem_ld_32x32b_x32(t_s + (c + 64 < cols ? c + 64 : 0), v[0]);  // after the last: the first again
          mb = max32(v[1], mb);
        }
        mb *= c1;
        const bool need = mb > m + RESCALE;
        if (__builtin_expect(__any_sync(0xffffffffu, need), 0)) {
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
        // P of the chunk from column c on goes over columns c / 2 .. c / 2 + 15, which earlier
        // chunks and this one alone cover.
        auto exps = [&](const uint32_t* x, int c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, o2), a0, a1);
            const float p0 = ex2(a0), p1 = ex2(a1);
            acc[i & 1] = f2_add(acc[i & 1], f2_pack(p0, p1));
            pk[i] = pack_bf162(p0, p1);
          }
          tmem_st_32x32b_x16(t_s + c / 2, pk);
        };
#pragma unroll 1
        for (int c = 0; c < cols; c += 64) {
          tmem_wait_ld_regs(v[0]);
          tmem_ld_32x32b_x32(t_s + c + 32u, v[1]);
          exps(v[0], c);
          tmem_wait_ld_regs(v[1]);
          if (c + 64 < cols) tmem_ld_32x32b_x32(t_s + c + 64u, v[0]);
          exps(v[1], c + 32);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(P_READY0 + g));
        float s0, s1;
        f2_unpack(f2_add(acc[0], acc[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      ok = warp_wait(bar(O_EMPTY0 + g), (on & 1u) ^ 1u, abort, limit);  // the last unit's have been read
      if (!ok) break;
      *ml = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ML_READY0 + g));
      ++on;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  } else if (warp >= OUT_WARP) {
    // ------------------------------------------------------------------ output
    // Row r of a tile lies at the same distance from its first row in every tile.
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t t_o = (static_cast<uint32_t>(quarter * 32) << 16) + TM_O;
    const uint32_t stage = base + SM_OUT + quarter * 4096u;  // this warp's 32 rows x 64 columns
    int64_t to[8];  // of rows 4 i + lane / 8 of the warp, and the lane's 8 columns
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = quarter * 32 + i * 4 + (lane >> 3), h = x / p.t.box;
      to[i] = h * p.a.o.head + (x - h * p.t.box) * p.a.o.token + (lane & 7) * 8;
    }
    const int64_t lse_at = static_cast<int64_t>(r / p.t.box) * p.a.q_tokens + r % p.t.box;
    uint32_t on = 0;  // units of each group, a bit each
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
#pragma unroll 1
      for (int g = 0; g < (u.second ? 2 : 1); ++g) {
        int head, token;
        tile_origin(p, u, u.tile0 + g, &head, &token);
        const int rows = p.t.pack > 1 ? p.t.pack * p.t.box : min(p.t.box, p.a.q_tokens - token);
        float* lse = p.a.lse + (static_cast<int64_t>(u.b) * p.a.heads + head) * p.a.q_tokens + token + lse_at;
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.a.o.data) + u.b * p.a.o.batch + head * p.a.o.head +
                           token * p.a.o.token;
        const int64_t part =
            (((static_cast<int64_t>(u.split) * p.a.batch + u.b) * p.a.kv_heads + u.kh) * p.t.tiles + u.tile0 + g) * TILE;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (u.count() > 0) {
          ok = warp_wait(bar(ML_READY0 + g), (on >> g) & 1u, abort, limit) &&
               warp_wait(bar(O_FULL0 + g), (on >> g) & 1u, abort, limit);
          if (!ok) break;
          on ^= 1u << g;
          tc_fence_after_sync();
          ml = reinterpret_cast<const float2*>(gbase + SM_ML)[g * TILE + r];
        }
        if (p.splits > 1) {
          if (r < rows) p.part_ml[part + r] = ml;
#pragma unroll 1
          for (int c = 0; c < TILE && u.count() > 0; c += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(t_o + g * 128u + c, v);
            tmem_wait_ld();
            float* po = p.part_o + (part + c) * TILE + r;
            if (r < rows) {
#pragma unroll
              for (int i = 0; i < 16; ++i) po[i * TILE] = __uint_as_float(v[i]);
            }
          }
        } else {
          if (r < rows) *lse = ml.x + log2f(ml.y);
          const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
          const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {  // column halves of 64, through the warp's staging rows
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              if (u.count() > 0) {
                tmem_ld_32x32b_x32(t_o + g * 128u + h * 64u + c * 32u, v);
                tmem_wait_ld();
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0u;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t pk[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  float a0, a1;
                  f2_unpack(f2_mul(f2_pack(__uint_as_float(v[8 * i + 2 * x]), __uint_as_float(v[8 * i + 2 * x + 1])), inv2),
                            a0, a1);
                  pk[x] = pack_bf162(a0, a1);
                }
                st_shared16(stage + swizzled(lane, c * 4 + i), pk[0], pk[1], pk[2], pk[3]);
              }
            }
            __syncwarp();
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = ld_shared16(stage + swizzled(i * 4 + (lane >> 3), lane & 7));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i)  // four rows of 128 bytes at a time
              if (quarter * 32 + i * 4 + (lane >> 3) < rows) *reinterpret_cast<uint4*>(o + to[i] + h * 64) = x[i];
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0 && u.count() > 0) mbar_arrive(bar(O_EMPTY0 + g));
      }
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  } else {
    if (warp == TMA_WARP) {
      // ------------------------------------------------------------------ TMA producer: Q, K
      uint32_t qn = 0, begun = 0, kn = 0;  // per group (a bit each): parity of the Q tiles, any; K tiles
      bool ok = true;
      const int halves = p.t.box * p.t.pack == TILE ? 1 : 2;  // copies of a Q tile
      for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
        const Unit u = decode(p, w);
        const int n = u.count();
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const uint32_t s = kn & 1u;
          ok = warp_wait(bar(STEP0 + s), ((kn >> 1) & 1u) ^ 1u, abort, limit);  // step kn - 2
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(K_FULL0 + s), TILE_BYTES);
            tma_load_5d(base + SM_K + s * TILE_BYTES, &tm_k, bar(K_FULL0 + s), 0, (u.t0 + j) * TILE, u.kh, 0,
                        p.a.k.batch ? u.b : 0);
          }
          __syncwarp();
          ++kn;
          if (j > 0) continue;
#pragma unroll 1
          for (int g = 0; g < (u.second ? 2 : 1); ++g) {
            ok = warp_wait(bar(Q_EMPTY0 + g), ((qn >> g) & 1u) ^ 1u, abort, limit);
            if (!ok) break;
            qn ^= 1u << g;
            begun |= 1u << g;
            int head, token;
            tile_origin(p, u, u.tile0 + g, &head, &token);
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(Q_FULL0 + g), tile_rows_bytes);
#pragma unroll 1
              for (int h = 0; h < halves; ++h)
                tma_load_5d(base + SM_Q + g * TILE_BYTES + h * (TILE_BYTES / 2), &tm_q, bar(Q_FULL0 + g), 0, token,
                            head, h, p.a.q.batch ? u.b : 0);
            }
            __syncwarp();
          }
          if (!ok) break;
        }
      }
      if (!ok && lane == 0) {
        raise_abort(abort, p.a.err);
        // Let the copies already issued land before the CTA's shared memory goes away.
        drain_copies(bar(K_FULL0), KV_STAGES, kn);
        if (begun & 1u) drain_copies(bar(Q_FULL0), 1, (qn & 1u) ? 1 : 2);
        if (begun & 2u) drain_copies(bar(Q_FULL0 + 1), 1, (qn & 2u) ? 1 : 2);
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
          if (vn >= KV_STAGES) ok = warp_wait(bar(STEP0 + ((vn - 1) & 1u)), ((vn - 1) >> 1) & 1u, abort, limit);
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
            ok = warp_wait(full, (tails - 1) & 1u, abort, limit);
            if (!ok) break;
            tails_seen = tails;
            zero_rows(tile, n, ceil64(n), lane);
            if (lane == 0) mbar_arrive(bar(V_FULL0 + s));
          }
          ++vn;
        }
      }
      if (!ok && lane == 0) {
        raise_abort(abort, p.a.err);
        if (tails > tails_seen) drain_copies(bar(V_TAIL), 1, tails);
        drain_copies(bar(V_FULL0), KV_STAGES, vn);
      }
      __syncwarp();
    } else if (warp == MMA_WARP) {
      // ------------------------------------------------------------------ UMMA issuer
      // The whole warp runs this role in lockstep; one elected lane issues.
      uint32_t x = 0;                    // step: K tile x, V tile x - 1
      uint32_t qn = 0, pn = 0, on = 0;   // parity of Q tiles, kv tiles and units, a bit per group
      bool ok = true, issued = false;
      // The products are negated (of A, bit 13) where the scale is negative.
      const uint32_t idesc_s = IDESC_S0 | (p.a.sm_scale < 0.f ? 1u << 13 : 0u);
      const uint64_t q_desc = sdesc_sw128(base + SM_Q, 16, 1024);
      const uint64_t k_desc = sdesc_sw128(base + SM_K, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(base + SM_V, TILE_BYTES / 2, 1024);
      // Step x: per group, O_g += P_g V with the kv tile of step x - 1 (pj of unit pu), then S_g of
      // the step's own (j of unit u).  One copy of the code for both groups and all steps: the
      // roles' code has to share the instruction caches, and with a copy per case this warp
      // waited for its instructions longer than the tensor core for it.
      Unit u{}, pu{};
      int w = static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x), j = 0, pj = 0;
      bool pv = false;  // P V of this step; S: unless w is past the last unit
      while (true) {
        if (j == u.count()) {  // to the next unit with keys
          j = 0;
#pragma unroll 1
          for (w += gridDim.x; w < p.total; w += gridDim.x) {
            u = decode(p, w);
            if (u.count() > 0) break;
          }
        }
        const bool s = w < p.total;
        if (!s && !pv) break;
        const uint32_t vx = x - 1;
        const int pkeys = pv ? pu.keys_of(pj) : 0;
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          if (pv && (g == 0 || pu.second)) {
            ok = warp_wait(bar(P_READY0 + g), (pn >> g) & 1u, abort, limit) &&
                 (g != 0 || warp_wait(bar(V_FULL0 + (vx & 1u)), (vx >> 1) & 1u, abort, limit)) &&
                 (pj != 0 || warp_wait(bar(O_EMPTY0 + g), ((on >> g) & 1u) ^ 1u, abort, limit));
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t vd = sdesc_advance(v_desc, (vx & 1u) * TILE_BYTES);
#pragma unroll 1
            for (int h = 0; h * 64 < pkeys; ++h)
              product_ts64<16>(tmem + TM_O + g * 128u, tmem + TM_S + g * 128u + h * 32u, sdesc_advance(vd, h * 8192u), IDESC_PV,
                           static_cast<uint32_t>(pj | h));
            pn ^= 1u << g;
            if (pj + 1 == pu.count()) {
              umma_commit_elect(bar(O_FULL0 + g));
              on ^= 1u << g;
            }
          }
          if (s && (g == 0 || u.second)) {
            ok = (g != 0 || warp_wait(bar(K_FULL0 + (x & 1u)), (x >> 1) & 1u, abort, limit)) &&
                 (j != 0 || warp_wait(bar(Q_FULL0 + g), (qn >> g) & 1u, abort, limit));
            if (!ok) break;
            tc_fence_after_sync();
            product_ss(tmem + TM_S + g * 128u, sdesc_advance(q_desc, g * TILE_BYTES),
                       sdesc_advance(k_desc, (x & 1u) * TILE_BYTES),
                       idesc_s | (static_cast<uint32_t>(ceil16(u.keys_of(j)) >> 3) << 17));
            umma_commit_elect(bar(S_FULL0 + g));
            if (j == 0) qn ^= 1u << g;
            if (j + 1 == u.count()) umma_commit_elect(bar(Q_EMPTY0 + g));
            issued = true;
          }
        }
        if (!ok) break;
        umma_commit_elect(bar(STEP0 + (x & 1u)));
        ++x;
        pv = s;
        pu = u;
        pj = j++;
        if (!s) break;
      }
      if (!ok && lane == 0) raise_abort(abort, p.a.err);
      if (issued) {
        // Every UMMA has completed before TMEM is released.
        umma_commit_elect(bar(DRAIN));
        volatile int never = 0;
        if (lane == 0) mbar_wait_bounded(bar(DRAIN), 0, &never, DRAIN_LIMIT_NS);
        __syncwarp();
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == TMA_WARP) tmem_dealloc(tmem, 512);
}

constexpr int JOIN_THREADS = 512;

// Threads for the rows of a tile, and groups of them for `splits` parts: one for up to 12 parts
// (three waits for loads), else as many as have 6 to 12 each.
__host__ __device__ inline int join_width(const QTiles& t) {
  const int rows = t.box * t.pack;
  return rows > 64 ? 128 : rows > 32 ? 64 : 32;
}
inline int join_threads(const QTiles& t, int splits) {
  int n = join_width(t);
  while (n < JOIN_THREADS && n * 12 < splits * join_width(t)) n *= 2;
  return n;
}

// Joins the parts of the keys: a CTA has 8 columns of a tile's rows.  Its threads are groups of as
// many as the tile has rows (in 32, 64 or 128); group g takes parts g, g + groups, .., four parts'
// loads at a time, and the groups are joined in shared memory in group order.  A part without a
// visible key (l = 0) is not read.  (The latency of the loads is what counts: with all parts of a
// row in one thread a single token of 8 heads on 32768 keys, 64 parts, took 8 us longer.)
__global__ void __launch_bounds__(JOIN_THREADS) cross_combine_kernel(const __grid_constant__ Params p) {
  __shared__ float sh_o[8][JOIN_THREADS];
  __shared__ float2 sh_ml[JOIN_THREADS];
  grid_dependency_wait();
  const int width = join_width(p.t), groups = blockDim.x / width;
  const int tile = blockIdx.x, r = threadIdx.x & (width - 1), g = threadIdx.x / width, c0 = blockIdx.y * 8;
  const int tiles = p.a.batch * p.a.kv_heads * p.t.tiles;
  const int x = tile % p.t.tiles, bk = tile / p.t.tiles, b = bk / p.a.kv_heads, kh = bk % p.a.kv_heads;
  const int rh = r / p.t.box;
  const int head = kh * p.t.share + x / p.t.blocks * p.t.pack + rh;
  const int token = x % p.t.blocks * p.t.box + r - rh * p.t.box;
  const bool valid = rh < p.t.pack && token < p.a.q_tokens;
  const float2* part_ml = p.part_ml + static_cast<int64_t>(tile) * TILE + r;
  const float* part_o = p.part_o + (static_cast<int64_t>(tile) * TILE + c0) * TILE + r;
  const int64_t step = static_cast<int64_t>(tiles) * TILE;
  float m = -INFINITY, l = 0.f, o[8] = {};
#pragma unroll 1
  for (int s0 = g; s0 < p.splits && valid; s0 += 4 * groups) {
    float y[4][8];
    float2 ml[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + k * groups;
      ml[k] = s < p.splits ? part_ml[s * step] : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[k][i] = ml[k].y == 0.f ? 0.f : part_o[(s0 + k * groups) * step * TILE + i * TILE];
    float mn = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) mn = fmaxf(mn, ml[k].x);
    const float ref = mn == -INFINITY ? 0.f : mn, f = ex2(m - ref);
    m = mn;
    l *= f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float w = ml[k].y == 0.f ? 0.f : ex2(ml[k].x - ref);  // NaN is kept
      l = fmaf(ml[k].y, w, l);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(y[k][i], w, o[i]);
    }
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.o.data) + b * p.a.o.batch + head * p.a.o.head +
                       token * p.a.o.token + c0;
  float* lse = p.a.lse + (static_cast<int64_t>(b) * p.a.heads + head) * p.a.q_tokens + token;
  if (groups == 1) {
    if (!valid) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf162(o[0] * inv, o[1] * inv), pack_bf162(o[2] * inv, o[3] * inv),
                                                pack_bf162(o[4] * inv, o[5] * inv), pack_bf162(o[6] * inv, o[7] * inv));
    if (c0 == 0) *lse = m + log2f(l);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sh_o[i][threadIdx.x] = o[i];
  sh_ml[threadIdx.x] = make_float2(m, l);
  __syncthreads();
  if (!valid) return;
  for (int i = g; i < 8; i += groups) {
    m = -INFINITY, l = 0.f;
    float sum = 0.f;
    for (int k = 0; k < groups; ++k) {
      const float2 ml = sh_ml[k * width + r];
      if (ml.y == 0.f) continue;
      float f, w;
      join(m, l, ml.x, ml.y, &f, &w);
      sum = sum * f + sh_o[i][k * width + r] * w;
    }
    out[i] = __float2bfloat16_rn(l == 0.f ? 0.f : sum / l);
    if (c0 + i == 0) *lse = m + log2f(l);
  }
}

struct Plan {
  QTiles t;
  int pairs, splits;
  size_t ml_off, total;  // workspace
};

// Parts of the keys: as many as give every SM at most one, down to a kv tile each (parts of at least
// two: 8 x 12 heads of 4 rows, 512 keys 10.9 instead of 9.9 us; 2 x 8 heads, 64 queries on 8191 keys
// 22.7 instead of 21.9).  From 77 units on that is one part, and up to half of the SMs have nothing to
// do: 2 x 8 heads, 1280 queries on 20000 keys are 80 units of 157 kv tiles and take 229 us, 48 % of the
// measured rate.  (Parts in several waves, weighed as cross_bwd.cu weighs its own, are not built here.)
Plan plan_of(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens) {
  Plan p{};
  p.t = q_tiles(heads, kv_heads, q_tokens);
  p.pairs = (p.t.tiles + 1) / 2;
  const int64_t units = static_cast<int64_t>(batch) * kv_heads * p.pairs;
  const int64_t kv_tiles = (kv_tokens + TILE - 1) / TILE;
  int64_t s = device_sm_count() / units;
  if (s > kv_tiles) s = kv_tiles;
  if (s > 1) {
    const int64_t per = (kv_tiles + s - 1) / s;
    s = (kv_tiles + per - 1) / per;  // no part without a tile
  }
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
  if (use_cross_token(heads, kv_heads, q_tokens))
    return cross_token_workspace(batch, heads, kv_heads, q_tokens, kv_tokens);
  return plan_of(batch, heads, kv_heads, q_tokens, kv_tokens).total;
}

cudaError_t launch_cross_fwd(const CrossArgs& a, cudaStream_t stream) {
  if (use_cross_token(a.heads, a.kv_heads, a.q_tokens)) return launch_cross_token(a, stream);
  const Plan plan = plan_of(a.batch, a.heads, a.kv_heads, a.q_tokens, a.kv_tokens);
  Params p{};
  p.a = a;
  p.t = plan.t;
  p.pairs = plan.pairs;
  p.splits = plan.splits;
  p.total = a.batch * a.kv_heads * plan.pairs * plan.splits;
  p.by_pairs = make_divisor(p.pairs);
  p.by_kv_heads = make_divisor(a.kv_heads);
  p.by_batch = make_divisor(a.batch);
  p.by_splits = make_divisor(p.splits);
  p.by_blocks = make_divisor(p.t.blocks);
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
  return launch_dependent(cross_combine_kernel, dim3(a.batch * a.kv_heads * p.t.tiles, 16), dim3(join_threads(p.t, p.splits)), 0,
                          stream, p);
}

}  // namespace vsa
