// cross_bwd.cu -- attention to an encoder's states of another length, backward.  With
//   P = 2^(q k^T sm_scale log2e - lse),  Delta = rowsum(O dO),  dS = P (dO v^T - Delta):
//   dQ = sm_scale dS k,  dV = P^T dO,  dK = sm_scale dS^T q.
//
// Two passes, each of which keeps its sums in tensor memory, so that nothing is added through
// global memory and the result does not depend on an order of arrival:
//   cross_dq_kernel   a 128-row query tile per CTA, over the kv tiles: S, dP, dQ += dS K
//                     (3 products); it also leaves Delta for the second pass;
//   cross_dkv_kernel  a 128-key kv tile per CTA, over the query tiles of every head that shares
//                     its key head: S^T, dP^T, dV += P^T dO, dK += dS^T Q (4 products).
// Together 7 products of 2 x 128 x 128 x 128 per tile pair, where one pass that adds its dQ parts
// through global memory has 5: for a few kv tiles (text) those fp32 parts would be as many bytes
// as all operands together, read and written once per kv tile.
//
// P and dS are rounded to bf16 as operands (kind::f16 takes one type for both operands, and q, k,
// dO are the caller's bf16); dS itself is computed from the unrounded P.
//
// Where the tiles are fewer than the SMs, the inner axis is split over CTAs (dq: the kv tiles,
// dkv: the query tiles): each part leaves fp32 sums in the workspace, and join kernels add them in
// part order (2 x 8 heads, 64 queries on 8191 keys: 52 us, without parts 103; 2 x 32 heads on 4 key
// heads, 16 queries: 38 us, without parts 94, without packing the heads that share keys 91).
//
// Measured: 32760 queries on 512 keys, 12 heads: 249 us in short bursts (1.03 PFLOP/s of the five
// products that the formulas have, 1.45 of the seven that are done), 267 to 276 us in a long run under
// the power cap; dQ 132 us, dK and dV 114 us, the join 7 us.
// What bounds dQ (tensor pipe 49 % active): an SM takes copies in at 34 to 45 bytes a cycle, and a
// step's 64 KB of K and V with its share of a unit's Q, dO and O are 2000 to 2500 cycles against
// 1554 of products; and its softmax warps are as long as its products (about 1580 cycles a step).
// Tried without gain: K and V multicast to pairs of CTAs (137 us), fewer and larger hand-overs
// (139), S, dQ, dP in this order, which frees a K tile earlier (148).
// What bounds dK and dV (tensor pipe 76 % active): the four products, and copies of 64 KB a step.
// Of the whole 249 us, leaving out dQ's exponentials or dK's and dV's saves nothing, dQ's output
// stores or its reads of O 5 us each, half of the dQ product 5 to 10.
#include "cross_common.cuh"

namespace vsa {

namespace {

// Warps: 0 TMEM owner and TMA producer, 1 UMMA issuer, 2 a second producer, 3 idle, 4-19 softmax;
// dq has 20-27 for what belongs to a unit and not to a step.  Softmax warp (quarter, col) has rows
// 32 quarter .. + 31 of a tile of scores, one per lane, and columns 32 col .. + 31.
constexpr int SOFTMAX_WARP = 4, SOFTMAX_WARPS = 16;
constexpr uint32_t IDESC_S0 = idesc_f16_f32acc(128, 0, false, false, true);  // N is added
constexpr uint32_t IDESC_ACC = idesc_f16_f32acc(128, 128, false, true, true);

__device__ __forceinline__ int ceil64(int n) { return (n + 63) & ~63; }
__device__ __forceinline__ uint32_t idesc_s(int n) { return IDESC_S0 | (static_cast<uint32_t>(n >> 3) << 17); }

struct Params {
  CrossArgs a;
  QTiles t;
  int kv_tiles;  // of kv_tokens
  int splits;    // parts of the inner axis
  int total;     // units
  Divisor by_tiles, by_kv_tiles, by_kv_heads, by_batch, by_splits, by_blocks, by_box;
  float* delta;  // [batch, heads, q_tokens]
  float* part;   // dq: [split][batch * kv_heads * tiles][128 columns][128 rows];
                 // dkv: [split][batch * kv_heads * kv_tiles][dV, dK][128 columns][128 keys]
};

__device__ __forceinline__ void load32(uint32_t taddr, uint32_t* v) {
  tmem_ld_32x32b_x32(taddr, v);
  tmem_wait_ld();
}
// Columns from n on of a thread's 32 become 0.
__device__ __forceinline__ void keep_columns(uint32_t* v, int n) {
  if (__builtin_expect(n < 32, 0)) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < n ? v[i] : 0u;
  }
}

// A dkv softmax warp's 32 rows x 32 columns of sums, scaled and rounded, to global memory: through 2
// KB of shared memory, so that 64 consecutive bytes of a row leave together.  `at`: distance of
// rows 8 i + lane / 4 from `out`, in elements; rows from `rows` on are not written.
__device__ __forceinline__ void write_rows(uint32_t stage, const uint32_t* v, float scale, __nv_bfloat16* out,
                                           const int64_t* at, int rows, int lane) {
  const uint64_t s2 = f2_pack(scale, scale);
  const uint32_t row = stage + lane * 64u, x = (lane >> 1) & 3u;  // chunks of 16 bytes, swizzled by row
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t pk[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a0, a1;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(v[8 * i + 2 * k]), __uint_as_float(v[8 * i + 2 * k + 1])), s2), a0, a1);
      pk[k] = pack_bf162(a0, a1);
    }
    st_shared16(row + ((i ^ x) << 4), pk[0], pk[1], pk[2], pk[3]);
  }
  __syncwarp();
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t rr = i * 8 + (lane >> 2);
    w[i] = ld_shared16(stage + rr * 64u + (((lane & 3u) ^ ((rr >> 1) & 3u)) << 4));
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i * 8 + (lane >> 2) < rows) reinterpret_cast<uint4*>(out + at[i])[lane & 3] = w[i];
}

// First head and token of a query tile, and how many rows it has (fewer in the last block of a
// head's tokens).
__device__ __forceinline__ void tile_origin(const Params& p, int kh, int tile, int* head, int* token) {
  const int g = p.by_blocks.quotient(tile);
  *head = kh * p.t.share + g * p.t.pack;
  *token = (tile - g * p.t.blocks) * p.t.box;
}
__device__ __forceinline__ int tile_rows(const Params& p, int token) {
  return p.t.pack > 1 ? p.t.pack * p.t.box : min(p.t.box, p.a.q_tokens - token);
}

// Row (head, token) of row r of a query tile, and whether it exists.
struct QRow {
  int head, token;
  bool valid;
};
__device__ __forceinline__ QRow q_row(const Params& p, int kh, int tile, int r) {
  const int g = tile / p.t.blocks, rh = r / p.t.box;
  QRow x;
  x.head = kh * p.t.share + g * p.t.pack + rh;
  x.token = (tile - g * p.t.blocks) * p.t.box + r - rh * p.t.box;
  x.valid = rh < p.t.pack && x.token < p.a.q_tokens;
  return x;
}

// Lane i of four neighbours has chunks 0 .. 3 of row i (chunk k: v[4 k] .. v[4 k + 3]) and gets chunk
// i of rows 0 .. 3.
__device__ __forceinline__ void transpose4(uint32_t* v, int lane) {
#pragma unroll
  for (int m = 1; m <= 2; m *= 2) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & m) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t& lo = v[4 * k + i];
        uint32_t& hi = v[4 * (k + m) + i];
        const uint32_t t = __shfl_xor_sync(0xffffffffu, up ? lo : hi, m);
        lo = up ? t : lo;
        hi = up ? hi : t;
      }
    }
  }
}

// s += the parts' 8 columns of a row, in part order; four parts' loads at a time.
__device__ __forceinline__ void add_parts(float* s, const float* part, int64_t stride, int parts) {
#pragma unroll 1
  for (int x = 0; x < parts; x += 4) {
    float t[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k][i] = x + k < parts ? part[(x + k) * stride + i * TILE] : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += t[k][i];
  }
}

// One query-side tile into shared memory, by one thread.
__device__ __forceinline__ void load_q_tile(const Params& p, const CUtensorMap* map, int64_t batch_stride, uint32_t dst,
                                            uint32_t full, int b, int head, int token) {
  const int rows = p.t.box * p.t.pack;
  mbar_arrive_expect_tx(full, static_cast<uint32_t>(rows) * 256u);
#pragma unroll 1
  for (int h = 0; h < (rows == TILE ? 1 : 2); ++h)
    tma_load_5d(dst + h * (TILE_BYTES / 2), map, full, 0, token, head, h, batch_stride ? b : 0);
}

// ================================================================================== dQ

namespace dq {

// K tiles are held from S to dQ of the same step, with the next step's S and dP in between, so
// three of them.  (With one V tile, its way from L2, 2000 cycles when all SMs load, set the pace.)
constexpr int K_STAGES = 3, V_STAGES = 2;
constexpr uint32_t SM_Q = 0, SM_DO = TILE_BYTES, SM_K = 2 * TILE_BYTES, SM_V = SM_K + K_STAGES * TILE_BYTES;
constexpr uint32_t SM_LSE = SM_V + V_STAGES * TILE_BYTES;  // [unit parity][128 rows] -lse, -Delta
constexpr uint32_t SM_DELTA = SM_LSE + 2 * TILE * 4;
constexpr uint32_t SM_BAR = SM_DELTA + 2 * TILE * 4;
constexpr int NUM_THREADS = 896, AUX_WARP = 20;
enum Bar : uint32_t {
  Q_FULL = 0,
  Q_EMPTY,
  DO_FULL,
  DO_EMPTY,  // the tensor core and the 8 warps that sum O dO
  K_FULL0,
  K_EMPTY0 = K_FULL0 + K_STAGES,
  V_FULL0 = K_EMPTY0 + K_STAGES,
  V_EMPTY0 = V_FULL0 + V_STAGES,
  S_FULL = V_EMPTY0 + V_STAGES,
  S_FREE,  // S has been read
  DP_FULL,
  DP_FREE,
  DS_READY0,  // two buffers
  DQ_FULL = DS_READY0 + 2,
  DQ_EMPTY,
  // One for even and one for odd units: a warp that fills may be a unit ahead of another that fills
  // or of one that waits, and two phases ahead of neither.
  LSE_FULL0,
  DELTA_FULL0 = LSE_FULL0 + 2,
  K_TAIL = DELTA_FULL0 + 2,
  DRAIN,
  NUM_BARS
};
constexpr uint32_t SM_TMEM_SLOT = SM_BAR + NUM_BARS * 8;
constexpr uint32_t SM_ABORT = SM_TMEM_SLOT + 4;
constexpr uint32_t SMEM_BYTES = SM_ABORT + 4;
static_assert(V_STAGES == 2, "stage = step & 1");
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DQ = 256, TM_DS = 384;  // dS: two buffers of 64 columns

struct Unit {
  int b, kh, tile, split, t0, t1, keys;
  __device__ __forceinline__ int count() const { return t1 - t0; }
  __device__ __forceinline__ int keys_of(int j) const { return min(TILE, keys - (t0 + j) * TILE); }
};

__device__ __forceinline__ Unit decode(const Params& p, int w) {
  Unit u;
  int q = p.by_tiles.quotient(w);
  u.tile = w - q * p.t.tiles;
  w = q;
  q = p.by_kv_heads.quotient(w);
  u.kh = w - q * p.a.kv_heads;
  u.split = p.by_batch.quotient(q);
  u.b = q - u.split * p.a.batch;
  u.keys = uniform(visible_keys(p.a.kv_len, u.b, p.a.kv_tokens, p.a.err));
  const int n = (u.keys + TILE - 1) / TILE, per = p.by_splits.quotient(n + p.splits - 1);
  u.t0 = min(u.split * per, n);
  u.t1 = min(u.t0 + per, n);
  return u;
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + SM_ABORT);
  auto bar = [&](uint32_t b) { return base + SM_BAR + 8u * b; };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint64_t limit = p.a.wait_ns;

  if (threadIdx.x == 0) {
    *abort = 0;
    for (uint32_t b = 0; b < NUM_BARS; ++b) {
      uint32_t count = 1;
      if (b == S_FREE || b == DP_FREE || b == DS_READY0 || b == DS_READY0 + 1) count = SOFTMAX_WARPS;
      if (b == DO_EMPTY) count = 9;
      if (b == DQ_EMPTY || b == DELTA_FULL0 || b == DELTA_FULL0 + 1) count = 8;
      if (b == LSE_FULL0 || b == LSE_FULL0 + 1) count = 4;
      mbar_init(bar(b), count);
    }
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(base + SM_TMEM_SLOT, 512);
    tmem_relinquish();
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_do);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  grid_dependency_wait();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they start at 0

  if (warp >= AUX_WARP) {
    // ------------------------------------------------------------------ lse, Delta, output
    // Off the softmax warps' path: a unit's -lse and -Delta are there before its first dS, and its
    // dQ leaves while the next unit is under way, straight from registers (shared memory has no
    // room left).
    const int quarter = warp & 3, half = (warp - AUX_WARP) >> 2, r = quarter * 32 + lane;
    const uint32_t t_dq = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TM_DQ + half * 64u;
    const int rh = r / p.t.box, rt = r - rh * p.t.box;
    int64_t at[4];  // of the four rows that the lane writes, and its 8 columns
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int y = (r & ~3) + i, h = p.by_box.quotient(y);
      at[i] = h * p.a.dq.head + (y - h * p.t.box) * p.a.dq.token + half * 64 + (lane & 3) * 8;
    }
    uint32_t un = 0;
    bool ok = true;
    Unit u{}, prev{};
    bool pending = false;  // dQ of `prev` is to be written
    for (int w = blockIdx.x; ok; w += gridDim.x) {
      const bool more = w < p.total;
      if (more) u = decode(p, w);
      const bool now = more && u.count() > 0;
      if (now) {
        int head, token;
        tile_origin(p, u.kh, u.tile, &head, &token);
        const int rows = tile_rows(p, token);
        const int64_t row = (static_cast<int64_t>(u.b) * p.a.heads + head) * p.a.q_tokens + token;
        // The buffers' last readers are done: dQ of the unit before the last has been put out.
        float* to_lse = reinterpret_cast<float*>(smem + SM_LSE) + (un & 1u) * TILE;
        float* to_delta = reinterpret_cast<float*>(smem + SM_DELTA) + (un & 1u) * TILE;
        // Delta of 16 rows a warp: four at a time, 8 lanes a row, 8 columns of each half a lane.
        const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(p.a.o.data) + u.b * p.a.o.batch +
                                 head * p.a.o.head + token * p.a.o.token + (lane & 7) * 8;
        const int y0 = quarter * 32 + half * 16 + (lane >> 3);
        uint4 ov[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int y = y0 + i * 4, h = p.by_box.quotient(y);
          const uint4* from = reinterpret_cast<const uint4*>(o + h * p.a.o.head + (y - h * p.t.box) * p.a.o.token);
          ov[2 * i] = y < rows ? from[0] : make_uint4(0u, 0u, 0u, 0u);
          ov[2 * i + 1] = y < rows ? from[8] : make_uint4(0u, 0u, 0u, 0u);
        }
        if (half == 0) {
          const float lse = r < rows ? p.a.lse[row + static_cast<int64_t>(rh) * p.a.q_tokens + rt] : 0.f;
          to_lse[r] = lse == -INFINITY ? 0.f : -lse;  // all scores -inf: P = 2^-inf = 0
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(LSE_FULL0 + (un & 1u)));
        }
        ok = warp_wait(bar(DO_FULL), un & 1u, abort, limit);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int y = y0 + i * 4;
          float s = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 d = ld_shared16(base + SM_DO + h * (TILE_BYTES / 2) + swizzled(y, lane & 7));
            const uint4 x = ov[2 * i + h];
            const uint32_t ow[4] = {x.x, x.y, x.z, x.w}, dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s = fmaf(__uint_as_float(ow[e] << 16), __uint_as_float(dw[e] << 16), s);
              s = fmaf(__uint_as_float(ow[e] & 0xffff0000u), __uint_as_float(dw[e] & 0xffff0000u), s);
            }
          }
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          s += __shfl_xor_sync(0xffffffffu, s, 4);
          if ((lane & 7) == 0) {
            to_delta[y] = -s;
            const int h = p.by_box.quotient(y);
            if (y < rows && u.t0 == 0) p.delta[row + static_cast<int64_t>(h) * p.a.q_tokens + y - h * p.t.box] = s;
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(DELTA_FULL0 + (un & 1u)));
          mbar_arrive(bar(DO_EMPTY));
        }
        ++un;
      }
      if (pending && (prev.count() > 0 || p.splits == 1)) {  // (split: the join kernel writes zeros)
        int head, token;
        tile_origin(p, prev.kh, prev.tile, &head, &token);
        const int rows = tile_rows(p, token);
        const bool any = prev.count() > 0;
        if (any) {
          ok = warp_wait(bar(DQ_FULL), (un - 1 - (now ? 1 : 0)) & 1u, abort, limit);
          if (!ok) break;
          tc_fence_after_sync();
        }
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.dq.data) + prev.b * p.a.dq.batch + head * p.a.dq.head +
                             token * p.a.dq.token;
        const int64_t part =
            ((static_cast<int64_t>(prev.split) * p.a.batch + prev.b) * p.a.kv_heads + prev.kh) * p.t.tiles + prev.tile;
        const float scale = any ? p.a.sm_scale : 1.f;
        const uint64_t s2 = f2_pack(scale, scale);
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          uint32_t v[32];
          if (any) {
            load32(t_dq + c, v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          if (p.splits > 1) {
            float* to = p.part + (part * TILE + half * 64 + c) * TILE + r;
            if (r < rows) {
#pragma unroll
              for (int i = 0; i < 32; ++i) to[i * TILE] = __uint_as_float(v[i]);
            }
            continue;
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a0, a1;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s2), a0, a1);
            pk[i] = pack_bf162(a0, a1);
          }
          // Four lanes turn their four rows of four 16-byte chunks over, so that each writes the
          // same chunk of all four: 64 bytes of a row in one piece (16 bytes of 32 rows at a time
          // took the load-store unit 4000 cycles a tile).
          transpose4(pk, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((r & ~3) + i < rows)
              *reinterpret_cast<uint4*>(out + at[i] + c) = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        }
        if (any) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(DQ_EMPTY));
        }
      }
      if (!more) break;
      prev = u;
      pending = true;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  } else if (warp >= SOFTMAX_WARP) {
    // ------------------------------------------------------------------ P, dS
    const int quarter = warp & 3, col = (warp - SOFTMAX_WARP) >> 2, r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t t_s = lanes + TM_S + col * 32u, t_dp = lanes + TM_DP + col * 32u, t_ds = lanes + TM_DS + col * 16u;
    const float c1 = p.a.sm_scale * LOG2E_F;
    const uint64_t c2 = f2_pack(c1, c1);
    uint32_t x = 0, un = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      const int n = u.count();
      if (n == 0) continue;
      ok = warp_wait(bar(LSE_FULL0 + (un & 1u)), (un >> 1) & 1u, abort, limit);
      if (!ok) break;
      const float nl = reinterpret_cast<const float*>(smem + SM_LSE)[(un & 1u) * TILE + r];
      float nd = 0.f;
      const uint64_t nl2 = f2_pack(nl, nl);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        ok = warp_wait(bar(S_FULL), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t v[32];
        load32(t_s, v);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S_FREE));
        float pr[32];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float a0, a1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2, nl2), a0, a1);
          pr[i] = ex2(a0);
          pr[i + 1] = ex2(a1);
        }
        if (j == 0) {
          ok = warp_wait(bar(DELTA_FULL0 + (un & 1u)), (un >> 1) & 1u, abort, limit);
          if (!ok) break;
          nd = reinterpret_cast<const float*>(smem + SM_DELTA)[(un & 1u) * TILE + r];
        }
        const uint64_t nd2 = f2_pack(nd, nd);
        ok = warp_wait(bar(DP_FULL), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t pk[16];
        load32(t_dp, v);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(DP_FREE));
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float a0, a1;
          f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), nd2),
                           f2_pack(pr[i], pr[i + 1])),
                    a0, a1);
          pk[i >> 1] = pack_bf162(a0, a1);
        }
        const int c = u.keys_of(j) - col * 32;  // columns of the warp that are visible
        if (__builtin_expect(c < 32, 0)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 2 * i + 1 < c ? pk[i] : 2 * i < c ? pk[i] & 0xffffu : 0u;
        }
        // The buffer's last reader, dQ of two steps ago, was issued before this dP.
        tmem_st_32x32b_x16(t_ds + (x & 1u) * 64u, pk);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(DS_READY0 + (x & 1u)));
        ++x;
      }
      ++un;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer: Q, dO, V
    uint32_t un = 0, vn = 0;
    bool ok = true, half = false;  // half: Q of a unit is loaded, its dO not
    Unit u{}, next{};
    for (int w = blockIdx.x; ok; w += gridDim.x) {  // unit u, and the one after it
      u = next;
      next = w < p.total ? decode(p, w) : Unit{};
      const int n = u.count();
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if (j == 0) {
          int head, token;
          tile_origin(p, u.kh, u.tile, &head, &token);
          ok = warp_wait(bar(Q_EMPTY), (un & 1u) ^ 1u, abort, limit);
          if (!ok) break;
          if (lane == 0) load_q_tile(p, &tm_q, p.a.q.batch, base + SM_Q, bar(Q_FULL), u.b, head, token);
          __syncwarp();
          half = true;
          ok = warp_wait(bar(DO_EMPTY), (un & 1u) ^ 1u, abort, limit);
          if (!ok) break;
          if (lane == 0) load_q_tile(p, &tm_do, p.a.dout.batch, base + SM_DO, bar(DO_FULL), u.b, head, token);
          __syncwarp();
          half = false;
          ++un;
          if (next.count() > 0 && lane == 0) {  // the next unit's tiles, into L2 (8 us of 254 at 32760 x 512)
            tile_origin(p, next.kh, next.tile, &head, &token);
#pragma unroll 1
            for (int h = 0; h < (p.t.box * p.t.pack == TILE ? 1 : 2); ++h) {
              tma_prefetch_5d(&tm_q, 0, token, head, h, p.a.q.batch ? next.b : 0);
              tma_prefetch_5d(&tm_do, 0, token, head, h, p.a.dout.batch ? next.b : 0);
              tma_prefetch_5d(&tm_o, 0, token, head, h, p.a.o.batch ? next.b : 0);
            }
          }
          __syncwarp();
        }
        const uint32_t s = vn & 1u;
        ok = warp_wait(bar(V_EMPTY0 + s), ((vn >> 1) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(V_FULL0 + s), TILE_BYTES);
          tma_load_5d(base + SM_V + s * TILE_BYTES, &tm_v, bar(V_FULL0 + s), 0, (u.t0 + j) * TILE, u.kh, 0,
                      p.a.v.batch ? u.b : 0);
        }
        __syncwarp();
        ++vn;
      }
      if (w >= p.total) break;
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.a.err);
      drain_copies(bar(Q_FULL), 1, un + (half ? 1 : 0));  // let the copies already issued land
      drain_copies(bar(DO_FULL), 1, un);
      drain_copies(bar(V_FULL0), V_STAGES, vn);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ TMA producer: K
    uint32_t kn = 0, tails = 0, tails_seen = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
#pragma unroll 1
      for (int j = 0; j < u.count(); ++j) {
        const uint32_t s = kn % K_STAGES, tile = base + SM_K + s * TILE_BYTES;
        ok = warp_wait(bar(K_EMPTY0 + s), ((kn / K_STAGES) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        // Rows past the last visible key may hold anything and meet dS = 0 in dS K: they are
        // zeroed here unless the copy itself fills them.
        const int n = u.keys_of(j);
        const bool patch = n < TILE && u.keys < p.a.kv_tokens;
        const uint32_t full = patch ? bar(K_TAIL) : bar(K_FULL0 + s);
        if (lane == 0) {
          mbar_arrive_expect_tx(full, TILE_BYTES);
          tma_load_5d(tile, &tm_k, full, 0, (u.t0 + j) * TILE, u.kh, 0, p.a.k.batch ? u.b : 0);
        }
        __syncwarp();
        if (patch) {
          ++tails;
          ok = warp_wait(full, (tails - 1) & 1u, abort, limit);
          if (!ok) break;
          tails_seen = tails;
          zero_rows(tile, n, ceil64(n), lane);
          if (lane == 0) mbar_arrive(bar(K_FULL0 + s));
        }
        ++kn;
      }
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.a.err);
      if (tails > tails_seen) drain_copies(bar(K_TAIL), 1, tails);
      drain_copies(bar(K_FULL0), K_STAGES, kn);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ UMMA issuer
    // Step x: S(x), dP(x), then dQ(x - 1); the first step of a unit: dQ(x - 1) of the last one first,
    // while Q and dO are on their way.
    const uint64_t q_desc = sdesc_sw128(base + SM_Q, 16, 1024), do_desc = sdesc_sw128(base + SM_DO, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(base + SM_K, 16, 1024), v_desc = sdesc_sw128(base + SM_V, 16, 1024);
    const uint64_t k_mn = sdesc_sw128(base + SM_K, TILE_BYTES / 2, 1024);
    uint32_t x = 0, un = 0, dqn = 0;    // steps; units begun; units whose dQ has begun
    uint32_t ks = 0, kph = 0, pks = 0;  // K stage and its phase; the last step's stage
    int prev_keys = 0;                  // the last step: its dQ is to come if > 0
    bool prev_first = false, prev_last = false, ok = true, issued = false;
    Unit u{};
    int w = static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x), j = 0;
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
      const int keys = s ? u.keys_of(j) : 0;
      const bool last = j + 1 == u.count();
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {
        if (prev_keys > 0 && turn == (s && j > 0 ? 1 : 0)) {
          // The step before this one, whose number is x - 1 until this one's S has been issued.
          const uint32_t y = x - 1 - turn;
          ok = warp_wait(bar(DS_READY0 + (y & 1u)), (y >> 1) & 1u, abort, limit) &&
               (!prev_first || warp_wait(bar(DQ_EMPTY), (dqn & 1u) ^ 1u, abort, limit));
          if (!ok) break;
          if (prev_first) ++dqn;
          tc_fence_after_sync();
#pragma unroll 1
          for (int h = 0; h * 64 < prev_keys; ++h)
            product_ts64<16>(tmem + TM_DQ, tmem + TM_DS + (y & 1u) * 64u + h * 32u,
                             sdesc_advance(k_mn, pks * TILE_BYTES + h * 8192u), IDESC_ACC, prev_first && h == 0 ? 0u : 1u);
          umma_commit_elect(bar(K_EMPTY0 + pks));
          if (prev_last) umma_commit_elect(bar(DQ_FULL));
        }
        if (s && turn == 0) {
          const uint32_t idesc = idesc_s((keys + 15) & ~15);
          ok = warp_wait(bar(K_FULL0 + ks), kph, abort, limit) &&
               (j != 0 || warp_wait(bar(Q_FULL), un & 1u, abort, limit)) &&
               warp_wait(bar(S_FREE), (x & 1u) ^ 1u, abort, limit);
          if (!ok) break;
          tc_fence_after_sync();
          product_ss(tmem + TM_S, q_desc, sdesc_advance(k_desc, ks * TILE_BYTES), idesc);
          umma_commit_elect(bar(S_FULL));
          issued = true;
          if (last) umma_commit_elect(bar(Q_EMPTY));
          ok = warp_wait(bar(V_FULL0 + (x & 1u)), (x >> 1) & 1u, abort, limit) &&
               (j != 0 || warp_wait(bar(DO_FULL), un & 1u, abort, limit)) &&
               warp_wait(bar(DP_FREE), (x & 1u) ^ 1u, abort, limit);
          if (!ok) break;
          tc_fence_after_sync();
          product_ss(tmem + TM_DP, do_desc, sdesc_advance(v_desc, (x & 1u) * TILE_BYTES), idesc);
          umma_commit_elect(bar(DP_FULL));
          umma_commit_elect(bar(V_EMPTY0 + (x & 1u)));
          if (last) {
            umma_commit_elect(bar(DO_EMPTY));
            ++un;
          }
          ++x;
        }
      }
      if (!ok || !s) break;
      prev_keys = keys;
      prev_first = j == 0;
      prev_last = last;
      pks = ks;
      if (++ks == K_STAGES) {
        ks = 0;
        kph ^= 1u;
      }
      ++j;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    if (issued) {
      umma_commit_elect(bar(DRAIN));  // every UMMA has completed before TMEM is released
      if (lane == 0) drain_copies(bar(DRAIN), 1, 1);
      __syncwarp();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// dQ of split tiles: the parts' sums in part order; a thread has one row and 8 columns.
__global__ void __launch_bounds__(TILE) cross_dq_join_kernel(const __grid_constant__ Params p) {
  grid_dependency_wait();
  const int tiles = p.a.batch * p.a.kv_heads * p.t.tiles;
  const int bk = blockIdx.x / p.t.tiles, b = bk / p.a.kv_heads, kh = bk % p.a.kv_heads, c0 = blockIdx.y * 8;
  const QRow q = q_row(p, kh, blockIdx.x % p.t.tiles, threadIdx.x);
  if (!q.valid) return;
  const int keys = visible_keys(p.a.kv_len, b, p.a.kv_tokens, p.a.err);
  const int n = (keys + TILE - 1) / TILE, per = (n + p.splits - 1) / p.splits;
  float s[8] = {};
  add_parts(s, p.part + (static_cast<int64_t>(blockIdx.x) * TILE + c0) * TILE + threadIdx.x,
            static_cast<int64_t>(tiles) * TILE * TILE, per > 0 ? (n + per - 1) / per : 0);
  const float c = p.a.sm_scale;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.dq.data) + b * p.a.dq.batch + q.head * p.a.dq.head +
                            q.token * p.a.dq.token + c0) =
      make_uint4(pack_bf162(s[0] * c, s[1] * c), pack_bf162(s[2] * c, s[3] * c), pack_bf162(s[4] * c, s[5] * c),
                 pack_bf162(s[6] * c, s[7] * c));
}

}  // namespace dq

// ================================================================================== dK, dV

namespace dkv {

constexpr int NUM_THREADS = 640;

// How the seven tiles of shared memory are used.  Many query tiles a unit: a Q tile is held from
// S^T to dK of the same step (with the next S^T in between), a dO tile from dP^T to dV, and the
// unit's output goes through K's space.  One query tile a unit (FEW; with one Q buffer a second
// S^T would wait for the first dK, which comes after it): what counts is the next unit's K and V,
// which get a second buffer, and the output has a space of its own (2 x 8 heads, 64 queries on 8191
// keys: the whole backward 52 us, with the other use of the tiles 59).
template <bool FEW>
struct Stages {
  static constexpr int KV = FEW ? 2 : 1, Q = FEW ? 1 : 3, DO = FEW ? 1 : 2;
  static constexpr uint32_t SM_K = 0, SM_V = KV * TILE_BYTES, SM_Q = 2 * KV * TILE_BYTES, SM_DO = SM_Q + Q * TILE_BYTES;
  static constexpr uint32_t SM_OUT = FEW ? SM_DO + DO * TILE_BYTES : SM_K;  // 16 warps x 2 KB
};
constexpr uint32_t SM_LSE = 7 * TILE_BYTES;           // 2 stages of -lse of 128 rows, fp32
constexpr uint32_t SM_DELTA = SM_LSE + 2 * TILE * 4;  // -Delta of 128 rows
constexpr uint32_t SM_BAR = SM_DELTA + TILE * 4;
enum Bar : uint32_t {
  KV_FULL0 = 0,
  KV_EMPTY0 = KV_FULL0 + 2,  // FEW: the tensor core; else the warps that write the unit out
  Q_FULL0 = KV_EMPTY0 + 2,
  Q_EMPTY0 = Q_FULL0 + 3,
  DO_FULL0 = Q_EMPTY0 + 3,
  DO_EMPTY0 = DO_FULL0 + 2,
  LSE_FULL0 = DO_EMPTY0 + 2,
  DELTA_FULL = LSE_FULL0 + 2,
  LSE_EMPTY0,
  DELTA_EMPTY = LSE_EMPTY0 + 2,
  S_FULL,
  P_READY,
  DP_FULL,
  DS_READY,
  ACC_FULL,
  ACC_EMPTY,
  DRAIN,
  NUM_BARS
};
constexpr uint32_t SM_TMEM_SLOT = SM_BAR + NUM_BARS * 8;
constexpr uint32_t SM_ABORT = SM_TMEM_SLOT + 4;
constexpr uint32_t SMEM_BYTES = SM_ABORT + 4;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 384;
constexpr float NO_ROW = -3.0e38f;  // -lse of a row that does not exist: P = 2^(0 - 3e38) = 0

struct Unit {
  int b, kh, j, split, q0, q1, keys;  // kv tile j; query tiles [q0, q1); visible keys of the tile
  __device__ __forceinline__ int count() const { return keys > 0 ? q1 - q0 : 0; }
};

__device__ __forceinline__ Unit decode(const Params& p, int w) {
  Unit u;
  int q = p.by_kv_tiles.quotient(w);
  u.j = w - q * p.kv_tiles;
  w = q;
  q = p.by_splits.quotient(w);
  u.split = w - q * p.splits;
  u.b = p.by_kv_heads.quotient(q);
  u.kh = q - u.b * p.a.kv_heads;
  const int per = p.by_splits.quotient(p.t.tiles + p.splits - 1);
  u.q0 = min(u.split * per, p.t.tiles);
  u.q1 = min(u.q0 + per, p.t.tiles);
  u.keys = max(0, min(TILE, uniform(visible_keys(p.a.kv_len, u.b, p.a.kv_tokens, p.a.err)) - u.j * TILE));
  return u;
}

template <bool FEW>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    cross_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ Params p) {
  using T = Stages<FEW>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + SM_ABORT);
  auto bar = [&](uint32_t b) { return base + SM_BAR + 8u * b; };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint64_t limit = p.a.wait_ns;

  if (threadIdx.x == 0) {
    *abort = 0;
    for (uint32_t b = 0; b < NUM_BARS; ++b) {
      const bool many = (!FEW && b >= KV_EMPTY0 && b < Q_FULL0) || b == P_READY || b == DS_READY || b == ACC_EMPTY ||
                        (b >= LSE_EMPTY0 && b < S_FULL);
      mbar_init(bar(b), many ? SOFTMAX_WARPS : 1);
    }
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(base + SM_TMEM_SLOT, 512);
    tmem_relinquish();
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_do);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  // Short tiles: the rows up to the next multiple of 64, which no copy writes, are multiplied as
  // zeros.
  const int full_rows = p.t.box * p.t.pack;
  if (full_rows % 64 != 0 && warp >= SOFTMAX_WARP && warp < SOFTMAX_WARP + T::Q + T::DO)
    zero_rows(base + T::SM_Q + (warp - SOFTMAX_WARP) * TILE_BYTES, full_rows, ceil64(full_rows), lane);
  grid_dependency_wait();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they start at 0

  if (warp >= SOFTMAX_WARP) {
    // ------------------------------------------------------------------ P^T, dS^T, output
    // Rows are keys, columns query rows.
    const int quarter = warp & 3, col = (warp - SOFTMAX_WARP) >> 2, r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col * 32u;
    const uint32_t stage = base + T::SM_OUT + (warp - SOFTMAX_WARP) * 2048u;
    const float c1 = p.a.sm_scale * LOG2E_F;
    const uint64_t c2 = f2_pack(c1, c1);
    uint32_t x = 0, un = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      const int n = u.count();
      uint32_t v[32];
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const float4* lse = reinterpret_cast<const float4*>(smem + SM_LSE) + (x & 1u) * (TILE / 4) + col * 8;
        ok = warp_wait(bar(LSE_FULL0 + (x & 1u)), (x >> 1) & 1u, abort, limit);
        if (!ok) break;
        // Query rows that do not exist are zeros in Q and dO, and times an infinite key or value NaN:
        // their scores and dP are taken as 0, of which NO_ROW makes P = dS = 0 (1.2 us of 248 at
        // 32760 x 512).  With one short query tile a unit, half of the warps may have no row at all.
        const int rows = __popc(__ballot_sync(0xffffffffu, reinterpret_cast<const float*>(lse)[lane] != NO_ROW));
        ok = warp_wait(bar(S_FULL), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t pk[16];
        float pr[32];
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = 0u;
        if (!FEW || rows > 0) {
          load32(lanes + TM_S, v);
          keep_columns(v, rows);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 nl = lse[c / 4];
            float a0, a1, a2, a3;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), c2, f2_pack(nl.x, nl.y)), a0, a1);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), c2, f2_pack(nl.z, nl.w)), a2, a3);
            pr[c] = ex2(a0), pr[c + 1] = ex2(a1), pr[c + 2] = ex2(a2), pr[c + 3] = ex2(a3);
            pk[c >> 1] = pack_bf162(pr[c], pr[c + 1]);
            pk[(c >> 1) + 1] = pack_bf162(pr[c + 2], pr[c + 3]);
          }
        }
        tmem_st_32x32b_x16(lanes + TM_S, pk);  // over the warp's own columns
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(P_READY));
          mbar_arrive(bar(LSE_EMPTY0 + (x & 1u)));
        }
        ok = warp_wait(bar(DELTA_FULL), x & 1u, abort, limit) && warp_wait(bar(DP_FULL), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        if (!FEW || rows > 0) {  // (else pk holds the zeros of P)
          load32(lanes + TM_DP, v);
          keep_columns(v, rows);
          const float4* delta = reinterpret_cast<const float4*>(smem + SM_DELTA) + col * 8;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 nd = delta[c / 4];
            float a0, a1, a2, a3;
            f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), f2_pack(nd.x, nd.y)),
                             f2_pack(pr[c], pr[c + 1])), a0, a1);
            f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), f2_pack(nd.z, nd.w)),
                             f2_pack(pr[c + 2], pr[c + 3])), a2, a3);
            pk[c >> 1] = pack_bf162(a0, a1);
            pk[(c >> 1) + 1] = pack_bf162(a2, a3);
          }
        }
        tmem_st_32x32b_x16(lanes + TM_DP, pk);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(DS_READY));
          mbar_arrive(bar(DELTA_EMPTY));
        }
        ++x;
      }
      if (!ok) break;
      if (n > 0) {
        ok = warp_wait(bar(ACC_FULL), un & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
      } else if (p.splits > 1) {
        continue;  // the join kernel writes
      }
      // Keys past the visible ones get exact zeros.  (Without a visible key the warp must not stage:
      // K's space may hold the next unit's already.)
      const int exist = min(TILE, p.a.kv_tokens - u.j * TILE);
      const int64_t part = ((static_cast<int64_t>(u.split) * p.a.batch + u.b) * p.a.kv_heads + u.kh) * p.kv_tiles + u.j;
#pragma unroll 1
      for (int y = 0; y < 2; ++y) {
        if (n > 0) {
          load32(lanes + (y == 0 ? TM_DV : TM_DK), v);
        } else {
          const HeadsView& out = y == 0 ? p.a.dv : p.a.dk;
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(out.data) + u.b * out.batch + u.kh * out.head +
                              (static_cast<int64_t>(u.j) * TILE + r) * out.token + col * 32;
          if (r < exist) {
#pragma unroll
            for (int c = 0; c < 4; ++c) reinterpret_cast<uint4*>(to)[c] = make_uint4(0u, 0u, 0u, 0u);
          }
          continue;
        }
        if (p.splits > 1) {
          float* to = p.part + ((part * 2 + y) * TILE + col * 32) * TILE + r;
          if (r < u.keys) {
#pragma unroll
            for (int c = 0; c < 32; ++c) to[c * TILE] = __uint_as_float(v[c]);
          }
          continue;
        }
        const HeadsView& out = y == 0 ? p.a.dv : p.a.dk;
        if (r >= u.keys) {
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = 0u;
        }
        int64_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = (quarter * 32 + i * 8 + (lane >> 2)) * out.token;
        // (A negative scale would turn the zeros into -0.)
        write_rows(stage, v, y == 0 || r >= u.keys ? 1.f : p.a.sm_scale,
                   static_cast<__nv_bfloat16*>(out.data) + u.b * out.batch + u.kh * out.head +
                       static_cast<int64_t>(u.j) * TILE * out.token + col * 32,
                   at, exist - quarter * 32, lane);
      }
      if (n == 0) continue;
      fence_proxy_async_smem();  // the staging writes before the next unit's copies
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(ACC_EMPTY));
        if (!FEW) mbar_arrive(bar(KV_EMPTY0));
      }
      ++un;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    uint32_t un = 0, qn = 0, dn = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0) continue;
      const uint32_t kv = un % T::KV;
      ok = warp_wait(bar(KV_EMPTY0 + kv), ((un / T::KV) & 1u) ^ 1u, abort, limit);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(KV_FULL0 + kv), 2 * TILE_BYTES);
        tma_load_5d(base + T::SM_K + kv * TILE_BYTES, &tm_k, bar(KV_FULL0 + kv), 0, u.j * TILE, u.kh, 0,
                    p.a.k.batch ? u.b : 0);
        tma_load_5d(base + T::SM_V + kv * TILE_BYTES, &tm_v, bar(KV_FULL0 + kv), 0, u.j * TILE, u.kh, 0,
                    p.a.v.batch ? u.b : 0);
      }
      __syncwarp();
      ++un;
#pragma unroll 1
      for (int i = u.q0; i < u.q1; ++i) {
        int head, token;
        tile_origin(p, u.kh, i, &head, &token);
        uint32_t s = qn % T::Q;
        ok = warp_wait(bar(Q_EMPTY0 + s), ((qn / T::Q) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        if (lane == 0) load_q_tile(p, &tm_q, p.a.q.batch, base + T::SM_Q + s * TILE_BYTES, bar(Q_FULL0 + s), u.b, head, token);
        __syncwarp();
        ++qn;
        s = dn % T::DO;
        ok = warp_wait(bar(DO_EMPTY0 + s), ((dn / T::DO) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        if (lane == 0)
          load_q_tile(p, &tm_do, p.a.dout.batch, base + T::SM_DO + s * TILE_BYTES, bar(DO_FULL0 + s), u.b, head, token);
        __syncwarp();
        ++dn;
      }
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.a.err);
      drain_copies(bar(KV_FULL0), T::KV, un);  // let the copies already issued land
      drain_copies(bar(Q_FULL0), T::Q, qn);
      drain_copies(bar(DO_FULL0), T::DO, dn);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ -lse and -Delta of the rows
    float* lse = reinterpret_cast<float*>(smem + SM_LSE);
    float* delta = reinterpret_cast<float*>(smem + SM_DELTA);
    int64_t at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int y = k * 32 + lane, h = y / p.t.box;
      at[k] = static_cast<int64_t>(h) * p.a.q_tokens + y - h * p.t.box;
    }
    uint32_t x = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0) continue;
#pragma unroll 1
      for (int i = u.q0; i < u.q1; ++i) {
        int head, token;
        tile_origin(p, u.kh, i, &head, &token);
        const int rows = tile_rows(p, token);
        const int64_t row = (static_cast<int64_t>(u.b) * p.a.heads + head) * p.a.q_tokens + token;
        float nl[4], nd[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          nl[k] = NO_ROW;
          nd[k] = 0.f;
          if (k * 32 + lane < rows) {
            const float l = p.a.lse[row + at[k]];
            nl[k] = l == -INFINITY ? 0.f : -l;  // all scores -inf: P = 2^-inf = 0
            nd[k] = -p.delta[row + at[k]];
          }
        }
        ok = warp_wait(bar(LSE_EMPTY0 + (x & 1u)), ((x >> 1) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) lse[(x & 1u) * TILE + k * 32 + lane] = nl[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(LSE_FULL0 + (x & 1u)));
        ok = warp_wait(bar(DELTA_EMPTY), (x & 1u) ^ 1u, abort, limit);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) delta[k * 32 + lane] = nd[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(DELTA_FULL));
        ++x;
      }
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ UMMA issuer
    // Turn i of a unit: dV(i - 1), S^T(i), dK(i - 1), dP^T(i).  P^T lies over S^T and dS^T over
    // dP^T, and products of one thread run in order.  Columns and rows count in halves of 64.
    const uint64_t k_desc = sdesc_sw128(base + T::SM_K, 16, 1024), v_desc = sdesc_sw128(base + T::SM_V, 16, 1024);
    const uint64_t q_desc = sdesc_sw128(base + T::SM_Q, 16, 1024), do_desc = sdesc_sw128(base + T::SM_DO, 16, 1024);
    const uint64_t q_mn = sdesc_sw128(base + T::SM_Q, TILE_BYTES / 2, 1024), do_mn = sdesc_sw128(base + T::SM_DO, TILE_BYTES / 2, 1024);
    uint32_t x = 0, un = 0;                 // steps begun; units
    uint32_t qs = 0, qph = 0, pqs = 0;      // Q stage and its phase; the last step's stage
    bool ok = true, issued = false;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0) continue;
      const uint32_t kv = un % T::KV;
      ok = warp_wait(bar(KV_FULL0 + kv), (un / T::KV) & 1u, abort, limit);
      int prev = 0;  // rows (in halves of 64) of the last step
#pragma unroll 1
      for (int i = u.q0; ok && i <= u.q1; ++i) {
        const uint32_t y = x - 1;  // the last step
        int rows = 0;
        if (i < u.q1) {
          int head, token;
          tile_origin(p, u.kh, i, &head, &token);
          rows = ceil64(tile_rows(p, token));
        }
        const uint32_t idesc = idesc_s(rows);
        if (prev > 0) {
          ok = warp_wait(bar(P_READY), y & 1u, abort, limit) &&
               (i != u.q0 + 1 || warp_wait(bar(ACC_EMPTY), (un & 1u) ^ 1u, abort, limit));
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll 1
          for (int h = 0; h * 64 < prev; ++h)
            product_ts64<32>(tmem + TM_DV, tmem + TM_S + h * 64u, sdesc_advance(do_mn, (y % T::DO) * TILE_BYTES + h * 8192u),
                             IDESC_ACC, i == u.q0 + 1 && h == 0 ? 0u : 1u);
          umma_commit_elect(bar(DO_EMPTY0 + y % T::DO));
        }
        if (rows > 0) {
          ok = warp_wait(bar(Q_FULL0 + qs), qph, abort, limit);
          if (!ok) break;
          tc_fence_after_sync();
          product_ss(tmem + TM_S, sdesc_advance(k_desc, kv * TILE_BYTES), sdesc_advance(q_desc, qs * TILE_BYTES), idesc);
          umma_commit_elect(bar(S_FULL));
          issued = true;
        }
        if (prev > 0) {
          ok = warp_wait(bar(DS_READY), y & 1u, abort, limit);
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll 1
          for (int h = 0; h * 64 < prev; ++h)
            product_ts64<32>(tmem + TM_DK, tmem + TM_DP + h * 64u, sdesc_advance(q_mn, pqs * TILE_BYTES + h * 8192u),
                             IDESC_ACC, i == u.q0 + 1 && h == 0 ? 0u : 1u);
          umma_commit_elect(bar(Q_EMPTY0 + pqs));
        }
        if (rows > 0) {
          ok = warp_wait(bar(DO_FULL0 + x % T::DO), (x / T::DO) & 1u, abort, limit);
          if (!ok) break;
          tc_fence_after_sync();
          product_ss(tmem + TM_DP, sdesc_advance(v_desc, kv * TILE_BYTES),
                     sdesc_advance(do_desc, (x % T::DO) * TILE_BYTES), idesc);
          umma_commit_elect(bar(DP_FULL));
          ++x;
          pqs = qs;
          if (++qs == T::Q) {
            qs = 0;
            qph ^= 1u;
          }
        }
        prev = rows;
      }
      if (!ok) break;
      umma_commit_elect(bar(ACC_FULL));
      if (FEW) umma_commit_elect(bar(KV_EMPTY0 + kv));
      ++un;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    if (issued) {
      umma_commit_elect(bar(DRAIN));  // every UMMA has completed before TMEM is released
      if (lane == 0) drain_copies(bar(DRAIN), 1, 1);
      __syncwarp();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// dV, dK of split tiles: the parts' sums in part order; a thread has one key and 8 columns.
__global__ void __launch_bounds__(TILE) cross_dkv_join_kernel(const __grid_constant__ Params p) {
  grid_dependency_wait();
  const int tiles = p.a.batch * p.a.kv_heads * p.kv_tiles;
  const int j = blockIdx.x % p.kv_tiles, bk = blockIdx.x / p.kv_tiles, b = bk / p.a.kv_heads, kh = bk % p.a.kv_heads;
  const int key = j * TILE + threadIdx.x, c0 = blockIdx.y * 8, y = blockIdx.z;
  if (key >= p.a.kv_tokens) return;
  const bool visible = key < visible_keys(p.a.kv_len, b, p.a.kv_tokens, p.a.err);
  const int per = (p.t.tiles + p.splits - 1) / p.splits;
  float s[8] = {};
  add_parts(s, p.part + ((static_cast<int64_t>(blockIdx.x) * 2 + y) * TILE + c0) * TILE + threadIdx.x,
            static_cast<int64_t>(tiles) * 2 * TILE * TILE, visible ? (p.t.tiles + per - 1) / per : 0);
  const HeadsView& out = y == 0 ? p.a.dv : p.a.dk;
  const float c = y == 0 || !visible ? 1.f : p.a.sm_scale;  // a hidden key's rows are +0
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out.data) + b * out.batch + kh * out.head + key * out.token + c0) =
      make_uint4(pack_bf162(s[0] * c, s[1] * c), pack_bf162(s[2] * c, s[3] * c), pack_bf162(s[4] * c, s[5] * c),
                 pack_bf162(s[6] * c, s[7] * c));
}

}  // namespace dkv

// Parts of an inner axis of `steps` for `units` tiles: the count with the least time by a model
// in units of one step (about 1 us): a wave of CTAs takes its steps and START for its first
// loads and its output; parts have to be written and read (`bytes` each way) and joined by
// another launch.  (Half and twice START and JOIN choose alike or as well at every size tried.)
int best_split(int64_t units, int steps, double bytes) {
  constexpr double START = 3.0, JOIN = 4.0, BYTES_PER_STEP = 6e6;
  const int sms = device_sm_count();
  int best = 1;
  double least = 0;
  for (int s = 1; s <= steps && s <= 64; ++s) {
    const int per = (steps + s - 1) / s;
    if (s > 1 && (steps + per - 1) / per != s) continue;  // the last part would be empty
    const int64_t waves = (units * s + sms - 1) / sms;
    const double t = waves * (per + START) + (s > 1 ? JOIN + 2 * units * s * bytes / BYTES_PER_STEP : 0.0);
    if (s == 1 || t < least) {
      best = s;
      least = t;
    }
  }
  return best;
}

struct Plan {
  QTiles t;
  int kv_tiles, dq_splits, dkv_splits;
  size_t part_off, total;  // Delta, then the parts of dQ and, over them, those of dK and dV
};

Plan plan_of(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens) {
  Plan p{};
  p.t = q_tiles(heads, kv_heads, q_tokens);
  p.kv_tiles = (kv_tokens + TILE - 1) / TILE;
  const int64_t bk = static_cast<int64_t>(batch) * kv_heads;
  constexpr double part = TILE * TILE * sizeof(float);
  p.dq_splits = best_split(bk * p.t.tiles, p.kv_tiles, part);
  p.dkv_splits = best_split(bk * p.kv_tiles, p.t.tiles, 2 * part);
  p.part_off = align_up(static_cast<size_t>(batch) * heads * q_tokens * sizeof(float), 256);
  const size_t dq = p.dq_splits > 1 ? static_cast<size_t>(p.dq_splits) * bk * p.t.tiles : 0;
  const size_t dkv = p.dkv_splits > 1 ? static_cast<size_t>(p.dkv_splits) * bk * p.kv_tiles * 2 : 0;
  p.total = p.part_off + (dq > dkv ? dq : dkv) * TILE * TILE * sizeof(float);
  return p;
}

}  // namespace

size_t cross_bwd_workspace(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens) {
  return plan_of(batch, heads, kv_heads, q_tokens, kv_tokens).total;
}

cudaError_t launch_cross_bwd(const CrossArgs& a, cudaStream_t stream) {
  const Plan plan = plan_of(a.batch, a.heads, a.kv_heads, a.q_tokens, a.kv_tokens);
  Params p{};
  p.a = a;
  p.t = plan.t;
  p.kv_tiles = plan.kv_tiles;
  p.delta = reinterpret_cast<float*>(a.workspace);
  p.part = reinterpret_cast<float*>(a.workspace + plan.part_off);
  CUtensorMap tq, td, to, tk, tv;
  cudaError_t e;
  if ((e = make_tmap_heads(&tq, a.q, a.q_tokens, a.batch, p.t.box, p.t.pack)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&td, a.dout, a.q_tokens, a.batch, p.t.box, p.t.pack)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&to, a.o, a.q_tokens, a.batch, p.t.box, p.t.pack)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&tk, a.k, a.kv_tokens, a.batch, TILE, 1)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&tv, a.v, a.kv_tokens, a.batch, TILE, 1)) != cudaSuccess) return e;
  static std::atomic<uint64_t> dq_smem{0}, dkv_smem{0}, dkv_few_smem{0};
  if ((e = ensure_smem_limit(dq::cross_dq_kernel, static_cast<int>(dq::SMEM_BYTES), dq_smem)) != cudaSuccess) return e;
  if ((e = ensure_smem_limit(dkv::cross_dkv_kernel<false>, static_cast<int>(dkv::SMEM_BYTES), dkv_smem)) != cudaSuccess ||
      (e = ensure_smem_limit(dkv::cross_dkv_kernel<true>, static_cast<int>(dkv::SMEM_BYTES), dkv_few_smem)) != cudaSuccess)
    return e;
  const int sms = device_sm_count(), bk = a.batch * a.kv_heads;
  p.by_tiles = make_divisor(p.t.tiles);
  p.by_kv_tiles = make_divisor(p.kv_tiles);
  p.by_kv_heads = make_divisor(a.kv_heads);
  p.by_batch = make_divisor(a.batch);
  p.by_blocks = make_divisor(p.t.blocks);
  p.by_box = make_divisor(p.t.box);
  p.splits = plan.dq_splits;
  p.by_splits = make_divisor(p.splits);
  p.total = bk * p.t.tiles * p.splits;
  e = launch_dependent(dq::cross_dq_kernel, dim3(p.total < sms ? p.total : sms), dim3(dq::NUM_THREADS), dq::SMEM_BYTES, stream,
                       tq, td, tk, tv, to, p);
  if (e != cudaSuccess) return e;
  if (p.splits > 1 &&
      (e = launch_dependent(dq::cross_dq_join_kernel, dim3(bk * p.t.tiles, 16), dim3(TILE), 0, stream, p)) != cudaSuccess)
    return e;
  p.splits = plan.dkv_splits;
  p.by_splits = make_divisor(p.splits);
  p.total = bk * p.kv_tiles * p.splits;
  const bool few = p.t.tiles <= p.splits && p.total > sms;  // one query tile a unit, several units a CTA
  e = launch_dependent(few ? dkv::cross_dkv_kernel<true> : dkv::cross_dkv_kernel<false>, dim3(p.total < sms ? p.total : sms), dim3(dkv::NUM_THREADS), dkv::SMEM_BYTES, stream,
                       tq, td, tk, tv, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_dependent(dkv::cross_dkv_join_kernel, dim3(bk * p.kv_tiles, 16, 2), dim3(TILE), 0, stream, p);
}

}  // namespace vsa
