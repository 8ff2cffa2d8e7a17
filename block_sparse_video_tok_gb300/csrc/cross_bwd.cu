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
// part order.
#include "cross_common.cuh"

namespace vsa {

namespace {

constexpr int NUM_THREADS = 384;  // warps are allocated in fours: the twelfth has no role
constexpr int SOFTMAX_WARPS = 8;
constexpr uint32_t IDESC_S0 = idesc_f16_f32acc(128, 0, false, false, true);  // N is added
constexpr uint32_t IDESC_ACC = idesc_f16_f32acc(128, 128, false, true, true);

__device__ __forceinline__ int ceil16(int n) { return (n + 15) & ~15; }
__device__ __forceinline__ uint32_t idesc_s(int n) {
  return IDESC_S0 | (static_cast<uint32_t>(ceil16(n) >> 3) << 17);
}

struct Params {
  CrossArgs a;
  QTiles t;
  int kv_tiles;  // of kv_tokens
  int splits;    // parts of the inner axis
  int total;     // units
  float* delta;  // [batch, heads, q_tokens]
  float* part;   // dq: [split][batch * kv_heads * tiles][128 columns][128 rows];
                 // dkv: [split][batch * kv_heads * kv_tiles][dV, dK][128 columns][128 keys]
};

// D (+)= A B: A of 16-bit pairs in tensor memory, `steps` of 16 along its columns (8 TMEM columns
// each; step 4 starts `half` columns after step 0), B an MN-major tile.
__device__ __forceinline__ void product_acc(uint32_t d, uint32_t a, uint32_t half, uint64_t b, bool fresh, int steps) {
  product_ts(d, a, b, IDESC_ACC, fresh ? 0u : 1u, min(steps, 4));
  if (steps > 4) product_ts(d, a + half, sdesc_advance(b, 8192u), IDESC_ACC, 1u, steps - 4);
}

// A warp's 32 rows x 64 fp32 columns (one row per lane), scaled and rounded, to global memory in
// whole lines through 4 KB of shared memory; `out` is each lane's row, written where `rows` has its bit.
__device__ __forceinline__ void write_rows(uint32_t stage, const uint32_t* v, float scale, __nv_bfloat16* out,
                                           unsigned rows, int lane) {
  const uint64_t s2 = f2_pack(scale, scale);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t pk[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float a0, a1;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(v[8 * i + 2 * x]), __uint_as_float(v[8 * i + 2 * x + 1])), s2), a0, a1);
      pk[x] = pack_bf162(a0, a1);
    }
    st_shared16(stage + swizzled(lane, i), pk[0], pk[1], pk[2], pk[3]);
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rr = i * 4 + (lane >> 3);
    const uint64_t to = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(out), rr);
    const uint4 x = ld_shared16(stage + swizzled(rr, lane & 7));
    if ((rows >> rr) & 1u) reinterpret_cast<uint4*>(to)[lane & 7] = x;
  }
  __syncwarp();
}

__device__ __forceinline__ void load64(uint32_t taddr, uint32_t* v) {
  tmem_ld_32x32b_x32(taddr, v);
  tmem_ld_32x32b_x32(taddr + 32u, v + 32);
  tmem_wait_ld();
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

// One query-side tile (rows packed as in QTiles) into shared memory, by one thread.
__device__ __forceinline__ void load_q_tile(const Params& p, const CUtensorMap* map, int64_t batch_stride, uint32_t dst,
                                            uint32_t full, int b, int kh, int tile) {
  const int g = tile / p.t.blocks;
  const int head = kh * p.t.share + g * p.t.pack, token = (tile - g * p.t.blocks) * p.t.box;
  const int rows = p.t.box * p.t.pack;
  mbar_arrive_expect_tx(full, static_cast<uint32_t>(rows) * 256u);
  for (int h = 0; h < (rows == TILE ? 1 : 2); ++h)
    tma_load_5d(dst + h * (TILE_BYTES / 2), map, full, 0, token, head, h, batch_stride ? b : 0);
}

// ================================================================================== dQ

namespace dq {

// K tiles are held from S to dQ of the same step, with the next step's S and dP in between, so
// three of them; a V tile serves one product.
constexpr int K_STAGES = 3;
constexpr uint32_t SM_Q = 0, SM_DO = TILE_BYTES, SM_K = 2 * TILE_BYTES, SM_V = SM_K + K_STAGES * TILE_BYTES;
constexpr uint32_t SM_OUT = SM_V + TILE_BYTES;       // 8 warps x 4 KB
constexpr uint32_t SM_XCH = SM_OUT + TILE_BYTES;     // [column half][128 rows] fp32
constexpr uint32_t SM_BAR = SM_XCH + 2 * TILE * 4;
enum Bar : uint32_t {
  Q_FULL = 0,
  Q_EMPTY,
  DO_FULL,
  DO_EMPTY,  // the tensor core and the 8 warps that sum O dO
  K_FULL0,
  K_EMPTY0 = K_FULL0 + K_STAGES,
  V_FULL = K_EMPTY0 + K_STAGES,
  V_EMPTY,
  S_FULL,
  S_FREE,  // S has been read
  DP_FULL,
  DP_FREE,
  DS_READY0,  // two buffers
  DQ_FULL = DS_READY0 + 2,
  DQ_EMPTY,
  XCH0,  // per lane quarter
  K_TAIL = XCH0 + 4,
  DRAIN,
  NUM_BARS
};
constexpr uint32_t SM_TMEM_SLOT = SM_BAR + NUM_BARS * 8;
constexpr uint32_t SM_ABORT = SM_TMEM_SLOT + 4;
constexpr uint32_t SMEM_BYTES = SM_ABORT + 4 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DQ = 256, TM_DS = 384;  // dS: two buffers of 64 columns

struct Unit {
  int b, kh, tile, split, t0, t1, keys;
  __device__ __forceinline__ int count() const { return t1 - t0; }
  __device__ __forceinline__ int keys_of(int j) const { return min(TILE, keys - (t0 + j) * TILE); }
};

__device__ __forceinline__ Unit decode(const Params& p, int w) {
  Unit u;
  u.tile = w % p.t.tiles;
  w /= p.t.tiles;
  u.kh = w % p.a.kv_heads;
  w /= p.a.kv_heads;
  u.b = w % p.a.batch;
  u.split = w / p.a.batch;
  u.keys = visible_keys(p.a.kv_len, u.b, p.a.kv_tokens, p.a.err);
  const int n = (u.keys + TILE - 1) / TILE, per = (n + p.splits - 1) / p.splits;
  u.t0 = min(u.split * per, n);
  u.t1 = min(u.t0 + per, n);
  return u;
}

__device__ __forceinline__ int next_unit(const Params& p, int w, Unit* u) {
  for (; w < p.total; w += gridDim.x) {
    *u = decode(p, w);
    if (u->count() > 0) break;
  }
  return w;
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ Params p) {
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
      uint32_t count = 1;
      if (b == S_FREE || b == DP_FREE || b == DS_READY0 || b == DS_READY0 + 1 || b == DQ_EMPTY) count = SOFTMAX_WARPS;
      if (b == DO_EMPTY) count = SOFTMAX_WARPS + 1;
      if (b >= XCH0 && b < K_TAIL) count = 2;
      mbar_init(bar(b), count);
    }
    fence_barrier_init();
  }
  if (warp == 8) {
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
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer: Q, dO, V
    uint32_t qn = 0, dn = 0, vn = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0) continue;
      ok = warp_wait(bar(Q_EMPTY), (qn & 1u) ^ 1u, abort, limit);
      if (!ok) break;
      if (lane == 0) load_q_tile(p, &tm_q, p.a.q.batch, base + SM_Q, bar(Q_FULL), u.b, u.kh, u.tile);
      __syncwarp();
      ++qn;
      ok = warp_wait(bar(DO_EMPTY), (dn & 1u) ^ 1u, abort, limit);
      if (!ok) break;
      if (lane == 0) load_q_tile(p, &tm_do, p.a.dout.batch, base + SM_DO, bar(DO_FULL), u.b, u.kh, u.tile);
      __syncwarp();
      ++dn;
      for (int j = 0; j < u.count(); ++j) {
        ok = warp_wait(bar(V_EMPTY), (vn & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(V_FULL), TILE_BYTES);
          tma_load_5d(base + SM_V, &tm_v, bar(V_FULL), 0, (u.t0 + j) * TILE, u.kh, 0, p.a.v.batch ? u.b : 0);
        }
        __syncwarp();
        ++vn;
      }
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.a.err);
      volatile int never = 0;  // let the copies already issued land
      if (qn > 0) mbar_wait_bounded(bar(Q_FULL), (qn - 1) & 1u, &never, DRAIN_LIMIT_NS);
      if (dn > 0) mbar_wait_bounded(bar(DO_FULL), (dn - 1) & 1u, &never, DRAIN_LIMIT_NS);
      if (vn > 0) mbar_wait_bounded(bar(V_FULL), (vn - 1) & 1u, &never, DRAIN_LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------------ TMA producer: K
    uint32_t kn = 0, tails = 0, tails_seen = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
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
          zero_rows(tile, n, ceil16(n), lane);
          if (lane == 0) mbar_arrive(bar(K_FULL0 + s));
        }
        ++kn;
      }
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.a.err);
      volatile int never = 0;
      if (tails > tails_seen) mbar_wait_bounded(bar(K_TAIL), (tails - 1) & 1u, &never, DRAIN_LIMIT_NS);
      for (uint32_t i = kn > K_STAGES ? kn - K_STAGES : 0; i < kn; ++i)
        mbar_wait_bounded(bar(K_FULL0 + i % K_STAGES), (i / K_STAGES) & 1u, &never, DRAIN_LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------------ UMMA issuer
    // Per step: S(x+1), dP(x+1), then dQ(x), across units.
    const uint64_t q_desc = sdesc_sw128(base + SM_Q, 16, 1024), do_desc = sdesc_sw128(base + SM_DO, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(base + SM_K, 16, 1024), v_desc = sdesc_sw128(base + SM_V, 16, 1024);
    const uint64_t k_mn = sdesc_sw128(base + SM_K, TILE_BYTES / 2, 1024);
    uint32_t x = 0, un = 0;  // steps issued (S and dP); units begun
    bool ok = true, issued = false;
    int prev_keys = 0;           // step x - 1: its dQ is to come if prev_keys > 0
    bool prev_first = false, prev_last = false;
    uint32_t dqn = 0;            // units whose dQ has begun
    auto issue_dq = [&]() {
      const uint32_t y = x - 1;
      if (!warp_wait(bar(DS_READY0 + (y & 1u)), (y >> 1) & 1u, abort, limit)) return false;
      if (prev_first && !warp_wait(bar(DQ_EMPTY), (dqn & 1u) ^ 1u, abort, limit)) return false;
      if (prev_first) ++dqn;
      tc_fence_after_sync();
      product_acc(tmem + TM_DQ, tmem + TM_DS + (y & 1u) * 64u, 32u,
                 sdesc_advance(k_mn, (y % K_STAGES) * TILE_BYTES), prev_first, ceil16(prev_keys) / 16);
      umma_commit_elect(bar(K_EMPTY0 + y % K_STAGES));
      if (prev_last) umma_commit_elect(bar(DQ_FULL));
      return true;
    };
    Unit u{};
    for (int w = next_unit(p, blockIdx.x, &u); w < p.total && ok; w = next_unit(p, w + gridDim.x, &u)) {
      const int n = u.count();
      for (int j = 0; j < n && ok; ++j) {
        const int keys = u.keys_of(j);
        const uint32_t idesc = idesc_s(keys);
        ok = warp_wait(bar(K_FULL0 + x % K_STAGES), (x / K_STAGES) & 1u, abort, limit) &&
             (j != 0 || warp_wait(bar(Q_FULL), un & 1u, abort, limit)) &&
             warp_wait(bar(S_FREE), (x & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        product_ss(tmem + TM_S, q_desc, sdesc_advance(k_desc, (x % K_STAGES) * TILE_BYTES), idesc);
        umma_commit_elect(bar(S_FULL));
        issued = true;
        if (j + 1 == n) umma_commit_elect(bar(Q_EMPTY));
        ok = warp_wait(bar(V_FULL), x & 1u, abort, limit) &&
             (j != 0 || warp_wait(bar(DO_FULL), un & 1u, abort, limit)) &&
             warp_wait(bar(DP_FREE), (x & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        product_ss(tmem + TM_DP, do_desc, v_desc, idesc);
        umma_commit_elect(bar(DP_FULL));
        umma_commit_elect(bar(V_EMPTY));
        if (j + 1 == n) umma_commit_elect(bar(DO_EMPTY));
        if (prev_keys > 0 && !(ok = issue_dq())) break;
        ++x;
        prev_keys = keys;
        prev_first = j == 0;
        prev_last = j + 1 == n;
      }
      ++un;
    }
    if (ok && prev_keys > 0) ok = issue_dq();
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    if (issued) {
      umma_commit_elect(bar(DRAIN));  // every UMMA has completed before TMEM is released
      volatile int never = 0;
      if (lane == 0) mbar_wait_bounded(bar(DRAIN), 0, &never, DRAIN_LIMIT_NS);
      __syncwarp();
    }
  } else if (warp < SOFTMAX_WARPS) {
    // ------------------------------------------------------------------ P, dS, Delta, output
    // Warp (quarter, half): rows 32 quarter .. + 31, one per lane; columns 64 half .. + 63.
    const int quarter = warp & 3, half = warp >> 2, r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + TM_S + half * 64u, t_dp = tmem + lane_off + TM_DP + half * 64u;
    const uint32_t t_ds = tmem + lane_off + TM_DS + half * 32u, t_dq = tmem + lane_off + TM_DQ + half * 64u;
    const uint32_t stage = base + SM_OUT + warp * 4096u;
    float* xch = reinterpret_cast<float*>(gbase + SM_XCH);
    const float c1 = p.a.sm_scale * LOG2E_F;
    const uint64_t c2 = f2_pack(c1, c1);
    uint32_t x = 0, un = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      const QRow q = q_row(p, u.kh, u.tile, r);
      const int64_t row = (static_cast<int64_t>(u.b) * p.a.heads + q.head) * p.a.q_tokens + q.token;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.dq.data) + u.b * p.a.dq.batch + q.head * p.a.dq.head +
                           q.token * p.a.dq.token + half * 64;
      if (u.count() == 0) {
        if (q.valid && u.split == 0 && p.splits == 1)
          for (int c = 0; c < 8; ++c) reinterpret_cast<uint4*>(out)[c] = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      const unsigned rows = __ballot_sync(0xffffffffu, q.valid);
      float lse = q.valid ? p.a.lse[row] : 0.f;
      if (lse == -INFINITY) lse = 0.f;  // a row whose scores are all -inf: P = 2^-inf = 0
      // This warp's share of Delta: 4 rows x 8 chunks of O at a time.
      const __nv_bfloat16* orow = static_cast<const __nv_bfloat16*>(p.a.o.data) + u.b * p.a.o.batch +
                                  q.head * p.a.o.head + q.token * p.a.o.token + half * 64;
      uint4 ov[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = i * 4 + (lane >> 3);
        const uint64_t from = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(orow), rr);
        ov[i] = (rows >> rr) & 1u ? reinterpret_cast<const uint4*>(from)[lane & 7] : make_uint4(0u, 0u, 0u, 0u);
      }
      ok = warp_wait(bar(DO_FULL), un & 1u, abort, limit);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = i * 4 + (lane >> 3);
        const uint4 d = ld_shared16(base + SM_DO + half * (TILE_BYTES / 2) + swizzled(quarter * 32 + rr, lane & 7));
        const uint32_t ow[4] = {ov[i].x, ov[i].y, ov[i].z, ov[i].w}, dw[4] = {d.x, d.y, d.z, d.w};
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s = fmaf(__uint_as_float(ow[k] << 16), __uint_as_float(dw[k] << 16), s);
          s = fmaf(__uint_as_float(ow[k] & 0xffff0000u), __uint_as_float(dw[k] & 0xffff0000u), s);
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        if ((lane & 7) == 0) xch[half * TILE + quarter * 32 + rr] = s;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(DO_EMPTY));
        mbar_arrive(bar(XCH0 + quarter));
      }
      ok = warp_wait(bar(XCH0 + quarter), un & 1u, abort, limit);
      if (!ok) break;
      // The next unit's sums come after this one's dQ, for which both warps have read these.
      const float delta = xch[r] + xch[TILE + r];
      if (half == 0 && q.valid && u.t0 == 0) p.delta[row] = delta;
      const uint64_t nl2 = f2_pack(-lse, -lse), nd2 = f2_pack(-delta, -delta);
      for (int j = 0; j < u.count(); ++j) {
        ok = warp_wait(bar(S_FULL), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t v[64];
        load64(t_s, v);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S_FREE));
        float pr[64];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float a0, a1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2, nl2), a0, a1);
          pr[i] = ex2(a0);
          pr[i + 1] = ex2(a1);
        }
        ok = warp_wait(bar(DP_FULL), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        load64(t_dp, v);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(DP_FREE));
        const int n = u.keys_of(j) - half * 64;  // columns of this half that are visible
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float a0, a1;
          f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), nd2),
                           f2_pack(pr[i], pr[i + 1])),
                    a0, a1);
          pk[i >> 1] = pack_bf162(a0, a1);
        }
        if (n < 64) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (2 * i >= n) pk[i] = 0u;
            else if (2 * i + 1 >= n) pk[i] &= 0xffffu;
          }
        }
        // The buffer's last reader, dQ of two steps ago, was issued before this dP.
        tmem_st_32x32b_x32(t_ds + (x & 1u) * 64u, pk);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(DS_READY0 + (x & 1u)));
        ++x;
      }
      if (!ok) break;
      ok = warp_wait(bar(DQ_FULL), un & 1u, abort, limit);
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t v[64];
      load64(t_dq, v);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(DQ_EMPTY));
      if (p.splits == 1) {
        write_rows(stage, v, p.a.sm_scale, out, rows, lane);
      } else if (q.valid) {
        const int64_t at = ((static_cast<int64_t>(u.split) * p.a.batch + u.b) * p.a.kv_heads + u.kh) * p.t.tiles + u.tile;
        float* to = p.part + (at * TILE + half * 64) * TILE + r;
#pragma unroll
        for (int i = 0; i < 64; ++i) to[i * TILE] = __uint_as_float(v[i]);
      }
      ++un;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 8) tmem_dealloc(tmem, 512);
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
  for (int x = 0; x < p.splits && x * per < n; ++x) {
    const float* from = p.part + ((static_cast<int64_t>(x) * tiles + blockIdx.x) * TILE + c0) * TILE + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += from[i * TILE];
  }
  const float c = p.a.sm_scale;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.dq.data) + b * p.a.dq.batch + q.head * p.a.dq.head +
                            q.token * p.a.dq.token + c0) =
      make_uint4(pack_bf162(s[0] * c, s[1] * c), pack_bf162(s[2] * c, s[3] * c), pack_bf162(s[4] * c, s[5] * c),
                 pack_bf162(s[6] * c, s[7] * c));
}

}  // namespace dq

// ================================================================================== dK, dV

namespace dkv {

// A Q tile is held from S^T to dK of the same step (with the next S^T in between), a dO tile from
// dP^T to dV.
constexpr int Q_STAGES = 3, DO_STAGES = 2;
constexpr uint32_t SM_K = 0, SM_V = TILE_BYTES, SM_Q = 2 * TILE_BYTES, SM_DO = SM_Q + Q_STAGES * TILE_BYTES;
constexpr uint32_t SM_LSE = SM_DO + DO_STAGES * TILE_BYTES;  // 2 stages of -lse of 128 rows, fp32
constexpr uint32_t SM_DELTA = SM_LSE + 2 * TILE * 4;         // -Delta of 128 rows
constexpr uint32_t SM_BAR = SM_DELTA + TILE * 4;
enum Bar : uint32_t {
  KV_FULL = 0,
  KV_EMPTY,  // the 8 warps that write the unit out (through K's and V's space)
  Q_FULL0,
  Q_EMPTY0 = Q_FULL0 + Q_STAGES,
  DO_FULL0 = Q_EMPTY0 + Q_STAGES,
  DO_EMPTY0 = DO_FULL0 + DO_STAGES,
  LSE_FULL0 = DO_EMPTY0 + DO_STAGES,
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
constexpr uint32_t SMEM_BYTES = SM_ABORT + 4 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 384;

struct Unit {
  int b, kh, j, split, q0, q1, keys;  // kv tile j; query tiles [q0, q1); visible keys of the tile
  __device__ __forceinline__ int count() const { return keys > 0 ? q1 - q0 : 0; }
};

__device__ __forceinline__ Unit decode(const Params& p, int w) {
  Unit u;
  u.j = w % p.kv_tiles;
  w /= p.kv_tiles;
  u.split = w % p.splits;
  w /= p.splits;
  u.kh = w % p.a.kv_heads;
  u.b = w / p.a.kv_heads;
  const int per = (p.t.tiles + p.splits - 1) / p.splits;
  u.q0 = min(u.split * per, p.t.tiles);
  u.q1 = min(u.q0 + per, p.t.tiles);
  u.keys = max(0, min(TILE, visible_keys(p.a.kv_len, u.b, p.a.kv_tokens, p.a.err) - u.j * TILE));
  return u;
}

// Rows of a query tile: fewer in the last block of a head's tokens.
__device__ __forceinline__ int rows_of(const Params& p, int tile) {
  if (p.t.pack > 1) return p.t.box * p.t.pack;
  return min(p.t.box, p.a.q_tokens - tile % p.t.blocks * p.t.box);
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    cross_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ Params p) {
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
      const bool eight = b == KV_EMPTY || b == P_READY || b == DS_READY || b == ACC_EMPTY ||
                         (b >= LSE_EMPTY0 && b < S_FULL);
      mbar_init(bar(b), eight ? SOFTMAX_WARPS : 1);
    }
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(base + SM_TMEM_SLOT, 512);
    tmem_relinquish();
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_do);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  // Short tiles: the rows up to the next multiple of 16, which no copy writes, are multiplied as
  // zeros in dV and dK.
  const int full_rows = p.t.box * p.t.pack;
  if (full_rows % 16 != 0 && warp < Q_STAGES + DO_STAGES)
    zero_rows(base + SM_Q + warp * TILE_BYTES, full_rows, ceil16(full_rows), lane);
  grid_dependency_wait();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    uint32_t un = 0, qn = 0, dn = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0) continue;
      ok = warp_wait(bar(KV_EMPTY), (un & 1u) ^ 1u, abort, limit);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(KV_FULL), 2 * TILE_BYTES);
        tma_load_5d(base + SM_K, &tm_k, bar(KV_FULL), 0, u.j * TILE, u.kh, 0, p.a.k.batch ? u.b : 0);
        tma_load_5d(base + SM_V, &tm_v, bar(KV_FULL), 0, u.j * TILE, u.kh, 0, p.a.v.batch ? u.b : 0);
      }
      __syncwarp();
      ++un;
      for (int i = u.q0; i < u.q1; ++i) {
        uint32_t s = qn % Q_STAGES;
        ok = warp_wait(bar(Q_EMPTY0 + s), ((qn / Q_STAGES) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        if (lane == 0) load_q_tile(p, &tm_q, p.a.q.batch, base + SM_Q + s * TILE_BYTES, bar(Q_FULL0 + s), u.b, u.kh, i);
        __syncwarp();
        ++qn;
        s = dn % DO_STAGES;
        ok = warp_wait(bar(DO_EMPTY0 + s), ((dn / DO_STAGES) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        if (lane == 0)
          load_q_tile(p, &tm_do, p.a.dout.batch, base + SM_DO + s * TILE_BYTES, bar(DO_FULL0 + s), u.b, u.kh, i);
        __syncwarp();
        ++dn;
      }
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.a.err);
      volatile int never = 0;  // let the copies already issued land
      if (un > 0) mbar_wait_bounded(bar(KV_FULL), (un - 1) & 1u, &never, DRAIN_LIMIT_NS);
      for (uint32_t i = qn > Q_STAGES ? qn - Q_STAGES : 0; i < qn; ++i)
        mbar_wait_bounded(bar(Q_FULL0 + i % Q_STAGES), (i / Q_STAGES) & 1u, &never, DRAIN_LIMIT_NS);
      for (uint32_t i = dn > DO_STAGES ? dn - DO_STAGES : 0; i < dn; ++i)
        mbar_wait_bounded(bar(DO_FULL0 + i % DO_STAGES), (i / DO_STAGES) & 1u, &never, DRAIN_LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------------ -lse and -Delta of the rows
    // A row that does not exist gets -lse = -inf: its P is 0.
    float* lse = reinterpret_cast<float*>(gbase + SM_LSE);
    float* delta = reinterpret_cast<float*>(gbase + SM_DELTA);
    uint32_t x = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0) continue;
      for (int i = u.q0; i < u.q1; ++i) {
        float nl[4], nd[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const QRow q = q_row(p, u.kh, i, k * 32 + lane);
          const int64_t row = (static_cast<int64_t>(u.b) * p.a.heads + q.head) * p.a.q_tokens + q.token;
          nl[k] = -INFINITY;
          nd[k] = 0.f;
          if (q.valid) {
            const float l = p.a.lse[row];
            nl[k] = l == -INFINITY ? 0.f : -l;  // all scores -inf: P = 2^-inf = 0
            nd[k] = -p.delta[row];
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
  } else if (warp == 9) {
    // ------------------------------------------------------------------ UMMA issuer
    // Per step: dV(g), S^T(g+1), dK(g), dP^T(g+1).  P^T lies over S^T and dS^T over dP^T (each
    // half of the query columns over its own columns), and products of one thread run in order.
    const uint64_t k_desc = sdesc_sw128(base + SM_K, 16, 1024), v_desc = sdesc_sw128(base + SM_V, 16, 1024);
    const uint64_t q_desc = sdesc_sw128(base + SM_Q, 16, 1024), do_desc = sdesc_sw128(base + SM_DO, 16, 1024);
    const uint64_t q_mn = sdesc_sw128(base + SM_Q, TILE_BYTES / 2, 1024), do_mn = sdesc_sw128(base + SM_DO, TILE_BYTES / 2, 1024);
    uint32_t x = 0, un = 0;  // steps begun with S^T; units
    bool ok = true, issued = false;
    auto issue_s = [&](uint32_t y, int rows) {
      const uint32_t s = y % Q_STAGES;
      if (!warp_wait(bar(Q_FULL0 + s), (y / Q_STAGES) & 1u, abort, limit)) return false;
      tc_fence_after_sync();
      product_ss(tmem + TM_S, k_desc, sdesc_advance(q_desc, s * TILE_BYTES), idesc_s(rows));
      umma_commit_elect(bar(S_FULL));
      issued = true;
      return true;
    };
    auto issue_dp = [&](uint32_t y, int rows) {
      const uint32_t s = y % DO_STAGES;
      if (!warp_wait(bar(DO_FULL0 + s), (y / DO_STAGES) & 1u, abort, limit)) return false;
      tc_fence_after_sync();
      product_ss(tmem + TM_DP, v_desc, sdesc_advance(do_desc, s * TILE_BYTES), idesc_s(rows));
      umma_commit_elect(bar(DP_FULL));
      return true;
    };
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      if (u.count() == 0) continue;
      int rows = rows_of(p, u.q0);
      ok = warp_wait(bar(KV_FULL), un & 1u, abort, limit) && issue_s(x, rows) && issue_dp(x, rows);
      for (int i = u.q0; i < u.q1 && ok; ++i) {
        const bool more = i + 1 < u.q1, fresh = i == u.q0;
        const int steps = ceil16(rows) / 16, next = more ? rows_of(p, i + 1) : 0;
        ok = warp_wait(bar(P_READY), x & 1u, abort, limit) &&
             (!fresh || warp_wait(bar(ACC_EMPTY), (un & 1u) ^ 1u, abort, limit));
        if (!ok) break;
        tc_fence_after_sync();
        product_acc(tmem + TM_DV, tmem + TM_S, 64u, sdesc_advance(do_mn, (x % DO_STAGES) * TILE_BYTES), fresh, steps);
        umma_commit_elect(bar(DO_EMPTY0 + x % DO_STAGES));
        if (more && !(ok = issue_s(x + 1, next))) break;
        ok = warp_wait(bar(DS_READY), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        product_acc(tmem + TM_DK, tmem + TM_DP, 64u, sdesc_advance(q_mn, (x % Q_STAGES) * TILE_BYTES), fresh, steps);
        umma_commit_elect(bar(Q_EMPTY0 + x % Q_STAGES));
        if (more && !(ok = issue_dp(x + 1, next))) break;
        ++x;
        rows = next;
      }
      if (!ok) break;
      umma_commit_elect(bar(ACC_FULL));
      ++un;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    if (issued) {
      umma_commit_elect(bar(DRAIN));  // every UMMA has completed before TMEM is released
      volatile int never = 0;
      if (lane == 0) mbar_wait_bounded(bar(DRAIN), 0, &never, DRAIN_LIMIT_NS);
      __syncwarp();
    }
  } else if (warp < SOFTMAX_WARPS) {
    // ------------------------------------------------------------------ P^T, dS^T, output
    // Warp (quarter, half): keys 32 quarter .. + 31, one per lane; query columns 64 half .. + 63.
    const int quarter = warp & 3, half = warp >> 2, r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + TM_S + half * 64u, t_dp = tmem + lane_off + TM_DP + half * 64u;
    const uint32_t t_dv = tmem + lane_off + TM_DV + half * 64u, t_dk = tmem + lane_off + TM_DK + half * 64u;
    const uint32_t stage = base + (warp < 4 ? SM_K : SM_V) + (warp & 3) * 4096u;
    const float c1 = p.a.sm_scale * LOG2E_F;
    const uint64_t c2 = f2_pack(c1, c1);
    uint32_t x = 0, un = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < p.total && ok; w += gridDim.x) {
      const Unit u = decode(p, w);
      const int key = u.j * TILE + r;
      const bool exists = key < p.a.kv_tokens, visible = r < u.keys;
      __nv_bfloat16* dk = static_cast<__nv_bfloat16*>(p.a.dk.data) + u.b * p.a.dk.batch + u.kh * p.a.dk.head +
                          key * p.a.dk.token + half * 64;
      __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(p.a.dv.data) + u.b * p.a.dv.batch + u.kh * p.a.dv.head +
                          key * p.a.dv.token + half * 64;
      if (p.splits == 1 && exists && !visible) {
        for (int c = 0; c < 8; ++c) {
          reinterpret_cast<uint4*>(dk)[c] = make_uint4(0u, 0u, 0u, 0u);
          reinterpret_cast<uint4*>(dv)[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (u.count() == 0) continue;
      for (int i = u.q0; i < u.q1; ++i) {
        const float* lse = reinterpret_cast<const float*>(gbase + SM_LSE) + (x & 1u) * TILE + half * 64;
        const float* delta = reinterpret_cast<const float*>(gbase + SM_DELTA) + half * 64;
        ok = warp_wait(bar(LSE_FULL0 + (x & 1u)), (x >> 1) & 1u, abort, limit) &&
             warp_wait(bar(S_FULL), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t v[64], pk[32];
        load64(t_s, v);
        float pr[64];
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float4 nl = *reinterpret_cast<const float4*>(lse + c);
          float a0, a1, a2, a3;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), c2, f2_pack(nl.x, nl.y)), a0, a1);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), c2, f2_pack(nl.z, nl.w)), a2, a3);
          pr[c] = ex2(a0), pr[c + 1] = ex2(a1), pr[c + 2] = ex2(a2), pr[c + 3] = ex2(a3);
          pk[c >> 1] = pack_bf162(pr[c], pr[c + 1]);
          pk[(c >> 1) + 1] = pack_bf162(pr[c + 2], pr[c + 3]);
        }
        tmem_st_32x32b_x32(t_s, pk);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(P_READY));
          mbar_arrive(bar(LSE_EMPTY0 + (x & 1u)));
        }
        ok = warp_wait(bar(DELTA_FULL), x & 1u, abort, limit) &&
             warp_wait(bar(DP_FULL), x & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        load64(t_dp, v);
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float4 nd = *reinterpret_cast<const float4*>(delta + c);
          float a0, a1, a2, a3;
          f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), f2_pack(nd.x, nd.y)),
                           f2_pack(pr[c], pr[c + 1])), a0, a1);
          f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), f2_pack(nd.z, nd.w)),
                           f2_pack(pr[c + 2], pr[c + 3])), a2, a3);
          pk[c >> 1] = pack_bf162(a0, a1);
          pk[(c >> 1) + 1] = pack_bf162(a2, a3);
        }
        tmem_st_32x32b_x32(t_dp, pk);
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
      ok = warp_wait(bar(ACC_FULL), un & 1u, abort, limit);
      if (!ok) break;
      tc_fence_after_sync();
      const unsigned rows = __ballot_sync(0xffffffffu, visible);
      const int64_t at = ((static_cast<int64_t>(u.split) * p.a.batch + u.b) * p.a.kv_heads + u.kh) * p.kv_tiles + u.j;
#pragma unroll 1
      for (int y = 0; y < 2; ++y) {
        uint32_t v[64];
        load64(y == 0 ? t_dv : t_dk, v);
        if (p.splits == 1) {
          write_rows(stage, v, y == 0 ? 1.f : p.a.sm_scale, y == 0 ? dv : dk, rows, lane);
        } else if (visible) {
          float* to = p.part + ((at * 2 + y) * TILE + half * 64) * TILE + r;
#pragma unroll
          for (int c = 0; c < 64; ++c) to[c * TILE] = __uint_as_float(v[c]);
        }
      }
      fence_proxy_async_smem();  // the staging writes before the next unit's copies
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(ACC_EMPTY));
        mbar_arrive(bar(KV_EMPTY));
      }
      ++un;
    }
    if (!ok && lane == 0) raise_abort(abort, p.a.err);
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 8) tmem_dealloc(tmem, 512);
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
  for (int x = 0; x < p.splits && x * per < p.t.tiles && visible; ++x) {
    const float* from = p.part + (((static_cast<int64_t>(x) * tiles + blockIdx.x) * 2 + y) * TILE + c0) * TILE + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += from[i * TILE];
  }
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
// another launch.
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
  CUtensorMap tq, td, tk, tv;
  cudaError_t e;
  if ((e = make_tmap_heads(&tq, a.q, a.q_tokens, a.batch, p.t.box, p.t.pack)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&td, a.dout, a.q_tokens, a.batch, p.t.box, p.t.pack)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&tk, a.k, a.kv_tokens, a.batch, TILE, 1)) != cudaSuccess) return e;
  if ((e = make_tmap_heads(&tv, a.v, a.kv_tokens, a.batch, TILE, 1)) != cudaSuccess) return e;
  static std::atomic<uint64_t> dq_smem{0}, dkv_smem{0};
  if ((e = ensure_smem_limit(dq::cross_dq_kernel, static_cast<int>(dq::SMEM_BYTES), dq_smem)) != cudaSuccess) return e;
  if ((e = ensure_smem_limit(dkv::cross_dkv_kernel, static_cast<int>(dkv::SMEM_BYTES), dkv_smem)) != cudaSuccess) return e;
  const int sms = device_sm_count(), bk = a.batch * a.kv_heads;
  p.splits = plan.dq_splits;
  p.total = bk * p.t.tiles * p.splits;
  e = launch_dependent(dq::cross_dq_kernel, dim3(p.total < sms ? p.total : sms), dim3(NUM_THREADS), dq::SMEM_BYTES, stream,
                       tq, td, tk, tv, p);
  if (e != cudaSuccess) return e;
  if (p.splits > 1 &&
      (e = launch_dependent(dq::cross_dq_join_kernel, dim3(bk * p.t.tiles, 16), dim3(TILE), 0, stream, p)) != cudaSuccess)
    return e;
  p.splits = plan.dkv_splits;
  p.total = bk * p.kv_tiles * p.splits;
  e = launch_dependent(dkv::cross_dkv_kernel, dim3(p.total < sms ? p.total : sms), dim3(NUM_THREADS), dkv::SMEM_BYTES, stream,
                       tq, td, tk, tv, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_dependent(dkv::cross_dkv_join_kernel, dim3(bk * p.kv_tiles, 16, 2), dim3(TILE), 0, stream, p);
}

}  // namespace vsa
