// gemm.cu -- matrix products on pairs of CTAs (tcgen05, cta_group::2), for vsa_linear.
//
// A pair of CTAs works on a tile of 256 x 256 results: each CTA stages its 128 rows of A and its 128 of
// B's 256 rows for 64 elements of k (32 KB a stage), and one UMMA of 256 x 256 x 16, issued by the
// pair's first CTA, reads both CTAs' shared memory, so every operand element is copied once per
// pair.  Each CTA's 128 x 256 sums lie in its tensor memory, twice: while the epilogue warps empty one
// tile, the next one's products run.
//
// Operands come row by row in k (K-major) or in m or n (MN-major) as the caller stores them; the copy
// and the descriptors differ, no operand is transposed in memory.
//
// Work: tiles in groups of GROUP_M rows of tiles (the operands of a wave of pairs, about 8 x 9 tiles,
// stay in L2), dealt to a persistent grid.  Tiles that do not fill a whole wave are split along k: the
// parts leave fp32 sums in the workspace, which gemm_join_kernel adds in part order and finishes.
// The same rule splits small problems, all of whose tiles are such a rest.
//
// Roles (384 or 640 threads): warp 0 TMA producer; warp 1 UMMA issuer (first CTA of the pair); warp 2 tensor
// memory; warp 3 biases; warps from 4 on epilogue, a half or a quarter of a row of the tile per thread: bias,
// activation, residual or slope in fp32, rounded once, through swizzled shared memory to TMA stores, which clip
// at the matrix's edges.  ACT: an activation (or its slope).  Without one it has kernels of its own: a branch
// around it in the epilogue took 32760 x 512 -> 1536 from 42 us to 47, with a residual from 58 to 65.
//
// Bound by the tensor cores (91 % of their cycles): 32760 x 1536 x 6144 with bias and gelu_tanh 324 us in
// bursts (1908 TFLOP/s, what the library reaches at 8192 x 8192 x 8192; at this size its plain product takes 304 us,
// 2030 TFLOP/s), 131040 rows 1267 (the library's 1210 to 1230); dx 328, dweight
// 305.  In runs of a second the power cap holds all of them to about 1650 TFLOP/s.  A residual or a
// slope to read adds 27 us, pre to write 45: the operands take about 18 TB/s between L2 and the SMs, and what
// the epilogue moves comes on top.  Four epilogue warps instead of eight: 455 us with bias and gelu_tanh.
#include <type_traits>

#include "act.cuh"
#include "cross_common.cuh"
#include "gemm.cuh"
#include "vec8.cuh"

namespace vsa {

namespace {

constexpr int BM = 256, BN = 256, BK = 64;  // of a pair
constexpr int GROUP_M = 8;
constexpr int TMA_WARP = 0, MMA_WARP = 1, TMEM_WARP = 2, BIAS_WARP = 3, EPI_WARP = 4;
constexpr int EPI_COLUMNS = 1024;  // of all epilogue warps together, a quarter of the rows each
constexpr uint32_t OPERAND_BYTES = 128 * BK * 2;  // a CTA's A or B of a stage
constexpr uint32_t STAGE_BYTES = 2 * OPERAND_BYTES;
constexpr uint32_t OUT_BYTES = 32 * 128;  // 32 rows x 64 results of an epilogue warp

constexpr int STAGES = 5;
// Buffers of the epilogue warps, one for each 64 results of their 32 rows.  With pre (and no operand to load) a
// warp of 128 columns has four of 32 results, two for pre and two for out, so that a store has the time of 32
// columns' work to leave its buffer: one of 64 for each of the two waited for its last store every time (32760 x
// 1536 x 6144, pre and gelu_tanh 373 us, now 366; gelu 384 and 371).  A warp of 64 columns has two of 32 and waits.
constexpr int BUFFERS = 16;

enum Bar : uint32_t {
  FULL0 = 0,                        // first CTA: both CTAs' copies of a stage have landed
  EMPTY0 = FULL0 + STAGES,          // each CTA: a stage's products are done
  ACC_FULL0 = EMPTY0 + STAGES,      // each CTA: a tile's products are done
  ACC_EMPTY0 = ACC_FULL0 + 2,       // first CTA: both CTAs' epilogues have read a tile
  AUX0 = ACC_EMPTY0 + 2,            // per epilogue warp and buffer
  DRAIN = AUX0 + BUFFERS,
  BIAS_FULL,                        // a tile's biases are in shared memory
  BIAS_EMPTY,                       // the epilogue warps have read them
  NUM_BARS
};
constexpr uint32_t SM_OUT = STAGES * STAGE_BYTES;
constexpr uint32_t SM_BIAS = SM_OUT + BUFFERS * OUT_BYTES;  // 256 floats
constexpr uint32_t SM_BAR = SM_BIAS + BN * 4;
constexpr uint32_t SMEM_BYTES = SM_BAR + NUM_BARS * 8 + 8 + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

struct Maps {
  CUtensorMap a, b, out, pre, aux;
};

struct Params {
  int m, n, steps;             // steps of BK along k
  int tiles_m, tiles_n;
  int full, tail;              // whole tiles; tiles in parts
  int splits, per;             // parts of one, and their steps
  int units;
  float* parts;                // [split][tail tile][CTA][256 columns][128 rows]
  const void* bias;
  bool bias_f32, has_pre;  // has_pre: in a kernel with PRE, or from the registers
  int act;
  MatrixView out, pre, aux;    // of the join
  uint32_t* err;
  uint64_t wait_ns;
};

// ------------------------------------------------------------------------------ pairs of CTAs

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the first CTA's copy of a shared-memory object of this one.
__device__ __forceinline__ uint32_t in_first_cta(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A box into this CTA's shared memory, counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src),
               "r"(c0), "r"(c1)
               : "memory");
}
// When the products issued so far are done: an arrival on the barrier at this offset in both CTAs.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 both;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "mov.b16 both, 3;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n\t}" ::"r"(
          bar)
      : "memory");
}
__device__ __forceinline__ void commit_first(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// The four UMMAs of a stage, issued by the lane elect.sync chooses of a converged warp.  AS, BS:
// descriptor steps of 16 elements of k.
template <int AS, int BS>
__device__ __forceinline__ void product_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, c, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 c, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, c;\n\t"
      "add.u64 a, %1, %5;\n\tadd.u64 b, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(AS), "n"(BS)
      : "memory");
}

// Byte offset of 16-byte chunk c of row r of 64 bytes, 64-byte swizzle.
__device__ __forceinline__ uint32_t swizzled64(uint32_t r, uint32_t c) { return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4); }

// ------------------------------------------------------------------------------ units

struct Unit {
  int m0, n0;  // of the pair's tile
  int k0, k1;  // steps
  int part;    // slot of its sums in the workspace, -1: a whole tile
};

__device__ __forceinline__ void tile_origin(const Params& p, int tile, int* m0, int* n0) {
  const int band = GROUP_M * p.tiles_n, g = tile / band, r = tile - g * band;
  const int rows = min(GROUP_M, p.tiles_m - g * GROUP_M);
  const int n = r / rows;
  *m0 = (g * GROUP_M + r - n * rows) * BM;
  *n0 = n * BN;
}

__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  Unit x;
  if (u < p.full) {
    tile_origin(p, u, &x.m0, &x.n0);
    x.k0 = 0;
    x.k1 = p.steps;
    x.part = -1;
  } else {
    const int v = u - p.full, split = v / p.tail, t = v - split * p.tail;
    tile_origin(p, p.full + t, &x.m0, &x.n0);
    x.k0 = split * p.per;
    x.k1 = min(x.k0 + p.per, p.steps);
    x.part = p.splits > 1 ? v : -1;
  }
  return x;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) { return pack_bf162(lo, hi); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename E>
__device__ __forceinline__ uint4 pack8(const float* z) {
  return make_uint4(pack2(z[0], z[1], E()), pack2(z[2], z[3], E()), pack2(z[4], z[5], E()), pack2(z[6], z[7], E()));
}

template <typename E>
__device__ __forceinline__ void add_bias(const void* bias, bool f32, int c, float* z) {
  float b[8];
  if (f32) load8(static_cast<const float*>(bias) + c, b);
  else load8(static_cast<const E*>(bias) + c, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += b[i];
}

// Busy for `ns` of wall time: longer than any copy takes to land.
__device__ __noinline__ void linger(uint64_t ns) {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < ns) {
  }
}

template <typename E, int OP, bool AUX, bool PRE, bool ACT, int EPI_WARPS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(128 + EPI_WARPS * 32, 1)
    gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  constexpr int COLUMNS = EPI_COLUMNS / EPI_WARPS, CHUNKS = COLUMNS / 64;  // of an epilogue warp; a buffer to each 64
  constexpr bool A_MN = OP == GEMM_DW, B_MN = OP != GEMM_FWD;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + SM_BAR + NUM_BARS * 8 + 4);
  auto bar = [&](uint32_t b) { return base + SM_BAR + 8u * b; };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = uniform(static_cast<int>(cluster_rank()));
  const int first = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const uint64_t limit = p.wait_ns;

  if (threadIdx.x == 32) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
    tma_prefetch_desc(&maps.out);
    if (PRE) tma_prefetch_desc(&maps.pre);
    if (AUX) tma_prefetch_desc(&maps.aux);
  }
  if (threadIdx.x == 0) {
    *abort = 0;
    for (uint32_t b = 0; b < NUM_BARS; ++b)
      mbar_init(bar(b), b >= ACC_EMPTY0 && b < AUX0 ? 2 * EPI_WARPS : b == BIAS_EMPTY ? EPI_WARPS : 1);
    fence_barrier_init();
  }
  if (warp == TMEM_WARP) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bar(NUM_BARS)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_dependency_wait();
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they start at 0

  if (warp == TMA_WARP) {
    // ------------------------------------------------------------------ TMA producer
    uint32_t it = 0;
    bool ok = true;
    for (int u = first; u < p.units && ok; u += pairs) {
      const Unit x = unit_of(p, u);
      const int m = x.m0 + rank * 128, n = x.n0 + rank * 128;
#pragma unroll 1
      for (int k = x.k0; k < x.k1; ++k) {
        const uint32_t s = it % STAGES;
        ok = warp_wait(bar(EMPTY0 + s), ((it / STAGES) & 1u) ^ 1u, abort, limit);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t full = in_first_cta(bar(FULL0 + s)), to = base + s * STAGE_BYTES;
          if (rank == 0) mbar_arrive_expect_tx(bar(FULL0 + s), 2 * STAGE_BYTES);
          if (A_MN) {
            tma_load_pair(to, &maps.a, full, m, k * BK);
            tma_load_pair(to + OPERAND_BYTES / 2, &maps.a, full, m + 64, k * BK);
          } else {
            tma_load_pair(to, &maps.a, full, k * BK, m);
          }
          if (B_MN) {
            tma_load_pair(to + OPERAND_BYTES, &maps.b, full, n, k * BK);
            tma_load_pair(to + OPERAND_BYTES + OPERAND_BYTES / 2, &maps.b, full, n + 64, k * BK);
          } else {
            tma_load_pair(to + OPERAND_BYTES, &maps.b, full, k * BK, n);
          }
        }
        __syncwarp();
        ++it;
      }
    }
    // The last products' arrivals, which the first CTA sends to both, come before either CTA ends.
    for (uint32_t i = it > STAGES ? it - STAGES : 0; i < it && ok; ++i)
      ok = warp_wait(bar(EMPTY0 + i % STAGES), (i / STAGES) & 1u, abort, limit);
    if (!ok && lane == 0) {
      raise_abort(abort, p.err);
      // Copies in flight land, of both CTAs, before the pair's shared memory goes away.
      if (rank == 0) drain_copies(bar(FULL0), STAGES, it);
      linger(1000000);
    }
    __syncwarp();
  } else if (warp == MMA_WARP && rank == 0) {
    // ------------------------------------------------------------------ UMMA issuer
    constexpr uint32_t IDESC = idesc_f16_f32acc(BM, BN, A_MN, B_MN, std::is_same<E, __nv_bfloat16>::value);
    const uint64_t a_desc = sdesc_sw128(base, A_MN ? OPERAND_BYTES / 2 : 16, 1024);
    const uint64_t b_desc = sdesc_sw128(base + OPERAND_BYTES, B_MN ? OPERAND_BYTES / 2 : 16, 1024);
    uint32_t it = 0, done = 0;
    bool ok = true;
    for (int u = first; u < p.units && ok; u += pairs) {
      const Unit x = unit_of(p, u);
      const uint32_t acc = done & 1u;
      ok = warp_wait(bar(ACC_EMPTY0 + acc), ((done >> 1) & 1u) ^ 1u, abort, limit);
      if (!ok) break;
      tc_fence_after_sync();
#pragma unroll 1
      for (int k = x.k0; k < x.k1; ++k) {
        const uint32_t s = it % STAGES;
        ok = warp_wait(bar(FULL0 + s), (it / STAGES) & 1u, abort, limit);
        if (!ok) break;
        tc_fence_after_sync();
        product_pair<A_MN ? 128 : 2, B_MN ? 128 : 2>(tmem + acc * BN, sdesc_advance(a_desc, s * STAGE_BYTES),
                                                     sdesc_advance(b_desc, s * STAGE_BYTES), IDESC, k > x.k0 ? 1u : 0u);
        commit_pair(bar(EMPTY0 + s));
        ++it;
      }
      if (!ok) break;
      commit_pair(bar(ACC_FULL0 + acc));
      ++done;
    }
    if (!ok && lane == 0) raise_abort(abort, p.err);
    if (it > 0) {
      // Every UMMA has completed before tensor memory is released.
      commit_first(bar(DRAIN));
      volatile int never = 0;
      if (lane == 0) mbar_wait_bounded(bar(DRAIN), 0, &never, DRAIN_LIMIT_NS);
      __syncwarp();
    }
  } else if (warp == BIAS_WARP && OP == GEMM_FWD && p.bias) {
    // ------------------------------------------------------------------ biases
    // 8 a lane, widened: loaded by the epilogue where it needs them they cost it a wait for every
    // 32 columns (32 rows, 256 -> 1536 features: 3 of 8.8 us).
    uint32_t done = 0;
    bool ok = true;
    for (int u = first; u < p.units && ok; u += pairs) {
      const Unit x = unit_of(p, u);
      if (x.part >= 0) continue;
      float b[8] = {};
      if (x.n0 + lane * 8 < p.n) {
        if (p.bias_f32) load8(static_cast<const float*>(p.bias) + x.n0 + lane * 8, b);
        else load8(static_cast<const E*>(p.bias) + x.n0 + lane * 8, b);
      }
      ok = warp_wait(bar(BIAS_EMPTY), (done & 1u) ^ 1u, abort, limit);
      if (!ok) break;
      float4* to = reinterpret_cast<float4*>(gbase + SM_BIAS) + lane * 2;
      to[0] = make_float4(b[0], b[1], b[2], b[3]);
      to[1] = make_float4(b[4], b[5], b[6], b[7]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BIAS_FULL));
      ++done;
    }
    if (!ok && lane == 0) raise_abort(abort, p.err);
    __syncwarp();
  } else if (warp >= EPI_WARP) {
    // ------------------------------------------------------------------ epilogue
    // A warp reads the quarter of tensor memory's rows that its number gives; two share it, 128 columns
    // each.
    const int e = warp - EPI_WARP, row0 = (warp & 3) * 32, col0 = (e >> 2) * COLUMNS;
    const uint32_t t_row = (static_cast<uint32_t>(row0) << 16) + col0;
    const uint32_t room = base + SM_OUT + e * CHUNKS * OUT_BYTES, aux_bar = bar(AUX0 + e * CHUNKS);
    const uint32_t acc_empty = in_first_cta(bar(ACC_EMPTY0));
    uint32_t done = 0, whole = 0;  // tiles; those that are not parts
    bool ok = true, pending = false;
    for (int u = first; u < p.units && ok; u += pairs) {
      const Unit x = unit_of(p, u);
      const int m0 = x.m0 + rank * 128 + row0;
      const uint32_t acc = done & 1u;
      if (AUX && x.part < 0) {
        // The epilogue's operand comes while the products run, each 64 columns into the buffer that
        // their results leave from; the last tile's stores have left them.
        if (lane == 0) {
          bulk_wait_read_all();
#pragma unroll 1
          for (int c = 0; c < CHUNKS; ++c) {
            mbar_arrive_expect_tx(aux_bar + 8u * c, OUT_BYTES);
            tma_load_2d(room + c * OUT_BYTES, &maps.aux, aux_bar + 8u * c, x.n0 + col0 + c * 64, m0);
          }
        }
        __syncwarp();
        pending = true;
      }
      ok = warp_wait(bar(ACC_FULL0 + acc), (done >> 1) & 1u, abort, limit);
      const bool bias = OP == GEMM_FWD && p.bias && x.part < 0;
      if (ok && bias) ok = warp_wait(bar(BIAS_FULL), whole & 1u, abort, limit);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t t_acc = tmem + t_row + acc * BN;
      if (x.part >= 0) {
        float* to = p.parts + ((static_cast<int64_t>(x.part) * 2 + rank) * BN + col0) * 128 + row0 + lane;
#pragma unroll 1
        for (int c = 0; c < COLUMNS && x.n0 + col0 + c < p.n && m0 < p.m; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(t_acc + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) to[(c + i) * 128] = __uint_as_float(v[i]);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < CHUNKS; ++c) {
          const int n0 = x.n0 + col0 + c * 64;
          const uint32_t out = room + c * OUT_BYTES;
          if (AUX) {
            ok = warp_wait(aux_bar + 8u * c, whole & 1u, abort, limit);
            if (!ok) break;
          } else if (!PRE) {
            if (lane == 0) bulk_wait_read<CHUNKS - 1>();  // all but the last 64 columns' stores
            __syncwarp();
          }
          if (n0 >= p.n || m0 >= p.m) {
            // Nothing of these 64 columns (131040 x 64 -> 64: 22.4 us, now 18.7): groups of no store, which are
            // counted all the same.
            if (lane == 0) {
              bulk_commit_group();
              if (PRE) bulk_commit_group();
            }
            continue;
          }
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(t_acc + c * 64 + h * 32, v);
            const int col = n0 + h * 32;
            // The other operands are on their way before the wait for tensor memory: the stores below
            // keep what follows them in order.
            float4 b4[8];
            if (bias) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                b4[j] = reinterpret_cast<const float4*>(gbase + SM_BIAS)[(col0 + c * 64 + h * 32) / 4 + j];
            }
            Raw<E> r[4];
            if (AUX) {
#pragma unroll
              for (int j = 0; j < 4; ++j) r[j].u[0] = ld_shared16(out + swizzled(lane, h * 4 + j));
            }
            tmem_wait_ld_regs(v);
            uint4 t[4], before[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float z[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) z[i] = __uint_as_float(v[8 * j + i]);
              if (OP == GEMM_FWD) {
                if (bias) {
                  z[0] += b4[2 * j].x, z[1] += b4[2 * j].y, z[2] += b4[2 * j].z, z[3] += b4[2 * j].w;
                  z[4] += b4[2 * j + 1].x, z[5] += b4[2 * j + 1].y, z[6] += b4[2 * j + 1].z, z[7] += b4[2 * j + 1].w;
                }
                if (PRE) {
                  before[j] = pack8<E>(z);
                } else if (AUX && p.has_pre && col + j * 8 < p.n && m0 + lane < p.m) {
                  // No room for a buffer of its own: straight from the registers.
                  store8(static_cast<E*>(p.pre.data) + (m0 + lane) * p.pre.stride + col + j * 8, z);
                }
                if (ACT) act8(p.act, z);
              }
              if (AUX) {
                float a[8];
                r[j].widen(a);
                if (OP == GEMM_FWD) {
#pragma unroll
                  for (int i = 0; i < 8; ++i) z[i] += a[i];
                } else {
                  slope8(p.act, a, z);
                }
              }
              t[j] = pack8<E>(z);
            }
            if (PRE) {
              if (lane == 0) bulk_wait_read<CHUNKS - 1>();  // all but the last 32 columns' stores
              __syncwarp();
              const uint32_t here = room + h % CHUNKS * OUT_BYTES;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t spot = here + swizzled64(lane, j);
                st_shared16(spot, before[j].x, before[j].y, before[j].z, before[j].w);
                st_shared16(spot + OUT_BYTES / 2, t[j].x, t[j].y, t[j].z, t[j].w);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (col < p.n && m0 < p.m) {
                  tma_store_2d(&maps.pre, here, col, m0);
                  tma_store_2d(&maps.out, here + OUT_BYTES / 2, col, m0);
                }
                bulk_commit_group();
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) st_shared16(out + swizzled(lane, h * 4 + j), t[j].x, t[j].y, t[j].z, t[j].w);
            }
          }
          if (PRE) continue;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (n0 < p.n && m0 < p.m) tma_store_2d(&maps.out, out, n0, m0);
            bulk_commit_group();
          }
        }
        if (!ok) break;
        pending = false;
        ++whole;
        if (bias) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BIAS_EMPTY));
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_cluster(acc_empty + 8u * acc);
      ++done;
    }
    if (!ok && lane == 0) {
      raise_abort(abort, p.err);
      volatile int never = 0;
      for (int c = 0; c < CHUNKS && pending; ++c)
        mbar_wait_bounded(aux_bar + 8u * c, whole & 1u, &never, DRAIN_LIMIT_NS);
    }
    if (lane == 0) bulk_wait_read_all();  // (the end of the grid waits for the writes)
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  if (warp == TMEM_WARP)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// The tiles in parts, added in part order; then 8 columns of a row a thread.  GROUPS 1: a CTA has 32 rows x 64
// columns of a tile, a warp 8 columns of every part (128-byte loads of 32 rows).  GROUPS 8, many parts: 8
// columns, a warp every eighth part, and their sums in warp order (dweight of 32760 rows, 128 x 128 in
// 76 parts: 34.3 us, now 11.7; 131040 rows, 64 x 64: 44.8 and 16.6).
template <typename E, int OP, int GROUPS>
__global__ void __launch_bounds__(256) gemm_join_kernel(const __grid_constant__ Params p) {
  constexpr int COLUMNS = 64 / GROUPS;
  __shared__ float sums[GROUPS][32][COLUMNS + 1];
  grid_dependency_wait();
  const int t = blockIdx.y, sub = blockIdx.x, rank = sub / (16 * GROUPS), r0 = (sub & 3) * 32;
  const int c0 = (sub >> 2) % (4 * GROUPS) * COLUMNS;
  int m0, n0;
  tile_origin(p, p.full + t, &m0, &n0);
  m0 += rank * 128 + r0;
  n0 += c0;
  if (m0 >= p.m || n0 >= p.n) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int group = GROUPS == 1 ? 0 : w, column = GROUPS == 1 ? w * 8 : 0;
  const float* from = p.parts + ((static_cast<int64_t>(t) * 2 + rank) * BN + c0 + column) * 128 + r0 + lane;
  const int64_t step = static_cast<int64_t>(p.tail) * 2 * BN * 128;
  float s[8] = {};
#pragma unroll 4
  for (int i = group; i < p.splits; i += GROUPS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += from[i * step + j * 128];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[group][lane][column + j] = s[j];
  __syncthreads();
  const int r = m0 + threadIdx.x * 8 / COLUMNS, c = n0 + threadIdx.x * 8 % COLUMNS;
  if (threadIdx.x * 8 >= 32 * COLUMNS || r >= p.m || c >= p.n) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[j] = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) s[j] += sums[g][threadIdx.x * 8 / COLUMNS][threadIdx.x * 8 % COLUMNS + j];
  }
  if (OP == GEMM_FWD) {
    if (p.bias) add_bias<E>(p.bias, p.bias_f32, c, s);
    if (p.pre.data) store8(static_cast<E*>(p.pre.data) + r * p.pre.stride + c, s);
    act8(p.act, s);
  }
  if (OP != GEMM_DW && p.aux.data) {
    float a[8];
    load8(static_cast<const E*>(p.aux.data) + r * p.aux.stride + c, a);
    if (OP == GEMM_FWD) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += a[j];
    } else {
      slope8(p.act, a, s);
    }
  }
  store8(static_cast<E*>(p.out.data) + r * p.out.stride + c, s);
}

// ------------------------------------------------------------------------------ plan

// The tiles of a last, incomplete wave in `splits` parts each.  Costs in steps of 64 along k (0.27 us): a
// unit's start and end about 5, the join 9 for its launch and 0.1 for each part it reads.
struct Plan {
  int tiles_m, tiles_n, steps, full, tail, splits, per, units, pairs;
  size_t bytes;
};
Plan plan_of(int m, int n, int k) {
  Plan q{};
  q.tiles_m = (m + BM - 1) / BM;
  q.tiles_n = (n + BN - 1) / BN;
  q.steps = (k + BK - 1) / BK;
  q.pairs = device_sm_count() > 1 ? device_sm_count() / 2 : 1;
  const int64_t tiles = static_cast<int64_t>(q.tiles_m) * q.tiles_n;
  q.full = static_cast<int>(tiles / q.pairs * q.pairs);
  q.tail = static_cast<int>(tiles - q.full);
  q.splits = 1;
  q.per = q.steps;
  if (q.tail > 0) {
    double best = q.steps + 5.0;
    // The parts that lengths of a part give (about 2 sqrt(steps) of them): s, then the next with shorter
    // ones.
    for (int s = 2; s <= q.steps && static_cast<int64_t>(s) * q.tail <= 2 * q.pairs;) {
      const int per = (q.steps + s - 1) / s;
      s = (q.steps + per - 1) / per;  // no part without a step
      if (static_cast<int64_t>(s) * q.tail > 2 * q.pairs) break;
      const int rounds = (s * q.tail + q.pairs - 1) / q.pairs;
      const double cost = rounds * (per + 5.0) + 9.0 + 0.1 * s * q.tail;
      if (cost < best) {
        best = cost;
        q.splits = s;
        q.per = per;
      }
      if (per == 1) break;
      s = (q.steps + per - 2) / (per - 1);
    }
  }
  q.units = q.full + q.tail * q.splits;
  if (q.units < q.pairs) q.pairs = q.units;
  q.bytes = q.splits > 1 ? static_cast<size_t>(q.tail) * q.splits * BM * BN * sizeof(float) : 0;
  return q;
}

template <typename E, int OP, bool AUX, bool PRE, bool ACT, int EPI_WARPS>
cudaError_t launch_main(const Maps& maps, const Params& p, int pairs, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  const auto kernel = gemm_kernel<E, OP, AUX, PRE, ACT, EPI_WARPS>;
  const cudaError_t e = ensure_smem_limit(kernel, static_cast<int>(SMEM_BYTES), smem_set);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(2 * pairs), dim3(128 + EPI_WARPS * 32), SMEM_BYTES, stream, maps, p);
}

// Twice the epilogue warps where activations or slopes would take longer than a tile's products.  Us with 8 and 16
// of them, 32760 rows -> 1536 features, by elements of k:
//   gelu_tanh            128: 54 and 44   512: 58 and 52   768: 63 and 59   1024: 69 and 71   1536: 94 and 97
//   the same + residual  128: 74 and 63   512: 77 and 68   768: 81 and 73   1024: 85 and 79   1536: 101 and 103
// Without an activation 16 win nothing (512: 40 and 42, with a residual 57 and 58).
template <typename E, int OP, bool AUX, bool PRE, bool ACT>
cudaError_t launch_kernel(const Maps& maps, const Params& p, int pairs, cudaStream_t stream) {
  cudaError_t e;
  if constexpr (ACT)
    e = p.steps <= (AUX ? 16 : 12) ? launch_main<E, OP, AUX, PRE, ACT, 16>(maps, p, pairs, stream)
                                   : launch_main<E, OP, AUX, PRE, ACT, 8>(maps, p, pairs, stream);
  else
    e = launch_main<E, OP, AUX, PRE, ACT, 8>(maps, p, pairs, stream);
  if (e != cudaSuccess || p.splits == 1) return e;
  if (p.splits >= 8) return launch_dependent(gemm_join_kernel<E, OP, 8>, dim3(256, p.tail), dim3(256), 0, stream, p);
  return launch_dependent(gemm_join_kernel<E, OP, 1>, dim3(32, p.tail), dim3(256), 0, stream, p);
}

template <typename E>
cudaError_t launch_typed(GemmOp op, const Maps& maps, const Params& p, int pairs, cudaStream_t stream) {
  const bool aux = p.aux.data != nullptr;
  switch (op) {
    case GEMM_FWD:
      if (!aux && p.has_pre) return launch_kernel<E, GEMM_FWD, false, true, true>(maps, p, pairs, stream);
      if (!p.act)
        return aux ? launch_kernel<E, GEMM_FWD, true, false, false>(maps, p, pairs, stream)
                   : launch_kernel<E, GEMM_FWD, false, false, false>(maps, p, pairs, stream);
      return aux ? launch_kernel<E, GEMM_FWD, true, false, true>(maps, p, pairs, stream)
                 : launch_kernel<E, GEMM_FWD, false, false, true>(maps, p, pairs, stream);
    case GEMM_DX:
      return aux ? launch_kernel<E, GEMM_DX, true, false, true>(maps, p, pairs, stream)
                 : launch_kernel<E, GEMM_DX, false, false, false>(maps, p, pairs, stream);
    default:
      return launch_kernel<E, GEMM_DW, false, false, false>(maps, p, pairs, stream);
  }
}

}  // namespace

double gemm_microseconds(int m, int n, int k) {
  const Plan q = plan_of(m, n, k);
  const int rounds = (q.tail * q.splits + q.pairs - 1) / q.pairs;
  return 7.5 + 0.27 * (static_cast<double>(q.full / q.pairs) * q.steps + static_cast<double>(rounds) * q.per) +
         (q.splits > 1 ? 3.5 : 0.0);
}

size_t gemm_workspace(int m, int n, int k) { return use_gemm_small(m, n, k) ? 0 : align_up(plan_of(m, n, k).bytes, 256); }

cudaError_t launch_gemm(GemmOp op, const GemmArgs& a, cudaStream_t stream) {
  if (use_gemm_small(a.m, a.n, a.k)) return launch_gemm_small(op, a, stream);
  const Plan q = plan_of(a.m, a.n, a.k);
  Params p{};
  p.m = a.m;
  p.n = a.n;
  p.steps = q.steps;
  p.tiles_m = q.tiles_m;
  p.tiles_n = q.tiles_n;
  p.full = q.full;
  p.tail = q.tail;
  p.splits = q.splits;
  p.per = q.per;
  p.units = q.units;
  p.parts = reinterpret_cast<float*>(a.workspace);
  p.bias = a.bias;
  p.bias_f32 = a.bias_f32;
  p.has_pre = a.pre.data != nullptr;
  p.act = a.act;
  p.out = a.out;
  p.pre = a.pre;
  p.aux = a.aux;
  p.err = a.err;
  p.wait_ns = a.wait_ns;
  const bool bf16 = a.dtype == VSA_BF16;
  Maps maps{};
  cudaError_t e;
  // Rows of A and B as stored: of m (n) with k along them, or of k with m (n) along them.
  e = op == GEMM_DW ? make_tmap_matrix(&maps.a, a.a, a.m, a.k, BK, bf16) : make_tmap_matrix(&maps.a, a.a, a.k, a.m, 128, bf16);
  if (e != cudaSuccess) return e;
  e = op == GEMM_FWD ? make_tmap_matrix(&maps.b, a.b, a.k, a.n, 128, bf16) : make_tmap_matrix(&maps.b, a.b, a.n, a.k, BK, bf16);
  if (e != cudaSuccess) return e;
  const bool narrow = op == GEMM_FWD && a.pre.data && !a.aux.data;  // PRE: boxes of 32 columns
  if ((e = make_tmap_matrix(&maps.out, a.out, a.n, a.m, 32, bf16, narrow)) != cudaSuccess) return e;
  if (narrow && (e = make_tmap_matrix(&maps.pre, a.pre, a.n, a.m, 32, bf16, true)) != cudaSuccess) return e;
  if (a.aux.data && (e = make_tmap_matrix(&maps.aux, a.aux, a.n, a.m, 32, bf16)) != cudaSuccess) return e;
  return bf16 ? launch_typed<__nv_bfloat16>(op, maps, p, q.pairs, stream) : launch_typed<__half>(op, maps, p, q.pairs, stream);
}

}  // namespace vsa
