// gemm_small.cu -- the products of vsa_linear where a tile of 256 x 256 results is too coarse: a CTA has
// 128 x 64 results of one tile, and a cluster shares the tile along k.
//
// Such calls are bound by what comes before and after the products and by single copies' time, not by traffic (1024 x
// 1536 -> 1536: L2 to the SMs 23 % of its peak over the kernel, 36 % on the busiest SM; issue slots 9 %): a pair
// of CTAs of gemm.cu takes 6.7 us
// for a tile with 256 elements of k, of which its products are 0.4 (two cluster barriers, the epilogue
// of 256 columns, TMA stores), and its tiles in parts a second kernel that adds them.  Here nothing is
// persistent: two warps copy and multiply, then all eight write the results; the CTAs of a cluster leave
// their sums in shared memory, and each adds a share of the tile's results over all of them, in rank
// order, through distributed shared memory.
//
// The 128 results of a tile's one side are those of m or of n, whichever fits better (swap: of n): few
// rows of x meet 128 features.  Either operand comes K-major or MN-major, as in gemm.cu.
//
// One launch takes the two products of a backward, dx and dweight, which do not depend on each other: a cluster
// has tiles of one of them, several where that one's tiles are shared by fewer CTAs.  How a tile is shared
// does not depend on the company, so neither do its bits.
#include <type_traits>

#include "act.cuh"
#include "cross_common.cuh"
#include "gemm.cuh"
#include "vec8.cuh"

namespace vsa {

namespace {

constexpr int TA = 128, TB = 64, BK = 64;  // results of a tile; elements of k of a stage
constexpr int STAGES = 4, WARPS = 8, THREADS = WARPS * 32;
constexpr int MAX_SHARE = 8;  // CTAs of a cluster
constexpr int TMA_WARP = 0, MMA_WARP = 1;
constexpr uint32_t A_BYTES = TA * BK * 2, B_BYTES = TB * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr uint32_t TMEM_COLUMNS = 64;

enum Bar : uint32_t { FULL0 = 0, EMPTY0 = FULL0 + STAGES, DONE = EMPTY0 + STAGES, NUM_BARS };
constexpr uint32_t SM_BAR = STAGES * STAGE_BYTES;
constexpr uint32_t SMEM_BYTES = SM_BAR + NUM_BARS * 8 + 8 + 1024;  // + alignment slack
constexpr int PITCH = TA + 4;  // of the sums, [64][128 + pad] fp32 where the stages were, theirs and the cluster's
static_assert(2 * TB * PITCH * 4 <= STAGES * STAGE_BYTES, "room for the sums");

struct Job {
  CUtensorMap map_a, map_b;
  bool a_mn, b_mn, swap;
  int m, n, steps;  // steps of BK along k
  int tiles_m, tiles;
  int share;        // CTAs of a tile
  const void* bias;
  bool bias_f32;
  int op, act;
  MatrixView out, pre, aux;
};
template <int JOBS>
struct Params {
  Job job[JOBS];
  int first;  // clusters of job 0
  uint32_t* err;
  uint64_t wait_ns;
};

// The four UMMAs of a stage; AS, BS: descriptor steps of 16 elements of k.
template <int AS, int BS>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, c, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 c, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, c;\n\t"
      "add.u64 a, %1, %5;\n\tadd.u64 b, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(AS), "n"(BS)
      : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void load4_cluster(uint32_t addr, float* v) {
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr));
}

// warp_wait, which also keeps a limit that is shorter than the time for which the hardware suspends a probe (some
// microseconds, the whole of such a product): barriers are then looked at without suspending.
constexpr uint64_t SUSPENDED_NS = 20000;
static __device__ __noinline__ bool poll_without_suspending(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!__all_sync(FULL, mbar_test_wait(bar, parity)))
    if (__any_sync(FULL, *abort != 0 || globaltimer_ns() - t0 > limit_ns)) return false;
  return true;
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (limit_ns < SUSPENDED_NS) return __all_sync(FULL, poll_without_suspending(bar, parity, abort, limit_ns));
  return warp_wait(bar, parity, abort, limit_ns);
}

// FORM of a lone product: A_MN + 2 B_MN + 4 swap, and its tiles are (y, z).  A pair reads these from its jobs, which
// costs a lone product up to 1.4 us (64 x 256 -> 256: 5.6 instead of 4.2).
constexpr int PAIR = 8;
template <typename E, int FORM>
__global__ void __launch_bounds__(THREADS) gemm_small_kernel(const __grid_constant__ Params<FORM == PAIR ? 2 : 1> params) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + SM_BAR + NUM_BARS * 8 + 4);
  auto bar = [&](uint32_t b) { return base + SM_BAR + 8u * b; };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  // Of the cluster's CTAs, `share` in a row have a tile.
  constexpr bool pair = FORM == PAIR;
  const int y = blockIdx.y;
  const bool second = pair && y >= params.first;
  const Job& p = params.job[second ? 1 : 0];
  const bool a_mn = pair ? p.a_mn : FORM & 1, b_mn = pair ? p.b_mn : FORM & 2, swap = pair ? p.swap : FORM & 4;
  const int cluster = pair ? static_cast<int>(gridDim.x) : p.share;
  const int peer0 = pair ? static_cast<int>(blockIdx.x) / p.share * p.share : 0, rank = static_cast<int>(blockIdx.x) - peer0;
  int tm = y, tn = blockIdx.z;
  bool has = true;
  if (pair) {
    const int tile = ((second ? y - params.first : y) * cluster + peer0) / p.share;
    has = tile < p.tiles;
    tn = tile / p.tiles_m;
    tm = tile - tn * p.tiles_m;
  }
  const int k0 = has ? rank * p.steps / p.share : 0, k1 = has ? (rank + 1) * p.steps / p.share : 0;
  const int a0 = (swap ? tn : tm) * TA, b0 = (swap ? tm : tn) * TB;
  const uint64_t limit = params.wait_ns;

  if (warp == TMA_WARP && lane == 0) {
    tma_prefetch_desc(&p.map_a);
    tma_prefetch_desc(&p.map_b);
    *abort = 0;
    for (uint32_t b = 0; b < NUM_BARS; ++b) mbar_init(bar(b), 1);
    fence_barrier_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(bar(NUM_BARS), TMEM_COLUMNS);
    tmem_relinquish();
  }
  grid_dependency_wait();
  // 8 results of a row a thread, at a time: a tile has 1024 such, the CTAs of the cluster write those of
  // equal shares of its 64 (swap: rows m of 16 such; else columns n, 128 rows of 1 to 8).  A thread's
  // columns stay the same.
  const int wide = swap ? TA / 8 : TB / 8 / p.share;  // such, side by side
  const int n_first = !has ? p.n : swap ? a0 + threadIdx.x % wide * 8 : b0 + (rank * wide + threadIdx.x % wide) * 8;
  float bias[8] = {};
  if (p.bias && n_first < p.n) {
    if (p.bias_f32) load8(static_cast<const float*>(p.bias) + n_first, bias);
    else load8(static_cast<const E*>(p.bias) + n_first, bias);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + SM_BAR + NUM_BARS * 8);

  bool ok = true;
  if (warp == TMA_WARP) {
    // ------------------------------------------------------------------ TMA producer
    uint32_t it = 0;
    for (int k = k0; k < k1; ++k, ++it) {
      const uint32_t s = it % STAGES, to = base + s * STAGE_BYTES, full = bar(FULL0 + s);
      ok = wait(bar(EMPTY0 + s), ((it / STAGES) & 1u) ^ 1u, abort, limit);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(full, STAGE_BYTES);
        if (a_mn) {
          tma_load_2d(to, &p.map_a, full, a0, k * BK);
          tma_load_2d(to + A_BYTES / 2, &p.map_a, full, a0 + 64, k * BK);
        } else {
          tma_load_2d(to, &p.map_a, full, k * BK, a0);
        }
        if (b_mn) tma_load_2d(to + A_BYTES, &p.map_b, full, b0, k * BK);
        else tma_load_2d(to + A_BYTES, &p.map_b, full, k * BK, b0);
      }
      __syncwarp();
    }
    // No copy is in flight when the CTA ends, also after the issuer has given up.
    if (lane == 0) {
      if (!ok) raise_abort(abort, params.err);
      drain_copies(bar(FULL0), STAGES, it);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------------ UMMA issuer
    const uint32_t idesc = idesc_f16_f32acc(TA, TB, a_mn, b_mn, std::is_same<E, __nv_bfloat16>::value);
    const uint64_t a_desc = sdesc_sw128(base, a_mn ? A_BYTES / 2 : 16, 1024);
    const uint64_t b_desc = sdesc_sw128(base + A_BYTES, b_mn ? B_BYTES : 16, 1024);
    auto stage = [&](uint64_t a, uint64_t b, uint32_t accumulate) {
      if (a_mn && b_mn) product<128, 128>(tmem, a, b, idesc, accumulate);
      else if (a_mn) product<128, 2>(tmem, a, b, idesc, accumulate);
      else if (b_mn) product<2, 128>(tmem, a, b, idesc, accumulate);
      else product<2, 2>(tmem, a, b, idesc, accumulate);
    };
    uint32_t it = 0;
    for (int k = k0; k < k1; ++k, ++it) {
      const uint32_t s = it % STAGES;
      ok = wait(bar(FULL0 + s), (it / STAGES) & 1u, abort, limit);
      if (!ok) break;
      tc_fence_after_sync();
      stage(sdesc_advance(a_desc, s * STAGE_BYTES), sdesc_advance(b_desc, s * STAGE_BYTES), k > k0 ? 1u : 0u);
      umma_commit_elect(bar(EMPTY0 + s));
    }
    if (!ok && lane == 0) raise_abort(abort, params.err);
    umma_commit_elect(bar(DONE));
  }
  // Every product is done, and every stage has been read.  (After an abort this CTA's sums do not leave it but
  // for the others of its cluster, whose results the error word declares invalid: the wait only keeps tensor
  // memory until they are there.)
  ok = wait(bar(DONE), 0, abort, limit) && ok;
  if (!ok) {
    if (lane == 0) {
      raise_abort(abort, params.err);
      volatile int never = 0;
      mbar_wait_bounded(bar(DONE), 0, &never, DRAIN_LIMIT_NS);
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ results
  tc_fence_after_sync();
  float* sums = reinterpret_cast<float*>(gbase);
  __syncthreads();  // both readers of the stages are past them, whichever way they ended
  ok = ok && *abort == 0;  // (the issuer commits DONE also where it has given up)
  {
    const int r = (warp & 3) * 32 + lane, c = (warp >> 2) * 32;
    uint32_t v[32];
    tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) sums[(c + i) * PITCH + r] = __uint_as_float(v[i]);
  }
  tc_fence_before_sync();
  const int mine = TB / p.share, first = rank * mine;  // of the tile's 64
  if (cluster > 1) cluster_sync();
  if (p.share > 1) {
    // Whole rows of 128 sums, 16 bytes a lane: other patterns are several times slower over the
    // cluster.  All CTAs' loads of a row are on their way before the first is added.
    const uint32_t at = smem_u32(sums) + lane * 16;
    float* total = sums + TB * PITCH;
    for (int c = first + warp; c < first + mine; c += WARPS) {
      float from[MAX_SHARE][4], z[4] = {};
#pragma unroll
      for (int r = 0; r < MAX_SHARE; ++r)
        if (r < p.share) load4_cluster(in_cta(at + c * PITCH * 4, peer0 + r), from[r]);
#pragma unroll
      for (int r = 0; r < MAX_SHARE; ++r)
        if (r < p.share) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] += from[r][i];
        }
      *reinterpret_cast<float4*>(total + c * PITCH + lane * 4) = make_float4(z[0], z[1], z[2], z[3]);
    }
    sums = total;
  }
  // The sums of a CTA stay until they have been read.
  if (cluster > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  __syncthreads();
  constexpr int MOST = TA * TB / 8 / THREADS;
  Raw<E> aux[MOST];
  auto here = [&](int i) { return ok && static_cast<int>(threadIdx.x) + i * THREADS < mine * (TA / 8) && n_first < p.n; };
  auto place = [&](int i, int* m) {  // of the thread's result i: its row, and where its sums are
    const int row = (threadIdx.x + i * THREADS) / wide;
    *m = swap ? b0 + first + row : a0 + row;
    return swap ? (first + row) * PITCH + threadIdx.x % wide * 8 : (first + threadIdx.x % wide * 8) * PITCH + row;
  };
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    int m;
    place(i, &m);
    if (here(i) && p.aux.data && m < p.m)
      aux[i].load(static_cast<const E*>(p.aux.data) + m * p.aux.stride + n_first);
  }
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    int m;
    const int at = place(i, &m);
    if (!here(i) || m >= p.m) continue;
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = sums[at + (swap ? j : j * PITCH)];
    if (p.op == GEMM_FWD) {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] += bias[j];
      if (p.pre.data) store8(static_cast<E*>(p.pre.data) + m * p.pre.stride + n_first, z);
      act8(p.act, z);
    }
    if (p.aux.data) {
      float a[8];
      aux[i].widen(a);
      if (p.op == GEMM_FWD) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += a[j];
      } else {
        slope8(p.act, a, z);
      }
    }
    store8(static_cast<E*>(p.out.data) + m * p.out.stride + n_first, z);
  }
  if (cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after_sync();
  if (warp == MMA_WARP) tmem_dealloc(tmem, TMEM_COLUMNS);
}

template <typename E, int FORM>
cudaError_t launch_form(const Params<FORM == PAIR ? 2 : 1>& p, dim3 grid, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = ensure_smem_limit(gemm_small_kernel<E, FORM>, static_cast<int>(SMEM_BYTES), smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = grid.x;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_small_kernel<E, FORM>, p);
}
template <typename E>
cudaError_t launch_typed(const Params<1>& p, dim3 grid, cudaStream_t stream) {
  const Job& j = p.job[0];
  switch (j.a_mn + 2 * j.b_mn + 4 * j.swap) {  // forward 0, 4; dx 2, 5; dweight 3, 7
    case 0: return launch_form<E, 0>(p, grid, stream);
    case 2: return launch_form<E, 2>(p, grid, stream);
    case 3: return launch_form<E, 3>(p, grid, stream);
    case 4: return launch_form<E, 4>(p, grid, stream);
    case 5: return launch_form<E, 5>(p, grid, stream);
    default: return launch_form<E, 7>(p, grid, stream);
  }
}

// How a product is cut: tiles of 128 along n and 64 along m or the other way round, whichever are
// fewer; a cluster of up to 8 while the CTAs do not fill two to an SM and each keeps four steps (with eight
// kept, 32 x 1536 -> 1536 features take 7.3 us instead of 5.8, with two 256 -> 1536 take 5.2 instead of 3.8).
struct Plan {
  bool swap;
  int64_t tiles;
  int steps, share, per;
};
Plan plan_of(int m, int n, int k) {
  Plan q;
  auto count = [](int x, int t) { return static_cast<int64_t>((x + t - 1) / t); };
  const int64_t swapped = count(n, TA) * count(m, TB), straight = count(m, TA) * count(n, TB);
  q.swap = swapped <= straight;
  q.tiles = q.swap ? swapped : straight;
  q.steps = (k + BK - 1) / BK;
  q.share = 1;
  while (q.share < MAX_SHARE && q.tiles * q.share * 2 <= 2 * device_sm_count() && q.steps >= q.share * 2 * 4) q.share *= 2;
  q.per = (q.steps + q.share - 1) / q.share;
  return q;
}

cudaError_t fill(Job* j, GemmOp op, const GemmArgs& a, const Plan& q) {
  const bool bf16 = a.dtype == VSA_BF16, m_mn = op == GEMM_DW, n_mn = op != GEMM_FWD;  // operands as stored
  const int box_m = q.swap ? TB : TA, box_n = q.swap ? TA : TB;
  CUtensorMap* map_m = q.swap ? &j->map_b : &j->map_a;
  CUtensorMap* map_n = q.swap ? &j->map_a : &j->map_b;
  cudaError_t e = m_mn ? make_tmap_matrix(map_m, a.a, a.m, a.k, BK, bf16) : make_tmap_matrix(map_m, a.a, a.k, a.m, box_m, bf16);
  if (e != cudaSuccess) return e;
  e = n_mn ? make_tmap_matrix(map_n, a.b, a.n, a.k, BK, bf16) : make_tmap_matrix(map_n, a.b, a.k, a.n, box_n, bf16);
  j->a_mn = q.swap ? n_mn : m_mn;
  j->b_mn = q.swap ? m_mn : n_mn;
  j->swap = q.swap;
  j->m = a.m;
  j->n = a.n;
  j->steps = q.steps;
  j->tiles_m = (a.m + box_m - 1) / box_m;
  j->tiles = static_cast<int>(q.tiles);
  j->share = q.share;
  j->bias = a.bias;
  j->bias_f32 = a.bias_f32;
  j->op = op;
  j->act = a.act;
  j->out = a.out;
  j->pre = a.pre;
  j->aux = a.aux;
  return e;
}

}  // namespace

// Where its CTAs fit on the GPU at once and its estimated time is the shorter.  Measured, us, here and
// with gemm.cu's tiles (forward, rows x in -> out features):
//   512 x 1536 -> 1536    8.0 and 11.2      512 x 4096 -> 1536   12.7 and 13.5
//   1024 x 1536 -> 1536   9.0 and 11.9      512 x 6144 -> 1536   16.4 and 15.1
//   256 x 1536 -> 9216   10.5 and 12.0      384 x 1536 -> 9216   17.8 and 12.5
// The estimate: 3 us for a call, 1.5 for a cluster, and for a step of 64 elements of k 0.2 where an SM has one
// CTA and 0.28 where it has two.
bool use_gemm_small(int m, int n, int k) {
  const Plan q = plan_of(m, n, k);
  const int64_t ctas = q.tiles * q.share;
  if (ctas > 2 * device_sm_count()) return false;
  return 3.0 + (q.share > 1 ? 1.5 : 0.0) + q.per * (ctas > device_sm_count() ? 0.28 : 0.2) <= gemm_microseconds(m, n, k);
}

cudaError_t launch_gemm_small(GemmOp op, const GemmArgs& a, cudaStream_t stream) {
  const Plan q = plan_of(a.m, a.n, a.k);
  Params<1> p{};
  const cudaError_t e = fill(&p.job[0], op, a, q);
  if (e != cudaSuccess) return e;
  p.first = static_cast<int>(q.tiles);
  p.err = a.err;
  p.wait_ns = a.wait_ns;
  const dim3 grid(q.share, p.job[0].tiles_m, p.job[0].tiles / p.job[0].tiles_m);
  return a.dtype == VSA_BF16 ? launch_typed<__nv_bfloat16>(p, grid, stream) : launch_typed<__half>(p, grid, stream);
}

// Where the CTAs of both fit on the GPU at once (us on the GPU, in one launch and in two: 64 x 256 -> 256 4.5 and 6.7,
// 512 x 512 -> 512 6.3 and 10.6, 1021 x 1000 -> 264 9.0 and 12.5; with 480 CTAs, 256 x 1536 -> 1536, 13.2 and 11.9).
bool use_gemm_small_pair(const GemmArgs& a, const GemmArgs& b) {
  if (!use_gemm_small(a.m, a.n, a.k) || !use_gemm_small(b.m, b.n, b.k)) return false;
  const Plan q = plan_of(a.m, a.n, a.k), r = plan_of(b.m, b.n, b.k);
  return q.tiles * q.share + r.tiles * r.share <= 2 * device_sm_count();
}

cudaError_t launch_gemm_small_pair(GemmOp op_a, const GemmArgs& a, GemmOp op_b, const GemmArgs& b, cudaStream_t stream) {
  const Plan q = plan_of(a.m, a.n, a.k), r = plan_of(b.m, b.n, b.k);
  Params<2> p{};
  cudaError_t e = fill(&p.job[0], op_a, a, q);
  if (e == cudaSuccess) e = fill(&p.job[1], op_b, b, r);
  if (e != cudaSuccess) return e;
  const int cluster = q.share > r.share ? q.share : r.share;
  p.first = static_cast<int>((q.tiles * q.share + cluster - 1) / cluster);
  p.err = a.err;
  p.wait_ns = a.wait_ns;
  const dim3 grid(cluster, static_cast<unsigned>(p.first + (r.tiles * r.share + cluster - 1) / cluster));
  return a.dtype == VSA_BF16 ? launch_form<__nv_bfloat16, PAIR>(p, grid, stream) : launch_form<__half, PAIR>(p, grid, stream);
}

}  // namespace vsa
