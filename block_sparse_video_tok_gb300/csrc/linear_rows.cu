// linear_rows.cu -- out = act(x W^T + bias) + residual for a few rows of x (single tokens, the embedding of
// a diffusion step).
//
// Bound by HBM: every weight is read once and used for a few rows.  The product runs on warp-level
// tensor instructions with the weights as their 16 rows, loaded straight from global memory into the
// fragments: which elements of k a fragment calls its first is free as long as both operands agree,
// so a lane's fragments of two instructions are 8 neighbouring elements (16 bytes) of a row, and
// nothing passes through shared memory.  (tcgen05 would stage the same bytes in shared memory for a
// tile of 128 rows or more of x: 8 rows, 1536 -> 9216 features took 20 us that way.)
//
// A CTA has 16 features; its 8 warps share k, 32 elements at a time in turn, all of a warp's loads in
// flight together.  Where there are fewer features than fill the GPU, the CTAs of a cluster share k
// too.  The warps' and CTAs' sums are added in their order, through shared memory.
//
// Measured: 8 x 1536 -> 9216 with silu 4.8 us where the call before left the weights (28 MB) in L2, 7.2 from HBM (58 %
// of the copy rate; 4096 -> 32768 85 %); 8 x 6144 -> 1536 5.0 and 7.9.  Where it stops: use_linear_rows.
#include "act.cuh"
#include "gemm.cuh"
#include "vec8.cuh"

namespace vsa {

namespace {

constexpr int WARPS = 8, FEATURES = 16, STEP = 32;

struct Params {
  LinearArgs a;
  int share;   // CTAs of a cluster, along k
  int blocks;  // of STEP elements of k
};

__device__ __forceinline__ void multiply(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, __nv_bfloat16) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void multiply(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, __half) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float load_cluster(uint32_t addr, uint32_t rank) {
  uint32_t there;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
  return v;
}

// TILES: of 8 rows of x.
template <typename E, int TILES>
__global__ void __launch_bounds__(WARPS * 32) linear_rows_kernel(const __grid_constant__ Params p) {
  constexpr int ROWS = 8 * TILES, UNROLL = TILES < 3 ? 6 : 3;  // as the registers allow
  __shared__ float sums[WARPS][FEATURES][ROWS + 1];
  __shared__ float total[FEATURES * ROWS];
  grid_dependency_wait();
  const LinearArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  const int n0 = blockIdx.y * FEATURES, rank = blockIdx.x;
  float c[TILES][4] = {};
  const E* w = static_cast<const E*>(a.weight.data) + (n0 + g) * a.weight.stride + j * 8;
  const bool has0 = n0 + g < a.out_features, has1 = n0 + g + 8 < a.out_features;
  const E* x[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) x[t] = static_cast<const E*>(a.x.data) + (t * 8 + g) * a.x.stride + j * 8;
  const int every = WARPS * p.share;
  for (int b0 = rank * WARPS + warp; b0 < p.blocks; b0 += every * UNROLL) {
    Raw<E> w0[UNROLL], w1[UNROLL], xs[UNROLL][TILES];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int k = (b0 + u * every) * STEP;
      const bool on = k + j * 8 < a.in;
      w0[u].zero();
      w1[u].zero();
      if (on && has0) w0[u].load(w + k);
      if (on && has1) w1[u].load(w + 8 * a.weight.stride + k);
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        xs[u][t].zero();
        if (on && t * 8 + g < a.rows) xs[u][t].load(x[t] + k);
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const uint4 f0 = w0[u].u[0], f1 = w1[u].u[0];
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const uint4 v = xs[u][t].u[0];
        multiply(c[t], f0.x, f1.x, f0.y, f1.y, v.x, v.y, E());
        multiply(c[t], f0.z, f1.z, f0.w, f1.w, v.z, v.w, E());
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][g + (i >> 1) * 8][t * 8 + 2 * j + (i & 1)] = c[t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < FEATURES * ROWS; i += WARPS * 32) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < WARPS; ++v) s += sums[v][i & 15][i >> 4];
    total[i] = s;
  }
  if (p.share > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (rank == 0) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(total));
    for (int i = threadIdx.x; i < FEATURES * ROWS; i += WARPS * 32) {
      const int m = i >> 4, n = n0 + (i & 15);
      if (m >= a.rows || n >= a.out_features) continue;
      float z = total[i];
      for (int r = 1; r < p.share; ++r) z += load_cluster(at + i * 4, r);
      if (a.bias) z += a.bias_dtype == VSA_F32 ? static_cast<const float*>(a.bias)[n] : widen16(static_cast<const E*>(a.bias)[n]);
      if (a.pre.data) narrow(z, static_cast<E*>(a.pre.data) + m * a.pre.stride + n);
      if (a.act == VSA_GELU) z = act_value<VSA_GELU>(z);
      else if (a.act == VSA_GELU_TANH) z = act_value<VSA_GELU_TANH>(z);
      else if (a.act == VSA_SILU) z = act_value<VSA_SILU>(z);
      if (a.residual.data) z += widen16(static_cast<const E*>(a.residual.data)[m * a.residual.stride + n]);
      narrow(z, static_cast<E*>(a.out.data) + m * a.out.stride + n);
    }
  }
  // The sums of a CTA stay until they have been read.
  if (p.share > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// CTAs of an SM: the registers of three tiles leave room for three.
constexpr int sm_ctas(int tiles) { return tiles < 3 ? 4 : 3; }

template <typename E, int TILES>
cudaError_t launch(const LinearArgs& a, cudaStream_t stream) {
  Params p;
  p.a = a;
  p.blocks = (a.in + STEP - 1) / STEP;
  const int features = (a.out_features + FEATURES - 1) / FEATURES;
  // CTAs of a cluster: while there are no more CTAs than run at once, up to four to an SM, and a warp has two blocks
  // or more.  (24 rows, 2048 -> 4096 with four instead of three to an SM: 13.8 us instead of 8.9.)
  p.share = 1;
  while (p.share < 8 && features * p.share * 2 <= sm_ctas(TILES) * device_sm_count() && p.blocks >= p.share * 2 * WARPS * 2)
    p.share *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.share, features);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.share;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_rows_kernel<E, TILES>, p);
}

template <typename E>
cudaError_t launch_rows(const LinearArgs& a, cudaStream_t stream) {
  return a.rows <= 8 ? launch<E, 1>(a, stream) : a.rows <= 16 ? launch<E, 2>(a, stream) : launch<E, 3>(a, stream);
}

}  // namespace

// Every CTA reads all of x, 1/2 to 3/2 of its weights' bytes: the more rows, the fewer weights.  Us here and with
// tiles (gemm_small.cu, or gemm.cu where those are too many), weights from HBM:
//   in -> out, million weights   8 rows            16 rows           24 rows
//    2048 ->  4096    8           6.8 and 10.0      8.4 and  9.6      8.9 and  9.6
//    8192 ->  1024    8                             8.7 and  9.9     10.6 and  9.9
//    1024 ->  8192    8                             6.8 and  8.9     10.9 and  8.9
//    1536 ->  7168   11                             8.2 and 10.0      8.0 and 10.0
//    1536 ->  9216   14           7.2 and 11.1      9.0 and 11.0     13.5 and 10.5
//    4096 ->  4096   17          10.3 and 12.3     12.5 and 11.8     19.9 and 11.8
//    4096 ->  5120   21          13.5 and 12.5     16.3 and 12.7     15.4 and 12.8
//    4096 ->  8192   34          15.3 and 15.5     18.8 and 15.5     29.7 and 15.5
//    6144 ->  6144   38          19.8 and 19.2     26.1 and 17.4     22.6 and 17.2
//    1536 -> 32768   50          20.7 and 20.7     26.5 and 20.9     34.8 and 20.6
//    8192 ->  8192   67          29.1 and 25.6     44.6 and 25.8     56.2 and 25.9
//   16384 ->  6144  101          50.3 and 35.8     79.9 and 35.7     62.9 and 35.9
//    4096 -> 32768  134          46.6 and 54.0     64.0 and 42.8     76.3 and 43.2
//   28672 ->  8192  235          92.1 and 72.5    146   and 72.8    199   and 72.6
// (1 and 4 rows take what 8 do here, and with tiles as much or more.)  Between 17 and 24 rows a second wave of CTAs
// costs more than it can win: there the features' CTAs are at most what runs at once (7168, not 8192).
bool use_linear_rows(int rows, int in, int out) {
  const int64_t weights = static_cast<int64_t>(in) * out;
  if (rows <= 8) return out <= FEATURES * 65535 && (weights <= 35000000 || in < 6144);
  if (rows <= 16) return weights <= 17000000;
  return rows <= 24 && weights <= 12000000 && (out + FEATURES - 1) / FEATURES <= sm_ctas(3) * device_sm_count();
}

cudaError_t launch_linear_rows(const LinearArgs& a, cudaStream_t stream) {
  return a.dtype == VSA_F16 ? launch_rows<__half>(a, stream) : launch_rows<__nv_bfloat16>(a, stream);
}

}  // namespace vsa
