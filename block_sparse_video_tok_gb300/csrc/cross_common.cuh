// cross_common.cuh -- what the cross-attention kernels share: how query rows are laid out in
// 128-row tiles, the tensor maps of operands of any strides, and small device helpers.
#pragma once

#include "layer_internal.cuh"
#include "ptx.cuh"

namespace vsa {

constexpr int TILE = 128;                        // rows of a query tile, keys of a kv tile
constexpr uint32_t TILE_BYTES = TILE * 128 * 2;  // one operand tile: two column halves of 16 KB

// Division of 0 <= n < 2^31 by a fixed d >= 1 as a multiply and a shift (the persistent kernels
// decode their units in every role, and the code of a 32-bit division there counts), after Granlund and
// Montgomery, "Division by invariant integers using multiplication" (1994): with 2^s >= d and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(n, m) + n) >> s.
struct Divisor {
  uint32_t d, m, s;
#ifdef __CUDACC__
  __device__ __forceinline__ int quotient(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> s);
  }
#endif
};
inline Divisor make_divisor(uint32_t d) {
  Divisor x{d, 0, 0};
  while ((1ull << x.s) < d) ++x.s;
  x.m = static_cast<uint32_t>((1ull << 32) * ((1ull << x.s) - d) / d + 1);
  return x;
}

// Query rows in tiles.  From 128 tokens on, a tile is 128 tokens of one head.  Below, a tile
// packs all tokens of `pack` neighbouring heads that read the same key head, so that the keys
// are read once for them: row r is token r % box of head r / box.  pack divides the number of
// heads that share a key head, so no tile reaches into another key head's.  (2 x 32 heads on 4 key
// heads, 16 queries on 8191 keys: forward 16 us, one head a tile 35; backward 38 and 91.)
struct QTiles {
  int box;     // tokens of one head in a tile
  int pack;    // heads in a tile
  int blocks;  // tiles along the tokens of a head
  int share;   // heads / kv_heads
  int tiles;   // tiles of one (batch, key head)
};

inline QTiles q_tiles(int heads, int kv_heads, int q_tokens) {
  QTiles t;
  t.share = heads / kv_heads;
  t.box = q_tokens < TILE ? q_tokens : TILE;
  t.blocks = (q_tokens + TILE - 1) / TILE;
  t.pack = 1;
  for (int p = 2; p <= t.share && p * t.box <= TILE; ++p)
    if (t.share % p == 0) t.pack = p;
  t.tiles = t.blocks * (t.share / t.pack);
  return t;
}

// Tensor map of x as (64 columns, tokens, heads, column half, batch), box (64, box_tokens,
// box_heads, 2, 1), 128-byte swizzle: one copy lands a tile of 128 rows as two column halves of
// box_heads x box_tokens rows of 128 bytes.  A box of fewer rows holds one column half (the
// halves of a tile in shared memory are 16 KB apart) and a tile takes two copies.  A broadcast dimension (stride 0) has extent 1 in the
// map, and its coordinate must be 0.
cudaError_t make_tmap_heads(CUtensorMap* map, const HeadsView& x, int tokens, int batch,
                            int box_tokens, int box_heads);

#ifdef __CUDACC__

// x, which all lanes hold alike, in a form that the compiler knows to be the same for the whole
// warp: what depends on it alone stays in uniform registers, where the tensor-core instructions
// take their operands from.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Wait of a converged warp for the phase of `bar` with the given parity; false if *abort was
// raised or `limit_ns` of wall time passed (a probe that fails has been suspended for a while, so
// the clock is read seldom).  The loop is a function of its own, not a copy in each of some twenty
// places: the code of all roles shares the instruction caches.
static __device__ __noinline__ bool warp_poll(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  uint64_t t0 = 0;
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (__any_sync(0xffffffffu, *abort != 0 || t - t0 > limit_ns)) return false;
  }
  return true;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  // (The vote tells the compiler that the result is the same for all lanes.)
  return __all_sync(0xffffffffu, warp_poll(bar, parity, abort, limit_ns));
}

// After an abort: the last `stages` of `count` copies, copy i counted on the barrier at full0 + 8
// (i % stages), have landed (one thread; gives up after DRAIN_LIMIT_NS).
static __device__ __noinline__ void drain_copies(uint32_t full0, uint32_t stages, uint32_t count) {
  volatile int never = 0;
  for (uint32_t i = count > stages ? count - stages : 0; i < count; ++i)
    mbar_wait_bounded(full0 + 8u * (i % stages), (i / stages) & 1u, &never, DRAIN_LIMIT_NS);
}

__device__ __forceinline__ void raise_abort(volatile int* abort, uint32_t* err) {
  *abort = 1;
  atomicOr(err, VSA_DEVERR_TIMEOUT);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Softmax statistics (m, l) and O += weight of another part: f scales the old, w the new.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2, float* f, float* w) {
  const float mn = fmaxf(m, m2), ref = mn == -INFINITY ? 0.f : mn;
  *f = ex2(m - ref);
  *w = ex2(m2 - ref);
  m = mn;
  l = l * *f + l2 * *w;
}

// Packed fp32 pairs: one instruction on both halves of a 64-bit register pair.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of row r in a column half of an operand tile.
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) {
  return r * 128u + ((c ^ (r & 7u)) << 4);
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// The rows [from, to) of an operand tile in shared memory become zero, for a whole warp to call;
// the writes are ordered before later tensor-core reads.
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int to, int lane) {
  for (int i = lane; i < (to - from) * 16; i += 32) {
    const uint32_t r = static_cast<uint32_t>(from + (i >> 4)), c = static_cast<uint32_t>(i & 15);
    st_shared_zero16(tile + (c >> 3) * (TILE_BYTES / 2) + r * 128u + (c & 7u) * 16u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// The UMMAs of a whole product in one block, issued by the lane elect.sync chooses of a converged
// warp.  The issuing warp shares its scheduler with two softmax warps, so what counts is how few
// instructions it takes: issued one by one, with an election and 64-bit descriptors each, a
// product of 8 UMMAs took the warp about 870 cycles, for 520 of the tensor core.

// D = A B^T over 128 columns: A, B K-major operand tiles (SWIZZLE_128B, column halves 16 KB apart).
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, f, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
      "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 1024;\n\tadd.u64 b, %2, 1024;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 1026;\n\tadd.u64 b, %2, 1026;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 1028;\n\tadd.u64 b, %2, 1028;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 1030;\n\tadd.u64 b, %2, 1030;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc)
      : "memory");
}

// D (+)= A B over 64 rows of B: A 16-bit pairs in tensor memory, 16 columns for 32 rows of B and the
// next 16 columns PAIR after them; B an MN-major tile (SWIZZLE_128B).  accumulate = 0: D is
// overwritten.
template <int PAIR>
__device__ __forceinline__ void product_ts64(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, c, t;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 c, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, c;\n\t"
      "add.u32 a, %1, %5;\n\tadd.u64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, %1, %6;\n\tadd.u64 b, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, %1, %7;\n\tadd.u64 b, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(8), "n"(PAIR), "n"(PAIR + 8)
      : "memory");
}

#endif

}  // namespace vsa
