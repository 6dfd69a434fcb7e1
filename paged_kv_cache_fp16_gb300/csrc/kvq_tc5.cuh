// Fifth-generation tensor core (tcgen05) and tensor-copy primitives of the tiled attention kernels.
//
// One thread issues the products; their accumulators, and the A operand of the second product of
// an attention tile, live in tensor memory (TMEM: 128 lanes x 512 columns of 32 bits per SM).
// Shared-memory operands are 128-byte rows in the 128-byte swizzle: the 16-byte piece c of row r
// lies at r * 128 + ((c ^ (r & 7)) * 16), which is how the tensor copies write them and the products
// read them.
#pragma once

#include <cstdint>

#include "kvq_warp.cuh"

namespace kvq {
namespace tc5 {

// ---- shared-memory matrix descriptors (128-byte swizzle, 1024-byte aligned row groups) ----------
// K-major operand (rows of 64 16-bit elements along the contraction): groups of 8 rows lie 1024
// bytes apart; a step of 16 along the contraction adds 32 bytes to the start.
// MN-major operand (rows of 64 elements along N, one row per contraction index): panels of 64
// along N lie `lbo` bytes apart, groups of 8 contraction rows 1024 bytes; a step of 16 along the
// contraction adds 2048 bytes to the start.
__device__ __forceinline__ uint64_t desc_base(uint32_t lbo_bytes) {
  return (static_cast<uint64_t>(lbo_bytes >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t smem_addr) {
  return base | static_cast<uint64_t>((smem_addr & 0x3ffffu) >> 4);
}

// Instruction descriptor: D float32, A and B both f16 or both bf16, M = 128, A K-major.
__host__ __device__ constexpr uint32_t idesc(bool bf16, int n, bool b_mn_major) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// True in one lane of a converged warp.  The products are issued inside `if (elect_one())`: the
// compiler then knows that one thread is active and hands their operands over as uniform
// registers directly (with `lane == 0` in its place each issue took 94 cycles).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[smem] B[smem]^T, 16 along the contraction; issued by one thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc ? 1u : 0u)
      : "memory");
}

// D[tmem] (+)= A[tmem] B[smem].
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc ? 1u : 0u)
      : "memory");
}

// One arrival on `bar` when every product this thread issued before has completed.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// Brings a tensor map to where the copies look for it.
__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Generic-proxy writes to shared memory before this are seen by the tensor cores and copies.
__device__ __forceinline__ void fence_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Whole-warp calls; `cols` a power of two >= 32.  The address of the columns goes to *dst.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

// Bounded wait for a barrier's phase: false when it did not complete within the limit, or when
// another role of the block has given up (*gave_up).  The drain of copies and products in flight
// uses mbar_wait_bounded.  A build may define a smaller limit (down to 0: give up at once) to run
// the way out.
#ifndef KVQ_TILE_WAIT_LIMIT
#define KVQ_TILE_WAIT_LIMIT (1 << 20)
#endif
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const volatile int* gave_up) {
  for (int i = 0; i < (KVQ_TILE_WAIT_LIMIT); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && *gave_up) return false;
  }
  return false;
}

// 32 columns of the warp's 32 lanes: thread = lane, r[i] = column i.  A load's registers hold
// their values after wait_ld32(r); further loads issued before that wait are covered by
// after_ld32(r), which only keeps the compiler from using r earlier.
#define KVQ_R32(r)                                                                               \
  "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), \
      "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),    \
      "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),               \
      "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]),               \
      "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
__device__ __forceinline__ void wait_ld32(uint32_t r[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KVQ_R32(r)::"memory");
}
__device__ __forceinline__ void after_ld32(uint32_t r[32]) { asm volatile("" : KVQ_R32(r)::"memory"); }
#undef KVQ_R32

__device__ __forceinline__ void ld32(uint32_t addr, uint32_t r[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void st32(uint32_t addr, const uint32_t r[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t addr, const uint32_t r[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A box of a 3-d tensor map to shared memory, completing its bytes on `bar`.
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// The two warps (of 8 softmax warps) that share the rows of quadrant `quad` meet.  Barrier numbers
// are spelt out: with a number in a register a kernel is charged all 16 of a block's barriers.
__device__ __forceinline__ void meet(int quad) {
  switch (quad) {
    case 0: asm volatile("bar.sync 2, 64;" ::: "memory"); break;
    case 1: asm volatile("bar.sync 3, 64;" ::: "memory"); break;
    case 2: asm volatile("bar.sync 4, 64;" ::: "memory"); break;
    default: asm volatile("bar.sync 5, 64;" ::: "memory"); break;
  }
}

// ---- the online softmax of a row held by one thread ---------------------------------------------
// Scores are taken to log2 units (x = s * scale * log2 e).  The row keeps a reference m that its
// weights 2^(x - m + kOff) are taken against, moved to the true maximum only when that has grown
// by more than kSlack: the sums (l and the accumulators in TMEM) are rescaled then, and only then.
// Weights reach 2^(kOff + kSlack) = 2^14 at most, inside fp16; those down to 2^-24 of the largest
// keep all of fp16's bits and smaller ones an absolute error of 2^-35 of it, so that a tail of
// 262,144 small weights is not lost.
constexpr float kOff = 10.f;
constexpr float kSlack = 4.f;

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The largest of N scores (float32 patterns); NaN only if all are.
template <int N>
__device__ __forceinline__ float row_max(const uint32_t s[N]) {
  const float ninf = __uint_as_float(0xff800000u);
  float m[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
  for (int i = 0; i < N; i += 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m[j] = max3(m[j], __uint_as_float(s[i + 2 * j]), __uint_as_float(s[i + 2 * j + 1]));
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16-bit pairs of float32 values, rounded to nearest even.
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The weights 2^(s c - mo) of 32 scores, rounded to 16 bits, to the 16 TMEM columns from `to` on;
// their float32 sums are added to the four in sum[2].  Two elements per multiply-add and per
// addition (packed float32).
template <bool BF>
__device__ __forceinline__ void weights32(const uint32_t s[32], float c, float mo, uint32_t to,
                                          uint64_t sum[2]) {
  const uint64_t c2 = pair(__float_as_uint(c), __float_as_uint(c));
  const uint64_t m2 = pair(__float_as_uint(-mo), __float_as_uint(-mo));
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    float x0, x1, x2, x3;
    unpair(fma2(pair(s[i], s[i + 1]), c2, m2), x0, x1);
    unpair(fma2(pair(s[i + 2], s[i + 3]), c2, m2), x2, x3);
    x0 = ex2_fast(x0);
    x1 = ex2_fast(x1);
    x2 = ex2_fast(x2);
    x3 = ex2_fast(x3);
    sum[0] = add2(sum[0], pair(__float_as_uint(x0), __float_as_uint(x1)));
    sum[1] = add2(sum[1], pair(__float_as_uint(x2), __float_as_uint(x3)));
    p[i / 2] = pack2<BF>(x0, x1);
    p[i / 2 + 1] = pack2<BF>(x2, x3);
  }
  st16(to, p);
}
__device__ __forceinline__ float sum_of(const uint64_t sum[2]) {
  float a, b;
  unpair(add2(sum[0], sum[1]), a, b);
  return a + b;
}

}  // namespace tc5
}  // namespace kvq
