// Selection of the next beams: of all tokens behind all of a sequence's beams, the num_out largest
//   t[b][v] = score[b] + x[b][v] - log sum_w exp x[b][w].
//
// One pass over the logits.  A block takes a slice of one row: it sums exponentials around a running
// maximum and keeps the slice's num_out largest logits (within a row the order of t is that of x).  A
// second kernel, a block per sequence, joins the slices' sums and picks among the kept logits.  The
// floor is one read of the logits: 9.9 us for 64 sequences of 4 beams over 131,072 bf16 logits, which take
// 27 us in the first kernel (2.5 TB/s; a block's start and end are about half of its time) and 29 a call.
//
// Keeping the largest: the first batch (four vectors of 16 bytes a thread) gives a bound by its warps'
// maxima that at least num_out elements reach; the num_out-th largest element of it is the bound for the
// later ones, so that an element costs little but its exponential and the warps need not meet.  (One warp
// finding that bound while the others go on with the old one: 36 instead of 29 us, the old one lets too many
// by.)  Where too many pass (logits that rise along the vocabulary), the slice is gone through again, meeting
// after every vector to raise the bound.  Two batches are on their way (asynchronous copies, a ring per warp)
// while one is worked on: with one, loaded to registers, the kernel waited for memory most of the time (26 us).
//
// Candidates of different beams are close, so the sums add little to what the exponentials are off (2^-22, and
// two roundings of their argument): the argument is multiplied by log2 e in two parts, the terms of a thread's
// batch are added in float32 and then to a pair of floats, and slices are joined in float64.  Against 64 bits a
// row's log-sum is 6e-8 off in ordinary rows, 2e-7 where all terms lie at one distance.  Where elements lie in
// the block's threads does not depend on the row's address, so that equal rows have equal sums (and ties
// between them stay ties).
#include <cstdint>
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_warp.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;                      // 16-byte vectors of a thread's batch
constexpr int kStages = 2;
constexpr int kVecBytes = 33 * 16;            // a warp's vector, and the word behind it
constexpr int kRingBytes = kWarps * kStages * kVecs * kVecBytes;
constexpr int kKeep = KVQ_MAX_BEAM_OUT;
constexpr int kList = 4096 + kKeep;           // the kept ones and one vector of 8 elements of every thread
#define kNegInf (-__int_as_float(0x7f800000))

struct SelectArgs {
  const void* logits;
  const float* scores;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  float4* part;       // per (row, slice): max, sum (high, low), number kept (as int bits)
  uint64_t* keys;     // per (row, slice): num_out keys
  int64_t stride;
  int beams, vocab, num_out, slices, slice;   // slice: elements, a multiple of a batch's vectors
};

// Floats in an order of unsigned integers; -0 and 0 are equal.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.));
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}

// Sums as pairs hi + lo.
struct Pair {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {          // exact sum of hi and x, rest into lo
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
  __device__ __forceinline__ void scale(float f) { hi *= f; lo *= f; }
};

// Sum over the warp, the same in every lane.
__device__ __forceinline__ void warp_sum(Pair& s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float h = __shfl_xor_sync(kFullMask, s.hi, o), l = __shfl_xor_sync(kFullMask, s.lo, o);
    // the same result in both partners: the larger part first
    const float big = fmaxf(s.hi, h), small = fminf(s.hi, h), sum = big + small;
    s.lo = (s.lo + l) + (small - (sum - big));
    s.hi = s.hi != s.hi || h != h ? s.hi + h : sum;
  }
}

template <typename T> struct Elem;
template <> struct Elem<__half> {
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
};
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <typename T> constexpr int kPer = 16 / sizeof(T);          // elements of a vector
template <typename T> constexpr int kSpread = kThreads * kPer<T>;   // of a vector of every thread

// The 16 bytes that start `off` bytes (a multiple of the element's) into the 32 of x.
template <typename T>
__device__ __forceinline__ void shifted(const uint32_t (&x)[8], int off, uint32_t (&w)[4]) {
  auto from = [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (sizeof(T) == 2 && (off & 2)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(x[K + i], x[K + i + 1], 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = x[K + i];
    }
  };
  switch (off >> 2) {
    case 0: from(std::integral_constant<int, 0>()); break;
    case 1: from(std::integral_constant<int, 1>()); break;
    case 2: from(std::integral_constant<int, 2>()); break;
    default: from(std::integral_constant<int, 3>());
  }
}

// Elements e .. e + kPer - 1 of a row (e a multiple of kPer), -inf behind its end.  Where rows do not start
// at 16 bytes, the two aligned 16-byte words that hold them are read and shifted: every word read holds an
// element of the row.
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int e, int end, uint32_t (&w)[4]) {
  if (e + kPer<T> <= end) {
    const char* at = reinterpret_cast<const char*>(row + e);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
    at -= off;
    const uint4 a = ld_nc_v4(at), b = off ? ld_nc_v4(at + 16) : a;
    uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    shifted<T>(x, off, w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = e + i < end ? __ldg(reinterpret_cast<const uint32_t*>(row + e + i)) : 0xff800000u;
      } else {
        constexpr uint32_t kLow = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;   // -inf
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row + e + 2 * i);
        const uint32_t lo = e + 2 * i < end ? __ldg(p) : kLow, hi = e + 2 * i + 1 < end ? __ldg(p + 1) : kLow;
        w[i] = lo | hi << 16;
      }
    }
  }
}

// A batch: kVecs vectors, one of every thread after the other.  The copies take the aligned 16-byte words
// from that on which holds the row's first element, as far as the row goes.
// mine: this thread's first word of the batch; left: bytes from the batch's first word to the slice's end.
__device__ __forceinline__ void copy_batch(const char* mine, int64_t left, uint32_t ring, int off) {
  const int lane = threadIdx.x & 31;
  const uint32_t dst = ring + 16 * lane;
  if (left >= kVecs * 16 * kThreads + 16) {  // the same in the whole block
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + v * kVecBytes),
                   "l"(mine + v * 16 * kThreads) : "memory");
      if (off && lane == 31)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + v * kVecBytes + 16),
                     "l"(mine + v * 16 * kThreads + 16) : "memory");
    }
  } else if (left > 0) {
    const int64_t here = left - static_cast<int>(threadIdx.x) * 16;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k && !(off && lane == 31)) continue;
        const int64_t rest = here - v * 16 * kThreads - 16 * k;
        const uint32_t n = rest >= 16 ? 16 : rest > 0 ? static_cast<uint32_t>(rest) : 0;
        if (n)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + v * kVecBytes + 16 * k),
                       "l"(mine + v * 16 * kThreads + 16 * k), "r"(n) : "memory");
      }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// A thread's vectors of the batch at `at` out of the ring; -inf behind the slice's end.
template <typename T>
__device__ __forceinline__ void take_batch(const uint8_t* ring, int at, int end, int off, uint32_t (&w)[kVecs][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    const uint4 a = *reinterpret_cast<const uint4*>(ring + v * kVecBytes + 16 * lane);
    w[v][0] = a.x; w[v][1] = a.y; w[v][2] = a.z; w[v][3] = a.w;
    if (off) {                               // the same in the whole block
      const uint4 b = *reinterpret_cast<const uint4*>(ring + v * kVecBytes + 16 * lane + 16);
      uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      shifted<T>(x, off, w[v]);
    }
  }
  if (at + kVecs * kSpread<T> > end) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = at + v * kSpread<T> + static_cast<int>(threadIdx.x) * kPer<T>;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          if (e + i >= end) w[v][i] = 0xff800000u;
        } else {
          constexpr uint32_t kNone = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;   // -inf
          if (e + 2 * i >= end) w[v][i] = kNone | kNone << 16;
          else if (e + 2 * i + 1 >= end) w[v][i] = (w[v][i] & 0xffffu) | kNone << 16;
        }
      }
    }
  }
}

// The largest of a vector's elements, NaN left out.
template <typename T>
__device__ __forceinline__ float largest(const uint32_t (&w)[4]) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])),
                 fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    auto two = [&](int i) { return *reinterpret_cast<const T2*>(&w[i]); };
    const T2 x = __hmax2(__hmax2(two(0), two(1)), __hmax2(two(2), two(3)));
    const float2 f = Elem<T>::two(*reinterpret_cast<const uint32_t*>(&x));
    return fmaxf(f.x, f.y);
  }
}

template <typename T>
__device__ __forceinline__ void unpack(const uint32_t (&w)[4], float (&x)[kPer<T>]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = Elem<T>::two(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = static_cast<float>(1.4426950408889634 - static_cast<double>(kLog2e));

// e^d for d <= 0 (NaN for NaN).
__device__ __forceinline__ float exp_of(float d) { return ex2_fast(fmaf(d, kLog2e, d * kLog2eLow)); }

// Two floats at once.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 exp2_of(float2 x, float2 minus) {   // e^(x + minus) of both
  const float2 d = add2(x, minus);
  const float2 t = fma2(d, make_float2(kLog2e, kLog2e), mul2(d, make_float2(kLog2eLow, kLog2eLow)));
  return make_float2(ex2_fast(t.x), ex2_fast(t.y));
}

// Keeps the k largest of the n (different) keys in `list`, in any order.  All threads call it; `other`
// has room for k keys.  Up to kThreads keys are ranked by counting the larger ones; more of them are
// first cut down by a search for the k-th largest.
__device__ __noinline__ int keep_largest(uint64_t* list, uint64_t* other, int n, int k, int* n_sm) {
  if (n <= k) return n;
  if (n > kThreads) {
    uint64_t lo = 0, hi = ~0ull;   // count(>= lo) >= k > count(>= hi + 1)
    while (lo < hi) {
      const uint64_t mid = lo + ((hi - lo) >> 1) + 1;
      int c = 0;
      for (int i = threadIdx.x; i < n; i += kThreads) c += list[i] >= mid;
      c = __reduce_add_sync(kFullMask, c);
      if (threadIdx.x == 0) *n_sm = 0;
      __syncthreads();
      if ((threadIdx.x & 31) == 0) atomicAdd(n_sm, c);
      __syncthreads();
      c = *n_sm;
      __syncthreads();
      if (c >= k) lo = mid; else hi = mid - 1;
      if (c == k) break;
    }
    if (threadIdx.x == 0) *n_sm = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (list[i] >= lo) {
        const int at = atomicAdd(n_sm, 1);
        if (at < k) other[at] = list[i];
      }
  } else {
    // a warp ranks the keys i, i + 16, ...: its lanes compare a 32nd of the list each
    for (int i = threadIdx.x >> 5; i < n; i += kWarps) {
      const uint64_t mine = list[i];
      int larger = 0;
      for (int j = threadIdx.x & 31; j < n; j += 32) larger += list[j] > mine;
      larger = __reduce_add_sync(kFullMask, larger);
      if (larger < k && (threadIdx.x & 31) == 0) other[larger] = mine;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < k; i += kThreads) list[i] = other[i];
  __syncthreads();
  return k;
}

// Puts the elements of at least `low` of those lanes' vectors in `hits` into the list, lane after lane, an
// element per lane.  e: this lane's first element.
template <typename T>
__device__ __noinline__ void push(uint4 v, int e, uint32_t hits, float low, uint64_t* list, int* n_list) {
  const int lane = threadIdx.x & 31;
  while (hits) {
    const int from = __ffs(hits) - 1;
    hits &= hits - 1;
    const uint32_t w0 = __shfl_sync(kFullMask, v.x, from), w1 = __shfl_sync(kFullMask, v.y, from),
                   w2 = __shfl_sync(kFullMask, v.z, from), w3 = __shfl_sync(kFullMask, v.w, from);
    const int e0 = __shfl_sync(kFullMask, e, from), at = lane * static_cast<int>(sizeof(T)) / 4;
    const uint32_t w = at & 2 ? (at & 1 ? w3 : w2) : (at & 1 ? w1 : w0);
    float x;
    if constexpr (sizeof(T) == 4) {
      x = __uint_as_float(w);
    } else {
      const float2 f = Elem<T>::two(w);
      x = lane & 1 ? f.y : f.x;
    }
    if (lane < kPer<T> && x >= low && x > kNegInf) {
      const int to = atomicAdd(n_list, 1);
      if (to < kList) list[to] = static_cast<uint64_t>(ordered(x)) << 32 | ~static_cast<uint32_t>(e0 + lane);
    }
  }
}

// The k largest of up to 32 kSome (different) keys, one after the other, by one warp: `got(i, key)` is called
// in all lanes.  A round costs two warp-wide maxima.
constexpr int kSome = 8, kFewOut = 16;
template <typename F>
__device__ __forceinline__ void warp_largest(const uint64_t* list, int n, int k, F got) {
  const int lane = threadIdx.x & 31;
  uint64_t key[kSome], best = 0;
#pragma unroll
  for (int j = 0; j < kSome; ++j) {
    key[j] = lane + 32 * j < n ? list[lane + 32 * j] : 0;
    best = key[j] > best ? key[j] : best;
  }
  for (int i = 0; i < k; ++i) {
    const uint32_t hi = __reduce_max_sync(kFullMask, static_cast<uint32_t>(best >> 32));
    const uint32_t lo = __reduce_max_sync(kFullMask, static_cast<uint32_t>(best >> 32) == hi
                                                         ? static_cast<uint32_t>(best) : 0u);
    const uint64_t top = static_cast<uint64_t>(hi) << 32 | lo;
    got(i, top);
    if (best == top) {                       // one lane
      best = 0;
#pragma unroll
      for (int j = 0; j < kSome; ++j) {
        key[j] = key[j] == top ? 0 : key[j];
        best = key[j] > best ? key[j] : best;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) select_slice_kernel(const __grid_constant__ SelectArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];            // the rings, then the list
  uint64_t* list = reinterpret_cast<uint64_t*>(smem + kRingBytes);
  __shared__ uint64_t other[kKeep];
  __shared__ float sm_max[kWarps], sm_low[kWarps];
  __shared__ float4 sm_sum[kWarps];
  __shared__ int n_list, n_tmp;
  constexpr int P = kPer<T>;
  static_assert(kKeep + kSpread<T> <= kList, "a vector of every thread fits");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.slices, sl = blockIdx.x - row * a.slices;
  asm volatile("griddepcontrol.wait;" ::: "memory");               // started while the work before it ends
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const T* x_row = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.stride;
  const int begin = sl * a.slice, end = begin + min(a.slice, a.vocab - begin);   // (begin + slice may leave int)
  const int K = a.num_out;
  const float score = __ldg(a.scores + row);
  float4* part = a.part + blockIdx.x;
  if (!(fabsf(score) < -kNegInf)) {   // a beam that continues nothing: its logits are not looked at
    if (tid == 0) *part = make_float4(kNegInf, 0.f, 0.f, __int_as_float(0));
    return;
  }
  if (tid == 0) n_list = 0;
  constexpr int kBatch = kVecs * kSpread<T>;
  // how far the row lies behind a 16-byte boundary
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x_row) & 15);
  constexpr int kBatchBytes = kVecs * 16 * kThreads;
  const char* mine = reinterpret_cast<const char*>(x_row + begin) - off + tid * 16;
  int64_t left = static_cast<int64_t>(end - begin) * sizeof(T) + off;
  uint8_t* ring = smem + warp * kStages * kVecs * kVecBytes;
#pragma unroll
  for (int i = 0; i < kStages; ++i) {
    copy_batch(mine, left, smem_u32(ring) + i * kVecs * kVecBytes, off);
    mine += kBatchBytes;
    left -= kBatchBytes;
  }
  uint32_t w[kVecs][4];

  float m = kNegInf, low = kNegInf;
  Pair s = {0.f, 0.f};
  // cuts the list down to num_out and raises the bound: later elements equal to the least kept one come
  // behind it
  auto cut = [&](int n) {
    n = keep_largest(list, other, n, K, &n_tmp);
    if (tid == 0) n_list = n;
    uint32_t least = 0xffffffffu;
    for (int i = lane; i < n; i += 32) least = min(least, static_cast<uint32_t>(list[i] >> 32));
    least = __reduce_min_sync(kFullMask, least);
    if (n == K) low = unordered(least + 1);
    return n;
  };
  int stage = 0, batch = 0;
  for (int at = begin; at < end; at += kBatch) {
    const bool more = at + kBatch < end;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();                            // every lane's copies are there
    uint8_t* here = ring + stage * kVecs * kVecBytes;
    stage ^= 1;
    take_batch<T>(here, at, end, off, w);
    __syncwarp();                            // every lane has its elements
    copy_batch(mine, left, smem_u32(here), off);
    mine += kBatchBytes;
    left -= kBatchBytes;
    float tops[kVecs], top = kNegInf;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      tops[v] = largest<T>(w[v]);
      top = fmaxf(top, tops[v]);
    }
    if (at == begin) {
      // the warps' share of num_out: each names the value that so many of its lanes reach
      uint32_t left = ordered(top), bound = 0, first = 0;
      const int share = (K + kWarps - 1) / kWarps;
      for (int i = 0; i < share; ++i) {
        bound = __reduce_max_sync(kFullMask, left);
        if (i == 0) first = bound;
        const uint32_t who = __ballot_sync(kFullMask, left == bound);
        if (lane == __ffs(who) - 1) left = 0;
      }
      if (lane == 0) {
        sm_max[warp] = unordered(first);
        sm_low[warp] = bound ? unordered(bound) : kNegInf;
      }
      __syncthreads();
      m = sm_max[lane & (kWarps - 1)];
      low = sm_low[lane & (kWarps - 1)];
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) {
        m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
        low = fminf(low, __shfl_xor_sync(kFullMask, low, o));
      }
    }
    // Warps without enough elements (short slices, masked regions) name nothing: then the num_out-th largest
    // of all threads' best, by the upper half of the order.
    if (at == begin && !(low > kNegInf)) {   // the same in all threads
      uint32_t mine = ordered(top), bound = 0;
      if (!(top > kNegInf)) mine = 0;
#pragma unroll 1
      for (int bit = 31; bit >= 16; --bit) {
        const uint32_t want = bound | 1u << bit;
        if (__syncthreads_count(mine >= want) >= K) bound = want;
      }
      if (bound) low = unordered(bound);
    }
    // m, low: the same in all threads at first; m grows where a thread meets more
    if (__any_sync(kFullMask, top >= low)) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const uint32_t hits = __ballot_sync(kFullMask, tops[v] >= low);
        if (hits)
          push<T>(make_uint4(w[v][0], w[v][1], w[v][2], w[v][3]), at + v * kSpread<T> + tid * P, hits, low,
                  list, &n_list);
      }
    }
    if (top > m) {
      s.scale(exp_of(m - top));           // m = -inf: nothing was added yet, 0 stays 0
      m = top;
    }
    const float ref = m == kNegInf ? 0.f : -m;
    const float2 minus = make_float2(ref, ref);
    float2 t[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float x[P];
      unpack<T>(w[v], x);
      t[v] = exp2_of(make_float2(x[0], x[1]), minus);
#pragma unroll
      for (int i = 2; i < P; i += 2) t[v] = add2(t[v], exp2_of(make_float2(x[i], x[i + 1]), minus));
    }
    const float2 all = add2(add2(t[0], t[1]), add2(t[2], t[3]));
    s.add(all.x + all.y);
    // after the first batch, and where many are kept (a cut costs what some tens of them do) after 2 and 4:
    // each later one brings as many as the bound is old
    if (more && (batch == 0 || (K > kFewOut && (batch == 1 || batch == 3)))) {
      __syncthreads();
      const int n = n_list;
      __syncthreads();
      if (n > K + K / 2 && n <= kList) cut(n);
      __syncthreads();
    }
    ++batch;
  }
  __syncthreads();
  if (n_list > kList) {                   // the same in all threads
    __syncthreads();
    if (tid == 0) n_list = 0;
    low = kNegInf;
    __syncthreads();
    for (int at = begin; at < end; at += kSpread<T>) {
      load_vec<T>(x_row, at + tid * P, end, w[0]);
      const uint32_t hits = __ballot_sync(kFullMask, largest<T>(w[0]) >= low);
      if (hits)
        push<T>(make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]), at + tid * P, hits, low, list, &n_list);
      __syncthreads();
      const int n = n_list;
      __syncthreads();
      if (n > K) cut(n);
      __syncthreads();
    }
  }
  // the threads' sums around their warp's maximum, then the warps' around the block's
  float M = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
  if (m != M) s.scale(m == kNegInf ? (s.hi == 0.f ? 0.f : s.hi) : exp_of(m - M));
  warp_sum(s);
  if (lane == 0) sm_sum[warp] = make_float4(M, s.hi, s.lo, 0.f);
  __syncthreads();
  int n = n_list;
  uint64_t* keys = a.keys + static_cast<int64_t>(blockIdx.x) * K;
  if (K <= kFewOut && n <= 32 * kSome) {
    n = min(n, K);
    if (warp == 1)
      warp_largest(list, n_list, n, [&](int i, uint64_t key) {
        if (lane == 0) keys[i] = key;
      });
  } else {
    n = keep_largest(list, other, n, K, &n_tmp);
    for (int i = tid; i < n; i += kThreads) keys[i] = list[i];
  }
  if (warp == 0) {
    float4 t = lane < kWarps ? sm_sum[lane] : make_float4(kNegInf, 0.f, 0.f, 0.f);
    float top = t.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
    s.hi = t.y;
    s.lo = t.z;
    if (t.x != top) s.scale(t.x == kNegInf ? (s.hi == 0.f ? 0.f : s.hi) : exp_of(t.x - top));
    warp_sum(s);
    if (lane == 0) *part = make_float4(top, s.hi, s.lo, __int_as_float(n));
  }
}

// ------------------------------------------------------------------------- a sequence's candidates
constexpr int kRound = 4 * kThreads;   // candidates looked at together

constexpr int kPairs = 16;

// e^d for d <= 0, to 2^-34: d = n ln 2 + r, the exponential series of r (|r| <= 0.35) up to r^9 / 9!, and the
// exponent n.  NaN for NaN; 0 below 2^-1000.
__device__ __forceinline__ double exp64(float d) {
  const float n = rintf(d * kLog2e);
  if (!(n > -1000.f)) return n != n ? static_cast<double>(n) : 0.;
  const double r = static_cast<double>(d) - static_cast<double>(n) * 0.69314718055994531;
  double y = 1. / 362880;
  y = y * r + 1. / 40320;
  y = y * r + 1. / 5040;
  y = y * r + 1. / 720;
  y = y * r + 1. / 120;
  y = y * r + 1. / 24;
  y = y * r + 1. / 6;
  y = y * r + 0.5;
  y = y * r + 1.;
  y = y * r + 1.;
  return __longlong_as_double(__double_as_longlong(y) + (static_cast<int64_t>(n) << 52));
}

// log x for a sum x of at least 1 (or 0, NaN), to 2^-33: float32's, and one step of Newton's iteration for
// e^y = x, whose error is the square of float32's.
__device__ __forceinline__ double log64(double x) {
  const float y = logf(static_cast<float>(x));
  if (!(fabsf(y) < -kNegInf)) return y;
  return y + (x * exp64(-y) - 1.);
}

// A candidate; its beam stands beside it.  Equal scores of one beam go by the logit first: different logits have
// equal t in float64 behind a far score, and where they are much nearer to each other than to the sum.
struct Cand {
  uint64_t score;   // ordered(double)
  uint64_t key;     // logit, then token: the larger one first
};

__global__ void __launch_bounds__(kThreads) select_join_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ double lse[KVQ_MAX_BEAMS], pair[KVQ_MAX_BEAMS][kPairs];
  __shared__ float most[KVQ_MAX_BEAMS];
  __shared__ Cand list[kRound + kKeep], other[kKeep];
  __shared__ uint8_t list_beam[kRound + kKeep], other_beam[kKeep];
  __shared__ int n_list;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x, K = a.num_out;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the slices are still worked on
  const int64_t row0 = static_cast<int64_t>(s) * a.beams;
  const int per_row = a.slices * K, all = a.beams * per_row;
  // a round of candidates: beam (-1: none), logit and token, score; the first is on its way before the sums
  struct Raw {
    int beam;
    float score;
    uint64_t key;
  } raw[kRound / kThreads];
  auto load = [&](int c0) {
#pragma unroll
    for (int j = 0; j < kRound / kThreads; ++j) {
      const int c = c0 + j * kThreads + tid;
      raw[j].beam = -1;
      if (c >= all) continue;
      const int b = c / per_row, rest = c - b * per_row, sl = rest / K, i = rest - sl * K;
      const int64_t at = (row0 + b) * a.slices + sl;
      raw[j].key = a.keys[at * K + i];       // garbage behind the slice's count
      raw[j].score = __ldg(a.scores + row0 + b);
      if (i < __float_as_int(a.part[at].w)) raw[j].beam = b;
    }
  };
  load(0);
  for (int b = warp; b < a.beams; b += kWarps) {
    const float4* part = a.part + (row0 + b) * a.slices;
    float M = kNegInf;
    for (int i = lane; i < a.slices; i += 32) M = fmaxf(M, __ldcg(&part[i].x));
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
    if (lane == 0) most[b] = M;
  }
  __syncthreads();
  // Float64 is slow, so its work is spread over as few warps as hold it: 16 (row, slice) pairs of a beam at a
  // time, then a lane per beam.
  for (int i0 = 0; i0 < a.slices; i0 += kPairs) {
    const int width = min(kPairs, a.slices - i0);
    for (int c = tid; c < a.beams * width; c += kThreads) {
      const int b = c / width, i = c - b * width;
      const float4 p = a.part[(row0 + b) * a.slices + i0 + i];
      const double v = static_cast<double>(p.y) + p.z;
      pair[b][i] = p.x == most[b] ? v : v * exp64(p.x - most[b]);
    }
    __syncthreads();
    if (tid < a.beams) {
      double sum = i0 ? lse[tid] : 0.;
      for (int i = 0; i < width; ++i) sum += pair[tid][i];
      lse[tid] = i0 + kPairs < a.slices ? sum : most[tid] + log64(sum);
    }
    __syncthreads();
  }
  if (tid == 0) n_list = 0;
  __syncthreads();
  int n = 0;
  uint64_t low = 0;        // a bound that num_out candidates reach
  for (int c0 = 0; c0 < all; c0 += kRound) {
    Cand mine[kRound / kThreads];
    if (c0) load(c0);
#pragma unroll
    for (int j = 0; j < kRound / kThreads; ++j) {
      mine[j].score = 0;
      if (raw[j].beam < 0) continue;
      const double x = static_cast<double>(unordered(static_cast<uint32_t>(raw[j].key >> 32)));
      const double t = (x - lse[raw[j].beam]) + raw[j].score;
      if (!(t > static_cast<double>(kNegInf))) continue;   // NaN and -inf
      mine[j] = Cand{ordered(t), raw[j].key};
    }
    if (c0 == 0 && all > 128) {
      // the num_out-th largest of the threads' best, by the upper half of the order (beams are so
      // different that the warps' shares would say little)
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kRound / kThreads; ++j) top = max(top, static_cast<uint32_t>(mine[j].score >> 32));
      uint32_t bound = 0;
#pragma unroll 1
      for (int bit = 31; bit >= 8; --bit) {
        const uint32_t want = bound | 1u << bit;
        if (__syncthreads_count(top >= want) >= K) bound = want;
      }
      low = static_cast<uint64_t>(bound) << 32;
    }
#pragma unroll
    for (int j = 0; j < kRound / kThreads; ++j)
      if (mine[j].score && mine[j].score >= low) {
        const int to = atomicAdd(&n_list, 1);
        list[to] = mine[j];
        list_beam[to] = static_cast<uint8_t>(raw[j].beam);
      }
    __syncthreads();
    n = n_list;
    for (int i = warp; i < n; i += kWarps) {
      const Cand x = list[i];
      const int beam = list_beam[i];
      int r = 0;
      for (int j = lane; j < n; j += 32) {
        const Cand o = list[j];
        r += o.score != x.score ? o.score > x.score
             : list_beam[j] != beam ? list_beam[j] < beam : o.key > x.key;
      }
      r = __reduce_add_sync(kFullMask, r);
      if (r < K && lane == 0) {
        other[r] = x;
        other_beam[r] = static_cast<uint8_t>(beam);
      }
    }
    n = min(n, K);
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      list[i] = other[i];
      list_beam[i] = other_beam[i];
    }
    if (tid == 0) n_list = n;
    if (n == K) low = other[K - 1].score;
    __syncthreads();
  }
  for (int i = tid; i < K; i += kThreads) {
    const int64_t o = static_cast<int64_t>(s) * K + i;
    float score = kNegInf;
    int parent = -1, token = -1;
    if (i < n) {
      const uint64_t u = list[i].score;
      score = static_cast<float>(__longlong_as_double(static_cast<long long>(
          u & 0x8000000000000000ull ? u ^ 0x8000000000000000ull : ~u)));
      parent = static_cast<int>(row0) + list_beam[i];
      token = static_cast<int>(~static_cast<uint32_t>(list[i].key));
    }
    a.out_scores[o] = score;
    a.out_parents[o] = parent;
    a.out_tokens[o] = token;
  }
}

// Slices per row, of `spread` elements times a whole number.  A block costs about as much as 3 microseconds
// of its stream for its start, the first bound and the end; a spread of every thread's 16 bytes takes 0.37
// where two blocks share an SM (both fitted to bf16 rows; float32's bytes go at the same rate, but half as
// many elements).  The fewest microseconds over the rounds of 304 blocks (two on each of 152 SMs) win.
// Rows are cut into kMostCut slices in all at most, so that a workspace serves every smaller call.
constexpr int64_t kMostCut = 2 * 304;

int slices_for(int64_t rows, int vocab, int spread) {
  const int chunks = (vocab + spread - 1) / spread;
  int best = 1;
  double least = 1e300;
  for (int per = chunks; per >= 1; per = per > 64 ? per / 2 : per - 1) {
    const int64_t n = (chunks + per - 1) / per;
    if (n > 1 && rows * n > kMostCut) break;
    const double cost = static_cast<double>((rows * n + 303) / 304) * (3. + 0.37 * per) + 0.02 * n;
    if (cost < least) {
      least = cost;
      best = static_cast<int>(n);
    }
  }
  return best;
}

size_t part_bytes(int64_t blocks) { return static_cast<size_t>(blocks) * sizeof(float4); }

template <typename T>
cudaError_t launch_slices(const SelectArgs& a, int blocks, cudaStream_t cs) {
  constexpr int kBytes = kRingBytes + kList * 8;
  static SmemOnce once;
  const cudaError_t e = once.allow(select_slice_kernel<T>, kBytes);
  if (e != cudaSuccess) return e;
  return launch_early(select_slice_kernel<T>, blocks, kThreads, kBytes, cs, a);
}

}  // namespace
}  // namespace kvq

extern "C" size_t kvq_beam_select_workspace(int nseq, int beams, int vocab, int num_out) {
  using namespace kvq;
  if (nseq < 1 || beams < 1 || beams > KVQ_MAX_BEAMS || vocab < 1 || num_out < 1 ||
      num_out > KVQ_MAX_BEAM_OUT || static_cast<int64_t>(nseq) * beams > KVQ_MAX_SEQS)
    return 0;
  const int64_t rows = static_cast<int64_t>(nseq) * beams;
  const int64_t chunks = (vocab + kSpread<float> - 1) / kSpread<float>;   // of the larger elements
  const int64_t blocks = std::max(rows, std::min(kMostCut, rows * chunks));
  return part_bytes(blocks) + static_cast<size_t>(blocks) * num_out * 8;
}

extern "C" kvq_status kvq_beam_select(kvq_dtype dtype, const void* logits, int64_t row_stride,
                                      const float* scores, int nseq, int beams, int vocab,
                                      int num_out, float* out_scores, int32_t* out_parents,
                                      int32_t* out_tokens, void* workspace, size_t workspace_bytes,
                                      kvq_stream_t stream) {
  using namespace kvq;
  const char* fn = "kvq_beam_select";
  if (dtype != KVQ_F16 && dtype != KVQ_BF16 && dtype != KVQ_F32)
    return fail(KVQ_ERR_SHAPE, "%s: dtype %d is none of KVQ_F16, KVQ_BF16, KVQ_F32", fn,
                static_cast<int>(dtype));
  if (beams < 1 || beams > KVQ_MAX_BEAMS)
    return fail(KVQ_ERR_SHAPE, "%s: beams %d not in [1, %d]", fn, beams, KVQ_MAX_BEAMS);
  if (num_out < 1 || num_out > KVQ_MAX_BEAM_OUT)
    return fail(KVQ_ERR_SHAPE, "%s: num_out %d not in [1, %d]", fn, num_out, KVQ_MAX_BEAM_OUT);
  if (vocab < 1 || vocab > INT32_MAX - 65536)
    return fail(KVQ_ERR_SHAPE, "%s: vocab %d", fn, vocab);
  if (row_stride < vocab)
    return fail(KVQ_ERR_SHAPE, "%s: rows overlap (stride %lld, vocab %d)", fn,
                static_cast<long long>(row_stride), vocab);
  if (nseq < 0 || static_cast<int64_t>(nseq) * beams > KVQ_MAX_SEQS)
    return fail(KVQ_ERR_RANGE, "%s: %d sequences of %d beams (at most %d rows)", fn, nseq, beams,
                KVQ_MAX_SEQS);
  if (nseq == 0) return ok();
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !workspace)
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  const size_t size = dtype == KVQ_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size || !aligned16(workspace))
    return fail(KVQ_ERR_ALIGN, "%s: logits or workspace not aligned", fn);
  for (const void* p : {static_cast<const void*>(scores), static_cast<const void*>(out_scores),
                        static_cast<const void*>(out_parents), static_cast<const void*>(out_tokens)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(KVQ_ERR_ALIGN, "%s: scores or outputs not aligned", fn);
  const size_t need = kvq_beam_select_workspace(nseq, beams, vocab, num_out);
  if (workspace_bytes < need)
    return fail(KVQ_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes,
                need);
  SelectArgs a;
  a.logits = logits; a.scores = scores;
  a.out_scores = out_scores; a.out_parents = out_parents; a.out_tokens = out_tokens;
  a.stride = row_stride; a.beams = beams; a.vocab = vocab; a.num_out = num_out;
  const int rows = nseq * beams;
  const int spread = dtype == KVQ_F32 ? kSpread<float> : kSpread<__half>;
  const int chunks = (vocab + spread - 1) / spread;
  a.slices = slices_for(rows, vocab, spread);
  const int per = (chunks + a.slices - 1) / a.slices;
  a.slice = per * spread;
  a.slices = (chunks + per - 1) / per;
  const int64_t blocks = static_cast<int64_t>(rows) * a.slices;
  if (blocks > INT32_MAX || static_cast<int64_t>(beams) * a.slices * num_out > INT32_MAX - kRound)
    return fail(KVQ_ERR_RANGE, "%s: %lld blocks", fn, static_cast<long long>(blocks));
  a.part = static_cast<float4*>(workspace);
  a.keys = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + part_bytes(blocks));
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int n = static_cast<int>(blocks);
  cudaError_t e = dtype == KVQ_F16 ? launch_slices<__half>(a, n, cs)
                : dtype == KVQ_BF16 ? launch_slices<__nv_bfloat16>(a, n, cs) : launch_slices<float>(a, n, cs);
  if (e == cudaSuccess) e = launch_early(select_join_kernel, nseq, kThreads, 0, cs, a);
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}
