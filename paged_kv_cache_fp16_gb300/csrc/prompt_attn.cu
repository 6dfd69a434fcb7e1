// Causal attention over whole prompts on the fifth-generation tensor cores.
//
// For a tile of 128 query rows and tiles of NB keys:
//   S = Q K^T            tcgen05.mma, both operands in shared memory, S (float32) in TMEM
//   p = 2^(S c - m)      one thread per row (c = softmax_scale log2 e), running maximum and sum
//   O += P V             tcgen05.mma, P (16 bits) and O in TMEM
// so the scores never leave the SM and a key is read once per tile of rows.
//
// Rows: a tile packs the G = Hq / H query heads of a KV head beside as many tokens as fit
// (128 / G tokens x G heads), so that a short prompt or a single token still shares each key among
// its heads.
// Roles of the 6 warps: 4 softmax warps (thread = row = TMEM lane), one that issues the products,
// one that issues the tensor copies.  K and V go through one ring of equal slots: a K tile as
// pieces along the channels, a V tile as pieces along its keys, each of which is handed back when
// its products are done.
//
// TMEM holds O, one score buffer (two at 64 channels) and two of weights.  Scores are formed over
// scores that the softmax has in registers, and weights are written over those of the product before
// last: every reuse follows a barrier, because only products of one shape and accumulator are
// promised to run in the order of their issue.  (Two score buffers with the weights over the scores,
// and a wait for the product that reads them before the next scores: 512 queries over 16,500 keys at
// 256 channels 168 us, this way 154; at 64 and 128 channels equal.)
// Per head dimension: at 256, O, S and P of 128 keys fill TMEM, one CTA per SM, and the softmax of
// one tile runs under the products of the next; at 128 and 64 two CTAs share an SM and cover each
// other's softmax.  What bounds it (one GB300, whole prompts of 16,384 tokens in short runs): at 256
// the tensor cores (1,730 to 1,760 TFLOP/s in fp16, 1,790 to 1,840 in bf16, by the chip's power;
// 1,490 to 1,520 in long runs); at 128 the tensor cores fed from shared memory (a product of 128 x 64
// x 16 with both operands there takes 48 cycles, not 32; 1,380 to 1,480 TFLOP/s); at 64 the
// softmax's chain of waits, exponentials and stores, 1,340 cycles per tile and CTA (860 to 960
// TFLOP/s, tensor and exponential units 35 % busy).  One token over 131,000 keys at 256 channels:
// 86.5 us, 6.2 TB/s.
//
// Keys that a row does not see: scores are set to -inf whatever they hold; in the tiles where some
// row's view ends, V rows that no row sees are zeroed and non-finite V values that only some rows
// see are zeroed too, and added to those rows' results at the end (0 * inf would reach the others).
//
// Few rows over many keys: the keys are split over CTAs, each leaves (m, l, O) and a second kernel
// joins them.
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_tc5.cuh"

namespace kvq {
namespace {

#define kNegInf (-__int_as_float(0x7f800000))

constexpr int kRows = 128;
constexpr int kSoftmaxThreads = 128;
constexpr int kThreads = 192;

// NB: keys per tile.  KD: channels of a K slot (NB rows).  VR: keys of a V slot (D channels).
// kSlots: ring slots.  kCtas: resident CTAs per SM.  kScores: score buffers.
// Measured against each other (16,384 tokens, TFLOP/s): at 128 channels one buffer of 128 keys
// 1,049, two of 64 1,354; at 64 channels two of 64 in 2 CTAs 972, one of 128 in 2 CTAs 790, two of
// 128 in 1 CTA 749, one of 64 in 4 CTAs 848 (buffers then held the weights too).
template <int D> struct Cfg;
template <> struct Cfg<256> {
  static constexpr int NB = 128, KD = 128, VR = 64, kSlots = 5, kCtas = 1, kScores = 1;
};
template <> struct Cfg<128> {
  static constexpr int NB = 64, KD = 128, VR = 64, kSlots = 5, kCtas = 2, kScores = 1;
};
template <> struct Cfg<64> {
  static constexpr int NB = 64, KD = 64, VR = 64, kSlots = 8, kCtas = 2, kScores = 2;
};

template <int D>
struct Lay {
  using C = Cfg<D>;
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kSlot = C::NB * C::KD * 2;
  static_assert(kSlot == C::VR * D * 2, "K and V slots are alike");
  static constexpr int kRing = kQ;
  static constexpr int kBars = kRing + C::kSlots * kSlot;
  static constexpr int kNumBars = 2 * C::kSlots + 9;
  static constexpr int kTotal = kBars + kNumBars * 8 + 16;
  static constexpr int kCols = 512 / C::kCtas;
  static constexpr int kS = D, kP = D + C::kScores * C::NB;   // TMEM columns: O at 0, S, two of P
  static_assert(kP + 2 * (C::NB / 2) <= kCols, "TMEM");
  static_assert(kRows * D * 4 <= kBars, "the results are staged over the operands");
  static constexpr int nk = D / C::KD, nv = C::NB / C::VR;
};

struct PromptArgs {
  const uint16_t* v;
  int64_t vs;
  const int32_t* cu_q;
  const int32_t* cu_k;
  uint16_t* out;
  float* lse;
  float* ws;
  int32_t* err;
  int nseq, total_q, total_k, max_q, max_k, Hq, H, G;
  int tpt;        // tokens per row tile
  int n_splits;   // CTAs along the keys
  int tps;        // key tiles per split
  float c;        // softmax_scale * log2(e)
  float inv;      // softmax_scale / c: from powers of 2 back, c's own rounding taken out
};

// One row tile of one KV head of one sequence.
struct Unit {
  int q0, lq, k0, lk, h, tile;
  bool found;
};

struct SeqSpan {
  int q0, lq, k0, lk, tiles;
};

// Sequence s's offsets and row tiles (none if it contradicts the call's bounds).
__device__ __forceinline__ SeqSpan span_of(const PromptArgs& a, int s, bool check) {
  SeqSpan x{0, 0, 0, 0, 0};
  if (s >= a.nseq) return x;
  const int q0 = __ldg(a.cu_q + s), q1 = __ldg(a.cu_q + s + 1);
  const int k0 = __ldg(a.cu_k + s), k1 = __ldg(a.cu_k + s + 1);
  if (q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k &&
      q1 - q0 <= a.max_q && k1 - k0 <= a.max_k)
    return SeqSpan{q0, q1 - q0, k0, k1 - k0, (q1 - q0 + a.tpt - 1) / a.tpt};
  if (check) report(a.err, KVQ_DEVERR_INDEX);
  return x;
}

__device__ __forceinline__ Unit unit_of(const SeqSpan& x, int src, int tile, int h) {
  Unit r;
  r.q0 = __shfl_sync(kFullMask, x.q0, src);
  r.lq = __shfl_sync(kFullMask, x.lq, src);
  r.k0 = __shfl_sync(kFullMask, x.k0, src);
  r.lk = __shfl_sync(kFullMask, x.lk, src);
  r.tile = tile;
  r.h = h;
  r.found = true;
  return r;
}

// The unit of linear index u, found by a whole warp.  Late tiles have the most keys, and the CTAs
// that start last should have the least to do: with up to 32 sequences the tiles of all of them go
// from the highest number to the lowest; with more, sequences go in order, the tiles of each from
// the last to the first.  For each tile, its KV heads.  With `check` set every sequence is looked
// at and reported.  A call's units fit 31 bits.
__device__ __forceinline__ Unit find_unit(const PromptArgs& a, int u, bool check) {
  const int lane = threadIdx.x & 31;
  const uint32_t at = static_cast<uint32_t>(u);
  if (a.nseq <= 32) {
    const SeqSpan x = span_of(a, lane, check);
    // units of tiles numbered t and more
    auto from = [&](int t) {
      return __reduce_add_sync(kFullMask, static_cast<uint32_t>(max(0, x.tiles - t))) * a.H;
    };
    if (at >= from(0)) return Unit{};
    int lo = 0, hi = __reduce_max_sync(kFullMask, x.tiles);   // from(lo) > at, from(hi) <= at
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (from(mid) > at) lo = mid;
      else hi = mid;
    }
    const uint32_t rem = at - from(lo + 1), k = rem / a.H;
    const unsigned with = __ballot_sync(kFullMask, x.tiles > lo);
    const unsigned hit = __ballot_sync(
        kFullMask, x.tiles > lo && __popc(with & ((1u << lane) - 1)) == static_cast<int>(k));
    return unit_of(x, __ffs(hit) - 1, lo, static_cast<int>(rem - k * a.H));
  }
  Unit r{};
  uint32_t before = 0;
  for (int base = 0; base < a.nseq; base += 32) {
    const SeqSpan x = span_of(a, base + lane, check);
    const uint32_t mine = static_cast<uint32_t>(x.tiles) * a.H;
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kFullMask, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t start = before + incl - mine;
    const unsigned hit = __ballot_sync(kFullMask, at >= start && at - start < mine);
    if (hit && !r.found) {
      const int src = __ffs(hit) - 1;
      const uint32_t rem = __shfl_sync(kFullMask, at - start, src);
      const uint32_t back = rem / a.H;
      r = unit_of(x, src, __shfl_sync(kFullMask, x.tiles, src) - 1 - static_cast<int>(back),
                  static_cast<int>(rem - back * a.H));
      if (!check) return r;
    }
    before += __shfl_sync(kFullMask, incl, 31);
  }
  return r;
}

// Keys that token i of the sequence sees.
__device__ __forceinline__ int keys_seen(const Unit& n, int i) {
  return max(0, min(n.lk, i + n.lk - n.lq + 1));
}

template <bool BF> __device__ __forceinline__ float to_f(uint16_t b) {
  if constexpr (BF) return __uint_as_float(static_cast<uint32_t>(b) << 16);
  else return h2f(b);
}
// Whether either 16-bit half of w is an infinity or NaN.
template <bool BF> __device__ __forceinline__ bool nonfinite2(uint32_t w) {
  constexpr uint32_t e = BF ? 0x7f80u : 0x7c00u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}
template <bool BF> __device__ __forceinline__ uint32_t finite2(uint32_t w) {
  constexpr uint32_t e = BF ? 0x7f80u : 0x7c00u;
  if ((w & e) == e) w &= 0xffff0000u;
  if ((w & (e << 16)) == (e << 16)) w &= 0x0000ffffu;
  return w;
}

// ln sum exp of a row from its reference m (in powers of 2) and its sum of 2^(s c - m + kOff).
__device__ __forceinline__ float row_lse(const PromptArgs& a, float m, float l) {
  constexpr float unit = 1.f / 1024.f;   // 2^-kOff: the offset goes out without a rounding
  static_assert(tc5::kOff == 10.f, "2^kOff");
  return l == 0.f ? kNegInf : (m + log2f(l * unit)) * a.inv;
}

// A whole warp's bounded wait: every lane goes the same way on.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          const volatile int* gave_up) {
  return __all_sync(kFullMask, tc5::wait(bar, parity, gave_up));
}

// A V slot before its product, in a tile where some row's view ends: row i of the slot is key
// t0 + i.  Keys no row sees are zeroed; non-finite values that only some rows see are zeroed and
// noted in *flag.  (A row's 128-byte pieces may be taken in any order: the swizzle stays inside.)
template <bool BF, int D, int VR>
__device__ __forceinline__ void clean_v(unsigned char* slot, int t0, int lim_min, int lim_max,
                                        int* flag) {
  constexpr int P = D / 8;   // 16-byte pieces of a key
  const int a = max(0, lim_min - t0), b = min(VR, max(a, lim_max - t0));
  auto at = [&](int row, int c) {
    return reinterpret_cast<uint4*>(slot + (c >> 3) * VR * 128 + row * 128 + (c & 7) * 16);
  };
  bool found = false;
  for (int i = threadIdx.x; i < (b - a) * P; i += kSoftmaxThreads) {
    uint4* p = at(a + i / P, i % P);
    uint4 w = *p;
    if (nonfinite2<BF>(w.x) || nonfinite2<BF>(w.y) || nonfinite2<BF>(w.z) || nonfinite2<BF>(w.w)) {
      w.x = finite2<BF>(w.x);
      w.y = finite2<BF>(w.y);
      w.z = finite2<BF>(w.z);
      w.w = finite2<BF>(w.w);
      *p = w;
      found = true;
    }
  }
  for (int i = threadIdx.x; i < (VR - b) * P; i += kSoftmaxThreads)
    *at(b + i / P, i % P) = make_uint4(0, 0, 0, 0);
  if (found) *flag = 1;
}

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtas)
prompt_attn_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap mq,
                   const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using C = Cfg<D>;
  using L = Lay<D>;
  constexpr int NB = C::NB, SL = C::kSlots;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBars);
  uint64_t *full = bars, *empty = bars + SL, *qfull = bars + 2 * SL, *odone = qfull + 1,
           *sfull = odone + 2, *sfree = sfull + 2, *pready = sfree + 1, *drain = pready + 2;
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(bars + L::kNumBars);
  volatile int* flags = reinterpret_cast<volatile int*>(tmem_ptr + 1);   // [0] gave up, [1] V

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 160) {   // the copying warp's
    tc5::prefetch_map(&mq);
    tc5::prefetch_map(&mk);
    tc5::prefetch_map(&mv);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < SL; ++i) { mbar_init(full + i, 1); mbar_init(empty + i, 1); }
    mbar_init(qfull, 1);
    mbar_init(odone, 1);
    mbar_init(odone + 1, 1);
    mbar_init(drain, 1);
    mbar_init(sfull, 1);
    mbar_init(sfull + 1, 1);
    mbar_init(sfree, kSoftmaxThreads / 32);
    mbar_init(pready, kSoftmaxThreads / 32);
    mbar_init(pready + 1, kSoftmaxThreads / 32);
    tc5::fence_barrier_init();
    flags[0] = 0;
    flags[1] = 0;
  }
  if (warp == 4) tc5::tmem_alloc(tmem_ptr, L::kCols);   // (while the unit is looked for)
  const Unit n = find_unit(a, blockIdx.x, blockIdx.x == 0 && blockIdx.y == 0 && warp == 0);
  const int i0 = n.tile * a.tpt, i1 = min(i0 + a.tpt, n.lq);      // the tile's tokens
  const int lim_min = keys_seen(n, i0), lim_max = keys_seen(n, i1 - 1);
  const int all = (lim_max + NB - 1) / NB;                         // key tiles any row sees
  const int j0 = blockIdx.y * a.tps, j1 = min(j0 + a.tps, all);
  const int nt = j1 - j0;
  const bool none = !n.found || (nt <= 0 && !(all == 0 && j0 == 0));
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = *tmem_ptr;
  if (none) {
    if (warp == 4) tc5::tmem_dealloc(tmem, L::kCols);
    return;
  }

  if (warp == 5) {
    // ---------------------------------------------------------------- tensor copies (one thread)
    if (nt > 0 && tc5::elect_one()) {
      mbar_expect_tx(qfull, (D / 64) * 128 * a.tpt * a.G);
      for (int p = 0; p < D / 64; ++p)
        tc5::tma_load_3d(sm + p * kRows * 128, &mq, p * 64, n.h * a.G, n.q0 + i0, qfull);
      int pos = 0;
      bool ok = true;
      auto slot_ready = [&]() {
        if (pos >= SL && !tc5::wait(empty + pos % SL, (pos / SL + 1) & 1, flags)) {
          flags[0] = 1;
          ok = false;
        }
        return ok;
      };
      auto load_k = [&](int j) {
        for (int i = 0; i < L::nk; ++i) {
          if (!slot_ready()) return;
          unsigned char* dst = sm + L::kRing + (pos % SL) * L::kSlot;
          mbar_expect_tx(full + pos % SL, L::kSlot);
#pragma unroll
          for (int p = 0; p < C::KD / 64; ++p)
            tc5::tma_load_3d(dst + p * NB * 128, &mk, i * C::KD + p * 64, n.h, n.k0 + (j0 + j) * NB,
                             full + pos % SL);
          ++pos;
        }
      };
      auto load_v = [&](int j) {
        for (int i = 0; i < L::nv; ++i) {
          if (!slot_ready()) return;
          unsigned char* dst = sm + L::kRing + (pos % SL) * L::kSlot;
          mbar_expect_tx(full + pos % SL, L::kSlot);
#pragma unroll
          for (int p = 0; p < D / 64; ++p)
            tc5::tma_load_3d(dst + p * C::VR * 128, &mv, p * 64, n.h,
                             n.k0 + (j0 + j) * NB + i * C::VR, full + pos % SL);
          ++pos;
        }
      };
      load_k(0);
      for (int j = 0; j < nt && ok; ++j) {
        if (j + 1 < nt) load_k(j + 1);
        if (ok) load_v(j);
      }
      // Whichever role gives up, and whether this one has by then issued everything or not: no copy
      // is in flight when the block ends.
      for (int i = max(0, pos - SL); i < pos; ++i) mbar_wait_bounded(full + i % SL, (i / SL) & 1);
      mbar_wait_bounded(qfull, 0);
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------------- products (one thread)
    if (nt > 0 && tc5::elect_one()) {
      const uint32_t base = smem_u32(sm), ring = base + L::kRing;
      const uint64_t dk = tc5::desc_base(16), dv = tc5::desc_base(C::VR * 128);
      constexpr uint32_t id_s = tc5::idesc(BF, NB, false), id_o = tc5::idesc(BF, D, true);
      int pos = 0;
      bool ok = tc5::wait(qfull, 0, flags);
      auto product_s = [&](int j) {
        for (int i = 0; i < L::nk; ++i, ++pos) {
          ok = ok && tc5::wait(full + pos % SL, (pos / SL) & 1, flags);
          if (C::kScores == 1 && i == 0 && j > 0) {   // (of two, tile j - 2's: pready told)
            ok = ok && tc5::wait(sfree, (j - 1) & 1, flags);
            tc5::fence_after();
          }
          if (!ok) return;
          const uint32_t kb = ring + (pos % SL) * L::kSlot;
#pragma unroll
          for (int k = 0; k < C::KD / 16; ++k) {
            const int kq = i * (C::KD / 16) + k;   // the contraction step within the row
            tc5::mma_ss(tmem + L::kS + j % C::kScores * NB,
                        tc5::desc_at(dk, base + (kq / 4) * kRows * 128 + (kq % 4) * 32),
                        tc5::desc_at(dk, kb + (k / 4) * NB * 128 + (k % 4) * 32), id_s, kq > 0);
          }
          tc5::commit(empty + pos % SL);
        }
        tc5::commit(sfull + (j & 1));   // completes when everything issued before has: O of tile j - 2 too
      };
      auto product_o = [&](int j) {
        ok = ok && tc5::wait(full + pos % SL, (pos / SL) & 1, flags);   // sooner than the weights
        ok = ok && tc5::wait(pready + (j & 1), (j >> 1) & 1, flags);
        if (!ok) return;
        tc5::fence_after();
        const uint32_t pb = tmem + L::kP + (j & 1) * (NB / 2);
        for (int i = 0; i < L::nv; ++i, ++pos) {
          if (i > 0) ok = ok && tc5::wait(full + pos % SL, (pos / SL) & 1, flags);
          if (!ok) return;
          const uint32_t vb = ring + (pos % SL) * L::kSlot;
#pragma unroll
          for (int k = 0; k < C::VR / 16; ++k)
            tc5::mma_ts(tmem, pb + (i * (C::VR / 16) + k) * 8, tc5::desc_at(dv, vb + k * 2048), id_o,
                        j > 0 || i > 0 || k > 0);
          tc5::commit(empty + pos % SL);
        }
        tc5::commit(odone + (j & 1));   // two, so that no wait is a whole turn of parity behind
      };
      if (ok) product_s(0);
      for (int j = 0; j < nt && ok; ++j) {
        if (j + 1 < nt) product_s(j + 1);
        if (ok) product_o(j);
      }
      if (!ok) flags[0] = 1;
      tc5::commit(drain);   // what was issued ends before the memory is given back, as above
      mbar_wait_bounded(drain, 0);
    }
  } else {
    // ------------------------------------------------------------------ softmax: thread = row
    const int r = threadIdx.x, ri = r / a.G;
    const int tok = i0 + ri;
    const bool live = ri < a.tpt && tok < i1;
    const int limit = live ? keys_seen(n, tok) : 0;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp) << 21);
    float m = kNegInf, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      ok = warp_wait(sfull + (j & 1), (j >> 1) & 1, flags);
      if (!ok) break;
      tc5::fence_after();
      const int t0 = (j0 + j) * NB;
      const bool edge = t0 + NB > lim_min;
      const int left = limit - t0;   // columns that the row sees
      uint32_t s[NB];
#pragma unroll
      for (int q = 0; q < NB / 32; ++q) tc5::ld32(lanes + L::kS + j % C::kScores * NB + q * 32, s + q * 32);
      tc5::wait_ld32(s);
#pragma unroll
      for (int q = 1; q < NB / 32; ++q) tc5::after_ld32(s + q * 32);
      if (edge) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
          if (i >= left) s[i] = 0xff800000u;
      }
      const float x = tc5::row_max<NB>(s) * a.c;
      if constexpr (C::kScores == 1) {   // the next scores may come (said before the maximum: slower)
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree);
      }
      if (j == 0) {
        m = x;
      } else {
        const bool up = x > m + tc5::kSlack;
        if (__any_sync(kFullMask, up)) {
          const float f = up ? ex2_fast(m - x) : 1.f;
          if (up) m = x;
          l *= f;
          ok = warp_wait(odone + ((j - 1) & 1), (j - 1) >> 1 & 1, flags);
          if (!ok) break;
          tc5::fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tc5::ld32(lanes + q * 32, o);
            tc5::wait_ld32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tc5::st32(lanes + q * 32, o);
          }
          tc5::wait_st();
        }
      }
      const float mo = m == kNegInf ? 0.f : m - tc5::kOff;
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int q = 0; q < NB / 32; ++q) {   // over the weights of tile j - 2: sfull told of their product
        tc5::weights32<BF>(s + q * 32, a.c, mo, lanes + L::kP + (j & 1) * (NB / 2) + q * 16, sum);
      }
      l += tc5::sum_of(sum);
      tc5::wait_st();
      if (edge) {
        // a slot's phase is told by its parity: the load before the one waited for must be known
        // to be over, and it is once the product of the tile before is
        if (j > 0) ok = warp_wait(odone + ((j - 1) & 1), (j - 1) >> 1 & 1, flags);
        const int at = min(j + 2, nt) * L::nk + j * L::nv;   // loaded before it
        for (int i = 0; i < L::nv; ++i) {
          const int pos = at + i;
          ok = ok && warp_wait(full + pos % SL, (pos / SL) & 1, flags);
          if (ok)
            clean_v<BF, D, C::VR>(sm + L::kRing + (pos % SL) * L::kSlot, t0 + i * C::VR, lim_min,
                                  lim_max, const_cast<int*>(flags) + 1);
        }
        if (!ok) break;
        tc5::fence_smem();
      }
      tc5::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready + (j & 1));   // one per warp: arrivals of lanes queue up
    }
    if (ok && nt > 0) ok = warp_wait(odone + ((nt - 1) & 1), (nt - 1) >> 1 & 1, flags);
    if (!ok) flags[0] = 1;
    tc5::fence_after();
    asm volatile("bar.sync 1, 128;" ::: "memory");   // every row's note on V is in
    const bool fix = flags[1] != 0;
    const bool whole = a.n_splits == 1 || all <= a.tps;
    const int head = n.h * a.G + (r - ri * a.G);
    const int64_t row = (static_cast<int64_t>(n.q0) + tok) * a.Hq + head;
    float* part = a.ws + ((static_cast<int64_t>(blockIdx.x) * a.n_splits + blockIdx.y) * kRows + r) *
                             (D + 4);
    if (fix && nt > 0) {   // apart from the rows' way out, which short calls run once, from cold
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tc5::ld32(lanes + q * 32, o);
        tc5::wait_ld32(o);
        for (int t = max(lim_min, j0 * NB); t < min(limit, j1 * NB); ++t) {
          const uint16_t* vr = a.v + (n.k0 + t) * a.vs + static_cast<int64_t>(n.h) * D + q * 32;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float v = to_f<BF>(vr[i]);
            if (!isfinite(v)) o[i] = __float_as_uint(__uint_as_float(o[i]) + v);
          }
        }
        __syncwarp();
        tc5::st32(lanes + q * 32, o);
      }
      tc5::wait_st();
    }
    const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
    // The rows go through shared memory, over the operands (all products are done), so that they
    // are written whole.  (Stored by each row's thread, 16 bytes here and there: prompts of 128 and
    // 1,024 tokens at 256 channels 10.0 and 24.5 us, this way 9.4 and 23.4.)
    const int row_bytes = whole ? D * 2 : D * 4;
    unsigned char* mine = sm + r * row_bytes;
    auto put = [&](int piece, uint4 w) {
      *reinterpret_cast<uint4*>(mine + (piece ^ (r & 7)) * 16) = w;
    };
    const int used = __popc(__ballot_sync(kFullMask, live));   // the warp's first rows
#pragma unroll 1
    for (int q = 0; q < (used ? D / 32 : 0); q += 2) {
      uint32_t o[64];
      __syncwarp();
      if (nt > 0) {
        tc5::ld32(lanes + q * 32, o);
        tc5::ld32(lanes + q * 32 + 32, o + 32);
        tc5::wait_ld32(o);
        tc5::after_ld32(o + 32);
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) o[i] = 0;
      }
      if (!live) continue;
#pragma unroll
      for (int i = 0; i < 64; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
      if (whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = tc5::pack2<BF>(__uint_as_float(o[i * 8 + e * 2]), __uint_as_float(o[i * 8 + e * 2 + 1]));
          put(q * 4 + i, make_uint4(w[0], w[1], w[2], w[3]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          put(q * 8 + i, make_uint4(o[i * 4], o[i * 4 + 1], o[i * 4 + 2], o[i * 4 + 3]));
      }
    }
    __syncwarp();
    // this warp's 32 rows, PR pieces of 16 bytes each
    auto write = [&](auto pieces, unsigned char* base, int64_t at) {   // at: own row's offset, -1: none
      constexpr int PR = decltype(pieces)::value;
      constexpr int rows = PR < 32 ? 32 / PR : 1;       // rows per step of the warp
      constexpr int batch = 8;
#pragma unroll 1
      for (int i = 0; i * 32 < used * PR; i += batch) {   // 32 pieces per step
        uint4 w[batch];
        int64_t to[batch];
#pragma unroll
        for (int e = 0; e < batch; ++e) {
          const int rr = PR < 32 ? (i + e) * rows + lane / PR : (i + e) / (PR / 32);
          const int p = PR < 32 ? lane % PR : lane + (i + e) % (PR / 32) * 32;
          to[e] = __shfl_sync(kFullMask, at, rr);
          if (to[e] >= 0) to[e] += p * 16;
          w[e] = *reinterpret_cast<const uint4*>(sm + (warp * 32 + rr) * (PR * 16) +
                                                 (p ^ (rr & 7)) * 16);
        }
#pragma unroll
        for (int e = 0; e < batch; ++e)
          if (to[e] >= 0) *reinterpret_cast<uint4*>(base + to[e]) = w[e];
      }
    };
    if (whole)
      write(std::integral_constant<int, D / 8>(), reinterpret_cast<unsigned char*>(a.out),
            live ? row * (D * 2) : -1);
    else
      write(std::integral_constant<int, D / 4>(), reinterpret_cast<unsigned char*>(part - r * (D + 4)),
            live ? static_cast<int64_t>(r) * (D + 4) * 4 : -1);
    if (live) {
      if (whole) {
        if (a.lse)
          a.lse[row] = row_lse(a, m, l);
      } else {
        part[D] = m;
        part[D + 1] = l;
      }
    }
    tc5::fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 4) {
    tc5::fence_after();
    tc5::tmem_dealloc(tmem, L::kCols);
  }
  if (threadIdx.x == 0 && flags[0]) report(a.err, KVQ_DEVERR_TIMEOUT);
}

// Joins the splits of a unit's rows: a thread holds 4 channels of a row and of one of S slices of
// the splits.  With up to 8 splits S = 1 and a block has several rows; with more, the slices of one
// row are joined in shared memory (one warp per row with the splits one after the other took 11 us
// for the 38 splits of a single token's rows; S > 1 for many rows of few splits took 10 us more
// than S = 1).
constexpr int kJoinThreads = 256;

template <bool BF, int D, int S>
__global__ void __launch_bounds__(kJoinThreads)
prompt_join_kernel(const __grid_constant__ PromptArgs a) {
  constexpr int NB = Cfg<D>::NB, T = D / 4, kRowsPer = kJoinThreads / (T * S);
  __shared__ float4 so[S][T];
  __shared__ float sm[S], sl[S];
  const Unit n = find_unit(a, blockIdx.x, false);
  if (!n.found) return;
  const int i0 = n.tile * a.tpt, i1 = min(i0 + a.tpt, n.lq);
  const int all = (keys_seen(n, i1 - 1) + NB - 1) / NB;
  if (all <= a.tps) return;
  const int live = (all + a.tps - 1) / a.tps;
  const int t = threadIdx.x % T, slice = S > 1 ? threadIdx.x / T : 0;
  constexpr int64_t step = static_cast<int64_t>(kRows) * (D + 4);
  // (with S > 1 all threads of a block have one row)
  for (int r = blockIdx.y * kRowsPer + (S > 1 ? 0 : threadIdx.x / T); r < (i1 - i0) * a.G;
       r += gridDim.y * kRowsPer) {
    const float* part = a.ws + (static_cast<int64_t>(blockIdx.x) * a.n_splits * kRows + r) * (D + 4);
    float M = kNegInf, l = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = slice; i < live; i += S) {
      const float* p = part + i * step;
      const float4 o = *reinterpret_cast<const float4*>(p + t * 4);
      const float2 ml = *reinterpret_cast<const float2*>(p + D);
      const float Mn = fmaxf(M, ml.x);
      const float f = M == kNegInf ? 0.f : ex2_fast(M - Mn);
      const float g = ml.x == kNegInf ? 0.f : ex2_fast(ml.x - Mn);
      l = l * f + ml.y * g;
      O.x = O.x * f + o.x * g;
      O.y = O.y * f + o.y * g;
      O.z = O.z * f + o.z * g;
      O.w = O.w * f + o.w * g;
      M = Mn;
    }
    if constexpr (S > 1) {
      so[slice][t] = O;
      if (t == 0) {
        sm[slice] = M;
        sl[slice] = l;
      }
      __syncthreads();
      if (slice == 0) {
        M = sm[0];
#pragma unroll
        for (int i = 1; i < S; ++i) M = fmaxf(M, sm[i]);
        l = 0.f;
        O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const float g = sm[i] == kNegInf ? 0.f : ex2_fast(sm[i] - M);
          const float4 o = so[i][t];
          l = fmaf(sl[i], g, l);
          O.x = fmaf(o.x, g, O.x);
          O.y = fmaf(o.y, g, O.y);
          O.z = fmaf(o.z, g, O.z);
          O.w = fmaf(o.w, g, O.w);
        }
      }
      __syncthreads();
    }
    if (slice == 0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t row = (static_cast<int64_t>(n.q0) + i0 + r / a.G) * a.Hq + n.h * a.G + r % a.G;
      *reinterpret_cast<uint2*>(a.out + row * D + t * 4) =
          make_uint2(tc5::pack2<BF>(O.x * inv, O.y * inv), tc5::pack2<BF>(O.z * inv, O.w * inv));
      if (a.lse && t == 0)
        a.lse[row] = row_lse(a, M, l);
    }
  }
}

// How a call is cut: row tiles (an upper bound: the lengths are on the device) and splits.
struct Plan {
  int tpt, tps, n_splits;
  int64_t units;
  int64_t most_parts;   // units x splits at most, of this call and any with smaller bounds; 0: never split
};

Plan plan_for(int nseq, int total_q, int num_q_heads, int num_kv_heads, int D, int max_q,
              int max_k) {
  const int nb = D == 256 ? 128 : 64, ctas = D == 256 ? 1 : 2;
  Plan p;
  p.tpt = kRows / (num_q_heads / num_kv_heads);
  const int64_t per = (static_cast<int64_t>(max_q) + p.tpt - 1) / p.tpt;
  const int64_t a = static_cast<int64_t>(nseq) * per, b = total_q / p.tpt + static_cast<int64_t>(nseq);
  p.units = (a < b ? a : b) * num_kv_heads;
  const int64_t tiles = (static_cast<int64_t>(max_k) + nb - 1) / nb;
  const int64_t slots = static_cast<int64_t>(sm_count() > 0 ? sm_count() : 152) * ctas;
  // Split only while the units leave SMs idle, and not below four tiles per split: a split costs
  // its start (about the time of two tiles) and its partial rows.
  int64_t want = p.units > 0 ? slots / p.units : 1;
  const int64_t most = (tiles + 3) / 4;
  // n_splits is at most `want`, so units * n_splits at most slots, and at most units * most; both
  // bounds fall with each of the call's
  p.most_parts = most <= 1 ? 0 : (p.units < slots / most ? p.units * most : slots);
  want = want > most ? most : want;
  if (want < 1) want = 1;
  p.tps = static_cast<int>((tiles + want - 1) / want);
  if (p.tps < 1) p.tps = 1;
  p.n_splits = tiles > 0 ? static_cast<int>((tiles + p.tps - 1) / p.tps) : 1;
  return p;
}

// Partial rows: O, m, l and two floats of padding, 128 rows of each part.
size_t parts_bytes(int64_t parts, int D) {
  return static_cast<size_t>(parts) * kRows * (D + 4) * sizeof(float);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::mutex mu;
  static EncodeFn fn = nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &st) == cudaSuccess && st == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  }
  return fn;
}

// Rows [tokens][heads][D] in boxes of 64 channels x `bh` heads x `bt` tokens, 128-byte swizzle.
bool encode(CUtensorMap* m, bool bf, const uint16_t* base, int64_t stride, int tokens, int heads,
            int D, int bh, int bt) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(bh), static_cast<cuuint32_t>(bt)};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode_fn()(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                     const_cast<uint16_t*>(base), dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF, int D>
kvq_status launch(const char* fn, PromptArgs& a, const Plan& p, const uint16_t* q, int64_t qs,
                  const uint16_t* k, int64_t ks, const uint16_t* v, int64_t vs, cudaStream_t cs) {
  using C = Cfg<D>;
  CUtensorMap mq, mk, mv;
  if (!encode_fn()) return fail(KVQ_ERR_CUDA, "%s: the driver has no cuTensorMapEncodeTiled", fn);
  bool ok = encode(&mq, BF, q, qs, a.total_q, a.Hq, D, a.G, p.tpt);
  if (a.total_k > 0) {
    ok = ok && encode(&mk, BF, k, ks, a.total_k, a.H, D, 1, C::NB) &&
         encode(&mv, BF, v, vs, a.total_k, a.H, D, 1, C::VR);
  } else {
    mk = mv = mq;   // no key: no copy is issued
  }
  if (!ok) return fail(KVQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled refused q, k or v", fn);
  cudaError_t e = cudaFuncSetAttribute(prompt_attn_kernel<BF, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kTotal);
  if (e == cudaSuccess) {
    const dim3 grid(static_cast<unsigned>(p.units), p.n_splits);
    prompt_attn_kernel<BF, D><<<grid, kThreads, Lay<D>::kTotal, cs>>>(a, mq, mk, mv);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && p.n_splits > 1) {
    constexpr int kSlices = kJoinThreads / (D / 4);
    const bool few = p.n_splits <= 8;
    int blocks = a.G * (a.max_q < p.tpt ? a.max_q : p.tpt);   // rows of a unit
    if (few) blocks = (blocks + kSlices - 1) / kSlices;
    const int64_t fill = 8192 / p.units;   // a few waves at most
    if (blocks > fill) blocks = fill < 1 ? 1 : static_cast<int>(fill);
    const dim3 grid(static_cast<unsigned>(p.units), blocks);
    if (few) prompt_join_kernel<BF, D, 1><<<grid, kJoinThreads, 0, cs>>>(a);
    else prompt_join_kernel<BF, D, kSlices><<<grid, kJoinThreads, 0, cs>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok ? kvq::ok() : KVQ_ERR_CUDA;
}

}  // namespace
}  // namespace kvq

extern "C" size_t kvq_prompt_attn_workspace(int nseq, int total_q, int num_q_heads,
                                            int num_kv_heads, int head_dim, int max_q,
                                            int max_k) {
  if (nseq < 1 || total_q < 0 || num_kv_heads < 1 || num_q_heads < num_kv_heads ||
      num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > kvq::kRows || max_q < 0 ||
      max_k < 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const kvq::Plan p =
      kvq::plan_for(nseq, total_q, num_q_heads, num_kv_heads, head_dim, max_q, max_k);
  return p.most_parts ? kvq::parts_bytes(p.most_parts, head_dim) : 16;
}

extern "C" kvq_status kvq_prompt_attn(kvq_dtype dtype, const uint16_t* q, int64_t q_stride,
                                      const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                      int64_t v_stride, int num_q_heads, int num_kv_heads,
                                      int head_dim, const int32_t* cu_q, const int32_t* cu_k,
                                      int nseq, int total_q, int total_k, int max_q, int max_k,
                                      float softmax_scale, uint16_t* out, float* lse,
                                      void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                      kvq_stream_t stream) {
  using namespace kvq;
  const char* fn = "kvq_prompt_attn";
  if (dtype != KVQ_F16 && dtype != KVQ_BF16)
    return fail(KVQ_ERR_SHAPE, "%s: dtype %d is neither KVQ_F16 nor KVQ_BF16", fn,
                static_cast<int>(dtype));
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(KVQ_ERR_SHAPE, "%s: head_dim %d unsupported (64, 128 or 256)", fn, head_dim);
  if (num_kv_heads < 1 || num_kv_heads > 65535 || num_q_heads < num_kv_heads ||
      num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 128)
    return fail(KVQ_ERR_SHAPE, "%s: num_q_heads %d must be a multiple of num_kv_heads %d, at most "
                "128 per KV head", fn, num_q_heads, num_kv_heads);
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kw = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_stride < qw || k_stride < kw || v_stride < kw || q_stride % 8 || k_stride % 8 ||
      v_stride % 8)
    return fail(KVQ_ERR_SHAPE, "%s: a token stride is below heads * head_dim or no multiple of 8",
                fn);
  if (nseq < 0 || total_q < 0 || total_k < 0 || max_q < 0 || max_k < 0)
    return fail(KVQ_ERR_RANGE, "%s: a count is negative", fn);
  if (total_k > INT32_MAX - kRows)
    return fail(KVQ_ERR_RANGE, "%s: total_k %d > 2^31 - 129", fn, total_k);
  const float c = softmax_scale * 1.4426950408889634f;   // of scores in powers of 2
  if (!std::isfinite(c) || softmax_scale <= 0)
    return fail(KVQ_ERR_RANGE, "%s: softmax_scale is not a finite value > 0 (2.3e38 at most)", fn);
  if (nseq == 0 || total_q == 0 || max_q == 0) return ok();
  if (!q || !cu_q || !cu_k || !out || !workspace || (total_k > 0 && (!k || !v)))
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      !aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(KVQ_ERR_ALIGN, "%s: a pointer is not 16-byte aligned (lse 4)", fn);
  const Plan p = plan_for(nseq, total_q, num_q_heads, num_kv_heads, head_dim, max_q, max_k);
  const size_t need = p.n_splits == 1 ? 16 : parts_bytes(p.units * p.n_splits, head_dim);
  if (workspace_bytes < need)
    return fail(KVQ_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, workspace_bytes, need);
  if (p.units > INT32_MAX)
    return fail(KVQ_ERR_RANGE, "%s: %lld row tiles exceed the grid", fn,
                static_cast<long long>(p.units));
  PromptArgs a;
  a.v = v; a.vs = v_stride; a.cu_q = cu_q; a.cu_k = cu_k; a.out = out; a.lse = lse;
  a.ws = static_cast<float*>(workspace); a.err = dev_err; a.nseq = nseq; a.total_q = total_q;
  a.total_k = total_k; a.max_q = max_q; a.max_k = max_k; a.Hq = num_q_heads; a.H = num_kv_heads;
  a.G = num_q_heads / num_kv_heads; a.tpt = p.tpt; a.n_splits = p.n_splits; a.tps = p.tps;
  a.c = c;
  a.inv = static_cast<float>(static_cast<double>(softmax_scale) / c);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto bf, auto d) {
    return launch<decltype(bf)::value, decltype(d)::value>(fn, a, p, q, q_stride, k, k_stride, v,
                                                           v_stride, cs);
  };
  auto by_dim = [&](auto bf) {
    if (head_dim == 256) return go(bf, std::integral_constant<int, 256>());
    if (head_dim == 128) return go(bf, std::integral_constant<int, 128>());
    return go(bf, std::integral_constant<int, 64>());
  };
  return dtype == KVQ_BF16 ? by_dim(std::true_type()) : by_dim(std::false_type());
}
