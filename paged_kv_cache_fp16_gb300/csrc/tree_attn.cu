// Attention of a tree of drafted tokens over the packed pages, on the fifth-generation tensor
// cores.
//
// A sequence's (draft, grouped query head) pairs of one KV head, draft by draft, are cut into row
// tiles of 128 (a draft's heads may lie in two: 64 drafts of 6 heads fill 3 tiles); per tile of 64
// tokens the packed codes are brought in once and become fp16 in shared memory, exactly as
// the dequantizer rounds them (k_hat = fp16(c * scale)):
//   S = Q K_hat^T       tcgen05.mma, Q (fp16) in TMEM, K_hat in shared memory
//   p = 2^(S c - m)     two threads per row, running maximum and sum; drafts outside the row's
//                       64-bit ancestor mask get weight 0
//   O += P V_hat        tcgen05.mma, P (fp16) in TMEM over the place of S, V_hat in shared memory
// TMEM is full: O 256 columns, two score buffers of 64, Q 128.  With Q in TMEM the first product
// reads only K_hat from shared memory, whose bandwidth is the scarcest after the codes' arrival.
//
// Roles of the 19 warps of a persistent CTA (one per SM): 8 softmax, 1 issues the products, 2
// bring codes and scales of K and of V (16-token groups of a page) into rings deep enough to cover
// the memory latency, 8 unpack.
//
// What bounds it: per tile of 64 tokens shared memory moves 178 KB at q6 (codes in and out, K_hat
// and V_hat in and out: 1,390 cycles), the unpacking and the softmax issue 5,300 warp instructions
// (1,340 cycles of the four schedulers), the products take 1,024 and the codes' arrival 1,060; they
// overlap to 2,500 cycles, the unpacking warps being busy for 2,000 of them (reads, arithmetic and
// the waits for the double buffers, which fill shared memory).  262,000 tokens and 16 drafts of 6
// heads: q6 142 us (2.87 TB/s, 726 TFLOP/s), q4 130 us; 8 x 20,000 tokens q8, 10 drafts 100 us
// (3.3 TB/s), 64 drafts (3 row tiles) 273 us.  The 96 registers that 19 warps leave are not quite
// enough (84 to 88 bytes of spills).  Measured against this: 16 unpacking warps (fewer registers
// each) and 4 softmax warps slower; two copying warps for each of K and V leave 80 registers, 158 us;
// a thread each for the two products, 8 ragged caches with 64 drafts at q8 214 instead of 189 us.
//
// Work: the tiles of all (layer, sequence, KV head, row tile) units in one line are dealt to the
// CTAs in equal contiguous shares, whatever the sequences' lengths (which only the device knows).
// A unit that lies inside one share is finished there; the at most two cut units of a share leave
// (m, l, O) and a second kernel joins them.  Short caches (8 tiles at most) are dealt whole units.
//
// Order of channels: unpacking is cheapest when it leaves pairs that lie 16 bits apart, so K_hat,
// V_hat and Q hold the channels of each group of 4 (q6) or 8 (q4) permuted; scores do not change,
// and O's columns are put back in order when they are stored.
#include <cmath>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_math.cuh"
#include "kvq_tc5.cuh"

namespace kvq {
namespace {

#define kNegInf (-__int_as_float(0x7f800000))

constexpr int kD = 256;
constexpr int kRows = 128;
constexpr int kTile = 64;             // tokens per tile
constexpr int kSoftmaxWarps = 8;      // warps 0-7: two threads per row, half of the columns each
constexpr int kMmaWarp = 8, kCopyWarp = 9, kUnpackWarp0 = 11, kUnpackWarps = 8;   // copies: K 9, V 10
constexpr int kThreads = (kUnpackWarp0 + kUnpackWarps) * 32;
constexpr int kRec = (kD + 2) * kRows;   // a partial record: O [256 / 4][128 rows][4], then m and l [128]
constexpr int kShortTiles = 8;        // caches of at most so many tiles are not cut
constexpr uint32_t kNoRow = 0xffffffffu;
constexpr int kMeta = 16;             // entries of the ring of group-validity bits
constexpr int kStage = kTile * kD * 2;
constexpr uint32_t kColS = 256, kColQ = 384, kCols = 512;   // TMEM: O at 0, S at 256 and 320, Q

struct TreePools {
  const uint8_t* kc;
  const uint16_t* ks;
  const uint8_t* vc;
  const uint16_t* vs;
  int64_t k_pages, v_pages;
};

// What a CTA leaves of the unit that its share cuts at the tail (the unit's first record): the
// join needs no search.  n = 0: none.
struct Cut {
  int n, row0, first, rows;   // records from this CTA on; out's row of the unit's sequence and KV
                              // head; the row tile's first row and its rows
};

struct TreeArgs {
  TreePools L[KVQ_MAX_TENSORS];
  const uint16_t* q;
  uint16_t* out;
  float* ws;
  const int32_t* pt;
  const int32_t* lens;
  const int32_t* cu;
  const int32_t* parents;
  int32_t* err;
  int n_layers, nseq, total, H, Hq, G, ps, max_pages, max_nodes, max_len;
  int grid;     // CTAs of the attention kernel
  int whole;    // deal whole units (short caches)
  uint32_t most_units, most_tiles;   // of a layer, by the call's bounds
  Cut* cuts;    // [grid]
  float c;      // softmax_scale * log2(e)
};

template <int BITS>
struct Lay {
  static constexpr int kPd = kD * BITS / 8;
  static constexpr int kRaw = kTile * kPd + 2 * kTile;   // codes and scales of K or V
  static constexpr int kRaws = BITS == 8 ? 3 : BITS == 6 ? 4 : 6;
  static constexpr int kK = 0, kV = 2 * kStage, kRawAt = 4 * kStage;
  static constexpr int kBars = kRawAt + 2 * kRaws * kRaw;
  static constexpr int kNumBars = 4 * kRaws + 4 * 2 + 3 * 2 + 2;
  static constexpr int kTail = kBars + kNumBars * 8;         // then: TMEM address, flags, meta,
  static constexpr int kParents = kTail + 16 + kMeta * 4;    // and the parents
  static constexpr int kHalves = kParents + KVQ_MAX_NODES;       // and the exchange [2][128]
  static constexpr int kConst = kHalves + 2 * kRows * 4;          // and the unpacking's constants
  static constexpr int kTotal = kConst + 16;
  static_assert(kTotal <= 232448, "shared memory");
};

// Where the element of natural index e of an aligned group of 8 channels is stored.
template <int BITS> __host__ __device__ constexpr int place(int e) {
  return BITS == 6 ? (e & 4) | ((e & 1) << 1) | ((e >> 1) & 1)
         : BITS == 4 ? ((e & 3) << 1) | (e >> 2) : e;
}

// The channel at place p of an aligned group of 32: the inverse.
template <int BITS> __host__ __device__ constexpr int channel(int p) {
  for (int e = 0; e < 8; ++e)
    if (place<BITS>(e) == (p & 7)) return (p & ~7) | e;
  return p;
}

struct Seq {
  int n0, n, len, tiles, rt;   // first draft, drafts, cached tokens, token tiles, row tiles
};

__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int s, bool check) {
  Seq q{0, 0, 0, 0, 0};
  if (s >= a.nseq) return q;
  const int n0 = __ldg(a.cu + s), n1 = __ldg(a.cu + s + 1), len = __ldg(a.lens + s);
  if (n0 >= 0 && n1 >= n0 && n1 <= a.total && n1 - n0 <= a.max_nodes && len >= 0 &&
      static_cast<int64_t>(len) + (n1 - n0) <= a.max_len) {
    q.n0 = n0;
    q.n = n1 - n0;
    q.len = len;
    if (q.n > 0) {
      q.tiles = (len + q.n + kTile - 1) / kTile;
      q.rt = (q.n * a.G + kRows - 1) / kRows;
    }
  } else if (check) {
    report(a.err, KVQ_DEVERR_INDEX);
  }
  return q;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFullMask, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {   // of sums below 2^51
  const uint64_t hi = __reduce_add_sync(kFullMask, static_cast<uint32_t>(x >> 24));
  return (hi << 24) + __reduce_add_sync(kFullMask, static_cast<uint32_t>(x) & 0xffffffu);
}

// Tiles and units of one layer (whole warp).  The call's fit 31 bits.  Offsets that fall and rise
// again can give the same drafts to many sequences, up to eight times (below 2^33) what the bounds
// allow and the line of tiles is numbered for: such a call is given no work.
__device__ __forceinline__ void layer_totals(const TreeArgs& a, bool check, uint32_t& tiles,
                                             uint32_t& units) {
  const int lane = threadIdx.x & 31;
  uint64_t t = 0, u = 0;
  for (int s = lane; s < a.nseq; s += 32) {
    const Seq q = seq_of(a, s, check);
    const uint64_t mine = static_cast<uint64_t>(q.rt) * a.H;
    u += mine;
    t += mine * q.tiles;
  }
  t = warp_sum(t);
  u = warp_sum(u);
  const bool bad = u > a.most_units || t > a.most_tiles;
  if (bad && check) report(a.err, KVQ_DEVERR_INDEX);
  tiles = bad ? 0 : static_cast<uint32_t>(t);
  units = bad ? 0 : static_cast<uint32_t>(u);
}

struct Unit {
  Seq q;
  int l, s, h, r;    // layer, sequence, KV head, row tile
  int tile;          // the tile sought
  uint32_t start;    // the unit's first tile in the line of all tiles
};

// The unit that holds tile `at` of the line of all tiles (BY_TILE), or unit number `at`; whole
// warp, `at` in range.
template <bool BY_TILE>
__device__ __forceinline__ Unit find_unit(const TreeArgs& a, uint32_t at, uint32_t layer_tiles,
                                          uint32_t layer_units) {
  const int lane = threadIdx.x & 31;
  Unit r;
  const uint32_t per = BY_TILE ? layer_tiles : layer_units;
  r.l = a.n_layers == 1 ? 0 : static_cast<int>(at / per);
  const uint32_t x = at - r.l * per;
  uint32_t before = 0, tiles_before = 0;
  for (int base = 0; base < a.nseq; base += 32) {
    const Seq q = seq_of(a, base + lane, false);
    const uint32_t units = static_cast<uint32_t>(q.rt) * a.H, tiles = units * q.tiles;
    const uint32_t mine = BY_TILE ? tiles : units;
    const uint32_t incl = warp_scan(mine), tincl = BY_TILE ? incl : warp_scan(tiles);
    const uint32_t start = before + incl - mine;
    const unsigned hit = __ballot_sync(kFullMask, x >= start && x - start < mine);
    if (hit) {
      const int src = __ffs(hit) - 1;
      r.s = base + src;
      r.q.n0 = __shfl_sync(kFullMask, q.n0, src);
      r.q.n = __shfl_sync(kFullMask, q.n, src);
      r.q.len = __shfl_sync(kFullMask, q.len, src);
      r.q.tiles = __shfl_sync(kFullMask, q.tiles, src);
      r.q.rt = __shfl_sync(kFullMask, q.rt, src);
      const uint32_t rem = x - __shfl_sync(kFullMask, start, src);
      const uint32_t tstart = tiles_before + __shfl_sync(kFullMask, tincl - tiles, src);
      const uint32_t u = BY_TILE ? rem / static_cast<uint32_t>(r.q.tiles) : rem;
      r.tile = BY_TILE ? static_cast<int>(rem - u * r.q.tiles) : 0;
      r.h = static_cast<int>(u / static_cast<uint32_t>(r.q.rt));
      r.r = static_cast<int>(u) - r.h * r.q.rt;
      r.start = r.l * layer_tiles + tstart + u * r.q.tiles;
      return r;
    }
    before += __shfl_sync(kFullMask, incl, 31);
    tiles_before += __shfl_sync(kFullMask, tincl, 31);
  }
  r.s = -1;   // not reached for `at` in range
  return r;
}

// A CTA's way through its share: segments (a unit's consecutive tiles).  Every role walks it.
struct Walk {
  uint32_t at, end, layer_tiles, layer_units;
  bool whole;
};

__device__ __forceinline__ uint32_t share_of(const TreeArgs& a, uint32_t layer_tiles) {
  return (layer_tiles * a.n_layers + a.grid - 1) / a.grid;
}

__device__ __forceinline__ Walk walk_of(const TreeArgs& a, bool check) {
  Walk w;
  layer_totals(a, check, w.layer_tiles, w.layer_units);
  w.whole = a.whole != 0;
  if (w.whole) {
    w.at = blockIdx.x;
    w.end = w.layer_units * a.n_layers;
  } else {
    const uint32_t share = share_of(a, w.layer_tiles), all = w.layer_tiles * a.n_layers;
    w.at = min(all, share * blockIdx.x);   // share * grid < all + grid: no overflow
    w.end = min(all, w.at + share);
  }
  return w;
}

struct Segment {
  Unit u;
  int count;   // tiles, from u.tile on
};

__device__ __forceinline__ bool next_segment(const TreeArgs& a, Walk& w, Segment& g) {
  if (w.at >= w.end) return false;
  if (w.whole) {
    g.u = find_unit<false>(a, w.at, w.layer_tiles, w.layer_units);
    g.count = g.u.q.tiles;
    w.at += a.grid;
  } else {
    g.u = find_unit<true>(a, w.at, w.layer_tiles, w.layer_units);
    g.count = static_cast<int>(min(static_cast<uint32_t>(g.u.q.tiles - g.u.tile), w.end - w.at));
    w.at += g.count;
  }
  return g.u.s >= 0;
}

// The constants of the unpacking, read from shared memory into registers once per warp: spelt out
// in the code, the compiler sets them anew at most uses (an instruction takes one immediate): 6,219
// warp instructions per tile instead of 5,344.
template <int BITS> __device__ __forceinline__ constexpr uint32_t unpack_constant(int i) {
  if (BITS == 8) return i == 0 ? 0x80808080u : i == 1 ? 0x64646464u : kHm1152;
  if (BITS == 6)
    return i == 0 ? 0x03F0003Fu : i == 1 ? 0x64006400u : i == 2 ? 0x2C003C00u : 0xD600E420u;
  return i == 0 ? 0x000F000Fu : i == 1 ? 0x64006400u : i == 2 ? kHm1032 : kHm72;
}

__device__ __forceinline__ uint32_t hadd2u(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// (x & m) | o in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t o) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(m), "r"(o));
  return r;
}

// 16 codes of a row (2 * BITS bytes in shared memory), and their product with the row's scale as
// two 16-byte pieces in the stored order of channels.
template <int BITS> struct Codes;

template <> struct Codes<8> {
  uint4 v;
  __device__ __forceinline__ void load(const unsigned char* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void unpack(uint32_t scale2, const uint32_t k[4], uint32_t o[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = w[i] ^ k[0];   // c + 128
      o[2 * i] = hmul2u(hadd2u(prmt(u, k[1], 0x4140), k[2]), scale2);
      o[2 * i + 1] = hmul2u(hadd2u(prmt(u, k[1], 0x4342), k[2]), scale2);
    }
  }
};

template <> struct Codes<6> {
  uint32_t w0, w1, w2;
  __device__ __forceinline__ void load(const unsigned char* p) {
    const uint32_t* x = reinterpret_cast<const uint32_t*>(p);
    w0 = x[0];
    w1 = x[1];
    w2 = x[2];
  }
  __device__ __forceinline__ void unpack(uint32_t scale2, const uint32_t k[4], uint32_t o[8]) const {
    // per group of 4: low half bytes 0-1 (u0 at bit 0, u1 at 6), high half bytes 1-2 (u2 at 4,
    // u3 at 10): the mask leaves (u0, 16 u2), and after a shift by 6 (u1, 16 u3); 1 and 1/16 and
    // the offsets 1056 and 96 make them codes
    const uint32_t x[4] = {prmt(w0, w0, 0x2110), prmt(w0, w1, 0x5443), prmt(w1, w2, 0x4332),
                           prmt(w2, w2, 0x3221)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = hmul2u(hfma2u(and_or(x[i], k[0], k[1]), k[2], k[3]), scale2);
      o[2 * i + 1] = hmul2u(hfma2u(and_or(x[i] >> 6, k[0], k[1]), k[2], k[3]), scale2);
    }
  }
};

template <> struct Codes<4> {
  uint2 v;
  __device__ __forceinline__ void load(const unsigned char* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void unpack(uint32_t scale2, const uint32_t k[4], uint32_t o[8]) const {
    const uint32_t w[2] = {v.x, v.y}, hi = k[0] << 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t y = w[i] >> 8;
      o[4 * i] = hmul2u(hadd2u(and_or(w[i], k[0], k[1]), k[2]), scale2);
      o[4 * i + 1] = hmul2u(hfma2u(and_or(w[i], hi, k[1]), kH16th, k[3]), scale2);
      o[4 * i + 2] = hmul2u(hadd2u(and_or(y, k[0], k[1]), k[2]), scale2);
      o[4 * i + 3] = hmul2u(hfma2u(and_or(y, hi, k[1]), kH16th, k[3]), scale2);
    }
  }
};

// v_hat of channel d of a packed row in global memory (the rare path of non-finite drafts).
template <int BITS>
__device__ __forceinline__ float value_at(const uint8_t* row, float sc, int d) {
  int c;
  if constexpr (BITS == 8) {
    c = static_cast<int8_t>(row[d]);
  } else if constexpr (BITS == 4) {
    c = static_cast<int>((row[d >> 1] >> ((d & 1) * 4)) & 15) - 8;
  } else {
    const uint8_t* b = row + d / 4 * 3;
    c = static_cast<int>(((b[0] | (b[1] << 8) | (b[2] << 16)) >> (6 * (d & 3))) & 63u) - 32;
  }
  return h2f(f2h(static_cast<float>(c) * sc));
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          const volatile int* gave_up) {
  return __all_sync(kFullMask, tc5::wait(bar, parity, gave_up));
}

template <int BITS>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_kernel(const __grid_constant__ TreeArgs a) {
  using L = Lay<BITS>;
  constexpr int R = L::kRaws;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBars);
  uint64_t *rawfull = bars, *rawempty = bars + 2 * R, *kfull = bars + 4 * R, *kempty = kfull + 2,
           *vfull = kempty + 2, *vempty = vfull + 2, *sfull = vempty + 2, *pready = sfull + 2,
           *odone = pready + 2, *qready = odone + 2, *drain = qready + 1;
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(sm + L::kTail);
  volatile int* flags = reinterpret_cast<volatile int*>(tmem_ptr + 1);   // [0] gave up, [1] V
  volatile int* meta = reinterpret_cast<volatile int*>(sm + L::kTail + 16);
  signed char* parents = reinterpret_cast<signed char*>(sm + L::kParents);
  float* halves = reinterpret_cast<float*>(sm + L::kHalves);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk w = walk_of(a, blockIdx.x == 0 && warp == 0);
  if (!w.whole && warp == kCopyWarp) {
    // the unit that holds this share's last tile, if it starts here and ends behind the share
    Cut cut{0, 0, 0, 0};
    if (w.at < w.end) {
      const Unit u = find_unit<true>(a, w.end - 1, w.layer_tiles, w.layer_units);
      if (u.start >= w.at && u.start + u.q.tiles > w.end)
        cut = Cut{static_cast<int>((u.start + u.q.tiles - 1) / share_of(a, w.layer_tiles)) -
                      static_cast<int>(blockIdx.x) + 1,
                  (u.l * a.total + u.q.n0) * a.Hq + u.h * a.G, u.r * kRows,
                  min(kRows, u.q.n * a.G - u.r * kRows)};
    }
    if (lane == 0) a.cuts[blockIdx.x] = cut;
  }
  if (w.at >= w.end) return;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * R; ++i) { mbar_init(rawfull + i, 1); mbar_init(rawempty + i, kUnpackWarps / 2); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + i, kUnpackWarps / 2);
      mbar_init(kempty + i, 1);
      mbar_init(vfull + i, kUnpackWarps / 2);
      mbar_init(vempty + i, 1);
      mbar_init(sfull + i, 1);
      mbar_init(pready + i, kSoftmaxWarps);
      mbar_init(odone + i, 1);
    }
    mbar_init(qready, kSoftmaxWarps);
    mbar_init(drain, 1);
    tc5::fence_barrier_init();
    flags[0] = 0;
    flags[1] = 0;
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint32_t*>(sm + L::kConst)[i] = unpack_constant<BITS>(i);
  }
  if (warp == kMmaWarp) tc5::tmem_alloc(tmem_ptr, kCols);
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = *tmem_ptr;
  Segment g;
  int it = 0;        // tiles done by this CTA
  bool ok = true;

  if (warp == kCopyWarp || warp == kCopyWarp + 1) {
    // ------------------------------------------------------------------------- copies
    // One warp for K and one for V, each with a ring of its own: the keys are used about two tiles
    // before the values, and would wait for them in a common one.  Eight tiles at a time: lane i
    // looks up the page of 16-token group i, then all lanes read those tiles' scales (two tokens
    // each; scales of tokens that are not there become 0, so that their rows unpack to zeros).
    // The next eight, of the next segment too, are looked up while the tiles of the present ones
    // go out, one bulk copy of codes per group.
    const int kind = warp - kCopyWarp;
    uint64_t *full = rawfull + kind * R, *empty = rawempty + kind * R;
    unsigned char* ring = sm + L::kRawAt + kind * R * L::kRaw;
    struct Batch {
      int first, total, n, l, h, s;   // first token, end of the sequence, tiles, unit
    };
    int b = 0;
    bool more = next_segment(a, w, g);
    auto next_batch = [&]() {
      Batch x{0, 0, 0, 0, 0, 0};
      if (more) {
        x = Batch{(g.u.tile + b) * kTile, g.u.q.len + g.u.q.n, min(8, g.count - b), g.u.l, g.u.h,
                  g.u.s};
        b += 8;
        if (b >= g.count) {
          b = 0;
          more = next_segment(a, w, g);
        }
      }
      return x;
    };
    auto page_of = [&](const Batch& x) {   // of group `lane`
      const int tg = x.first + lane * 16;
      if ((lane >> 2) >= x.n || tg >= x.total) return -2;
      const int lp = tg / a.ps;
      return lp < a.max_pages ? __ldg(a.pt + static_cast<int64_t>(x.s) * a.max_pages + lp) : -1;
    };
    // Row numbers fit 32 bits: 2^32 - 1 rows of 128 bytes are more than the device's memory.
    auto row_of = [&](const Batch& x, int page) -> uint32_t {
      if (page == -2) return kNoRow;
      if (page < 0 || page >= a.L[x.l].k_pages || page >= a.L[x.l].v_pages) {
        if (kind == 0) report(a.err, KVQ_DEVERR_PAGE_RANGE);
        return kNoRow;
      }
      const int tg = x.first + lane * 16;
      return (static_cast<uint32_t>(page) * a.H + x.h) * a.ps + tg % a.ps;
    };
    auto load_scales = [&](const Batch& x, uint32_t rows, uint32_t v[8]) {
      const uint16_t* scales = kind ? a.L[x.l].vs : a.L[x.l].ks;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t r = __shfl_sync(kFullMask, rows, j * 4 + (lane >> 3));
        v[j] = r != kNoRow ? ld_nc_u32(scales + r + (lane & 7) * 2) : 0u;
      }
    };
    Batch cur = next_batch();
    uint32_t rows = row_of(cur, page_of(cur));
    uint32_t x[8], nx[8];
    load_scales(cur, rows, x);
    while (ok && cur.n > 0) {
      const uint8_t* codes = kind ? a.L[cur.l].vc : a.L[cur.l].kc;
      Batch nxt = next_batch();
      const int page = page_of(nxt);
      uint32_t next_rows = kNoRow;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j == 4 || (j == 0 && cur.n <= 4)) {
          next_rows = row_of(nxt, page);
          load_scales(nxt, next_rows, nx);
        }
        if (!ok || j >= cur.n) continue;
        const int st = it % R;
        if (it >= R) ok = warp_wait(empty + st, (it / R + 1) & 1, flags);
        if (!ok) continue;
        unsigned char* dst = ring + st * L::kRaw;
        const int left = cur.total - (cur.first + j * kTile + lane * 2);   // tokens still there
        if (left < 2) x[j] &= left < 1 ? 0u : 0x0000ffffu;
        *reinterpret_cast<uint32_t*>(dst + kTile * L::kPd + lane * 4) = x[j];
        uint32_t r[4];
        unsigned have = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[i] = __shfl_sync(kFullMask, rows, j * 4 + i);
          have |= (r[i] != kNoRow ? 1u : 0u) << i;
        }
        __syncwarp();
        if (tc5::elect_one()) {   // copies by several lanes at once take 100 cycles each
          if (kind == 0) meta[it % kMeta] = static_cast<int>(have);
          mbar_expect_tx(full + st, __popc(have) * (16 * L::kPd));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (r[i] != kNoRow)
              bulk_g2s(dst + i * 16 * L::kPd, codes + static_cast<uint64_t>(r[i]) * L::kPd,
                       16 * L::kPd, full + st);
        }
        __syncwarp();
        ++it;
      }
      cur = nxt;
      rows = next_rows;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = nx[j];
    }
    // Whichever role gives up, and whether this one has by then issued everything or not: no copy is
    // in flight when the block ends.
    for (int i = max(0, it - R); i < it; ++i) mbar_wait_bounded(full + i % R, (i / R) & 1);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- products (one thread)
    const uint32_t base = smem_u32(sm);
    const uint64_t dk = tc5::desc_base(16), dv = tc5::desc_base(kTile * 128);
    constexpr uint32_t id_s = tc5::idesc(false, kTile, false), id_o = tc5::idesc(false, kD, true);
    int seg = 0;
    while (ok && next_segment(a, w, g)) {
      if (tc5::elect_one()) {
        auto product_s = [&](int i) {
          ok = ok && tc5::wait(kfull + (i & 1), (i >> 1) & 1, flags);
          // These scores go over the weights of tile i - 2, once their product is done: only products
          // of one shape and accumulator are promised to run in the order of their issue.  (The first
          // two tiles of a segment follow on qready, before which all products were done.)
          if (i >= it + 2) ok = ok && tc5::wait(odone + (i & 1), (i - 2) >> 1 & 1, flags);
          if (!ok) return;
          tc5::fence_after();
          const uint32_t kb = base + L::kK + (i & 1) * kStage;
#pragma unroll
          for (int k = 0; k < kD / 16; ++k)
            tc5::mma_ts(tmem + kColS + (i & 1) * kTile, tmem + kColQ + k * 8,
                        tc5::desc_at(dk, kb + (k / 4) * kTile * 128 + (k % 4) * 32), id_s, k > 0);
          tc5::commit(kempty + (i & 1));
          tc5::commit(sfull + (i & 1));
        };
        auto product_o = [&](int i, bool first) {
          ok = ok && tc5::wait(vfull + (i & 1), (i >> 1) & 1, flags);
          ok = ok && tc5::wait(pready + (i & 1), (i >> 1) & 1, flags);
          if (!ok) return;
          tc5::fence_after();
          const uint32_t vb = base + L::kV + (i & 1) * kStage;
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            tc5::mma_ts(tmem, tmem + kColS + (i & 1) * kTile + k * 8,
                        tc5::desc_at(dv, vb + k * 2048), id_o, !first || k > 0);
          tc5::commit(vempty + (i & 1));
          tc5::commit(odone + (i & 1));
        };
        ok = tc5::wait(qready, seg & 1, flags);
        tc5::fence_after();
        if (ok) product_s(it);
        for (int j = 0; ok && j < g.count; ++j) {
          if (j + 1 < g.count) product_s(it + j + 1);
          if (ok) product_o(it + j, j == 0);
        }
      }
      ok = __all_sync(kFullMask, ok);
      it += g.count;
      ++seg;
    }
    if (!ok) flags[0] = 1;
    if (tc5::elect_one()) {   // what was issued ends before the memory is given back, as above
      tc5::commit(drain);
      mbar_wait_bounded(drain, 0);
    }
  } else if (warp >= kUnpackWarp0) {
    // ------------------------------------------------------------------------------- unpack
    // Half the warps for K and half for V, so that neither waits for the other's products.  A warp's
    // step takes two rows: lanes 8q .. 8q+7 hold panel q (64 channels) of both, four 16-channel
    // units each, which spreads a quarter-warp's 16-byte stores over all banks.  A tile's codes
    // are all read before the first is stored: reads and stores would otherwise alternate, each
    // waiting for the other.
    constexpr int W = kUnpackWarps / 2;
    const int kv = (warp - kUnpackWarp0) / W, uw = (warp - kUnpackWarp0) % W;
    const int q = lane >> 3, rr = (lane >> 2) & 1, u = lane & 3;
    const int src = (q * 4 + u) * 2 * BITS;
    uint32_t k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      k[i] = reinterpret_cast<const volatile uint32_t*>(sm + L::kConst)[i];
    uint64_t *full = kv ? vfull : kfull, *empty = kv ? vempty : kempty;
    uint64_t *rfull = rawfull + kv * R, *rempty = rawempty + kv * R;
    const unsigned char* ring = sm + L::kRawAt + kv * R * L::kRaw;
    unsigned char* stages = sm + (kv ? L::kV : L::kK) + q * kTile * 128;
    constexpr int S = kTile / 2 / W;   // steps
    while (ok && next_segment(a, w, g)) {
      const int len = g.u.q.len;
      for (int j = 0; j < g.count; ++j, ++it) {
        const int st = it % R, t0 = (g.u.tile + j) * kTile;
        ok = warp_wait(rfull + st, (it / R) & 1, flags);
        if (!ok) break;
        const unsigned char* raw = ring + st * L::kRaw;
        const uint16_t* sc = reinterpret_cast<const uint16_t*>(raw + kTile * L::kPd);
        Codes<BITS> c[S];
        uint32_t s1[S];
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int row = (i * W + uw) * 2 + rr;
          c[i].load(raw + row * L::kPd + src);
          s1[i] = sc[row];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(rempty + st);   // all read: the next copies may come
        if (it >= 2) ok = warp_wait(empty + (it & 1), (it / 2 + 1) & 1, flags);
        if (!ok) break;
        unsigned char* dst = stages + (it & 1) * kStage;
        auto store = [&](int row, const uint32_t o[8]) {
          unsigned char* p = dst + row * 128;
          const int at = ((2 * u) ^ (row & 7)) * 16;
          *reinterpret_cast<uint4*>(p + at) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(p + (at ^ 16)) = make_uint4(o[4], o[5], o[6], o[7]);
        };
        bool found = false;
        if (!(kv && t0 + kTile > len)) {   // no branch inside: the steps overlap
#pragma unroll
          for (int i = 0; i < S; ++i) {
            uint32_t o[8];
            c[i].unpack(s1[i] | (s1[i] << 16), k, o);
            store((i * W + uw) * 2 + rr, o);
          }
        } else {   // drafts among the values: 0 * inf must not reach the rows that do not see them
#pragma unroll
          for (int i = 0; i < S; ++i) {
            const int row = (i * W + uw) * 2 + rr;
            uint32_t o[8];
            c[i].unpack(s1[i] | (s1[i] << 16), k, o);
            if (t0 + row >= len) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if (nonfinite2(o[e])) found = true;
                if ((o[e] & 0x7c00u) == 0x7c00u) o[e] &= 0xffff0000u;
                if ((o[e] & 0x7c000000u) == 0x7c000000u) o[e] &= 0x0000ffffu;
              }
            }
            store(row, o);
          }
        }
        if (found) flags[1] = 1;
        tc5::fence_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + (it & 1));
      }
    }
  } else {
    // ------------------------------------- softmax: two threads per row, half the columns each
    const int quad = warp & 3, half = warp >> 2, r = quad * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad) << 21);
    // the other half's value, through shared memory: the row's two warps meet after the write and
    // after the read
    auto other = [&](float v) {
      halves[half * kRows + r] = v;
      tc5::meet(quad);
      v = halves[(half ^ 1) * kRows + r];
      tc5::meet(quad);
      return v;
    };
    auto node_of_row = [&]() { return (g.u.r * kRows + r) / a.G; };
    auto has_drafts = [&]() { return (g.u.tile + g.count) * kTile > g.u.q.len; };
    int met = 0;   // where this warp gave up: its exchanges of the present segment so far
    while (ok && next_segment(a, w, g)) {
      const Seq& q = g.u.q;
      const int node = node_of_row();
      const bool live = node < q.n;
      const bool idle = !__any_sync(kFullMask, live);
      const int64_t row = (static_cast<int64_t>(g.u.l) * a.total + q.n0 + node) * a.Hq +
                          g.u.h * a.G + (g.u.r * kRows + r - node * a.G);
      // Q of this row into TMEM, channels in the stored order
#pragma unroll 1
      for (int b = half * 2; b < half * 2 + 2; ++b) {
        uint32_t x[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live) v = ld_nc_v4(a.q + row * kD + b * 64 + i * 8);
          if constexpr (BITS == 8) {
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
          } else if constexpr (BITS == 6) {
            x[4 * i] = prmt(v.x, v.y, 0x5410);
            x[4 * i + 1] = prmt(v.x, v.y, 0x7632);
            x[4 * i + 2] = prmt(v.z, v.w, 0x5410);
            x[4 * i + 3] = prmt(v.z, v.w, 0x7632);
          } else {
            x[4 * i] = prmt(v.x, v.z, 0x5410);
            x[4 * i + 1] = prmt(v.x, v.z, 0x7632);
            x[4 * i + 2] = prmt(v.y, v.w, 0x5410);
            x[4 * i + 3] = prmt(v.y, v.w, 0x7632);
          }
        }
        tc5::st32(lanes + kColQ + b * 32, x);
      }
      tc5::wait_st();
      tc5::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);
      // the ancestors, if drafts are among this segment's tokens
      uint64_t seen = 0;
      const bool drafts = has_drafts();
      if (drafts) {
        asm volatile("bar.sync 1, 256;" ::: "memory");   // the previous unit's are no longer read
        if (half == 0 && r < q.n) {
          int p = __ldg(a.parents + q.n0 + r);
          if (p < -1 || p >= r) {
            report(a.err, KVQ_DEVERR_INDEX);
            p = -1;
          }
          parents[r] = static_cast<signed char>(p);
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (live)
          for (int i = node; i >= 0; i = parents[i]) seen |= 1ull << i;
      }
      float m = kNegInf, l = 0.f;
      for (int j = 0; j < g.count; ++j, ++it) {
        ok = warp_wait(sfull + (it & 1), (it >> 1) & 1, flags);
        if (!ok) {
          met = idle ? 0 : j;
          break;
        }
        tc5::fence_after();
        if (idle) {   // no row of this warp is used: its weights may be anything
          if (lane == 0) mbar_arrive(pready + (it & 1));
          continue;
        }
        const uint32_t sb = lanes + kColS + (it & 1) * kTile;
        const int t0 = (g.u.tile + j) * kTile;
        uint32_t s[32];
        tc5::ld32(sb + half * 32, s);
        const unsigned have = static_cast<unsigned>(meta[it % kMeta]);
        tc5::wait_ld32(s);
        if (t0 + kTile > q.len || have != 15u) {
          const int d0 = t0 - q.len;   // node number of the tile's first token
          uint64_t v = d0 >= 0 ? (d0 < 64 ? seen >> d0 : 0)
                     : d0 > -64 ? (seen << -d0) | ((1ull << -d0) - 1) : ~0ull;
#pragma unroll
          for (int gi = 0; gi < 4; ++gi)
            if (!(have >> gi & 1)) v &= ~(0xffffull << (16 * gi));
          const uint32_t vis = static_cast<uint32_t>(v >> (32 * half));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(vis >> i & 1)) s[i] = 0xff800000u;
        }
        float x = tc5::row_max<32>(s) * a.c;
        x = fmaxf(x, other(x));
        if (j == 0) {
          m = x;
        } else {
          const bool up = x > m + tc5::kSlack;   // the same in both halves
          if (__any_sync(kFullMask, up)) {
            const float f = up ? ex2_fast(m - x) : 1.f;
            if (up) m = x;
            l *= f;
            ok = warp_wait(odone + ((it - 1) & 1), (it - 1) >> 1 & 1, flags);
            if (!ok) {
              met = j + 1;
              break;
            }
            tc5::fence_after();
#pragma unroll 1
            for (int b = half * 4; b < half * 4 + 4; ++b) {
              uint32_t o[32];
              tc5::ld32(lanes + b * 32, o);
              tc5::wait_ld32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tc5::st32(lanes + b * 32, o);
            }
            tc5::wait_st();
          }
        }
        const float mo = m == kNegInf ? 0.f : m - tc5::kOff;
        uint64_t sum[2] = {0, 0};
        // both halves' scores have been read (the exchange above), so the weights may go over them
        tc5::weights32<false>(s, a.c, mo, sb + half * 16, sum);
        l += tc5::sum_of(sum);
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pready + (it & 1));
      }
      if (!ok) break;
      ok = warp_wait(odone + ((it - 1) & 1), (it - 1) >> 1 & 1, flags);
      if (!ok) {
        met = idle ? 0 : g.count;
        break;
      }
      tc5::fence_after();
      l += other(l);
      const bool whole = g.count == q.tiles;
      const bool fix = drafts && flags[1] != 0;
      if (fix) {   // apart from the rows' way out, which short calls run once, from cold
#pragma unroll 1
        for (int b = half * 4; b < half * 4 + 4; ++b) {
          uint32_t o[32];
          tc5::ld32(lanes + b * 32, o);
          tc5::wait_ld32(o);
          const TreePools& P = a.L[g.u.l];
          const int lo = max(0, g.u.tile * kTile - q.len);
          const int hi = min(q.n, (g.u.tile + g.count) * kTile - q.len);
          for (int d = lo; d < hi; ++d) {
            if (!(seen >> d & 1)) continue;
            const int64_t at =   // (a page that only one of K and V has is not attended)
                locate_row(a.pt, a.max_pages, a.ps, a.H, min(P.k_pages, P.v_pages), g.u.s,
                           static_cast<int64_t>(q.len) + d, g.u.h, nullptr);
            if (at < 0) continue;
            const float vs = h2f(P.vs[at]);
#pragma unroll
            for (int i = 0; i < 32; ++i) {   // o[i]: the channel stored at place i
              const float v = value_at<BITS>(P.vc + at * L::kPd, vs, b * 32 + channel<BITS>(i));
              if (!isfinite(v)) o[i] = __float_as_uint(__uint_as_float(o[i]) + v);
            }
          }
          __syncwarp();
          tc5::st32(lanes + b * 32, o);
        }
        tc5::wait_st();
      }
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      // a cut unit at the head of the share is its first record, one at the tail its second
      float* part = a.ws + (static_cast<int64_t>(blockIdx.x) * 2 + (g.u.tile > 0 ? 0 : 1)) * kRec;
#pragma unroll 1
      for (int b = half * 4; b < half * 4 + 4; ++b) {
        uint32_t o[32];
        __syncwarp();
        tc5::ld32(lanes + b * 32, o);
        tc5::wait_ld32(o);
        if (!live) continue;
        uint32_t x[32];   // in natural order
#pragma unroll
        for (int i = 0; i < 32; ++i)
          x[i] = __float_as_uint(__uint_as_float(o[(i & ~7) | place<BITS>(i & 7)]) * inv);
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * kD + b * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = pack_h2(__uint_as_float(x[i * 8 + e * 2]), __uint_as_float(x[i * 8 + e * 2 + 1]));
            dst[i] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(part) + b * 8 * kRows + r;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i * kRows] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
      }
      if (live && !whole && half == 0) {
        part[kD * kRows + r] = m;
        part[(kD + 1) * kRows + r] = l;
      }
      tc5::fence_before();
    }
    if (!ok) {
      // Another warp may have seen the phase complete whose wait ran out here.  It goes on to the
      // barriers of the walk, which have no limit of their own, until one of its own waits fails:
      // so a warp that gave up goes on meeting the others there, to the walk's end (every warp
      // walks the same segments), and waits for nothing else.
      flags[0] = 1;
      auto exchanges = [&]() {   // of a segment: one per tile that has rows of this warp, and l's
        return (__any_sync(kFullMask, node_of_row() < g.u.q.n) ? g.count : 0) + 1;
      };
      int owed = exchanges() - met;
      for (;;) {
        for (; owed > 0; --owed) other(0.f);
        if (!next_segment(a, w, g)) break;
        if (has_drafts()) {
          asm volatile("bar.sync 1, 256;" ::: "memory");
          asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        owed = exchanges();
      }
    }
  }
  if (!ok) flags[0] = 1;
  __syncwarp();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc5::fence_after();
    tc5::tmem_dealloc(tmem, kCols);
  }
  if (threadIdx.x == 0 && flags[0]) report(a.err, KVQ_DEVERR_TIMEOUT);
}

// Joins the records of a cut unit.  A block takes kJoinCols channels of all rows: thread = (row,
// slice of the records), so that every read is along the rows as the records were written.
constexpr int kJoinCols = 8, kJoinSlices = 4;

__global__ void __launch_bounds__(kRows * kJoinSlices)
tree_join_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ float part_sm[kJoinSlices][kJoinCols + 2][kRows];
  // the block's unit: the blockIdx.x-th CTA that left a cut one
  __shared__ int counts[kRows * kJoinSlices / 32], mine;
  const bool has = threadIdx.x < a.grid && a.cuts[threadIdx.x].n > 0;
  const unsigned votes = __ballot_sync(kFullMask, has);
  if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = __popc(votes);
  if (threadIdx.x == 0) mine = -1;
  __syncthreads();
  int rank = __popc(votes & ((1u << (threadIdx.x & 31)) - 1));
  for (int i = 0; i < static_cast<int>(threadIdx.x >> 5); ++i) rank += counts[i];
  if (has && rank == static_cast<int>(blockIdx.x)) mine = threadIdx.x;
  __syncthreads();
  if (mine < 0) return;
  const Cut cut = a.cuts[mine];
  const int c0 = mine, c1 = c0 + cut.n - 1;
  const int r = threadIdx.x % kRows, slice = threadIdx.x / kRows, col = blockIdx.y * kJoinCols;
  const int node = (cut.first + r) / a.G;
  const bool live = r < cut.rows;
  float M = kNegInf, l = 0.f, O[kJoinCols];
#pragma unroll
  for (int e = 0; e < kJoinCols; ++e) O[e] = 0.f;
  if (live) {
#pragma unroll 4
    for (int c = c0 + slice; c <= c1; c += kJoinSlices) {
      // its first record is the tail one of c0, the others the head ones
      const float* p = a.ws + (static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * kRec;
      const float mi = p[kD * kRows + r], li = p[(kD + 1) * kRows + r];
      float4 o4[kJoinCols / 4];
#pragma unroll
      for (int e = 0; e < kJoinCols / 4; ++e)
        o4[e] = reinterpret_cast<const float4*>(p)[(col / 4 + e) * kRows + r];
      const float* o = reinterpret_cast<const float*>(o4);
      const float Mn = fmaxf(M, mi);
      const float f = M == kNegInf ? 0.f : ex2_fast(M - Mn), fi = mi == kNegInf ? 0.f : ex2_fast(mi - Mn);
      l = l * f + li * fi;
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e) O[e] = O[e] * f + o[e] * fi;
      M = Mn;
    }
  }
#pragma unroll
  for (int e = 0; e < kJoinCols; ++e) part_sm[slice][e][r] = O[e];
  part_sm[slice][kJoinCols][r] = M;
  part_sm[slice][kJoinCols + 1][r] = l;
  __syncthreads();
  if (slice > 0 || !live) return;
  float Mx = M;
#pragma unroll
  for (int i = 1; i < kJoinSlices; ++i) Mx = fmaxf(Mx, part_sm[i][kJoinCols][r]);
  l = 0.f;
#pragma unroll
  for (int e = 0; e < kJoinCols; ++e) O[e] = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinSlices; ++i) {
    const float mi = part_sm[i][kJoinCols][r], f = mi == kNegInf ? 0.f : ex2_fast(mi - Mx);
    l = fmaf(part_sm[i][kJoinCols + 1][r], f, l);
#pragma unroll
    for (int e = 0; e < kJoinCols; ++e) O[e] = fmaf(part_sm[i][e][r], f, O[e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t row = static_cast<int64_t>(cut.row0) + node * a.Hq + (cut.first + r - node * a.G);
  uint32_t y[kJoinCols / 2];
#pragma unroll
  for (int e = 0; e < kJoinCols; e += 2) y[e / 2] = pack_h2(O[e] * inv, O[e + 1] * inv);
#pragma unroll
  for (int e = 0; e < kJoinCols / 8; ++e)
    *reinterpret_cast<uint4*>(a.out + row * kD + col + e * 8) =
        make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
}

// How a call is cut; the units are an upper bound (the lengths are on the device).
struct Plan {
  int grid;
  bool whole;
  int64_t units;
};

Plan plan_for(int n_layers, int nseq, int total_nodes, int H, int Hq, int max_nodes, int max_len) {
  Plan p;
  const int G = Hq / H;
  const int64_t per = (max_nodes * G + kRows - 1) / kRows;
  const int64_t a = static_cast<int64_t>(nseq) * per;
  const int64_t b = static_cast<int64_t>(total_nodes) * G / kRows + nseq;
  p.units = (a < b ? a : b) * H * n_layers;
  const int64_t tiles = (static_cast<int64_t>(max_len) + kTile - 1) / kTile;
  p.whole = tiles <= kShortTiles;
  int sms = sm_count() > 0 ? sm_count() : 152;
  if (sms > kRows * kJoinSlices) sms = kRows * kJoinSlices;   // the join's block looks at all CTAs
  const int64_t work = p.whole ? p.units : p.units * tiles;
  p.grid = static_cast<int>(work < sms ? (work < 1 ? 1 : work) : sms);
  return p;
}

template <int BITS>
cudaError_t launch(const TreeArgs& a, const Plan& p, cudaStream_t cs) {
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<BITS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Lay<BITS>::kTotal);
  if (e != cudaSuccess) return e;
  tree_attn_kernel<BITS><<<p.grid, kThreads, Lay<BITS>::kTotal, cs>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.whole) return e;
  const unsigned cuts = static_cast<unsigned>(p.units < p.grid ? p.units : p.grid);
  tree_join_kernel<<<dim3(cuts, kD / kJoinCols), kRows * kJoinSlices, 0, cs>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace kvq

extern "C" size_t kvq_tree_attn_workspace(int n_layers, int nseq, int total_nodes,
                                          int num_kv_heads, int num_q_heads, int head_dim,
                                          int max_nodes, int max_seq_len) {
  (void)head_dim;
  if (n_layers < 1 || nseq < 1 || total_nodes < 0 || num_kv_heads < 1 ||
      num_q_heads < num_kv_heads || num_q_heads % num_kv_heads ||
      num_q_heads / num_kv_heads > kvq::kRows || max_nodes < 1 || max_nodes > KVQ_MAX_NODES ||
      max_seq_len < 0)
    return 0;
  const kvq::Plan p = kvq::plan_for(n_layers, nseq, total_nodes, num_kv_heads, num_q_heads,
                                    max_nodes, max_seq_len);
  if (p.whole) return 16;
  return static_cast<size_t>(p.grid) * (2 * kvq::kRec * sizeof(float) + sizeof(kvq::Cut));
}

extern "C" kvq_status kvq_tree_attn(const kvq_pool* k_pools, const kvq_pool* v_pools, int n_layers,
                                    const uint16_t* q, int num_q_heads, const int32_t* page_table,
                                    int max_pages, const int32_t* seq_lens,
                                    const int32_t* cu_nodes, const int32_t* parents, int nseq,
                                    int total_nodes, int max_nodes, int max_seq_len,
                                    float softmax_scale, uint16_t* out, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_err,
                                    kvq_stream_t stream) {
  using namespace kvq;
  const char* fn = "kvq_tree_attn";
  if (n_layers < 1 || n_layers > KVQ_MAX_TENSORS)
    return fail(KVQ_ERR_RANGE, "%s: n_layers %d not in [1, %d]", fn, n_layers, KVQ_MAX_TENSORS);
  kvq_status st = check_pools_uniform(k_pools, n_layers, fn);
  if (st != KVQ_OK) return st;
  st = check_pools_uniform(v_pools, n_layers, fn);
  if (st != KVQ_OK) return st;
  const kvq_pool& k0 = k_pools[0];
  const kvq_pool& v0 = v_pools[0];
  if (v0.bits != k0.bits || v0.num_heads != k0.num_heads || v0.head_dim != k0.head_dim ||
      v0.page_size != k0.page_size)
    return fail(KVQ_ERR_SHAPE, "%s: K and V pools differ in shape", fn);
  if (k0.head_dim != kD)
    return fail(KVQ_ERR_SHAPE, "%s: head_dim %d unsupported (256 only)", fn, k0.head_dim);
  if (k0.page_size % 16)
    return fail(KVQ_ERR_SHAPE, "%s: page_size %d must be a multiple of 16", fn, k0.page_size);
  const int H = k0.num_heads;
  if (num_q_heads < H || num_q_heads % H || num_q_heads / H > 16)
    return fail(KVQ_ERR_SHAPE, "%s: num_q_heads %d must be a multiple of %d, at most 16 per KV "
                "head", fn, num_q_heads, H);
  if (nseq < 0 || total_nodes < 0 || max_pages < 1 || max_seq_len < 0)
    return fail(KVQ_ERR_RANGE, "%s: bad nseq/total_nodes/max_pages/max_seq_len", fn);
  if (max_nodes < 1 || max_nodes > KVQ_MAX_NODES)
    return fail(KVQ_ERR_RANGE, "%s: max_nodes %d not in [1, %d]", fn, max_nodes, KVQ_MAX_NODES);
  if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_pages) * k0.page_size)
    return fail(KVQ_ERR_RANGE, "%s: max_seq_len exceeds max_pages * page_size", fn);
  if (max_seq_len > INT32_MAX - kTile)
    return fail(KVQ_ERR_RANGE, "%s: max_seq_len %d > 2^31 - 65", fn, max_seq_len);
  const float c = softmax_scale * 1.4426950408889634f;   // of scores in powers of 2
  if (!std::isfinite(c) || softmax_scale <= 0)
    return fail(KVQ_ERR_RANGE, "%s: softmax_scale is not a finite value > 0 (2.3e38 at most)", fn);
  if (nseq == 0 || total_nodes == 0) return ok();
  if (!q || !page_table || !seq_lens || !cu_nodes || !parents || !out || !workspace)
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return fail(KVQ_ERR_ALIGN, "%s: q/out/workspace must be 16-byte aligned", fn);
  const size_t need = kvq_tree_attn_workspace(n_layers, nseq, total_nodes, H, num_q_heads, kD,
                                              max_nodes, max_seq_len);
  if (workspace_bytes < need)
    return fail(KVQ_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, workspace_bytes, need);
  const Plan p = plan_for(n_layers, nseq, total_nodes, H, num_q_heads, max_nodes, max_seq_len);
  const int64_t seq_tiles = (static_cast<int64_t>(max_seq_len) + kTile - 1) / kTile;
  if (p.units > INT32_MAX / 2 || p.units * (seq_tiles < 1 ? 1 : seq_tiles) > INT32_MAX / 2)
    return fail(KVQ_ERR_RANGE, "%s: %lld units (layers x KV heads x tiles of 128 rows) of up to "
                "%lld tiles of 64 tokens exceed 2^30 tiles", fn, static_cast<long long>(p.units),
                static_cast<long long>(seq_tiles));
  TreeArgs a;
  for (int i = 0; i < KVQ_MAX_TENSORS; ++i)
    a.L[i] = i < n_layers ? TreePools{k_pools[i].codes, k_pools[i].scales, v_pools[i].codes,
                                      v_pools[i].scales, k_pools[i].num_pages,
                                      v_pools[i].num_pages}
                          : TreePools{nullptr, nullptr, nullptr, nullptr, 0, 0};
  a.q = q; a.out = out; a.ws = static_cast<float*>(workspace); a.pt = page_table;
  a.lens = seq_lens; a.cu = cu_nodes; a.parents = parents; a.err = dev_err;
  a.n_layers = n_layers; a.nseq = nseq; a.total = total_nodes; a.H = H; a.Hq = num_q_heads;
  a.G = num_q_heads / H; a.ps = k0.page_size; a.max_pages = max_pages; a.max_nodes = max_nodes;
  a.max_len = max_seq_len; a.grid = p.grid; a.whole = p.whole ? 1 : 0;
  a.most_units = static_cast<uint32_t>(p.units / n_layers);
  a.most_tiles = static_cast<uint32_t>(p.units / n_layers * seq_tiles);
  a.cuts = reinterpret_cast<Cut*>(a.ws + static_cast<int64_t>(p.grid) * 2 * kRec);
  a.c = c;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = k0.bits == 8 ? launch<8>(a, p, cs)
                        : k0.bits == 6 ? launch<6>(a, p, cs) : launch<4>(a, p, cs);
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}
