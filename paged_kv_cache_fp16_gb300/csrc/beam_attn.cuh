// Decode attention over a cache held in 4 bits, for heads of 64, 128 and 256 channels, of sequences
// that may come in groups sharing a prefix (beams): the prefix is read once for the whole group.
//
//   out[s][j] = sum_t softmax(scale q[s][j] . k_t)_t v_t,   k_t = code_t * scale_t,   h = j / (Hq / H)
//
// Work: units are (shared prefix of a group, for all heads of all its sequences, or the own tokens of a
// sequence) x KV head x layer, cut into granules of 128 tokens.  The granules of all prefixes in one line,
// and those of all own tokens in another, are dealt out to the resident blocks in contiguous shares of
// equal cost, so lengths of any kind load the GPU evenly; every block finds its share from the lengths by
// itself.  Where a unit has more columns than a block, neighbouring blocks take the same tokens at the same
// time.  A block's four warps take a granule's steps of 32 tokens, each with a ring of asynchronous copies
// of its own.  Where the call's bound says that no sequence has more own tokens than a granule, a unit of them
// is one warp's: it costs more to start and end than to attend (63 groups of 8 beams with up to 107 own
// tokens: 89 to 63 us).  Tokens are the products' M:
//   S^T[16 x 8 NT] = K[16 x D] Q^T,  online softmax per column,  O^T[D x 8 NT] += V^T[D x 16] P^T
// What bounds it is the unpacking of the codes, so that is spent once per NT column tiles, and little:
//   - a 4-bit code u = c + 8 in bits 0-3 of a 16-bit lane, with fp16's 1024 set above it, is 1024 + u,
//     from which one packed addition of two lanes leaves c; in bits 4-7 it is 1024 + 16 u.  V's high
//     nibbles become c by a packed fma; K's are used as they are, with 1/16 in the queries, and
//     72 sum_d q_d over those channels is where the score's sum starts (the others' 1032 would cost it
//     bits).  Fp16 subnormals need no 1024, but a product of theirs loses bits in the tensor cores:
//     outputs were off by 2^-13 of 8 codes.
//   - ldmatrix hands out K's words as a product's A operand, and transposed V's as its pairs of tokens,
//     so that no bytes have to be brought together.  Copies of 16 bytes go to places that make it free
//     of bank conflicts.
//   - keys' scales multiply the scores in float32, so no product is rounded: the cache stands for
//     code * scale exactly.  V's scales multiply the weights, and the products are rounded to fp16; the
//     exponentials' reference keeps the largest of them between some 2^10 and 2^15, so that all but those
//     below 2^-24 of it keep fp16's 11 bits, whatever the scales are.
// Queries are put into fp16 with one power of two per row (that of the largest entry), so bf16 queries
// lose nothing that a float32 sum of the row would keep.
//
// A block joins its warps per unit and writes one record (O, reference, sum per column) to the workspace, or,
// where it had the whole of a row, the result; a second kernel joins the records of a sequence's prefix
// and own tokens in a fixed order.  Record unit + place of the block in its line is nobody else's: from
// one piece of the line to the next one of the two rises.
#pragma once

#include <cstdint>
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_math.cuh"
#include "kvq_warp.cuh"

namespace kvq {
namespace beam {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;
constexpr int kStep = 2 * kTile;             // tokens of a warp's step
constexpr int kGranule = kWarps * kStep;     // tokens of a block's step
constexpr int kMostBlocks = 152 * 3;
// Cost of starting and ending a unit in a block; a granule's is 2 (unpacking) and 1 per column tile.  (Fitted
// at 128 channels: 5 gave equal times, 12 gave 47 instead of 45 us for 64 sequences.)
constexpr int kUnitCost = 8;
// Where own tokens are one granule at most, a unit is a warp's, four of a sequence a block's at once.
// (With fewer units than blocks a block's four warps end one sooner: 4 beams of 300 tokens 14.4 against 17 us.)
constexpr int kSoloCost = 5, kSoloUnits = 400;
#define kNegInf (-__int_as_float(0x7f800000))
#define kMaxFloor (-3.402823466e38f)   // floor of the exponentials' reference; one still at it saw no token

struct LayerPools {
  const uint8_t* kc;
  const uint16_t* ks;
  const uint8_t* vc;
  const uint16_t* vs;
  int64_t pages;
};

// A line of granules: `who` prefixes or sequences, `rep` = layers x heads units of each.
struct Line {
  int n, rep, blocks;                  // column blocks of a unit
  int weight, most;                    // cost of a granule; blocks of one column block in the line at most
  int solo;                            // units (of one granule) are a warp's
  int64_t units, first_unit, first_rec;
};

struct BeamArgs {
  LayerPools L[KVQ_MAX_TENSORS];
  const uint16_t* q;
  uint16_t* out;
  int64_t* head;                       // [0]: cost of a block's share; then each unit's place in its line
  float* ws;                           // records
  const int32_t *pt, *lens, *shared;
  int32_t* err;
  int nseq, beams, groups, H, G, Hq, ps, max_pages, n_layers;
  Line line[2];                        // prefixes, own tokens
  int max_shared, max_own, max_len;    // max_len: what a row of the table holds
  uint32_t magic;
  float scale;                         // softmax_scale * log2(e)
};

// Column tiles a block holds at most: the accumulators O^T take D / 4 * NT registers (128 at most), and
// 8 tiles of 64 channels do not fit beside the 8 tiles' other state.
__host__ __device__ constexpr int most_tiles(int D) { return D == 256 ? 2 : 4; }

template <int D, int NT>
struct Lay {
  static constexpr int kPd = D / 2;
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;
  // a step's codes of K and of V, then the scales of K and of V
  static constexpr int kStage = 2 * kStep * kPd + 4 * kStep;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kQ = kRing;                              // query fragments [D/16][NT][32] x 8
  // (one column tile for each warp where the warps work alone)
  static constexpr int kTiles = NT > kWarps ? NT : kWarps;
  static constexpr int kCol = kQ + D / 16 * kTiles * 32 * 8;    // per column: correction, factor
  static constexpr int kMain = kCol + 8 * kTiles * 8;
  // the join of the warps reuses the ring: the warps' O of one column tile, then max and sum of all
  static constexpr int kJoin = kWarps * 8 * D * 4 + kWarps * 8 * NT * 8;
  static constexpr int kTotal = kMain > kJoin ? kMain : kJoin;
};

// Where 16-byte piece `ch` of row `r` of a tile's codes lies: the pieces that one ldmatrix reads (8 rows,
// one ch) fall into different banks.
template <int D>
__device__ __forceinline__ int piece_at(int r, int ch) {
  if constexpr (D == 256) return r * 128 + ((ch ^ (r & 7)) << 4);
  else if constexpr (D == 128) return (r >> 1) * 128 + ((((r & 1) << 2) | (ch ^ ((r >> 1) & 3))) << 4);
  else return (r >> 2) * 128 + ((((r & 3) << 1) | (ch ^ ((r >> 2) & 1))) << 4);
}

// ----- the line of granules
// What a prefix or a sequence's own tokens come to: tokens [begin, end), granules from the tile that
// holds the first of them.
// Nothing of a group whose lengths contradict the bounds is attended.
struct Span {
  int begin, end, granules;
};

__device__ __forceinline__ Span span_from(int begin, int end, bool ok) {
  Span s;
  s.begin = ok ? begin : 0;
  s.end = ok ? end : 0;
  // (unsigned: the last tokens of the range of int do not overflow)
  s.granules = s.end > s.begin ? static_cast<int>((static_cast<uint32_t>(s.end - s.begin / kTile * kTile) +
                                                   (kGranule - 1)) / kGranule)
                               : 0;
  return s;
}

// Whether a group's lengths agree with the bounds; sh gets its prefix.
__device__ __forceinline__ bool group_ok(const BeamArgs& a, int g, int& sh) {
  sh = a.shared ? __ldg(a.shared + g) : 0;
  bool ok = true;
#pragma unroll 4
  for (int i = 0; i < a.beams; ++i) {
    const int len = __ldg(a.lens + g * a.beams + i);
    ok = ok && len >= sh && len - sh <= a.max_own && len <= a.max_len;
  }
  return ok && sh >= 0 && sh <= a.max_shared;
}

__device__ __forceinline__ Span span_of(const BeamArgs& a, bool shared, int who) {
  int sh;
  const bool ok = group_ok(a, shared ? who : who / a.beams, sh);
  return shared ? span_from(0, sh, ok) : span_from(sh, __ldg(a.lens + who), ok);
}

// Places in the line: a unit starts with its first granule, whose cost has that of starting and ending a
// unit added (kUnitCost), then the others follow.
__device__ __forceinline__ int64_t unit_cost(int granules, const Line& L) {
  if (granules && L.solo) return kSoloCost;
  return granules ? kUnitCost + static_cast<int64_t>(granules) * L.weight : 0;
}
__device__ __forceinline__ int64_t granule_at(int k, int weight) {
  return k ? kUnitCost + static_cast<int64_t>(k) * weight : 0;
}
// n / d for n >= 0, d > 0: both are mostly short, and the long division takes a microsecond.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  return ((n | d) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d)) : n / d;
}
// Granules that start before place x of a unit.
__device__ __forceinline__ int granules_before(int64_t x, int granules, int weight) {
  if (x <= 0) return 0;
  if (x <= kUnitCost + weight) return 1;
  const int64_t k = quotient(x - kUnitCost + weight - 1, weight);
  return k < granules ? static_cast<int>(k) : granules;
}

// A piece of a unit: what a block has of it.
struct Piece {
  int seq;                 // the sequence, or the group's first one
  int layer, h, x0, cols;  // its columns: heads of the group's sequences
  int tok0, tok1, tile0;   // tokens, and the tile that the first granule starts with
};

// Row of q and out of column x of a piece.
__device__ __forceinline__ int64_t col_row(const BeamArgs& a, const Piece& u, int x) {
  const int beam = x / a.G;   // 0 for own units
  return (static_cast<int64_t>(u.layer) * a.nseq + u.seq + beam) * a.Hq + u.h * a.G + (x - beam * a.G);
}

template <bool BF>
__device__ __forceinline__ float to_float(uint16_t b) {
  if constexpr (BF) return __uint_as_float(static_cast<uint32_t>(b) << 16);
  else return h2f(b);
}
template <bool BF>
__device__ __forceinline__ uint16_t from_float(float f) {
  if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  else return f2h(f);
}

// Codes in bits 0-3 (or 4-7) of the 16-bit lanes of w: as fp16, exact; or the latter as 16 (c + 72).
// `magic` is 0x64006400 out of the kernel's arguments: as a constant it costs an instruction of its own
// beside the mask.
__device__ __forceinline__ uint32_t masked(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));   // (w & mask) | magic
  return r;
}
__device__ __forceinline__ uint32_t low_codes(uint32_t w, uint32_t magic) {
  return hfma2u(masked(w, 0x000F000Fu, magic), kH1, kHm1032);
}
__device__ __forceinline__ uint32_t high_raw(uint32_t w, uint32_t magic) {
  return masked(w, 0x00F000F0u, magic);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w, uint32_t magic) {
  return hfma2u(high_raw(w, magic), kH16th, kHm72);
}

// 16 bytes from global to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 2^e as a product of two factors, |e| < 250.
__device__ __forceinline__ float pow2_half(int e) { return __int_as_float((e / 2 + 127) << 23); }
__device__ __forceinline__ float pow2_rest(int e) { return __int_as_float((e - e / 2 + 127) << 23); }

// Blocks per SM: fewer than the registers allow.  Every block more makes the shares shorter, of which each
// costs its start and end (7 + 2 us): 64 sequences of up to 8,192 tokens of 128 channels 44.8 us with 4,
// 41.8 with 3, 42.5 with 2; up to 32,768 tokens 123, 114 and 120.  (Measured at one column tile; 64 channels
// with one and two take the same three.)
template <int D, int NT> constexpr int kResident = NT * D >= 256 ? 2 : 3;

// d = a b + c and d += a b, free to be scheduled among each other.
__device__ __forceinline__ void product_from(float (&d)[4], const float (&c)[2], uint32_t a0, uint32_t a1,
                                             uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void product(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One piece: its granules' softmax and O, joined over the warps, to the record `rec` or (rec NULL) the
// result.  LT: the kernel's column tiles, NT: the piece's.  SOLO: the piece is the warp's alone (every warp
// has another), and nothing is joined.
template <int D, int LT, int NT, bool BF, bool SOLO = false>
__device__ __forceinline__ void run_piece(const BeamArgs& a, const Piece& u, float* rec, uint8_t* smem) {
  using Ly = Lay<D, LT>;
  constexpr int kPd = Ly::kPd, S = Ly::kStages;
  constexpr int CH = D / 32;     // 16-byte pieces of a row
  constexpr int kTileBytes = kTile * kPd;
  // tiles whose scores are held at once
  constexpr int TP = NT >= 4 ? 1 : 2;
  constexpr int WN = SOLO ? 1 : kWarps;     // warps that share the piece
  static_assert(!SOLO || NT == 1, "one column tile per warp");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int part = SOLO ? 0 : warp;         // this warp among those
  const LayerPools& P = a.L[u.layer];
  const uint32_t magic = a.magic;
  const int tile1 = (u.tok1 + kTile - 1) / kTile;
  const int n_steps = (tile1 - u.tile0 + 1) / 2;
  const int n_mine = n_steps > part ? (n_steps - part + WN - 1) / WN : 0;

  const uint32_t ring = smem_u32(smem) + warp * S * Ly::kStage;
  // Places (in tiles) of this warp's tiles, 16 steps of two tiles at a time, one per lane, and which of
  // them there are (the last steps' ones stay known for a while).
  uint32_t place = 0, there = 0, there_before = 0;
  // this lane's part of a tile's copies
  const uint8_t* k_src = P.kc + 16 * lane;
  const uint8_t* v_src = P.vc + 16 * lane;
  const uint8_t* s_src = reinterpret_cast<const uint8_t*>(lane & 2 ? P.vs : P.ks) + 16 * (lane & 1);
  const uint32_t s_dst = 4 * kTileBytes + (lane >> 1 & 1) * 2 * kStep + 16 * (lane & 1);
  constexpr int kCopies = kTile * CH / 32;
  uint32_t code_dst[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) code_dst[i] = piece_at<D>((i * 32 + lane) / CH, (i * 32 + lane) % CH);
  int st_in = 0;                 // stage of the next copies
  int page_next = -1, lp_tok = 0;
  auto look_up = [&](int j) {    // starts the loads of the next list's page ids
    const int jl = j + (lane >> 1), tile = u.tile0 + (jl * WN + part) * 2 + (lane & 1);
    page_next = -2;              // no tile
    if (jl < n_mine && tile < tile1) {
      const int tok = tile * kTile, lp = tok / a.ps;
      lp_tok = tok - lp * a.ps;
      page_next = lp < a.max_pages ? __ldg(a.pt + static_cast<int64_t>(u.seq) * a.max_pages + lp) : -1;
    }
  };
  auto issue = [&](int j) {
    if ((j & 15) == 0) {
      there_before = there;
      const bool ok = page_next >= 0 && page_next < P.pages;
      if (ok)
        place = static_cast<uint32_t>(((static_cast<int64_t>(page_next) * a.H + u.h) * a.ps + lp_tok) / kTile);
      else if (page_next != -2)
        report(a.err, KVQ_DEVERR_PAGE_RANGE);
      there = __ballot_sync(kFullMask, ok);
      look_up(j + 16);
    }
    const uint32_t dst = ring + st_in * Ly::kStage;
    st_in = st_in == S - 1 ? 0 : st_in + 1;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int from = (j & 15) * 2 + t;
      const uint64_t tile = __shfl_sync(kFullMask, place, from);
      if (there >> from & 1u) {  // the same in the whole warp
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          copy16(dst + t * kTileBytes + code_dst[i], k_src + tile * kTileBytes + 512 * i);
          copy16(dst + (2 + t) * kTileBytes + code_dst[i], v_src + tile * kTileBytes + 512 * i);
        }
        if (lane < 4) copy16(dst + s_dst + t * 2 * kTile, s_src + tile * (2 * kTile));
      }
    }
  };
  look_up(0);
  // the queries of this warp's columns, on their way while the first copies are started
  constexpr int N = D / 32;                 // a lane's channels N lane .. N lane + N - 1
  constexpr int Y = 8 * NT / WN;            // this warp's columns
  uint32_t qw[Y][N / 2];
#pragma unroll
  for (int y = 0; y < Y; ++y) {
    const int x = y * WN + part;
    const uint16_t* qp = a.q + col_row(a, u, u.x0 + min(x, u.cols - 1)) * D + N * lane;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) qw[y][i] = x < u.cols ? ld_nc_u32(qp + 2 * i) : 0;
  }
#pragma unroll
  for (int j = 0; j < S - 1; ++j) {
    if (j < n_mine) issue(j);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // ---- the queries' fragments and the columns' factors, a warp per column in turn
  uint32_t* qf = reinterpret_cast<uint32_t*>(smem + Ly::kQ + (SOLO ? warp * (D / 16 * 32 * 8) : 0));
  float2* col = reinterpret_cast<float2*>(smem + Ly::kCol) + (SOLO ? warp * 8 : 0);
#pragma unroll
  for (int y = 0; y < Y; ++y) {
    const int x = y * WN + part;
    float v[N];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      v[i] = to_float<BF>(static_cast<uint16_t>(qw[y][i / 2]));
      v[i + 1] = to_float<BF>(static_cast<uint16_t>(qw[y][i / 2] >> 16));
      most = fmaxf(most, fmaxf(fabsf(v[i]), fabsf(v[i + 1])));
    }
    most = __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(most)));
    // 2^e times the row has its largest entry in [2^13, 2^14) (below, where that is subnormal)
    const int exponent = static_cast<int>(__float_as_uint(most) >> 23);
    const int e = most > 0.f && exponent < 255 ? 13 + 127 - exponent : 0;
    const float f0 = pow2_half(e), f1 = pow2_rest(e);
    float sum = 0.f;
    // Channel 8 w + nib is of piece w / 4 of a row, thread w % 4's word of it; masks pair nibbles (0,4) (1,5)
    // and, shifted, (2,6) (3,7).  A lane has whole words (D 256), halves or quarters of one.
    const int w = N * lane / 8, nib0 = N == 8 ? 0 : (N * lane) & 7;
    uint32_t* at = qf + ((w / 4 * 2 * NT + (x >> 3)) * 32 + (x & 7) * 4 + w % 4) * 2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // the nibble in bits 4-7 of its lane (odd channels) stands for 16 (c + 72)
      const float y = v[i] * f0 * f1;
      const __half hy = __float2half_rn(i & 1 ? y * 0.0625f : y);
      if (i & 1) sum += __half2float(hy);
      const int nib = nib0 + i;
      reinterpret_cast<__half*>(at + (nib >> 1 & 1) * NT * 64 + (i & 1))[nib >> 2] = hy;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    // score in powers of two: (products - 16 * 72 sum) * factor * scale_t
    if (lane == 0) col[x] = make_float2(-1152.f * sum, a.scale * pow2_half(-e) * pow2_rest(-e));
  }
  if constexpr (SOLO) __syncwarp();
  else __syncthreads();
  float corr[NT][2], fac[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 f = col[8 * n + 2 * c + i];
      corr[n][i] = f.x;
      fac[n][i] = f.y;
    }
  const uint32_t qaddr = smem_u32(qf) + 8 * lane;
  // one column tile's fragments stay in registers where they are few
  constexpr bool kQRegs = NT == 1 && D <= 128;
  uint2 qr[kQRegs ? D / 16 : 1];
  auto q_pair = [&](int ks, int n) -> uint2 {
    if constexpr (kQRegs) {
      return qr[ks];
    } else {
      uint2 b;
      asm("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(b.x), "=r"(b.y) : "r"(qaddr + (ks * NT + n) * 256));
      return b;
    }
  };
  if constexpr (kQRegs) {
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) qr[ks] = reinterpret_cast<const uint2*>(qf)[ks * 32 + lane];
  }

  float acc[D / 16][NT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = kMaxFloor;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][n][k] = 0.f;
  }
  // this lane's addresses for ldmatrix: K's matrices are rows 0-7 and 8-15 of two pieces, V's too
  uint32_t at[CH / 2];
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) at[i] = piece_at<D>(lane & 15, 2 * i + (lane >> 4));

  int st = 0;
  for (int j = 0; j < n_mine; ++j) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncwarp();                           // all lanes' copies are there, the last stage has been read
    if (j + S - 1 < n_mine) issue(j + S - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    // the copies run up to S - 1 steps ahead: their list may be the next one already
    const uint32_t list = min(j + S - 1, n_mine - 1) >> 4 == j >> 4 ? there : there_before;
    const uint32_t bits = list >> (2 * (j & 15)) & 3u;
    const uint32_t stage = ring + st * Ly::kStage;
    const uint16_t* sc = reinterpret_cast<const uint16_t*>(smem + (warp * S + st) * Ly::kStage +
                                                           4 * kTileBytes) + g;
    st = st == S - 1 ? 0 : st + 1;
    const int t0 = (u.tile0 + (j * WN + part) * 2) * kTile;
    const bool full = bits == 3u && t0 >= u.tok0 && t0 + kStep <= u.tok1;
#pragma unroll
    for (int tp = 0; tp < 2; tp += TP) {
      // ---- scores
      float s[TP][NT][4];
#pragma unroll
      for (int t = 0; t < TP; ++t) {
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          uint32_t k[4];     // piece 2 i of rows g and g + 8, piece 2 i + 1 of them
          ldsm_x4(stage + (tp + t) * kTileBytes + at[i], k);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t ra = q & 1 ? k[q & 2] >> 8 : k[q & 2],
                           rb = q & 1 ? k[(q & 2) + 1] >> 8 : k[(q & 2) + 1];
            const uint32_t a0 = low_codes(ra, magic), a1 = low_codes(rb, magic);
            const uint32_t a2 = high_raw(ra, magic), a3 = high_raw(rb, magic);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 b = q_pair(4 * i + q, n);
              if (i == 0 && q == 0) product_from(s[t][n], corr[n], a0, a1, a2, a3, b.x, b.y);
              else product(s[t][n], a0, a1, a2, a3, b.x, b.y);
            }
          }
        }
      }
      // ---- weights
      float ks[2 * TP], vs[2 * TP];           // tokens g, g + 8, ...
#pragma unroll
      for (int i = 0; i < 2 * TP; ++i) {
        ks[i] = h2f(sc[8 * i + tp * kTile]);
        vs[i] = h2f(sc[kStep + 8 * i + tp * kTile]);
      }
      uint32_t out_of = 0;                    // tokens that are not attended
      if (!full) {
#pragma unroll
        for (int i = 0; i < 2 * TP; ++i) {
          const int tok = t0 + tp * kTile + g + 8 * i;
          if (!(tok >= u.tok0 && tok < u.tok1 && (bits >> (tp + (i >> 1)) & 1u))) {
            out_of |= 1u << i;
            vs[i] = 0.f;
          }
        }
      }
      // The products weight * scale of V are rounded to fp16, so the reference m follows score + exponent of the
      // scale (of this lane's largest one; 0 counts as the smallest that fp16 has): m is taken up anew, to 10 below
      // that, when it is more than 14 below, so that products stay below 2^15 and the largest do not fall far
      // below 2^10.  (Not at every new maximum: those of all 8 columns change in most of a run's first steps.)
      // Scores whose neighbours are further apart than that: the differences taken here are exact, and m is
      // rounded up, but never above the score, so that the largest weight is 1 or more.
      float v_most = fmaxf(fabsf(vs[0]), fabsf(vs[1]));
      if constexpr (TP == 2) v_most = fmaxf(v_most, fmaxf(fabsf(vs[2]), fabsf(vs[3])));
      const float v_exp = static_cast<float>(max((__float_as_int(v_most) >> 23) - 127, -24));
      const float v_below = fminf(v_exp, 10.f) - 10.f;
      uint32_t pb[NT][2 * TP];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[2 * TP][2];
#pragma unroll
        for (int i = 0; i < 2 * TP; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) x[i][k] = s[i >> 1][n][2 * (i & 1) + k] * (fac[n][k] * ks[i]);
        if (!full) {
#pragma unroll
          for (int i = 0; i < 2 * TP; ++i)
            if (out_of >> i & 1u) x[i][0] = x[i][1] = kNegInf;
        }
        float m0 = fmaxf(x[0][0], x[1][0]), m1 = fmaxf(x[0][1], x[1][1]);
        if constexpr (TP == 2) {
          m0 = fmaxf(m0, fmaxf(x[2][0], x[3][0]));
          m1 = fmaxf(m1, fmaxf(x[2][1], x[3][1]));
        }
        if (__any_sync(kFullMask, m0 - m[n][0] + v_exp > 14.f || m1 - m[n][1] + v_exp > 14.f)) {
          float n0 = fmaxf(m[n][0], __fadd_ru(m0, v_below)), n1 = fmaxf(m[n][1], __fadd_ru(m1, v_below));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(kFullMask, n0, o));
            n1 = fmaxf(n1, __shfl_xor_sync(kFullMask, n1, o));
          }
          const float f[2] = {ex2_fast(m[n][0] - n0), ex2_fast(m[n][1] - n1)};
          m[n][0] = n0;
          m[n][1] = n1;
          l[n][0] *= f[0];
          l[n][1] *= f[1];
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][n][k] *= f[k & 1];
        }
#pragma unroll
        for (int i = 0; i < 2 * TP; ++i) {
          const float p0 = ex2_fast(x[i][0] - m[n][0]), p1 = ex2_fast(x[i][1] - m[n][1]);
          l[n][0] += p0;
          l[n][1] += p1;
          pb[n][i] = movtrans(pack_h2(p0 * vs[i], p1 * vs[i]));
        }
      }
      // ---- O^T: a product's row g is channel 32 j + 4 g + (its nibble) of piece j, row g + 8 two on
#pragma unroll
      for (int t = 0; t < TP; ++t) {
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          uint32_t v[4];     // tokens 2c, 2c + 1 and 2c + 8, 2c + 9 of piece 2 i, then of piece 2 i + 1
          ldsm_x4_trans(stage + (2 + tp + t) * kTileBytes + at[i], v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w0 = v[2 * h], w1 = v[2 * h + 1], y0 = w0 >> 8, y1 = w1 >> 8;
            const uint32_t a0 = low_codes(w0, magic), a1 = low_codes(y0, magic), a2 = low_codes(w1, magic), a3 = low_codes(y1, magic);
            const uint32_t b0 = high_codes(w0, magic), b1 = high_codes(y0, magic), b2 = high_codes(w1, magic),
                           b3 = high_codes(y1, magic);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                product(acc[4 * i + 2 * h][n], a0, a1, a2, a3, pb[n][2 * t], pb[n][2 * t + 1]);
              product(acc[4 * i + 2 * h + 1][n], b0, b1, b2, b3, pb[n][2 * t], pb[n][2 * t + 1]);
            }
          }
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[n][i] += __shfl_xor_sync(kFullMask, l[n][i], o);
  if constexpr (SOLO) {
    // a lane has channels 32 j + 4 g .. + 3 of columns 2 c and 2 c + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x = 2 * c + i;
      if (x >= u.cols) continue;
      const float M = m[0][i], sum = l[0][i];
      const float inv = M == kMaxFloor && sum == 0.f ? 0.f : 1.f / sum;
      uint16_t* out = a.out + col_row(a, u, u.x0 + x) * D + 4 * g;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const float y[4] = {acc[2 * j][0][i], acc[2 * j + 1][0][i], acc[2 * j][0][2 + i], acc[2 * j + 1][0][2 + i]};
        if (rec) {
          float2* to = reinterpret_cast<float2*>(rec + x * (D + 2) + 32 * j + 4 * g);
          to[0] = make_float2(y[0], y[1]);
          to[1] = make_float2(y[2], y[3]);
        } else {
          uint2 w;
          w.x = from_float<BF>(y[0] * inv) | static_cast<uint32_t>(from_float<BF>(y[1] * inv)) << 16;
          w.y = from_float<BF>(y[2] * inv) | static_cast<uint32_t>(from_float<BF>(y[3] * inv)) << 16;
          *reinterpret_cast<uint2*>(out + 32 * j) = w;
        }
      }
      if (rec && g == 0) {
        rec[x * (D + 2) + D] = M;
        rec[x * (D + 2) + D + 1] = sum;
      }
    }
    return;
  }
  // ---- the warps' parts: common maximum and sum, then O, one column tile at a time
  float* so = reinterpret_cast<float*>(smem);                       // [warp][8][D]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * 8 * D);     // [warp][8 NT]
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (8 * n >= u.cols) continue;
    if (n) __syncthreads();
    float2* ml = sml + 8 * n;
    if (g == 0) {
      ml[warp * 8 * NT + 2 * c] = make_float2(m[n][0], l[n][0]);
      ml[warp * 8 * NT + 2 * c + 1] = make_float2(m[n][1], l[n][1]);
    }
    // channel 32 (i / 2) + 4 g + low, its low bits by the column, so that a warp's 32 values fall into
    // different banks
    float* mine = so + (warp * 8 + 2 * c) * D + 4 * g;
#pragma unroll
    for (int low = 0; low < 4; ++low) {
      float* to = mine + (low ^ c);
#pragma unroll
      for (int i = low & 1; i < D / 16; i += 2) {
        to[32 * (i >> 1)] = acc[i][n][low & 2];
        to[32 * (i >> 1) + D] = acc[i][n][(low & 2) + 1];
      }
    }
    __syncthreads();
    // warp w finishes columns w and w + 4
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int y = warp + 4 * h, x = 8 * n + y;
      if (x >= u.cols) continue;
      float2 p[kWarps];
      float M = kMaxFloor, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        p[w] = ml[w * 8 * NT + y];
        M = fmaxf(M, p[w].x);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        p[w].x = ex2_fast(p[w].x - M);
        sum += p[w].y * p[w].x;
      }
      const float inv = M == kMaxFloor && sum == 0.f ? 0.f : 1.f / sum;
      uint16_t* out = a.out + col_row(a, u, u.x0 + x) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int d = 32 * i + lane;
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) o += so[(w * 8 + y) * D + (d ^ (y >> 1))] * p[w].x;
        if (rec) rec[x * (D + 2) + d] = o;
        else out[d] = from_float<BF>(o * inv);
      }
      if (rec && lane == 0) {
        rec[x * (D + 2) + D] = M;
        rec[x * (D + 2) + D + 1] = sum;
      }
    }
  }
  __syncthreads();                          // the next piece's copies overwrite what was joined
}

// ALONE: own tokens are a granule at most in the whole call, and their units the warps'.  (In one kernel
// with the others they cost those their registers and places in the instruction cache: 8 groups of 4 beams
// 42.5 instead of 38.8 us.)
template <int D, int NT, bool BF, bool ALONE>
__global__ void __launch_bounds__(kThreads, (kResident<D, NT>)) beam_attn_kernel(const __grid_constant__ BeamArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");               // started while the work before it ends
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // ---- this block's share of a line: every warp finds it by itself, a lane adds up a run of groups
  const int run = (a.groups + 31) / 32;
  const int g0 = min(a.groups, lane * run), g1 = min(a.groups, g0 + run);
  int64_t mine[2] = {0, 0}, before[2], total[2];
  for (int g = g0; g < g1; ++g) {
    const int sh = a.shared ? __ldg(a.shared + g) : 0;
    bool ok = sh >= 0 && sh <= a.max_shared;
    int64_t own = 0;
#pragma unroll 4
    for (int i = 0; i < a.beams; ++i) {
      const int len = __ldg(a.lens + g * a.beams + i);
      ok = ok && len >= sh && len - sh <= a.max_own && len <= a.max_len;
      own += unit_cost(span_from(sh, len, ok).granules, a.line[1]);
    }
    if (ok) {
      mine[0] += unit_cost(span_from(0, sh, true).granules, a.line[0]);
      mine[1] += own;
    } else if (blockIdx.x == 0 && threadIdx.x < 32) {
      report(a.err, KVQ_DEVERR_INDEX);
    }
  }
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    mine[kind] *= a.line[kind].rep;
    before[kind] = mine[kind];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFullMask, before[kind], o);
      if (lane >= o) before[kind] += y;
    }
    total[kind] = __shfl_sync(kFullMask, before[kind], 31);
    before[kind] -= mine[kind];
  }
  // both lines' last blocks may be partly filled; no two granules of a unit start further apart than a share
  const int64_t cost = total[0] * a.line[0].blocks + total[1] * a.line[1].blocks;
  const int room = gridDim.x - a.line[0].blocks - a.line[1].blocks;
  const int64_t share = max(quotient(cost + room - 1, room),
                            static_cast<int64_t>(kUnitCost + max(a.line[0].weight, a.line[1].weight)));
  if (blockIdx.x == 0 && threadIdx.x == 0) a.head[0] = share;
  const int64_t n_prefix = quotient(total[0] + share - 1, share) * a.line[0].blocks;
  const int kind = blockIdx.x < n_prefix ? 0 : 1;
  const Line& L = a.line[kind];
  const int cta = blockIdx.x - (kind ? static_cast<int>(n_prefix) : 0);
  const int place = cta / L.blocks, blk = cta - place * L.blocks;
  const int64_t begin = share * place, end = min(kind ? total[1] : total[0], begin + share);
  if (begin >= (kind ? total[1] : total[0])) return;
  Span sp = {0, 0, 0};
  int w = 0;
  int64_t at = kind ? before[1] : before[0];   // place of entry w's first unit
  const int64_t ours = kind ? mine[1] : mine[0];
  const bool here = begin >= at && begin < at + ours;
  if (here) {
    for (w = kind ? g0 * a.beams : g0;; ++w) {
      sp = span_of(a, kind == 0, w);
      const int64_t c = unit_cost(sp.granules, L) * L.rep;
      if (begin < at + c) break;
      at += c;
    }
  }
  const int from = __ffs(__ballot_sync(kFullMask, here)) - 1;   // one lane has it
  w = __shfl_sync(kFullMask, w, from);
  at = __shfl_sync(kFullMask, at, from);
  sp.begin = __shfl_sync(kFullMask, sp.begin, from);
  sp.end = __shfl_sync(kFullMask, sp.end, from);
  sp.granules = __shfl_sync(kFullMask, sp.granules, from);
  int64_t unit = unit_cost(sp.granules, L);
  int r = static_cast<int>(quotient(begin - at, unit));
  at += r * unit;                           // place of unit r
  int k0 = granules_before(begin - at, sp.granules, L.weight);
  while (at < end) {
    const int k1 = granules_before(end - at, sp.granules, L.weight);
    int units = 1;                          // that this turn ends
    const bool solo = ALONE && kind == 1 && k0 == 0;
    if (solo) {
      units = static_cast<int>(min(static_cast<int64_t>(min(kWarps, L.rep - r)), quotient(end - at + unit - 1, unit)));
    }
    const int mine_r = solo ? r + static_cast<int>(threadIdx.x >> 5) : r;
    if (k0 < k1 && mine_r < r + units) {
      Piece u;
      u.seq = kind == 0 ? w * a.beams : w;
      u.h = mine_r % a.H;
      u.layer = mine_r / a.H;
      u.x0 = blk * 8 * NT;
      u.cols = min(8 * NT, (kind == 0 ? a.beams : 1) * a.G - u.x0);
      u.tile0 = sp.begin / kTile + k0 * (kGranule / kTile);
      u.tok0 = max(sp.begin, u.tile0 * kTile);
      u.tok1 = k1 == sp.granules ? sp.end : (sp.begin / kTile + k1 * (kGranule / kTile)) * kTile;
      const int64_t number = static_cast<int64_t>(w) * L.rep + mine_r;
      const bool whole = kind == 1 && sp.begin == 0 && k0 == 0 && k1 == sp.granules;
      if (k0 == 0 && blk == 0 && (solo ? lane : static_cast<int>(threadIdx.x)) == 0)
        a.head[1 + L.first_unit + number] = at + (mine_r - r) * unit;
      float* rec = a.ws + (L.first_rec + blk * (L.units + L.most) + number + place) * (8 * NT) * (D + 2);
      if (whole) rec = nullptr;
      // own tokens mostly have fewer columns than the prefixes' tiles
      if constexpr (ALONE) {
        if (solo) run_piece<D, NT, 1, BF, true>(a, u, rec, smem);
        else run_piece<D, NT, NT, BF>(a, u, rec, smem);
      } else {
        if (NT > 1 && u.cols <= 8) run_piece<D, NT, 1, BF>(a, u, rec, smem);
        else run_piece<D, NT, NT, BF>(a, u, rec, smem);
      }
    }
    if (ALONE && solo) {
      __syncthreads();                      // the next turn's copies and join may be other warps'
      r += units - 1;
      at += (units - 1) * unit;
    }
    k0 = 0;
    at += unit;
    if (++r == L.rep) {
      r = 0;
      do {
        if (++w == L.n) return;
        sp = span_of(a, kind == 0, w);
      } while (sp.granules == 0);
      unit = unit_cost(sp.granules, L);
    }
  }
}

// ---- joins the records: a warp per 64 channels of a row of out, two of them per lane
template <int D, int NT, bool BF>
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int kParts = D / 64;
  constexpr int64_t kStep = 8 * NT * (D + 2);
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int d = static_cast<int>(item % kParts) * 64 + 2 * lane;
  const int64_t row = item / kParts;
  if (row >= static_cast<int64_t>(a.n_layers) * a.nseq * a.Hq) return;
  int i = static_cast<int>(row);
  const int j = i % a.Hq;
  i /= a.Hq;
  const int s = i % a.nseq, layer = i / a.nseq;
  const int h = j / a.G, g = s / a.beams;
  int sh;
  const bool ok = group_ok(a, g, sh);
  const Span span[2] = {span_from(0, sh, ok), span_from(sh, __ldg(a.lens + s), ok)};
  asm volatile("griddepcontrol.wait;" ::: "memory");   // started while the attention still runs
  const int64_t share = a.head[0];
  // the records of the prefix, then those of the own tokens
  const float* rec[2] = {nullptr, nullptr};
  int n[2] = {0, 0};
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const Line& L = a.line[kind];
    if (span[kind].granules == 0 || L.n == 0) continue;
    const int who = kind == 0 ? g : s;
    const int x = kind == 0 ? (s - g * a.beams) * a.G + (j - h * a.G) : j - h * a.G;
    const int64_t number = static_cast<int64_t>(who) * L.rep + layer * a.H + h;
    const int64_t at = a.head[1 + L.first_unit + number];
    const int64_t first = quotient(at, share),
                  last = quotient(at + granule_at(span[kind].granules - 1, L.weight), share);
    n[kind] = static_cast<int>(last - first + 1);
    rec[kind] = a.ws + (L.first_rec + x / (8 * NT) * (L.units + L.most) + number + first) * kStep +
                x % (8 * NT) * (D + 2);
  }
  const int all = n[0] + n[1];
  if (span[1].begin == 0 && n[0] == 0 && n[1] == 1) return;   // written by the block that had all of it
  float M = kMaxFloor, sum = 0.f;
  float2 o = make_float2(0.f, 0.f);
  for (int k0 = 0; k0 < all; k0 += 32) {
    // each lane takes a record's maximum and sum
    const int k = k0 + lane;
    const float* mine = k < n[0] ? rec[0] + k * kStep : rec[1] + (k - n[0]) * kStep;
    float m = kMaxFloor, l = 0.f;
    if (k < all) {
      const float2 ml = *reinterpret_cast<const float2*>(mine + D);
      m = ml.x;
      l = ml.y;
    }
    float top = fmaxf(M, m);
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
    const float f = k < all ? ex2_fast(m - top) : 0.f;
    l *= f;
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(kFullMask, l, x);
    const float old = ex2_fast(M - top);
    M = top;
    sum = sum * old + l;
    o.x *= old;
    o.y *= old;
    const int most = min(32, all - k0);
    for (int y = 0; y < most; y += 8) {
      float2 v[8];
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        const int q = k0 + y + z;
        const float* r = q < n[0] ? rec[0] + q * kStep : rec[1] + (q - n[0]) * kStep;
        v[z] = y + z < most ? *reinterpret_cast<const float2*>(r + d) : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        const float w = __shfl_sync(kFullMask, f, (y + z) & 31);
        if (y + z < most) {
          o.x += w * v[z].x;
          o.y += w * v[z].y;
        }
      }
    }
  }
  const bool none = M == kMaxFloor && sum == 0.f;
  const uint32_t lo = from_float<BF>(none ? 0.f : o.x / sum), hi = from_float<BF>(none ? 0.f : o.y / sum);
  *reinterpret_cast<uint32_t*>(a.out + row * D + d) = lo | hi << 16;
}

// ----------------------------------------------------------------------------------------- launches
template <int D, int NT, bool BF, bool ALONE>
cudaError_t launch_attn(const BeamArgs& a, int blocks, cudaStream_t cs) {
  using Ly = Lay<D, NT>;
  static_assert(kResident<D, NT> * (Ly::kTotal + 1024) <= 227 * 1024, "shared memory");
  static_assert(152 * kResident<D, NT> <= kMostBlocks, "records");
  static SmemOnce once;
  const cudaError_t e = once.allow(beam_attn_kernel<D, NT, BF, ALONE>, Ly::kTotal);
  return e != cudaSuccess ? e
                          : launch_early(beam_attn_kernel<D, NT, BF, ALONE>, blocks, kThreads, Ly::kTotal, cs, a);
}

template <int D, int NT, bool BF>
cudaError_t launch(const BeamArgs& a, int64_t granules, cudaStream_t cs) {
  // one block more for the partly filled ones at the end of each line and column block
  const int64_t most = granules + a.line[0].blocks + a.line[1].blocks;
  const int blocks = static_cast<int>(std::min<int64_t>(152 * kResident<D, NT>, most));
  const cudaError_t e = a.line[1].solo ? launch_attn<D, NT, BF, true>(a, blocks, cs)
                                       : launch_attn<D, NT, BF, false>(a, blocks, cs);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.n_layers) * a.nseq * a.Hq * (D / 64);
  return launch_early(beam_join_kernel<D, NT, BF>, static_cast<unsigned>((items + kWarps - 1) / kWarps), kThreads, 0,
                      cs, a);
}

template <int D, bool BF>
cudaError_t by_tiles(const BeamArgs& a, int nt, int64_t granules, cudaStream_t cs) {
  if (nt == 1) return launch<D, 1, BF>(a, granules, cs);
  if (nt == 2) return launch<D, 2, BF>(a, granules, cs);
  if constexpr (most_tiles(D) == 4) return launch<D, 4, BF>(a, granules, cs);
  return cudaErrorInvalidValue;
}


template <bool BF>
cudaError_t by_dim(const BeamArgs& a, int D, int nt, int64_t granules, cudaStream_t cs) {
  return D == 64 ? by_tiles<64, BF>(a, nt, granules, cs)
       : D == 128 ? by_tiles<128, BF>(a, nt, granules, cs) : by_tiles<256, BF>(a, nt, granules, cs);
}

// The kernels of either type are compiled in a unit of their own.
cudaError_t run_f16(const BeamArgs& a, int D, int nt, int64_t granules, cudaStream_t cs);
cudaError_t run_bf16(const BeamArgs& a, int D, int nt, int64_t granules, cudaStream_t cs);

}  // namespace beam
}  // namespace kvq
