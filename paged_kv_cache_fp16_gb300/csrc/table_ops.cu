// Page tables that share pages: the update between two steps (sequences forked, continued, dropped,
// extended; pages shared, copied, freed and taken) and the compaction of the pages in use.
//
// The count of a page's owners is the only state: a page is free where it is 0.  Both operators read
// tables and counts and write new ones, so that nothing has to be undone and a call can be repeated.
// Each is two launches (one, where there is little of both): a plan, whose blocks meet between its phases,
// and the moves of pages and rows of the tables by the whole GPU, started early.  What bounds them: the
// phases' meetings and chains of dependent reads where little is to be moved (4 beams, one layer: 8.5 us in a
// graph; 64 beams over 262,000 tokens: 24.6 us, 21 of them the plan that reads 2.9 MB), the copied pages'
// bytes where much is (32 pools, 3,200 pages of each: 53 us, 49 of them moves at 6.3 TB/s).
//
//   update:  counts copied; every block learns all sequences, counts children and finds page writers in
//            its shared memory | every table entry changes its page's count by (children - 1) | pages
//            without owners counted per block of 1,024, needs of all sequences summed | the i-th needed
//            page is the i-th free one.  Then: rows of tables, started pages of sequences that part
//   compact: pages in use counted per block of 1,024 | free places below their number and used pages
//            above it ranked.  Then: the i-th such page moves to the i-th such place, tables follow
//
// The plan runs as one block, a cluster of eight or a cooperative grid, by the number of table entries and
// pages.  The order in which atomics arrive changes nothing: sums, minima and ranks only.
#include <cstdint>
#include <algorithm>
#include <initializer_list>

#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_warp.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = kThreads;       // pages counted together
constexpr int kChunk = 128;            // entries of a row that a warp takes at once
constexpr int kCluster = 8;            // blocks of the middle variant
constexpr int kMoveThreads = 256;
// table entries and pages up to which the plan is one block, one cluster
constexpr int64_t kBlockWork = 1 << 12, kClusterWork = 1 << 17;
constexpr int64_t kBlockBytes = 1 << 18;   // copies up to which one block makes them, too
// what becomes of a sequence's started page: kept (0), copied, or copied while the counts contradict
// the tables (then they are left as they are)
constexpr int kCopy = 1, kCopyUncounted = 2;

struct Pools {
  PoolRef p[KVQ_MAX_TENSORS];
  int n, H, ps, pd;
};

struct TableArgs {
  const int32_t *table, *lens, *held, *refs, *parents, *room;
  int32_t *table_out, *lens_out, *held_out, *refs_out, *live_out;
  int32_t* err;
  int32_t* bar;                        // a grid's plan: arrivals
  int32_t* blk;                        // free (update) or used (compact) pages per block
  int32_t *place, *from;               // compact: place of rank i, page of rank i
  int32_t* rank;                       // compact: per page
  int2* copy;                          // update, per new sequence: its copied page and where to, or -1
  int2* count;                         // x: moves (compact); new sequences whose rows are written (update)
                                       // y: blocks that gave up waiting
  int ps, max_pages, n_in, n_out, num_pages, n_blk, hash;   // hash: slots, a power of two
};

struct MoveArgs {
  Pools pools;
  TableArgs t;
};

// ------------------------------------------------------------------- how the blocks of a call meet
// One block.
struct BlockMeet {
  static constexpr bool kSure = true;
  __device__ explicit BlockMeet(const TableArgs&) {}
  __device__ bool operator()() {
    __threadfence_block();
    __syncthreads();
    return true;
  }
};

// One cluster: the hardware's barrier.
struct ClusterMeet {
  static constexpr bool kSure = true;
  __device__ explicit ClusterMeet(const TableArgs&) {}
  __device__ bool operator()() {
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    return true;
  }
};

// Polls of a meeting before a block gives up; a build may define a smaller limit (down to 0: give up at
// once) to run that path.
#ifndef KVQ_MEET_WAIT_LIMIT
#define KVQ_MEET_WAIT_LIMIT (1LL << 22)
#endif

// A cooperative grid: arrivals counted in global memory (zeroed before the launch, as `count` is), with a
// bounded wait.  A block that gave up leaves the others to their own limits, reports it and is counted: the
// blocks that met after all do not know of it, so the moves look whether there was one.
struct GridMeet {
  static constexpr bool kSure = false;
  int32_t *bar, *gone, *err;
  int goal = 0;
  __device__ explicit GridMeet(const TableArgs& a) : bar(a.bar), gone(&a.count->y), err(a.err) {}
  __device__ bool operator()() {
    goal += gridDim.x;
    __threadfence();
    __syncthreads();
    bool met = true;
    if (threadIdx.x == 0) {
      atomicAdd(bar, 1);
      met = false;
      for (long long i = 0; i < static_cast<long long>(KVQ_MEET_WAIT_LIMIT) && !met; ++i) {
        int v;
        asm volatile("ld.acquire.gpu.s32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
        met = v >= goal;
      }
      if (!met) {
        atomicAdd(gone, 1);
        report(err, KVQ_DEVERR_TIMEOUT);
      }
      __threadfence();
    }
    return __syncthreads_and(met);
  }
};

// Data that this launch writes and reads back goes through L2.
__device__ __forceinline__ int ld(const int32_t* p) { return __ldcg(p); }
__device__ __forceinline__ void st(int32_t* p, int v) { __stcg(p, v); }

// What the plan leaves to the moves.  Where a block gave up, what it had to write holds anything, and nothing
// is moved.
template <typename Meet>
__device__ __forceinline__ void put_count(const TableArgs& a, int n) {
  if constexpr (Meet::kSure) *a.count = make_int2(n, 0);
  else a.count->x = n;
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ int block_sum(int v, int* sm) {
  v = __reduce_add_sync(kFullMask, v);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = __reduce_add_sync(kFullMask, sm[threadIdx.x & 31]);
  __syncthreads();
  return v;
}

// Exclusive prefix over the block's threads; total gets the sum.
template <typename T>
__device__ __forceinline__ T block_prefix(T v, T* sm, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFullMask, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  T w = sm[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFullMask, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(kFullMask, w, 31);
  const T before = __shfl_sync(kFullMask, w, (warp + 31) & 31);
  __syncthreads();
  return x - v + (warp ? before : 0);
}

// Sum of blk[0 .. n).
__device__ __forceinline__ int sum_of(const int32_t* blk, int n, int* sm) {
  int v = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) v += ld(blk + i);
  return block_sum(v, sm);
}

// Copies n bytes (a multiple of sizeof(U)), one warp: 8 pieces of every lane on their way at once.
template <typename U>
__device__ __forceinline__ void warp_copy(void* dst, const void* src, int64_t n) {
  const int lane = threadIdx.x & 31;
  const U* s = static_cast<const U*>(src);
  U* d = static_cast<U*>(dst);
  const int64_t m = n / static_cast<int64_t>(sizeof(U));
  for (int64_t i = lane; i < m; i += 256) {
    U v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + 32 * k < m) v[k] = s[i + 32 * k];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + 32 * k < m) d[i + 32 * k] = v[k];
  }
}

// --------------------------------------------------------------------------------- table update
// An old sequence: the pages it hands on (keep) and those it has (held).  What contradicts the
// bounds holds nothing.
struct Old {
  int len, keep, held;
  bool bad;
};

__device__ __forceinline__ Old old_seq(const TableArgs& a, int p) {
  Old o;
  o.len = __ldg(a.lens + p);
  o.held = __ldg(a.held + p);
  o.keep = o.len > 0 ? (o.len - 1) / a.ps + 1 : 0;
  o.bad = o.len < 0 || o.held < 0 || o.held > a.max_pages || o.keep > o.held;
  if (o.bad) o.len = o.keep = o.held = 0;
  return o;
}

// A new sequence: its parent, the pages it takes over, and those it ends with.
struct New {
  int parent, len, keep, total;
  bool bad, writes;    // writes: into a page that has been started
};

__device__ __forceinline__ New new_seq(const TableArgs& a, int s) {
  New n;
  n.parent = __ldg(a.parents + s);
  int64_t room = __ldg(a.room + s);
  n.bad = n.parent < -1 || n.parent >= a.n_in;
  if (n.bad) n.parent = -1;
  n.len = n.keep = 0;
  if (n.parent >= 0) {
    const Old o = old_seq(a, n.parent);
    n.len = o.len;
    n.keep = o.keep;
  }
  if (room < 0 || room + n.len > static_cast<int64_t>(a.max_pages) * a.ps) {
    n.bad = true;
    room = 0;
  }
  n.total = room > 0 ? static_cast<int>((n.len + room - 1) / a.ps + 1) : n.keep;
  n.writes = room > 0 && n.len % a.ps != 0;
  return n;
}

// What every block knows of all sequences, in shared memory: [n_out] each, then children of the old ones
// and a hash table of the pages about to be written into.
struct Known {
  int *need, *keep, *tail, *start, *copy, *slot, *children, *key, *first, *count;
  __device__ Known(const TableArgs& a, int* sm) {
    auto take = [&](int n) {
      int* p = sm;
      sm += n;
      return p;
    };
    need = take(a.n_out);
    keep = take(a.n_out);
    tail = take(a.n_out);
    start = take(a.n_out);
    copy = take(a.n_out);
    slot = take(a.n_out);
    children = take(a.n_in);
    key = take(a.hash);
    first = take(a.hash);
    count = take(a.hash);
  }
};

template <typename Meet>
__device__ __forceinline__ void update_body(const TableArgs& a) {
  extern __shared__ int dyn[];
  __shared__ int sm[kWarps];
  __shared__ int64_t sm64[kWarps];
  Meet meet(a);
  const Known k(a, dyn);
  const int n_cta = gridDim.x, cta = blockIdx.x, tid = threadIdx.x;
  const int all = n_cta * kThreads, me = cta * kThreads + tid;

  for (uint32_t i = me; i < static_cast<uint32_t>(a.num_pages); i += all)   // (the last step may leave int)
    st(a.refs_out + i, __ldg(a.refs + i));
  for (int i = tid; i < a.n_in; i += kThreads) k.children[i] = 0;
  for (int i = tid; i < a.hash; i += kThreads) {
    k.key[i] = -1;
    k.first[i] = INT32_MAX;
    k.count[i] = 0;
  }
  __syncthreads();
  for (int s = tid; s < a.n_out; s += kThreads) {
    const New n = new_seq(a, s);
    if (n.bad && cta == 0) report(a.err, KVQ_DEVERR_INDEX);
    k.keep[s] = n.keep;
    k.need[s] = n.total - n.keep;
    int tail = -1;
    if (n.writes) {
      tail = __ldg(a.table + static_cast<int64_t>(n.parent) * a.max_pages + n.keep - 1);
      if (tail < 0 || tail >= a.num_pages) tail = -1;
    }
    k.tail[s] = tail;
    if (n.parent >= 0) atomicAdd(k.children + n.parent, 1);
    if (tail >= 0) {
      int at = static_cast<int>(static_cast<uint32_t>(tail) * 0x9E3779B1u >> 8) & (a.hash - 1);
      while (true) {       // at most n_out of the 2 n_out or more slots are ever taken
        const int was = atomicCAS(k.key + at, -1, tail);
        if (was == -1 || was == tail) break;
        at = (at + 1) & (a.hash - 1);
      }
      k.slot[s] = at;
      atomicMin(k.first + at, s);
      atomicAdd(k.count + at, 1);
    }
    if (cta == s % n_cta) {
      a.lens_out[s] = n.len;
      a.held_out[s] = n.total;
    }
  }
  if (!meet()) return;

  // every entry's page loses its owner and gains the owner's heirs; a warp takes 128 entries of a row
  const int lane = tid & 31, per_row = (a.max_pages - 1) / kChunk + 1;
  const int64_t chunks = static_cast<int64_t>(a.n_in) * per_row;
  for (int64_t ch = me >> 5; ch < chunks; ch += all >> 5) {
    const int p = static_cast<int>(ch / per_row), j0 = static_cast<int>(ch - static_cast<int64_t>(p) * per_row) * kChunk;
    const Old o = old_seq(a, p);
    if (o.bad && j0 == 0 && lane == 0) report(a.err, KVQ_DEVERR_INDEX);
    const int c = k.children[p] - 1;
    const int32_t* row = a.table + static_cast<int64_t>(p) * a.max_pages + j0;
    const int left = o.held - j0;
    int page[kChunk / 32];
#pragma unroll
    for (int i = 0; i < kChunk / 32; ++i) page[i] = lane + 32 * i < left ? __ldg(row + lane + 32 * i) : -1;
#pragma unroll
    for (int i = 0; i < kChunk / 32; ++i) {
      const int j = lane + 32 * i;
      if (j >= left) continue;
      const int d = j0 + j < o.keep ? c : -1;
      if (page[i] < 0 || page[i] >= a.num_pages) report(a.err, KVQ_DEVERR_PAGE_RANGE);
      else if (d != 0) atomicAdd(a.refs_out + page[i], d);
    }
  }
  if (!meet()) return;

  for (int b = cta; b < a.n_blk; b += n_cta) {
    const int i = b * kBlock + tid, r = i < a.num_pages ? ld(a.refs_out + i) : 1;
    if (r < 0) report(a.err, KVQ_DEVERR_INDEX);
    const int free = __syncthreads_count(r == 0);
    if (tid == 0) st(a.blk + b, free);
  }
  int64_t total = 0;
  for (int s0 = 0; s0 < a.n_out; s0 += kThreads) {
    const int s = s0 + tid;
    int64_t need = 0;
    int copy = 0;
    if (s < a.n_out) {
      const int tail = k.tail[s];
      if (tail >= 0) {
        // the first writer keeps the page where nobody but writers has it
        const int at = k.slot[s], spare = ld(a.refs_out + tail) - k.count[at];
        if (spare != 0 || k.first[at] != s) copy = spare < 0 ? kCopyUncounted : kCopy;
        if (spare < 0 && cta == 0) report(a.err, KVQ_DEVERR_INDEX);   // fewer owners counted than there are
      }
      need = k.need[s] + (copy != 0);
    }
    int64_t t;
    const int64_t at = total + block_prefix<int64_t>(need, sm64, t);
    total += t;
    if (s < a.n_out) {
      k.start[s] = static_cast<int>(at < INT32_MAX ? at : INT32_MAX);
      k.copy[s] = copy;
      // the page of a copy is taken below, by whoever has it
      if (!copy && cta == s % n_cta) a.copy[s] = make_int2(-1, -1);
    }
  }
  if (!meet()) return;

  const bool enough = total <= sum_of(a.blk, a.n_blk, sm);   // the same in every block
  if (me == 0) {
    if (!enough) report(a.err, KVQ_DEVERR_NO_PAGES);
    put_count<Meet>(a, enough ? a.n_out : 0);
  }
  if (!enough) return;
  for (int b = cta; b < a.n_blk; b += n_cta) {
    const int before = sum_of(a.blk, b, sm);
    if (before >= total) break;               // the same in the whole block
    const int i = b * kBlock + tid;
    const bool is = i < a.num_pages && ld(a.refs_out + i) == 0;
    int t;
    const int at = before + block_prefix<int>(is, sm, t);
    if (is && at < total) {
      int lo = 0, hi = a.n_out - 1;           // the last sequence whose needs start at or before at
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (k.start[mid] <= at) lo = mid; else hi = mid - 1;
      }
      const int copy = k.copy[lo] != 0, nth = at - k.start[lo];
      a.table_out[static_cast<int64_t>(lo) * a.max_pages + k.keep[lo] - copy + nth] = i;
      if (copy && nth == 0) a.copy[lo] = make_int2(k.tail[lo], i);
      st(a.refs_out + i, 1);
    }
  }
  // one owner fewer; somebody is left, so that no block sees the page as free meanwhile
  for (int s = me; s < a.n_out; s += all)
    if (k.copy[s] == kCopy) atomicSub(a.refs_out + k.tail[s], 1);
}

// The rows that sequences take over, and the started pages' rows of those that part.
template <typename U>
__device__ __forceinline__ void update_move(const MoveArgs& m, int64_t me, int64_t warps) {
  const TableArgs& a = m.t;
  const Pools& P = m.pools;
  const int2 count = __ldcg(a.count);
  if (count.x == 0 || count.y != 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t per_seq = static_cast<int64_t>(P.n) * P.H, pages = a.n_out * per_seq;
  for (int64_t it = me; it < pages; it += warps) {
    const int s = static_cast<int>(it / per_seq);
    const int2 c = __ldcg(a.copy + s);
    if (c.x < 0) continue;
    const int rest = static_cast<int>(it - s * per_seq), t = rest / P.H, h = rest - t * P.H;
    const int rows = __ldg(a.lens + __ldg(a.parents + s)) % P.ps;
    const int64_t from = (static_cast<int64_t>(c.x) * P.H + h) * P.ps;
    const int64_t to = (static_cast<int64_t>(c.y) * P.H + h) * P.ps;
    warp_copy<U>(P.p[t].codes + to * P.pd, P.p[t].codes + from * P.pd, static_cast<int64_t>(rows) * P.pd);
    warp_copy<uint16_t>(P.p[t].scales + to, P.p[t].scales + from, 2 * rows);
  }
  constexpr int kRow = 256;                   // entries of a row that a warp takes at once
  const int per_row = (a.max_pages - 1) / kRow + 1;
  const int64_t rows = static_cast<int64_t>(a.n_out) * per_row;
  for (int64_t it = me; it < rows; it += warps) {
    const int s = static_cast<int>(it / per_row), j0 = static_cast<int>(it - static_cast<int64_t>(s) * per_row) * kRow;
    const int parent = __ldg(a.parents + s);
    if (parent < 0 || parent >= a.n_in) continue;
    const int left = old_seq(a, parent).keep - (__ldcg(a.copy + s).x >= 0) - j0;   // (j0 + 256 may leave int)
    const int32_t* from = a.table + static_cast<int64_t>(parent) * a.max_pages + j0;
    int32_t* to = a.table_out + static_cast<int64_t>(s) * a.max_pages + j0;
    int v[kRow / 32];
#pragma unroll
    for (int i = 0; i < kRow / 32; ++i)
      if (32 * i + lane < left) v[i] = __ldg(from + 32 * i + lane);
#pragma unroll
    for (int i = 0; i < kRow / 32; ++i)
      if (32 * i + lane < left) to[32 * i + lane] = v[i];
  }
}

// -------------------------------------------------------------------------------- compaction
template <typename Meet>
__device__ __forceinline__ void compact_body(const TableArgs& a) {
  __shared__ int sm[kWarps];
  Meet meet(a);
  const int n_cta = gridDim.x, cta = blockIdx.x, tid = threadIdx.x;
  for (int b = cta; b < a.n_blk; b += n_cta) {
    const int i = b * kBlock + tid;
    const int used = __syncthreads_count(i < a.num_pages && __ldg(a.refs + i) != 0);
    if (tid == 0) st(a.blk + b, used);
  }
  if (!meet()) return;

  const int n = sum_of(a.blk, a.n_blk, sm);
  // of the used pages, those below n stay
  const int bn = n / kBlock, in = bn * kBlock + tid;
  const int stay = sum_of(a.blk, bn, sm) + __syncthreads_count(in < n && __ldg(a.refs + in) != 0);
  for (int b = cta; b < a.n_blk; b += n_cta) {
    const int before = sum_of(a.blk, b, sm);
    const int i = b * kBlock + tid, refs = i < a.num_pages ? __ldg(a.refs + i) : 0;
    int t;
    const int at = before + block_prefix<int>(refs != 0, sm, t);   // used pages before i
    if (i >= a.num_pages) continue;
    if (i < n) {
      if (refs == 0) a.place[i - at] = i;
      else a.refs_out[i] = refs;
    } else {
      if (refs != 0) a.from[at - stay] = i;
      a.rank[i] = refs != 0 ? at - stay : -1;
      a.refs_out[i] = 0;
    }
  }
  if (cta == 0 && tid == 0) {
    *a.live_out = n;
    put_count<Meet>(a, n - stay);
  }
}

template <typename U>
__device__ __forceinline__ void compact_move(const MoveArgs& m, int64_t me, int64_t warps) {
  const TableArgs& a = m.t;
  const Pools& P = m.pools;
  const int2 count = __ldcg(a.count);
  const int moves = count.x, n = ld(a.live_out);
  if (count.y != 0) return;
  const int lane = threadIdx.x & 31;
  // a page of one pool is one run of bytes: its heads' rows lie one after the other
  const int64_t codes = static_cast<int64_t>(P.H) * P.ps * P.pd, scales = static_cast<int64_t>(P.H) * P.ps;
  const int64_t pages = static_cast<int64_t>(moves) * P.n;
  for (int64_t it = me; it < pages; it += warps) {
    const int i = static_cast<int>(it / P.n), t = static_cast<int>(it - static_cast<int64_t>(i) * P.n);
    const int64_t from = ld(a.from + i), to = ld(a.place + i);
    warp_copy<U>(P.p[t].codes + to * codes, P.p[t].codes + from * codes, codes);
    warp_copy<uint16_t>(P.p[t].scales + to * scales, P.p[t].scales + from * scales, 2 * scales);
  }
  for (int64_t i = me * 32 + lane; i < moves; i += warps * 32)
    a.refs_out[ld(a.place + i)] = __ldg(a.refs + ld(a.from + i));
  constexpr int kRow = 256;
  const int per_row = (a.max_pages - 1) / kRow + 1;
  const int64_t rows = static_cast<int64_t>(a.n_in) * per_row;
  for (int64_t it = me; it < rows; it += warps) {
    const int s = static_cast<int>(it / per_row), j0 = static_cast<int>(it - static_cast<int64_t>(s) * per_row) * kRow;
    int held = __ldg(a.held + s);
    if (held < 0 || held > a.max_pages) {
      if (lane == 0 && j0 == 0) report(a.err, KVQ_DEVERR_INDEX);
      held = 0;
    }
    const int64_t row = static_cast<int64_t>(s) * a.max_pages + j0;
    const int left = held - j0;
#pragma unroll
    for (int i = 0; i < kRow / 32; ++i) {
      const int j = 32 * i + lane;
      if (j >= left) continue;
      int page = __ldg(a.table + row + j);
      if (page < 0 || page >= a.num_pages) {
        report(a.err, KVQ_DEVERR_PAGE_RANGE);
      } else if (page >= n) {
        const int r = ld(a.rank + page);
        if (r >= 0) page = ld(a.place + r);
        else report(a.err, KVQ_DEVERR_INDEX);              // an entry whose page has no owners
      } else if (__ldg(a.refs + page) == 0) {
        report(a.err, KVQ_DEVERR_INDEX);
      }
      a.table_out[row + j] = page;
    }
  }
}

template <bool UPDATE, typename U>
__device__ __forceinline__ void move(const MoveArgs& m, int64_t me, int64_t warps) {
  if constexpr (UPDATE) update_move<U>(m, me, warps);
  else compact_move<U>(m, me, warps);
}
template <bool UPDATE, typename U>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ MoveArgs m) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  move<UPDATE, U>(m, static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5),
                  static_cast<int64_t>(gridDim.x) * (kMoveThreads / 32));
}

template <bool UPDATE, typename Meet>
__device__ __forceinline__ void plan_body(const TableArgs& a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // started while the work before it ends
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (UPDATE) update_body<Meet>(a);
  else compact_body<Meet>(a);
}
template <bool UPDATE>
__global__ void __launch_bounds__(kThreads, 1) plan_block_kernel(const __grid_constant__ TableArgs a) {
  plan_body<UPDATE, BlockMeet>(a);
}
// Plan and moves in one launch: a launch less, where a block's own copies take no longer than that.
template <bool UPDATE, typename U>
__global__ void __launch_bounds__(kThreads, 1) whole_kernel(const __grid_constant__ MoveArgs m) {
  plan_body<UPDATE, BlockMeet>(m.t);
  __threadfence_block();
  __syncthreads();
  move<UPDATE, U>(m, threadIdx.x >> 5, kWarps);
}
template <bool UPDATE>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(kCluster, 1, 1)
    plan_cluster_kernel(const __grid_constant__ TableArgs a) {
  plan_body<UPDATE, ClusterMeet>(a);
}
template <bool UPDATE>
__global__ void __launch_bounds__(kThreads, 1) plan_grid_kernel(const __grid_constant__ TableArgs a) {
  plan_body<UPDATE, GridMeet>(a);
}

// ------------------------------------------------------------------------------------ host side
struct Plan {
  size_t bar, count, place, from, rank, blk, copy, bytes;
};

Plan plan(int64_t num_pages, int64_t nseq) {
  Plan p;
  size_t at = 0;
  auto take = [&](int64_t n) {
    const size_t here = at;
    at += (static_cast<size_t>(n) * 4 + 15) / 16 * 16;
    return here;
  };
  p.bar = take(4);
  p.count = take(4);       // (behind bar: they are zeroed together)
  p.place = take(num_pages);
  p.from = take(num_pages);
  p.rank = take(num_pages);
  p.blk = take((num_pages + kBlock - 1) / kBlock);
  p.copy = take(2 * nseq);
  p.bytes = at;
  return p;
}

// What both entry points check and fill in the same way.
kvq_status common(const char* fn, MoveArgs& m, const kvq_pool* pools, int n_tensors,
                  const int32_t* table, int max_pages, const int32_t* held, const int32_t* refs,
                  int n_in, int n_out, int32_t* table_out, int32_t* refs_out, void* workspace,
                  size_t workspace_bytes, int32_t* dev_err) {
  if (n_tensors < 1 || n_tensors > KVQ_MAX_TENSORS)
    return fail(KVQ_ERR_RANGE, "%s: n_tensors %d not in [1, %d]", fn, n_tensors, KVQ_MAX_TENSORS);
  const kvq_status st = check_pools_uniform(pools, n_tensors, fn);
  if (st != KVQ_OK) return st;
  for (int i = 1; i < n_tensors; ++i)
    if (pools[i].num_pages != pools[0].num_pages)
      return fail(KVQ_ERR_SHAPE, "%s: pool %d has another number of pages than pool 0", fn, i);
  if (pools[0].num_pages > INT32_MAX - 2 * kBlock)
    return fail(KVQ_ERR_RANGE, "%s: %lld pages", fn, static_cast<long long>(pools[0].num_pages));
  if (n_in < 0 || n_out < 0 || max_pages < 1 || n_in > KVQ_MAX_TABLE_SEQS || n_out > KVQ_MAX_TABLE_SEQS)
    return fail(KVQ_ERR_RANGE, "%s: bad number of sequences (at most %d) or max_pages", fn,
                KVQ_MAX_TABLE_SEQS);
  if (!refs || !refs_out || (n_in > 0 && (!table || !held)) || !workspace)
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned16(workspace)) return fail(KVQ_ERR_ALIGN, "%s: workspace is not 16-byte aligned", fn);
  for (const int32_t* p : {table, held, refs, static_cast<const int32_t*>(table_out), static_cast<const int32_t*>(refs_out)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(KVQ_ERR_ALIGN, "%s: tables and counts must be aligned", fn);
  const size_t need = kvq_table_workspace(pools[0].num_pages, std::max(n_in, n_out));
  if (workspace_bytes < need)
    return fail(KVQ_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes,
                need);
  for (int i = 0; i < KVQ_MAX_TENSORS; ++i)
    m.pools.p[i] = i < n_tensors ? PoolRef{pools[i].codes, pools[i].scales, pools[i].num_pages}
                                 : PoolRef{nullptr, nullptr, 0};
  m.pools.n = n_tensors;
  m.pools.H = pools[0].num_heads;
  m.pools.ps = pools[0].page_size;
  m.pools.pd = kvq_packed_dim(pools[0].head_dim, pools[0].bits);
  TableArgs& a = m.t;
  a.ps = pools[0].page_size;
  a.num_pages = static_cast<int>(pools[0].num_pages);
  a.n_blk = (a.num_pages + kBlock - 1) / kBlock;
  a.table = table;
  a.held = held;
  a.refs = refs;
  a.table_out = table_out;
  a.refs_out = refs_out;
  a.err = dev_err;
  a.max_pages = max_pages;
  a.n_in = n_in;
  a.n_out = n_out;
  const Plan p = plan(a.num_pages, std::max(n_in, n_out));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto at = [&](size_t o) { return reinterpret_cast<int32_t*>(ws + o); };
  a.bar = at(p.bar); a.count = reinterpret_cast<int2*>(ws + p.count); a.place = at(p.place); a.from = at(p.from);
  a.rank = at(p.rank); a.blk = at(p.blk);
  a.copy = reinterpret_cast<int2*>(ws + p.copy);
  a.hash = 64;
  while (a.hash < 2 * n_out) a.hash *= 2;
  return KVQ_OK;
}

// What the largest update's Known takes.
constexpr int kMostSmem = (6 + 1 + 3 * 2) * KVQ_MAX_TABLE_SEQS * 4;

template <bool UPDATE>
size_t plan_smem(const TableArgs& a) {
  return UPDATE ? (6 * static_cast<size_t>(a.n_out) + a.n_in + 3 * static_cast<size_t>(a.hash)) * 4 : 0;
}
// Table entries and pages that the plan's blocks go through.
template <bool UPDATE>
int64_t plan_work(const TableArgs& a) {
  return a.num_pages + (UPDATE ? static_cast<int64_t>(a.n_in) * a.max_pages : 0);
}

template <bool UPDATE>
cudaError_t launch_plan(const TableArgs& a, cudaStream_t cs) {
  const size_t smem = plan_smem<UPDATE>(a);
  const int64_t work = plan_work<UPDATE>(a);
  static SmemOnce block, cluster, grid;
  cudaError_t e;
  if (work <= kBlockWork) {
    e = block.allow(plan_block_kernel<UPDATE>, kMostSmem);
    return e != cudaSuccess ? e : launch_early(plan_block_kernel<UPDATE>, 1, kThreads, smem, cs, a);
  }
  if (work <= kClusterWork) {
    e = cluster.allow(plan_cluster_kernel<UPDATE>, kMostSmem);
    return e != cudaSuccess ? e : launch_early(plan_cluster_kernel<UPDATE>, kCluster, kThreads, smem, cs, a);
  }
  e = grid.allow(plan_grid_kernel<UPDATE>, kMostSmem);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(a.bar, 0, 32, cs);   // bar and count
  if (e != cudaSuccess) return e;
  TableArgs copy = a;
  void* args[] = {&copy};
  e = cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(&plan_grid_kernel<UPDATE>), dim3(sm_count()),
                                  dim3(kThreads), args, smem, cs);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

// warps: what the moves can use at most; bytes: what they copy at most.
template <bool UPDATE, typename U>
cudaError_t launch(const MoveArgs& m, int64_t warps, int64_t bytes, cudaStream_t cs) {
  const int64_t entries = static_cast<int64_t>(UPDATE ? m.t.n_out : m.t.n_in) * m.t.max_pages;
  if (plan_work<UPDATE>(m.t) <= kBlockWork && entries <= kBlockWork && bytes <= kBlockBytes) {
    static SmemOnce whole;
    const cudaError_t e = whole.allow(whole_kernel<UPDATE, U>, kMostSmem);
    return e != cudaSuccess ? e : launch_early(whole_kernel<UPDATE, U>, 1, kThreads, plan_smem<UPDATE>(m.t), cs, m);
  }
  const cudaError_t e = launch_plan<UPDATE>(m.t, cs);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (warps + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
  const unsigned n = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(blocks, 152 * 8)));
  return launch_early(move_kernel<UPDATE, U>, n, kMoveThreads, 0, cs, m);
}

template <bool UPDATE>
kvq_status run(const char* fn, const MoveArgs& m, int64_t warps, int64_t bytes, kvq_stream_t stream) {
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  // the widest piece that divides what is copied (a row of one head, a whole page)
  const int64_t unit = UPDATE ? m.pools.pd : static_cast<int64_t>(m.pools.H) * m.pools.ps * m.pools.pd;
  const cudaError_t e = unit % 16 == 0 ? launch<UPDATE, uint4>(m, warps, bytes, cs)
                      : unit % 4 == 0 ? launch<UPDATE, uint32_t>(m, warps, bytes, cs)
                                      : launch<UPDATE, uint8_t>(m, warps, bytes, cs);
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

}  // namespace
}  // namespace kvq

extern "C" size_t kvq_table_workspace(int64_t num_pages, int nseq) {
  if (num_pages < 1 || num_pages > INT32_MAX || nseq < 0 || nseq > KVQ_MAX_TABLE_SEQS) return 0;
  return kvq::plan(num_pages, nseq).bytes;
}

extern "C" kvq_status kvq_table_update(const kvq_pool* pools, int n_tensors, const int32_t* table,
                                       int max_pages, const int32_t* lens, const int32_t* held,
                                       int n_in, const int32_t* refs, const int32_t* parents,
                                       const int32_t* room, int n_out, int32_t* table_out,
                                       int32_t* lens_out, int32_t* held_out, int32_t* refs_out,
                                       void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                       kvq_stream_t stream) {
  using namespace kvq;
  const char* fn = "kvq_table_update";
  MoveArgs m = {};
  const kvq_status st = common(fn, m, pools, n_tensors, table, max_pages, held, refs, n_in, n_out,
                               table_out, refs_out, workspace, workspace_bytes, dev_err);
  if (st != KVQ_OK) return st;
  if ((n_in > 0 && !lens) || (n_out > 0 && (!parents || !room || !table_out || !lens_out || !held_out)))
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  for (const int32_t* p : {lens, parents, room, static_cast<const int32_t*>(lens_out),
                           static_cast<const int32_t*>(held_out)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(KVQ_ERR_ALIGN, "%s: lengths must be aligned", fn);
  if (refs == refs_out || (n_in > 0 && n_out > 0 && (table == table_out || lens == lens_out || held == held_out)))
    return fail(KVQ_ERR_RANGE, "%s: an output is the input of the same kind", fn);
  m.t.lens = lens;
  m.t.parents = parents;
  m.t.room = room;
  m.t.lens_out = lens_out;
  m.t.held_out = held_out;
  const int64_t page = static_cast<int64_t>(m.pools.H) * m.pools.ps * m.pools.pd * n_tensors;
  return run<true>(fn, m, static_cast<int64_t>(n_out) * std::max<int64_t>(n_tensors * m.pools.H,
                                                                         (max_pages - 1) / 256 + 1),
                   n_out * page, stream);
}

extern "C" kvq_status kvq_table_compact(const kvq_pool* pools, int n_tensors, const int32_t* table,
                                        int max_pages, const int32_t* held, int nseq,
                                        const int32_t* refs, int32_t* table_out, int32_t* refs_out,
                                        int32_t* live, void* workspace, size_t workspace_bytes,
                                        int32_t* dev_err, kvq_stream_t stream) {
  using namespace kvq;
  const char* fn = "kvq_table_compact";
  MoveArgs m = {};
  const kvq_status st = common(fn, m, pools, n_tensors, table, max_pages, held, refs, nseq, 0,
                               table_out, refs_out, workspace, workspace_bytes, dev_err);
  if (st != KVQ_OK) return st;
  if (!live || (nseq > 0 && !table_out)) return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  if (refs == refs_out || (nseq > 0 && table == table_out))
    return fail(KVQ_ERR_RANGE, "%s: an output is the input of the same kind", fn);
  if (reinterpret_cast<uintptr_t>(live) % 4) return fail(KVQ_ERR_ALIGN, "%s: live must be aligned", fn);
  m.t.live_out = live;
  return run<false>(fn, m, std::max(static_cast<int64_t>(m.t.num_pages) / 2 * n_tensors,
                                    static_cast<int64_t>(nseq) * ((max_pages - 1) / 256 + 1)),
                    static_cast<int64_t>(m.t.num_pages) / 2 * m.pools.H * m.pools.ps * m.pools.pd * n_tensors,
                    stream);
}
