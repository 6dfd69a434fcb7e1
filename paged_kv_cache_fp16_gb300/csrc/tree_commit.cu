// Keep the accepted drafts of a tree: their packed rows move to the places behind the cached text.
//
// Pure data movement, a few rows per (sequence, head, pool): the time is the launch and three
// dependent reads (accepted node, page id, row), so one block takes all of a (sequence, head,
// pool)'s rows at once: every thread reads its pieces into registers, the block meets, and then
// writes them.  The barrier between is what makes any order of accepted nodes safe in place.
// One sequence's accepted path in one layer: 3.1 us on the device; those of 64 sequences in 16
// layers (8,192 blocks): 16.7 us.
#include <cstdint>

#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;

struct CommitArgs {
  PoolRef pools[KVQ_MAX_TENSORS];
  const int32_t* pt;
  const int32_t* lens;
  const int32_t* cu;
  const int32_t* accept;
  int32_t* err;
  int H, ps, max_pages, total, pd;
};

// U: the piece a thread moves at once (the widest that divides a row's bytes, so that every piece
// is aligned); NP: pieces per thread that the largest case (64 rows of 256 / U-multiple bytes)
// needs.
template <typename U, int NP>
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const __grid_constant__ CommitArgs a) {
  __shared__ int64_t from[KVQ_MAX_NODES], to[KVQ_MAX_NODES];
  const int s = blockIdx.x, h = blockIdx.y;
  const PoolRef P = a.pools[blockIdx.z];
  const int c0 = __ldg(a.cu + s), c1 = __ldg(a.cu + s + 1);
  const int len = __ldg(a.lens + s);
  if (c0 < 0 || c1 < c0 || c1 > a.total || c1 - c0 > KVQ_MAX_NODES || len < 0) {
    if (threadIdx.x == 0) report(a.err, KVQ_DEVERR_INDEX);
    return;
  }
  const int n = c1 - c0;
  if (n == 0) return;
  if (threadIdx.x < n) {
    const int i = threadIdx.x, node = __ldg(a.accept + c0 + i);
    int64_t f = -1, g = -1;
    if (node < 0 || node >= KVQ_MAX_NODES) {
      report(a.err, KVQ_DEVERR_INDEX);
    } else if (node != i) {   // a row already in its place stays
      f = locate_row(a.pt, a.max_pages, a.ps, a.H, P.num_pages, s,
                     static_cast<int64_t>(len) + node, h, a.err);
      g = locate_row(a.pt, a.max_pages, a.ps, a.H, P.num_pages, s,
                     static_cast<int64_t>(len) + i, h, a.err);
      if (f < 0 || g < 0) f = g = -1;
    }
    from[i] = f;
    to[i] = g;
  }
  __syncthreads();
  const int per_row = a.pd / static_cast<int>(sizeof(U));
  U* codes = reinterpret_cast<U*>(P.codes);
  U v[NP];
  uint16_t sc = 0;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = j * kThreads + threadIdx.x, r = c / per_row;
    if (r < n && from[r] >= 0) v[j] = codes[from[r] * per_row + (c - r * per_row)];
  }
  if (threadIdx.x < n && from[threadIdx.x] >= 0) sc = P.scales[from[threadIdx.x]];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = j * kThreads + threadIdx.x, r = c / per_row;
    if (r < n && to[r] >= 0) codes[to[r] * per_row + (c - r * per_row)] = v[j];
  }
  if (threadIdx.x < n && to[threadIdx.x] >= 0) P.scales[to[threadIdx.x]] = sc;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_tree_commit(const kvq_pool* pools, int n_tensors,
                                      const int32_t* page_table, int max_pages,
                                      const int32_t* seq_lens, const int32_t* cu_accept,
                                      const int32_t* accept, int nseq, int total_accept,
                                      int32_t* dev_err, kvq_stream_t stream) {
  using namespace kvq;
  const char* fn = "kvq_tree_commit";
  if (n_tensors < 1 || n_tensors > KVQ_MAX_TENSORS)
    return fail(KVQ_ERR_RANGE, "%s: n_tensors %d not in [1, %d]", fn, n_tensors, KVQ_MAX_TENSORS);
  const kvq_status st = check_pools_uniform(pools, n_tensors, fn);
  if (st != KVQ_OK) return st;
  if (nseq < 0 || total_accept < 0 || max_pages < 1)
    return fail(KVQ_ERR_RANGE, "%s: bad nseq/total_accept/max_pages", fn);
  if (pools[0].num_heads > 65535)
    return fail(KVQ_ERR_RANGE, "%s: num_heads %d > 65535", fn, pools[0].num_heads);
  if (nseq == 0 || total_accept == 0) return ok();
  if (!page_table || !seq_lens || !cu_accept || !accept)
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  CommitArgs a;
  for (int i = 0; i < KVQ_MAX_TENSORS; ++i)
    a.pools[i] = i < n_tensors ? PoolRef{pools[i].codes, pools[i].scales, pools[i].num_pages}
                               : PoolRef{nullptr, nullptr, 0};
  a.pt = page_table; a.lens = seq_lens; a.cu = cu_accept; a.accept = accept; a.err = dev_err;
  a.H = pools[0].num_heads; a.ps = pools[0].page_size; a.max_pages = max_pages;
  a.total = total_accept; a.pd = kvq_packed_dim(pools[0].head_dim, pools[0].bits);
  const dim3 grid(nseq, a.H, n_tensors);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (a.pd % 16 == 0) tree_commit_kernel<uint4, 4><<<grid, kThreads, 0, cs>>>(a);
  else if (a.pd % 4 == 0) tree_commit_kernel<uint32_t, 16><<<grid, kThreads, 0, cs>>>(a);
  else tree_commit_kernel<uint8_t, 64><<<grid, kThreads, 0, cs>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}
