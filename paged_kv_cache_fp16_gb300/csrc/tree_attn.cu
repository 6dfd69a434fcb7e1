// Attention of drafted tokens over the packed pages: one warp per (layer, node, query head).
#include <cmath>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kD = 256;

struct TreePools {
  const uint8_t* kc;
  const uint16_t* ks;
  const uint8_t* vc;
  const uint16_t* vs;
  int64_t k_pages, v_pages;
};

struct TreeArgs {
  TreePools L[KVQ_MAX_TENSORS];
  const uint16_t* q;
  uint16_t* out;
  const int32_t* pt;
  const int32_t* lens;
  const int32_t* cu;
  const int32_t* parents;
  int32_t* err;
  int n_layers, nseq, total, H, Hq, ps, max_pages, max_nodes, max_len;
  float scale;
};

template <int BITS>
__device__ __forceinline__ float value(const uint8_t* row, float sc, int d) {
  int c;
  if constexpr (BITS == 8) {
    c = static_cast<int8_t>(row[d]);
  } else if constexpr (BITS == 4) {
    c = static_cast<int>((row[d >> 1] >> ((d & 1) * 4)) & 15) - 8;
  } else {
    const uint8_t* b = row + d / 4 * 3;
    const uint32_t w = b[0] | (b[1] << 8) | (b[2] << 16);
    c = static_cast<int>((w >> (6 * (d & 3))) & 63u) - 32;
  }
  return h2f(f2h(static_cast<float>(c) * sc));
}

template <int BITS>
__global__ void __launch_bounds__(256) tree_rows_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int PD = kD * BITS / 8;
  const int lane = threadIdx.x & 31;
  const int64_t n_rows = static_cast<int64_t>(a.n_layers) * a.total * a.Hq;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < n_rows;
       row += step) {
    const int j = static_cast<int>(row % a.Hq);
    const int t = static_cast<int>(row / a.Hq % a.total);
    const TreePools& P = a.L[row / a.Hq / a.total];
    const int s = find_seq_from(a.cu, a.nseq, t, 0);
    const int n0 = a.cu[s], n1 = a.cu[s + 1], len = a.lens[s];
    if (t < n0 || t >= n1) continue;
    if (n0 < 0 || n1 > a.total || n1 - n0 > a.max_nodes || len < 0 ||
        static_cast<int64_t>(len) + n1 - n0 > a.max_len) {
      report(a.err, KVQ_DEVERR_INDEX);
      continue;
    }
    uint64_t seen = 0;
    for (int i = t - n0; i >= 0;) {
      seen |= 1ull << i;
      int p = a.parents[n0 + i];
      if (p < -1 || p >= i) {
        report(a.err, KVQ_DEVERR_INDEX);
        p = -1;
      }
      i = p;
    }
    const int h = j / (a.Hq / a.H);
    float qf[8], o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      qf[e] = h2f(a.q[row * kD + lane * 8 + e]);
      o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < len + n1 - n0; ++i) {
      if (i >= len && !((seen >> (i - len)) & 1)) continue;
      const int64_t kr = locate_row(a.pt, a.max_pages, a.ps, a.H, P.k_pages, s, i, h, a.err);
      const int64_t vr = locate_row(a.pt, a.max_pages, a.ps, a.H, P.v_pages, s, i, h, a.err);
      if (kr < 0 || vr < 0) continue;
      const float ks = h2f(P.ks[kr]), vs = h2f(P.vs[vr]);
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x = fmaf(qf[e], value<BITS>(P.kc + kr * PD, ks, lane * 8 + e), x);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(kFullMask, x, w);
      x *= a.scale;
      const float mn = fmaxf(m, x);
      const float f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(x - mn);
      l = l * f + p;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = o[e] * f + p * value<BITS>(P.vc + vr * PD, vs, lane * 8 + e);
      m = mn;
    }
    const float inv = m > -INFINITY ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) a.out[row * kD + lane * 8 + e] = f2h(o[e] * inv);
  }
}

}  // namespace
}  // namespace kvq

extern "C" size_t kvq_tree_attn_workspace(int n_layers, int nseq, int total_nodes,
                                          int num_kv_heads, int num_q_heads, int head_dim,
                                          int max_nodes, int max_seq_len) {
  (void)head_dim; (void)max_nodes;
  if (n_layers < 1 || nseq < 1 || total_nodes < 0 || num_kv_heads < 1 || num_q_heads < 1 ||
      max_seq_len < 0)
    return 0;
  return 16;
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
  if (!std::isfinite(softmax_scale) || softmax_scale <= 0)
    return fail(KVQ_ERR_RANGE, "%s: softmax_scale is not a finite value > 0", fn);
  if (nseq == 0 || total_nodes == 0) return ok();
  if (!q || !page_table || !seq_lens || !cu_nodes || !parents || !out || !workspace)
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return fail(KVQ_ERR_ALIGN, "%s: q/out/workspace must be 16-byte aligned", fn);
  const size_t need = kvq_tree_attn_workspace(n_layers, nseq, total_nodes, H, num_q_heads, kD,
                                              max_nodes, max_seq_len);
  if (workspace_bytes < need)
    return fail(KVQ_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, workspace_bytes, need);
  TreeArgs a;
  for (int i = 0; i < KVQ_MAX_TENSORS; ++i)
    a.L[i] = i < n_layers ? TreePools{k_pools[i].codes, k_pools[i].scales, v_pools[i].codes,
                                      v_pools[i].scales, k_pools[i].num_pages,
                                      v_pools[i].num_pages}
                          : TreePools{nullptr, nullptr, nullptr, nullptr, 0, 0};
  a.q = q; a.out = out; a.pt = page_table; a.lens = seq_lens; a.cu = cu_nodes;
  a.parents = parents; a.err = dev_err; a.n_layers = n_layers; a.nseq = nseq;
  a.total = total_nodes; a.H = H; a.Hq = num_q_heads; a.ps = k0.page_size;
  a.max_pages = max_pages; a.max_nodes = max_nodes; a.max_len = max_seq_len;
  a.scale = softmax_scale;
  const int64_t warps = static_cast<int64_t>(n_layers) * total_nodes * num_q_heads;
  const int64_t want = (warps + 7) / 8, cap = 152 * 8;
  const int blocks = static_cast<int>(want < cap ? want : cap);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (k0.bits == 8) tree_rows_kernel<8><<<blocks, 256, 0, cs>>>(a);
  else if (k0.bits == 6) tree_rows_kernel<6><<<blocks, 256, 0, cs>>>(a);
  else tree_rows_kernel<4><<<blocks, 256, 0, cs>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}
