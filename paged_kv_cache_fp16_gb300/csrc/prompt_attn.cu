// Causal attention over whole prompts: one warp per (token, query head), online softmax.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

struct PromptArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t qs, ks, vs;
  const int32_t* cu_q;
  const int32_t* cu_k;
  uint16_t* out;
  float* lse;
  int32_t* err;
  int nseq, total_q, total_k, max_q, max_k, Hq, H;
  float scale;
};

template <bool BF> __device__ __forceinline__ float to_f(uint16_t b) {
  if constexpr (BF) return __uint_as_float(static_cast<uint32_t>(b) << 16);
  else return h2f(b);
}
template <bool BF> __device__ __forceinline__ uint16_t from_f(float f) {
  if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  else return f2h(f);
}

template <bool BF, int D>
__global__ void __launch_bounds__(256) prompt_rows_kernel(const PromptArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t n_rows = static_cast<int64_t>(a.total_q) * a.Hq;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < n_rows;
       row += step) {
    const int t = static_cast<int>(row / a.Hq), j = static_cast<int>(row % a.Hq);
    const int s = find_seq_from(a.cu_q, a.nseq, t, 0);
    const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
    if (t < q0 || t >= q1) continue;
    if (q0 < 0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k || q1 - q0 > a.max_q ||
        k1 - k0 > a.max_k) {
      report(a.err, KVQ_DEVERR_INDEX);
      continue;
    }
    const int end = t - q0 + (k1 - k0) - (q1 - q0) + 1;   // keys seen
    const int h = j / (a.Hq / a.H);
    float qf[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      qf[e] = to_f<BF>(a.q[t * a.qs + static_cast<int64_t>(j) * D + lane * E + e]);
      o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < end; ++i) {
      const uint16_t* kr = a.k + (k0 + i) * a.ks + static_cast<int64_t>(h) * D + lane * E;
      const uint16_t* vr = a.v + (k0 + i) * a.vs + static_cast<int64_t>(h) * D + lane * E;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x = fmaf(qf[e], to_f<BF>(kr[e]), x);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(kFullMask, x, w);
      x *= a.scale;
      const float mn = fmaxf(m, x);
      const float f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(x - mn);
      l = l * f + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * to_f<BF>(vr[e]);
      m = mn;
    }
    const float inv = end > 0 ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      a.out[(static_cast<int64_t>(t) * a.Hq + j) * D + lane * E + e] = from_f<BF>(o[e] * inv);
    if (a.lse && lane == 0)
      a.lse[static_cast<int64_t>(t) * a.Hq + j] = end > 0 ? m + logf(l) : -INFINITY;
  }
}

template <bool BF>
void launch(const PromptArgs& a, int D, int blocks, cudaStream_t cs) {
  if (D == 256) prompt_rows_kernel<BF, 256><<<blocks, 256, 0, cs>>>(a);
  else if (D == 128) prompt_rows_kernel<BF, 128><<<blocks, 256, 0, cs>>>(a);
  else prompt_rows_kernel<BF, 64><<<blocks, 256, 0, cs>>>(a);
}

}  // namespace
}  // namespace kvq

extern "C" size_t kvq_prompt_attn_workspace(int nseq, int total_q, int num_q_heads,
                                            int num_kv_heads, int head_dim, int max_q,
                                            int max_k) {
  (void)head_dim;
  if (nseq < 1 || total_q < 0 || num_q_heads < 1 || num_kv_heads < 1 || max_q < 0 || max_k < 0)
    return 0;
  return 16;
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
  if (!std::isfinite(softmax_scale) || softmax_scale <= 0)
    return fail(KVQ_ERR_RANGE, "%s: softmax_scale is not a finite value > 0", fn);
  if (nseq == 0 || total_q == 0 || max_q == 0) return ok();
  if (!q || !cu_q || !cu_k || !out || !workspace || (total_k > 0 && (!k || !v)))
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      !aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(KVQ_ERR_ALIGN, "%s: a pointer is not 16-byte aligned (lse 4)", fn);
  const size_t need = kvq_prompt_attn_workspace(nseq, total_q, num_q_heads, num_kv_heads,
                                                head_dim, max_q, max_k);
  if (workspace_bytes < need)
    return fail(KVQ_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, workspace_bytes, need);
  PromptArgs a{q, k, v, q_stride, k_stride, v_stride, cu_q, cu_k, out, lse, dev_err, nseq, total_q,
               total_k, max_q, max_k, num_q_heads, num_kv_heads, softmax_scale};
  const int64_t warps = static_cast<int64_t>(total_q) * num_q_heads;
  const int64_t want = (warps + 7) / 8, cap = 152 * 8;
  const int blocks = static_cast<int>(want < cap ? want : cap);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == KVQ_BF16) launch<true>(a, head_dim, blocks, cs);
  else launch<false>(a, head_dim, blocks, cs);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}
