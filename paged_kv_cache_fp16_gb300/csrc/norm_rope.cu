// Per-head norm of queries and keys with the position rotation, one pass over the rows.
//
// For a row x of D values: y_d = x_d * rsqrt(mean_d x_d^2 + eps) * w_d, then pairs (a, b) of the
// first rotary_dim values turn by the angle positions[t] * inv_freq[i].  Written per element,
//   y'_d = r * (x_d * (w_d cos) + x_p * (+-w_p sin)),      r = rsqrt(mean x^2 + eps), p = partner
// so the two bracketed factors depend on the token and the lane's channels only: they are formed
// once per token and used by all of its heads, which leaves two multiply-adds and one multiply
// per element of a row.
//
// A row is held by D / 8 lanes (8 channels = 16 bytes each; the next power of two of lanes is set
// aside for it, so a warp holds 1, 2 or 4 rows of 256, 128 or 64 channels).  The mean is a
// shuffle tree over those lanes; the partner's values come by four more shuffles of the packed
// words (pairs half a row apart) or are the lane's own (interleaved).
//
// The angle in turns is position * phase mod 2^64 with the phase in units of 2^-64 turn: exact to
// 2^-33 turn for every 32-bit position.  Its sine and cosine are the hardware approximations of
// an argument already inside [-pi, pi], where their absolute error is at most 2^-21.2 (CUDA's
// bound for __sinf and __cosf there): a thousandth of half an fp16 step of the pair's magnitude,
// for a twentieth of the instructions of the accurate forms.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

struct NormRopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* qo;
  uint16_t* ko;
  int64_t qs, ks, qos, kos;   // elements per token
  const int32_t* pos;
  const uint64_t* phases;
  const float* qw;
  const float* kw;
  float eps;
  int tokens, Hq, H, D, rd;
  int rows_per_task, tasks_per_token;
};

__device__ __forceinline__ uint4 ld_v4(const void* p) {
  return *reinterpret_cast<const uint4*>(p);
}

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& v, float x[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float x[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a lane keeps for one token: its channels' own and partner factors, and where its partner is.
template <int LPR, bool INTER>
struct Lane {
  int sub;        // lane within the row
  bool live;      // holds channels (sub * 8 < D)
  bool rot;       // its channels are rotated (8 at a time: rotary_dim is a multiple of 16)
  int src;        // the lane that holds the partners
  float c[8], s[8];
};

template <int LPR, bool INTER>
__device__ __forceinline__ void token_factors(Lane<LPR, INTER>& L, const NormRopeArgs& a, int t) {
  const int64_t p = __ldg(a.pos + t);
  const int half = a.rd >> 1, d0 = L.sub * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) { L.c[e] = 1.f; L.s[e] = 0.f; }
  if (!L.rot) return;
  const int i0 = INTER ? (d0 >> 1) : (d0 < half ? d0 : d0 - half);
  const bool second = !INTER && d0 >= half;
#pragma unroll
  for (int i = 0; i < (INTER ? 4 : 8); ++i) {
    const uint64_t turn = static_cast<uint64_t>(p) * __ldg(a.phases + i0 + i) + 0x80000000ull;
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) *
                    1.4629180792671596e-9f;   // 2 pi / 2^32
    const float c = __cosf(x), s = __sinf(x);
    if constexpr (INTER) {
      L.c[2 * i] = L.c[2 * i + 1] = c;
      L.s[2 * i] = -s;
      L.s[2 * i + 1] = s;
    } else {
      L.c[i] = c;
      L.s[i] = second ? s : -s;
    }
  }
}

// The rows [0, n) at x (D apart) to y, with the norm's weights w (NULL: no norm).
template <bool BF, int LPR, bool INTER>
__device__ __forceinline__ void rows(const Lane<LPR, INTER>& L, const NormRopeArgs& a,
                                     const uint16_t* x, uint16_t* y, const float* w, int n,
                                     int n_max) {
  const int d0 = L.sub * 8;
  float wc[8], ws[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) { wc[e] = L.c[e]; ws[e] = L.s[e]; }
  if (w != nullptr && L.live) {
    const int half = a.rd >> 1;
    const int dp = INTER || !L.rot ? d0 : (d0 < half ? d0 + half : d0 - half);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      wc[e] *= __ldg(w + d0 + e);
      ws[e] *= __ldg(w + (INTER ? (d0 + (e ^ 1)) : (dp + e)));
    }
  }
  const float inv_d = 1.f / static_cast<float>(a.D);
  constexpr int U = 4;   // rows in flight per group of lanes
  for (int r0 = 0; r0 < n_max; r0 += U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (L.live && r0 + u < n) v[u] = ld_v4(x + static_cast<int64_t>(r0 + u) * a.D + d0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8], g[8];
      unpack8<BF>(v[u], f);
      float r = 1.f;
      if (w != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o, LPR);
        r = rsqrtf(fmaf(ss, inv_d, a.eps));
      }
      if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = L.rot ? f[e ^ 1] : 0.f;
      } else {
        uint4 pv;
        pv.x = __shfl_sync(kFullMask, v[u].x, L.src, LPR);
        pv.y = __shfl_sync(kFullMask, v[u].y, L.src, LPR);
        pv.z = __shfl_sync(kFullMask, v[u].z, L.src, LPR);
        pv.w = __shfl_sync(kFullMask, v[u].w, L.src, LPR);
        if (!L.rot) pv = make_uint4(0, 0, 0, 0);   // a zero partner: 0 * 0 adds nothing
        unpack8<BF>(pv, g);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaf(g[e], ws[e], f[e] * wc[e]) * r;
      if (L.live && r0 + u < n)
        *reinterpret_cast<uint4*>(y + static_cast<int64_t>(r0 + u) * a.D + d0) = pack8<BF>(f);
    }
  }
}

// A task is one token and rows_per_task of its Hq + H rows; groups of LPR lanes take tasks in
// turn.  Groups of one warp run the same number of steps, so every shuffle has all its lanes.
template <bool BF, int LPR, bool INTER>
__global__ void __launch_bounds__(256) norm_rope_kernel(const NormRopeArgs a) {
  Lane<LPR, INTER> L;
  const int lane = threadIdx.x & 31;
  L.sub = lane & (LPR - 1);
  L.live = L.sub * 8 < a.D;
  L.rot = L.sub * 8 < a.rd;
  const int hl = a.rd >> 4;   // lanes per half of the rotated part
  L.src = L.rot ? (L.sub < hl ? L.sub + hl : L.sub - hl) : L.sub;
  constexpr int GPW = 32 / LPR;
  const int64_t n_tasks = static_cast<int64_t>(a.tokens) * a.tasks_per_token;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x >> 5) * GPW;
  for (int64_t base = warp * GPW; base < n_tasks; base += step) {
    const int64_t task = base + lane / LPR;
    const bool on = task < n_tasks;
    const int64_t tk = on ? task : n_tasks - 1;
    const int t = static_cast<int>(tk / a.tasks_per_token);
    const int r0 = static_cast<int>(tk - static_cast<int64_t>(t) * a.tasks_per_token) *
                   a.rows_per_task;
    const int r1 = min(r0 + a.rows_per_task, a.Hq + a.H);
    token_factors(L, a, t);
    const int q0 = min(r0, a.Hq), q1 = min(r1, a.Hq);
    const int k0 = max(r0, a.Hq) - a.Hq, k1 = max(r1, a.Hq) - a.Hq;
    int nq = on ? q1 - q0 : 0, nk = on ? k1 - k0 : 0;
    int mq = nq, mk = nk;
    if constexpr (GPW > 1) {
      mq = __reduce_max_sync(kFullMask, nq);
      mk = __reduce_max_sync(kFullMask, nk);
    }
    rows<BF>(L, a, a.q + t * a.qs + static_cast<int64_t>(q0) * a.D,
             a.qo + t * a.qos + static_cast<int64_t>(q0) * a.D, a.qw, nq, mq);
    rows<BF>(L, a, a.k + t * a.ks + static_cast<int64_t>(k0) * a.D,
             a.ko + t * a.kos + static_cast<int64_t>(k0) * a.D, a.kw, nk, mk);
  }
}

template <bool BF, int LPR>
void launch(const NormRopeArgs& a, bool inter, int blocks, cudaStream_t cs) {
  if (inter) norm_rope_kernel<BF, LPR, true><<<blocks, 256, 0, cs>>>(a);
  else norm_rope_kernel<BF, LPR, false><<<blocks, 256, 0, cs>>>(a);
}

template <bool BF>
void launch_lanes(const NormRopeArgs& a, bool inter, int lpr, int blocks, cudaStream_t cs) {
  if (lpr == 32) launch<BF, 32>(a, inter, blocks, cs);
  else if (lpr == 16) launch<BF, 16>(a, inter, blocks, cs);
  else launch<BF, 8>(a, inter, blocks, cs);
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_rope_phases(const double* inv_freq, int n, uint64_t* phases) {
  using namespace kvq;
  if (n < 0 || n > 128) return fail(KVQ_ERR_RANGE, "kvq_rope_phases: n %d not in [0, 128]", n);
  if (n > 0 && (!inv_freq || !phases)) return fail(KVQ_ERR_NULL, "kvq_rope_phases: NULL pointer");
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i]) || inv_freq[i] < 0)
      return fail(KVQ_ERR_RANGE, "kvq_rope_phases: inv_freq[%d] is not a finite value >= 0", i);
  for (int i = 0; i < n; ++i) {
    // turns per position in extended precision; whole turns do not matter
    long double t = static_cast<long double>(inv_freq[i]) *
                    0.15915494309189533576888376337251436203L;
    t -= floorl(t);
    const long double u = floorl(t * 18446744073709551616.0L + 0.5L);
    phases[i] = u >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(u);
  }
  return ok();
}

extern "C" kvq_status kvq_qk_norm_rope(kvq_dtype dtype, const uint16_t* q, int64_t q_stride,
                                       const uint16_t* k, int64_t k_stride, uint16_t* q_out,
                                       int64_t q_out_stride, uint16_t* k_out,
                                       int64_t k_out_stride, int num_tokens, int num_q_heads,
                                       int num_kv_heads, int head_dim, int rotary_dim,
                                       int interleaved, const int32_t* positions,
                                       const uint64_t* phases, const float* q_weight,
                                       const float* k_weight, float eps, kvq_stream_t stream) {
  using namespace kvq;
  const char* fn = "kvq_qk_norm_rope";
  if (dtype != KVQ_F16 && dtype != KVQ_BF16)
    return fail(KVQ_ERR_SHAPE, "%s: dtype %d is neither KVQ_F16 nor KVQ_BF16", fn,
                static_cast<int>(dtype));
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads > 65535 || num_kv_heads > 65535)
    return fail(KVQ_ERR_SHAPE, "%s: %d query and %d KV heads not in [1, 65535]", fn, num_q_heads,
                num_kv_heads);
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(KVQ_ERR_SHAPE, "%s: head_dim %d is not a multiple of 8 in [8, 256]", fn, head_dim);
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16)
    return fail(KVQ_ERR_SHAPE, "%s: rotary_dim %d is not a multiple of 16 in [0, head_dim]", fn,
                rotary_dim);
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kw = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_stride < qw || q_out_stride < qw || k_stride < kw || k_out_stride < kw || q_stride % 8 ||
      q_out_stride % 8 || k_stride % 8 || k_out_stride % 8)
    return fail(KVQ_ERR_SHAPE, "%s: a token stride is below heads * head_dim or no multiple of 8",
                fn);
  if (num_tokens < 0) return fail(KVQ_ERR_RANGE, "%s: num_tokens %d < 0", fn, num_tokens);
  if (!std::isfinite(eps) || eps < 0) return fail(KVQ_ERR_RANGE, "%s: eps is not finite or < 0", fn);
  if (num_tokens == 0) return ok();
  if (!q || !k || !q_out || !k_out || !positions || (rotary_dim > 0 && !phases))
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(q_weight) || !aligned16(k_weight) ||
      (reinterpret_cast<uintptr_t>(phases) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return fail(KVQ_ERR_ALIGN, "%s: a pointer is not aligned (rows and weights 16 bytes)", fn);
  if ((q == q_out && q_stride != q_out_stride) || (k == k_out && k_stride != k_out_stride))
    return fail(KVQ_ERR_SHAPE, "%s: in place needs equal strides", fn);
  NormRopeArgs a;
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  a.qs = q_stride; a.ks = k_stride; a.qos = q_out_stride; a.kos = k_out_stride;
  a.pos = positions; a.phases = phases; a.qw = q_weight; a.kw = k_weight; a.eps = eps;
  a.tokens = num_tokens; a.Hq = num_q_heads; a.H = num_kv_heads; a.D = head_dim; a.rd = rotary_dim;
  const int lpr = head_dim > 128 ? 32 : head_dim > 64 ? 16 : 8;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  // Whole tokens per task when they fill the machine (the factors are then formed once per
  // token); with fewer, a token's rows go to several tasks, four at least (one batch of loads).
  const int64_t slots = static_cast<int64_t>(sms) * 64 * (32 / lpr);   // groups resident at once
  const int total = num_q_heads + num_kv_heads;
  int64_t split = slots / num_tokens;
  const int most = (total + 3) / 4;
  split = split < 1 ? 1 : split > most ? most : split;
  a.rows_per_task = static_cast<int>((total + split - 1) / split);
  a.tasks_per_token = (total + a.rows_per_task - 1) / a.rows_per_task;
  const int64_t groups = static_cast<int64_t>(num_tokens) * a.tasks_per_token;
  const int64_t warps = (groups + 32 / lpr - 1) / (32 / lpr);
  const int64_t want = (warps + 7) / 8, cap = static_cast<int64_t>(sms) * 8;
  const int blocks = static_cast<int>(want < cap ? want : cap);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == KVQ_BF16) launch_lanes<true>(a, interleaved != 0, lpr, blocks, cs);
  else launch_lanes<false>(a, interleaved != 0, lpr, blocks, cs);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}
