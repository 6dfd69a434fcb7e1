// Per-head norm of queries and keys with the position rotation, one pass over the rows.
//
// For a row x of D values: y_d = x_d * rsqrt(mean_d x_d^2 + eps) * w_d, then pairs (a, b) of the
// first rotary_dim values turn by the angle positions[t] * inv_freq[i].  Written per element,
//   y'_d = r * (x_d * (w_d cos) + x_p * (+-w_p sin)),      r = rsqrt(mean x^2 + eps), p = partner
// so the two bracketed factors depend on the token and the lane's channels only: they are formed
// once per token and used by all of its heads, which leaves two multiply-adds and one multiply
// per element of a row.
//
// A row is held by D / 8 lanes, 8 channels each (the next power of two of lanes is set aside for
// it, so a warp holds 1, 2 or 4 rows of 256, 128 or 64 channels).  A lane's channels are two runs
// of 4 so chosen that both channels of a pair are its own: for pairs half a rotated part apart,
// one run from each half; a row then costs two 8-byte loads and stores and no exchange but the
// mean's shuffle tree.  For neighbouring pairs the runs are neighbours too and move as 16 bytes
// (5,003 tokens of 40 rows of 64 channels: 17.1 us as two loads, 16.3 so).
//
// What bounds it is the arithmetic as much as the memory: 32,768 tokens of 28 rows of 256 channels
// (940 MB) would take 139 us at the copy rate.  Measured there: with the partner's channels
// fetched by shuffles and 16-byte loads 202 us (126 registers, 2 blocks per SM), in this form 155.
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
#include "kvq_tc5.cuh"

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

// Two 16-bit values as float32.
template <bool BF>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  if constexpr (BF) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  }
}

// Where a lane's two runs of 4 channels start, and what their pairs turn by.
struct Lane {
  int a, b;       // channels a .. a+3 and b .. b+3
  int pair0;      // its first pair's number
  bool live;      // holds channels
  bool rot;       // they are rotated (8 at a time: rotary_dim is a multiple of 16)
};

// A lane's 8 values are held as the first of its four pairs, then the second (e < 4 and e >= 4):
// with INTER pair i is the neighbours 2i, 2i + 1 of its 8 channels, otherwise one value of each
// run.  The factors: y_e = x_e own[e] + x_(e^4) part[e].
template <bool INTER>
__device__ __forceinline__ void factors(const Lane& L, const float c[4], const float s[4],
                                        const float* w, uint64_t own[4], uint64_t part[4]) {
  float wt[8], o[8], p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    wt[e] = w != nullptr && L.live
                ? __ldg(w + (INTER ? L.a + 2 * (e & 3) + (e >> 2) : e < 4 ? L.a + e : L.b + e - 4))
                : 1.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    o[e] = wt[e] * c[e & 3];
    p[e] = e < 4 ? -(wt[e + 4] * s[e]) : wt[e - 4] * s[e - 4];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    own[i] = tc5::pair(__float_as_uint(o[2 * i]), __float_as_uint(o[2 * i + 1]));
    part[i] = tc5::pair(__float_as_uint(p[2 * i]), __float_as_uint(p[2 * i + 1]));
  }
}

constexpr int kThreads = 128;
constexpr int kU = 4;   // rows in flight per group of lanes

// Rows r0 .. r0 + kU - 1 of the n at x (D apart).
template <bool INTER>
__device__ __forceinline__ void load_rows(const Lane& L, const NormRopeArgs& a, const uint16_t* x,
                                          int r0, int n, uint2 v[kU][2]) {
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    v[u][0] = v[u][1] = make_uint2(0, 0);
    if (L.live && r0 + u < n) {
      const uint16_t* p = x + static_cast<int64_t>(r0 + u) * a.D;
      if constexpr (INTER) {   // the runs are neighbours
        const uint4 w = *reinterpret_cast<const uint4*>(p + L.a);
        v[u][0] = make_uint2(w.x, w.y);
        v[u][1] = make_uint2(w.z, w.w);
      } else {
        v[u][0] = *reinterpret_cast<const uint2*>(p + L.a);
        v[u][1] = *reinterpret_cast<const uint2*>(p + L.b);
      }
    }
  }
}

// The rows [0, n) at x, of which v holds the first batch, to y; NORM: divided by their root mean
// square.
template <bool BF, int LPR, bool INTER, bool NORM>
__device__ __forceinline__ void rows(const Lane& L, const NormRopeArgs& a, const uint16_t* x,
                                     uint16_t* y, const uint64_t own[4], const uint64_t part[4],
                                     int n, int n_max, uint2 v[kU][2]) {
  const float inv_d = 1.f / static_cast<float>(a.D);
#pragma unroll 1
  for (int r0 = 0; r0 < n_max; r0 += kU) {
    if (r0 > 0) load_rows<INTER>(L, a, x, r0, n, v);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float f[8];
      if constexpr (INTER) {
        unpack2<BF>(v[u][0].x, f[0], f[4]);
        unpack2<BF>(v[u][0].y, f[1], f[5]);
        unpack2<BF>(v[u][1].x, f[2], f[6]);
        unpack2<BF>(v[u][1].y, f[3], f[7]);
      } else {
        unpack2<BF>(v[u][0].x, f[0], f[1]);
        unpack2<BF>(v[u][0].y, f[2], f[3]);
        unpack2<BF>(v[u][1].x, f[4], f[5]);
        unpack2<BF>(v[u][1].y, f[6], f[7]);
      }
      uint64_t f2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f2[i] = tc5::pair(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
      uint64_t y2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y2[i] = tc5::fma2(f2[i ^ 2], part[i], tc5::mul2(f2[i], own[i]));
      if (!L.rot) {   // (a partner times 0 could still be a NaN)
#pragma unroll
        for (int i = 0; i < 4; ++i) y2[i] = tc5::mul2(f2[i], own[i]);
      }
      if constexpr (NORM) {
        uint64_t ss2 = tc5::mul2(f2[0], f2[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) ss2 = tc5::fma2(f2[i], f2[i], ss2);
        float s0, s1;
        tc5::unpair(ss2, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o, LPR);
        const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
        const uint64_t r2 = tc5::pair(__float_as_uint(r), __float_as_uint(r));
#pragma unroll
        for (int i = 0; i < 4; ++i) y2[i] = tc5::mul2(y2[i], r2);
      }
      if (L.live && r0 + u < n) {
        float g[8];
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) tc5::unpair(y2[i], g[2 * i], g[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = INTER ? tc5::pack2<BF>(g[i], g[i + 4]) : tc5::pack2<BF>(g[2 * i], g[2 * i + 1]);
        uint16_t* p = y + static_cast<int64_t>(r0 + u) * a.D;
        if constexpr (INTER) {
          *reinterpret_cast<uint4*>(p + L.a) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          *reinterpret_cast<uint2*>(p + L.a) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(p + L.b) = make_uint2(w[2], w[3]);
        }
      }
    }
  }
}

template <bool BF, int LPR, bool INTER>
__device__ __forceinline__ void rows_of(const Lane& L, const NormRopeArgs& a, const float c[4],
                                        const float s[4], const uint16_t* x, uint16_t* y,
                                        const float* w, int n, int n_max, uint2 v[kU][2]) {
  uint64_t own[4], part[4];
  factors<INTER>(L, c, s, w, own, part);
  if (w != nullptr) rows<BF, LPR, INTER, true>(L, a, x, y, own, part, n, n_max, v);
  else rows<BF, LPR, INTER, false>(L, a, x, y, own, part, n, n_max, v);
}

// 64 registers (and 68 to 92 bytes of spills) and 32 warps per SM: loads in flight and other warps'
// arithmetic cover each other.  32,768 tokens: 155 us, 6.05 TB/s (24 warps 162 us; 40 warps, which
// spill far more, 238 us).
template <bool BF, int LPR, bool INTER>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) norm_rope_kernel(const NormRopeArgs a) {
  Lane L;
  const int lane = threadIdx.x & 31, sub = lane & (LPR - 1), half = a.rd >> 1;
  L.live = sub * 8 < a.D;
  L.rot = sub * 8 < a.rd;
  L.a = INTER || !L.rot ? sub * 8 : sub * 4;
  L.b = INTER || !L.rot ? sub * 8 + 4 : half + sub * 4;
  L.pair0 = sub * 4;
  constexpr int GPW = 32 / LPR;
  // tasks fit 32 bits: a token has several only where tokens are few
  const uint32_t n_tasks = static_cast<uint32_t>(a.tokens) * a.tasks_per_token;
  const uint32_t warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const uint32_t step = (gridDim.x * blockDim.x >> 5) * GPW;
  for (uint32_t base = warp * GPW; base < n_tasks; base += step) {
    const uint32_t task = base + lane / LPR;
    const bool on = task < n_tasks;
    const uint32_t tk = on ? task : n_tasks - 1;
    const int t = a.tasks_per_token == 1 ? tk : tk / static_cast<uint32_t>(a.tasks_per_token);
    const int r0 = static_cast<int>(tk - static_cast<uint32_t>(t) * a.tasks_per_token) *
                   a.rows_per_task;
    const int r1 = min(r0 + a.rows_per_task, a.Hq + a.H);
    const int q0 = min(r0, a.Hq), q1 = min(r1, a.Hq);
    const int k0 = max(r0, a.Hq) - a.Hq, k1 = max(r1, a.Hq) - a.Hq;
    const int nq = on ? q1 - q0 : 0, nk = on ? k1 - k0 : 0;
    int mq = nq, mk = nk;
    if constexpr (GPW > 1) {
      mq = __reduce_max_sync(kFullMask, nq);
      mk = __reduce_max_sync(kFullMask, nk);
    }
    const uint16_t* xq = a.q + t * a.qs + static_cast<int64_t>(q0) * a.D;
    const uint16_t* xk = a.k + t * a.ks + static_cast<int64_t>(k0) * a.D;
    uint2 v[kU][2];   // the first rows are on their way while the factors are formed
    if (mq > 0) load_rows<INTER>(L, a, xq, 0, nq, v);
    else load_rows<INTER>(L, a, xk, 0, nk, v);
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (L.rot) {
      const int64_t p = __ldg(a.pos + t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t turn = static_cast<uint64_t>(p) * __ldg(a.phases + L.pair0 + i) + 0x80000000ull;
        const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) *
                        1.4629180792671596e-9f;   // 2 pi / 2^32
        c[i] = __cosf(x);
        s[i] = __sinf(x);
      }
    }
    if (mq > 0) {
      rows_of<BF, LPR, INTER>(L, a, c, s, xq, a.qo + t * a.qos + static_cast<int64_t>(q0) * a.D,
                              a.qw, nq, mq, v);
      if (mk > 0) load_rows<INTER>(L, a, xk, 0, nk, v);
    }
    if (mk > 0)
      rows_of<BF, LPR, INTER>(L, a, c, s, xk, a.ko + t * a.kos + static_cast<int64_t>(k0) * a.D,
                              a.kw, nk, mk, v);
  }
}

template <bool BF, int LPR>
void launch(const NormRopeArgs& a, bool inter, int blocks, cudaStream_t cs) {
  if (inter) norm_rope_kernel<BF, LPR, true><<<blocks, kThreads, 0, cs>>>(a);
  else norm_rope_kernel<BF, LPR, false><<<blocks, kThreads, 0, cs>>>(a);
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
  const int64_t slots = static_cast<int64_t>(sms) * 32 * (32 / lpr);   // groups resident at once
  const int total = num_q_heads + num_kv_heads;
  int64_t split = slots / num_tokens;
  const int most = (total + 3) / 4;
  split = split < 1 ? 1 : split > most ? most : split;
  a.rows_per_task = static_cast<int>((total + split - 1) / split);
  a.tasks_per_token = (total + a.rows_per_task - 1) / a.rows_per_task;
  const int64_t groups = static_cast<int64_t>(num_tokens) * a.tasks_per_token;
  const int64_t warps = (groups + 32 / lpr - 1) / (32 / lpr);
  constexpr int kWarps = kThreads / 32;
  const int64_t want = (warps + kWarps - 1) / kWarps;
  const int64_t cap = static_cast<int64_t>(sms) * (64 / kWarps);
  const int blocks = static_cast<int>(want < cap ? want : cap);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == KVQ_BF16) launch_lanes<true>(a, interleaved != 0, lpr, blocks, cs);
  else launch_lanes<false>(a, interleaved != 0, lpr, blocks, cs);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}
