/*
 * kvq.h -- C ABI of libkvq: quantized paged KV cache kernels for NVIDIA GB300 (sm_103a).
 *
 * Operations (each defined on the page cited at its declaration):
 *   kvq_quant_pack_paged   symmetric per-token-per-head quantize + pack into paged storage
 *   kvq_dequant_paged      gather + unpack + dequantize back to fp16
 *   kivi_quant_dequant     KIVI asymmetric group quantize->dequantize, in place
 *   kvq_decode_attn        decode attention that reads the packed pages directly
 *   kvq_append_decode_attn one decode step: append the new token, then attend, in one launch
 *   kivi_pack, kivi_decode_attn   packed KIVI storage and decode attention over it
 *   kivi_update, kivi_trim, kivi_packed_update, kivi_packed_trim   the KIVI cache protocol
 *   kvq_*_side             fp16 attention sinks and outlier side channel on the symmetric path
 *   kvq_qk_norm_rope       per-head norm of queries and keys with the position rotation
 *   kvq_prompt_attn        causal attention over whole prompts, packed sequences
 *   kvq_tree_attn, kvq_tree_commit   attention of drafted tokens over the packed pages, and the
 *                          move of the accepted ones into place
 *   kvq_beam_select, kvq_table_update, kvq_table_compact, kvq_beam_attn   beam search: the next beams,
 *                          tables that share pages, and attention that reads a shared prefix once
 * plus host helpers: packed_dim, the KIVI residual boundary, and a page allocator.
 *
 * Conventions shared by every entry point
 *   - The caller owns all memory.  The library never allocates or frees device memory and never
 *     synchronizes a stream.  Pointers documented "device" must be device (or managed) memory;
 *     "host" pointers are read before the call returns.
 *   - fp16 values are passed as their 16-bit patterns (uint16_t).
 *   - Every GPU entry point validates its arguments on the host first and returns a status
 *     without launching anything if they are invalid.  Otherwise it enqueues its kernels on
 *     `stream` (NULL = the legacy default stream) and returns KVQ_OK, or KVQ_ERR_CUDA if a launch
 *     was rejected.  Asynchronous device faults surface at the caller's next synchronization.
 *   - Kernels that read a page table check every page id they use against the pool size.  An id
 *     outside [0, num_pages) or a logical page beyond max_pages is skipped (nothing is read or
 *     written for that row) and, if `dev_err` is non-NULL, bit KVQ_DEVERR_PAGE_RANGE is OR-ed
 *     into *dev_err (device int32, caller zeroes it).  The kernels never trap.
 *   - kvq_last_error() returns a thread-local message describing the last non-OK status.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define KVQ_API __attribute__((visibility("default")))
#else
#define KVQ_API
#endif

/* Same object as cudaStream_t. */
typedef struct CUstream_st* kvq_stream_t;

typedef enum kvq_status {
  KVQ_OK = 0,
  KVQ_ERR_BITS = 1,      /* bit width not in {8, 6, 4} (the explicit width table)            */
  KVQ_ERR_SHAPE = 2,     /* head_dim / heads / group / range shape not supported              */
  KVQ_ERR_NULL = 3,      /* a required pointer is NULL                                        */
  KVQ_ERR_ALIGN = 4,     /* a device pointer is not 16-byte aligned                           */
  KVQ_ERR_RANGE = 5,     /* a count or index is out of range                                  */
  KVQ_ERR_CUDA = 6,      /* a CUDA launch or query failed                                     */
  KVQ_ERR_NOMEM = 7,     /* the host page allocator has too few free pages                    */
  KVQ_ERR_WORKSPACE = 8  /* the caller's workspace is too small                               */
} kvq_status;

/* Bits OR-ed into the optional device error word. */
#define KVQ_DEVERR_PAGE_RANGE 1  /* a page id or logical page was out of range (row skipped)   */
#define KVQ_DEVERR_TIMEOUT 2     /* a bounded wait for an asynchronous copy gave up (the
                                    affected output is invalid; the kernel returned normally)  */
#define KVQ_DEVERR_INDEX 4       /* a length, offset, parent or node number in device memory
                                    contradicts the call's bounds (what it concerns is skipped) */
#define KVQ_DEVERR_NO_PAGES 8    /* fewer free pages than a table update needs (it changed nothing) */

/* Maximum number of tensors one quant/dequant/KIVI call may batch, and of layers per decode
 * attention call. */
#define KVQ_MAX_TENSORS 64

/*
 * One page pool: the packed storage of one (layer, K-or-V) tensor.
 *   codes  : device uint8  [num_pages][num_heads][page_size][packed_dim(head_dim, bits)]
 *   scales : device fp16   [num_pages][num_heads][page_size]  (one scale per token per head)
 * Token `pos` of sequence `s` lives in physical page page_table[s * max_pages + pos / page_size],
 * slot pos % page_size.  Both arrays must be 16-byte aligned.  Within one page, the rows of one
 * head are contiguous (page_size * packed_dim bytes).
 */
typedef struct kvq_pool {
  int32_t bits;       /* 8, 6 or 4 */
  int32_t num_heads;  /* KV heads H */
  int32_t head_dim;   /* D <= 256 with kvq_packed_dim(D, bits) > 0: any D at q8, even at q4,
                         a multiple of 4 at q6 (the decode attention takes D = 256 only) */
  int32_t page_size;  /* tokens per page, >= 1 */
  int64_t num_pages;
  uint8_t* codes;
  uint16_t* scales;
} kvq_pool;

/* ---------------------------------------------------------------------------------------------
 * Host helpers
 * ------------------------------------------------------------------------------------------ */

/* Library version string. */
KVQ_API const char* kvq_version(void);

/* Thread-local message for the last non-OK status returned on this thread ("" if none). */
KVQ_API const char* kvq_last_error(void);

/* Name of a status code. */
KVQ_API const char* kvq_status_string(kvq_status status);

/*
 * The address under which kernels read page-locked host memory (cudaHostAlloc, or
 * cudaHostRegister with the mapped flag; on systems with unified addressing all page-locked memory
 * is mapped).  Any entry point documented to take "device" input may be given this address: its
 * kernels then read the host memory directly over the host link (NVLink-C2C on Grace systems)
 * instead of the caller copying it to the device first.  A device or managed pointer is returned
 * as is; other memory is refused with KVQ_ERR_RANGE (no kernel ever sees an unmapped address).
 * No counterpart on the pages: a host-memory convenience of this library.
 */
KVQ_API kvq_status kvq_host_device_view(const void* host_ptr, void** device_ptr);

/*
 * Bytes per packed row.  MTPLX pull request #267, "feat(kv-cache): add q6 paged KV
 * quantization", description, packed_dim sentence: packed_dim(D, 6) = D*3/4 and q6 needs
 * D % 4 == 0; q8 stores one code per byte, q4 two per byte (D % 2 == 0).
 * Returns -1 for an unknown width or an unsupported D (no error state is set).
 */
KVQ_API int kvq_packed_dim(int head_dim, int bits);

/*
 * KIVI residual-window boundary.  VeloxQuant-MLX source page "veloxquant_mlx.cache.kivi_cache",
 * KIVIKVCache._quantization_boundary: the tokens older than the newest `residual_length`,
 * snapped down to a multiple of `group_size`: ((max(0, offset - residual_length)) / group_size)
 * * group_size.  Returns -1 if group_size < 1 or residual_length < 0.
 */
KVQ_API int kivi_boundary(int offset, int residual_length, int group_size);

/*
 * Host page allocator over page ids [0, num_pages) (a LIFO free list; not thread-safe).
 * The pages themselves are the caller's kvq_pool memory; this only hands out ids.
 * MTPLX pull request #267, description: cache allocation is width-generic through packed_dim --
 * the allocator deals in pages, never in bytes.
 */
typedef struct kvq_allocator kvq_allocator;

/* Returns NULL on bad size or host allocation failure. */
KVQ_API kvq_allocator* kvq_alloc_create(int64_t num_pages);
KVQ_API void kvq_alloc_destroy(kvq_allocator* a);
KVQ_API int64_t kvq_alloc_free_count(const kvq_allocator* a);

/* Take n page ids into out_ids (host int32[n]).  All or nothing: KVQ_ERR_NOMEM if fewer than n
 * are free (nothing taken). */
KVQ_API kvq_status kvq_alloc_pages(kvq_allocator* a, int64_t n, int32_t* out_ids);

/* Return n page ids.  KVQ_ERR_RANGE (nothing returned) if an id is out of range, not currently
 * allocated, or repeated in `ids`. */
KVQ_API kvq_status kvq_free_pages(kvq_allocator* a, int64_t n, const int32_t* ids);

/*
 * Map the pages that an append of new_tokens[s] tokens at position cur_len[s] needs, for every
 * sequence s: every logical page in [cur_len[s] / page_size, ceil((cur_len[s] + new_tokens[s]) /
 * page_size)) whose entry in the host table page_table[s * max_pages + p] is negative gets a
 * fresh page id.  Entries already >= 0 are kept (a partially filled tail page is appended into).
 * All or nothing: on KVQ_ERR_NOMEM or KVQ_ERR_RANGE (a page beyond max_pages) the table is left
 * unchanged.  The caller then copies the table to the device.
 */
KVQ_API kvq_status kvq_table_reserve(kvq_allocator* a, int32_t* page_table, int max_pages, int page_size,
                             const int32_t* cur_len, const int32_t* new_tokens, int nseq);

/* ---------------------------------------------------------------------------------------------
 * Quantize + pack into pages
 * ------------------------------------------------------------------------------------------ */

/*
 * MTPLX pull request #267, "feat(kv-cache): add q6 paged KV quantization", description:
 * symmetric per-token-per-head quantizer with one fp16 scale per row, qmax 127 / 31 / 7 for
 * 8 / 6 / 4 bits (bit-width table paragraph); q6 codes biased by +32 and packed four per three
 * bytes, byte0 = u0 | (u1 & 3) << 6, byte1 = (u1 >> 2) | (u2 & 15) << 4,
 * byte2 = (u2 >> 4) | (u3 & 63) << 2 (byte-layout formula).
 *
 * Per row x (one token, one KV head, D fp16):
 *   scale = fp16_rne(float32(max_d |x_d|) / qmax)           (IEEE float32 divide)
 *   c_d   = clamp(rint_half_even(float32(x_d) / float32(scale)), -qmax, qmax), or 0 if scale == 0
 *   q8: byte = int8 two's complement of c; q6: u = c + 32, 4 -> 3 bytes as above;
 *   q4: u = c + 8, element 2i in the low nibble of byte i.
 *
 * pools      host array [n_tensors]: the destination pools (all with the same bits, num_heads,
 *            head_dim, page_size).
 * x          host array [n_tensors] of device pointers, each fp16 [total_new_tokens][H][D],
 *            16-byte aligned: the new rows of every sequence, sequence s owning rows
 *            cu_new_tokens[s] .. cu_new_tokens[s+1]-1, which are its tokens start_pos[s],
 *            start_pos[s]+1, ...
 * page_table device int32 [nseq][max_pages], shared by every tensor of the call.
 * cu_new_tokens device int32 [nseq+1], non-decreasing, cu[0] = 0, cu[nseq] = total_new_tokens.
 * start_pos  device int32 [nseq].
 * dev_err    optional device int32 error word (see the file header).
 * Rows are independent; a row's packed bytes and scale are written whole.  Two rows of one call
 * mapping to the same (page, slot) race (a caller error).
 * Head dims that are not a multiple of 16 run a one-warp-per-row kernel (same arithmetic).
 * Errors: KVQ_ERR_BITS, KVQ_ERR_SHAPE (kvq_packed_dim(D, bits) < 1, D > 256, mismatched pools),
 * KVQ_ERR_NULL, KVQ_ERR_ALIGN, KVQ_ERR_RANGE (n_tensors not in [1, KVQ_MAX_TENSORS], nseq < 0,
 * total_new_tokens < 0, max_pages < 1), KVQ_ERR_CUDA.
 */
KVQ_API kvq_status kvq_quant_pack_paged(const kvq_pool* pools, const uint16_t* const* x, int n_tensors,
                                const int32_t* page_table, int max_pages,
                                const int32_t* cu_new_tokens, const int32_t* start_pos, int nseq,
                                int total_new_tokens, int32_t* dev_err, kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Gather + unpack + dequantize
 * ------------------------------------------------------------------------------------------ */

/*
 * MTPLX pull request #267, description: dequantization runs over the active window; the inverse
 * of kvq_quant_pack_paged: x_hat_d = fp16_rne(float32(c_d) * float32(scale)) (the product is
 * exact in float32).
 *
 * Same addressing as kvq_quant_pack_paged: out[i] (host array of device pointers, each fp16
 * [total_tokens][H][D], 16-byte aligned) receives rows cu_tokens[s] .. cu_tokens[s+1]-1 =
 * tokens start_pos[s], start_pos[s]+1, ... of sequence s.  Rows whose page id is out of range
 * are left untouched.  Errors as for kvq_quant_pack_paged.
 */
KVQ_API kvq_status kvq_dequant_paged(const kvq_pool* pools, uint16_t* const* out, int n_tensors,
                             const int32_t* page_table, int max_pages, const int32_t* cu_tokens,
                             const int32_t* start_pos, int nseq, int total_tokens,
                             int32_t* dev_err, kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * KIVI group quantize -> dequantize, in place
 * ------------------------------------------------------------------------------------------ */

/*
 * VeloxQuant-MLX source page "veloxquant_mlx.cache.kivi_cache", KIVIKVCache._quant_dequant_along
 * and update_and_fetch.  For every tensor i, the token slice [lo, hi) of x[i] (device fp16
 * [B][H][S][D], 16-byte aligned, modified in place) is round-tripped in float32:
 *   keys   (is_key[i] != 0): per channel, groups of group_size tokens starting at lo;
 *   values (is_key[i] == 0): per token, groups of group_size channels starting at channel 0;
 *   a ragged last group uses only its real elements (the page pads it with its last element,
 *   which leaves min and max unchanged);
 *   scale = max((gmax - gmin) / levels, eps); c = clamp(rint_half_even((x - gmin) / scale), 0,
 *   levels); y = fp16_rne((c * scale) + gmin) with two roundings (no fused multiply-add).
 * is_key     host int32 [n_tensors].
 * levels     2^b - 1 for b-bit KIVI (the page's default b = 2 gives 3); >= 1.
 * eps        the page's 1e-8 (as float32).
 * Use kivi_boundary() for hi and the previous frontier for lo (update_and_fetch).
 * Errors: KVQ_ERR_SHAPE (D % 8, D > 256, 0 <= lo <= hi <= S violated, group_size < 1,
 * levels < 1), KVQ_ERR_NULL, KVQ_ERR_ALIGN, KVQ_ERR_RANGE (n_tensors, B, H, S), KVQ_ERR_CUDA.
 * An empty slice (lo == hi) launches nothing and returns KVQ_OK.
 */
KVQ_API kvq_status kivi_quant_dequant(uint16_t* const* x, const int32_t* is_key, int n_tensors, int B,
                              int H, int S, int D, int lo, int hi, int group_size, int levels,
                              float eps, kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Decode attention over packed pages
 * ------------------------------------------------------------------------------------------ */

/*
 * Attention for one decode query per sequence over that sequence's whole packed cache, reading
 * the packed pages directly (MTPLX pull request #267, description: the reference path instead
 * dequantizes to fp16 and runs SDPA; this computes the same function without materialising fp16).
 * For layer l, sequence s, query head j (KV head h = j / (Hq / H)):
 *   s_t = softmax_scale * sum_d q[l][s][j][d] * k_hat_t[d],   t in [0, seq_lens[s])
 *   out[l][s][j][:] = sum_t softmax(s)_t * v_hat_t[:]    (float32 accumulation)
 * where k_hat, v_hat are the fp16 dequantized rows of k_pools[l], v_pools[l].
 * k_pools, v_pools host arrays [n_layers] (same bits/H/D/page_size for all).
 * q          device fp16 [n_layers][nseq][num_q_heads][D], 16-byte aligned.
 * out        device float32 [n_layers][nseq][num_q_heads][D]; a sequence of length 0 gets 0.
 * page_table device int32 [nseq][max_pages] (shared by all layers); seq_lens device int32 [nseq].
 * max_seq_len host upper bound on seq_lens (sizes the split over tokens).
 * workspace  device scratch of at least kvq_decode_attn_workspace(...) bytes, 16-byte aligned;
 *            its contents need no initialisation and are garbage afterwards.
 * Errors: KVQ_ERR_SHAPE (num_q_heads % H, num_q_heads / H > 8, D != 256 for now), KVQ_ERR_BITS,
 * KVQ_ERR_NULL, KVQ_ERR_ALIGN, KVQ_ERR_RANGE, KVQ_ERR_WORKSPACE, KVQ_ERR_CUDA.
 */
KVQ_API size_t kvq_decode_attn_workspace(int n_layers, int nseq, int num_kv_heads, int num_q_heads,
                                 int head_dim, int page_size, int max_seq_len);

KVQ_API kvq_status kvq_decode_attn(const kvq_pool* k_pools, const kvq_pool* v_pools, int n_layers,
                           const uint16_t* q, int num_q_heads, const int32_t* page_table,
                           int max_pages, const int32_t* seq_lens, int nseq, int max_seq_len,
                           float softmax_scale, float* out, void* workspace,
                           size_t workspace_bytes, int32_t* dev_err, kvq_stream_t stream);

/*
 * One decode step with the append fused in: for every sequence s, quantize its new token's K and
 * V rows (k_new[l], v_new[l]: device fp16 [nseq][H][256] per layer, 16-byte aligned) exactly as
 * kvq_quant_pack_paged would, store them at position seq_lens[s] of the pools (page
 * page_table[s][seq_lens[s] / page_size], which the caller has mapped, e.g. with
 * kvq_table_reserve), and attend over the seq_lens[s] + 1 tokens that result -- one launch (plus
 * the split merge).  MTPLX pull request #267, description: quantize on write, and attention over
 * the active window; the pages run the two as separate steps (write, then dequantize + SDPA).
 * seq_lens holds the lengths BEFORE the append and is not modified: the caller advances it.
 * max_seq_len bounds seq_lens[s] + 1.  The page size must be a multiple of 16.  Other arguments,
 * the workspace (kvq_decode_attn_workspace with that max_seq_len) and the errors are those of
 * kvq_decode_attn; the pools are written, so they must not be read by other work in flight.
 */
KVQ_API kvq_status kvq_append_decode_attn(const kvq_pool* k_pools, const kvq_pool* v_pools,
                                          int n_layers, const uint16_t* const* k_new,
                                          const uint16_t* const* v_new, const uint16_t* q,
                                          int num_q_heads, const int32_t* page_table,
                                          int max_pages, const int32_t* seq_lens, int nseq,
                                          int max_seq_len, float softmax_scale, float* out,
                                          void* workspace, size_t workspace_bytes,
                                          int32_t* dev_err, kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * fp16 side channels: attention sinks and dense-and-sparse outliers
 * ------------------------------------------------------------------------------------------ */

#define KVQ_MAX_OUTLIERS 8
#define KVQ_MAX_SINKS 16

/*
 * VeloxQuant-MLX API docs, "veloxquant_mlx.cache.kvquant_cache module": per-vector
 * dense-and-sparse outlier isolation with an fp16 side channel (value + position index), and
 * Attention Sink-Aware quantization (the first n_sink tokens of a sequence restored to exact
 * fp16), applied to the symmetric quantizer above.  One kvq_side accompanies one kvq_pool:
 *   a row's n_outlier largest-magnitude elements (ties: the lower position) are stored as fp16
 *   value + uint8 position, ascending by position, in out_val / out_idx at the row's physical
 *   index; the rest of the row (outliers set to 0) is quantized as usual -- its scale comes from
 *   the (n_outlier + 1)-th largest magnitude and the outlier positions hold code 0;
 *   rows at positions < n_sink are also copied exactly into sink, which dequantization and
 *   attention read instead of the pages.
 * The page's fraction 0.01 gives n_outlier = ceil(0.01 * head_dim) (3 at 256).
 */
typedef struct kvq_side {
  int32_t n_outlier;  /* outliers per row, 0..KVQ_MAX_OUTLIERS, < head_dim */
  int32_t n_sink;     /* sink tokens per sequence, 0..KVQ_MAX_SINKS */
  int32_t max_seqs;   /* sequences the sink buffer holds (>= nseq of every call) */
  uint16_t* out_val;  /* fp16 [num_pages][H][page_size][n_outlier], 16-byte aligned */
  uint8_t* out_idx;   /* uint8 [num_pages][H][page_size][n_outlier], 16-byte aligned */
  uint16_t* sink;     /* fp16 [max_seqs][n_sink][H][D], 16-byte aligned */
} kvq_side;

/*
 * kvq_quant_pack_paged with the side channels: same arguments plus sides[i] for pools[i]
 * (uniform n_outlier and n_sink).  Any head_dim a pool accepts.  Errors: those of
 * kvq_quant_pack_paged, KVQ_ERR_RANGE (n_outlier, n_sink, max_seqs < nseq).
 */
KVQ_API kvq_status kvq_quant_pack_paged_side(const kvq_pool* pools, const kvq_side* sides,
                                             const uint16_t* const* x, int n_tensors,
                                             const int32_t* page_table, int max_pages,
                                             const int32_t* cu_new_tokens,
                                             const int32_t* start_pos, int nseq,
                                             int total_new_tokens, int32_t* dev_err,
                                             kvq_stream_t stream);

/* kvq_dequant_paged with the side channels: outliers written back, sink rows exact. */
KVQ_API kvq_status kvq_dequant_paged_side(const kvq_pool* pools, const kvq_side* sides,
                                          uint16_t* const* out, int n_tensors,
                                          const int32_t* page_table, int max_pages,
                                          const int32_t* cu_tokens, const int32_t* start_pos,
                                          int nseq, int total_tokens, int32_t* dev_err,
                                          kvq_stream_t stream);

/*
 * kvq_decode_attn over pools with side channels: the keys and values of a row are the dense
 * reconstruction with its outliers written back, and the sink positions (< n_sink) use the exact
 * fp16 rows of the sink buffer.  k_sides[l] / v_sides[l] accompany k_pools[l] / v_pools[l]
 * (uniform n_outlier and n_sink; max_seqs >= nseq).  The page size must be a multiple of 16.
 * Other arguments, the workspace and the errors are those of kvq_decode_attn.
 */
KVQ_API kvq_status kvq_decode_attn_side(const kvq_pool* k_pools, const kvq_pool* v_pools,
                                        const kvq_side* k_sides, const kvq_side* v_sides,
                                        int n_layers, const uint16_t* q, int num_q_heads,
                                        const int32_t* page_table, int max_pages,
                                        const int32_t* seq_lens, int nseq, int max_seq_len,
                                        float softmax_scale, float* out, void* workspace,
                                        size_t workspace_bytes, int32_t* dev_err,
                                        kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Packed KIVI storage and decode attention over it
 * ------------------------------------------------------------------------------------------ */

/*
 * VeloxQuant-MLX source page "veloxquant_mlx.cache.kivi_cache": the page keeps the KIVI cache in
 * fp16 and estimates the bytes of a packed form (module docstring, _quantized_bytes,
 * _account_bytes): b-bit codes plus an fp16 (scale, zero) pair per group -- per (token group,
 * channel) for keys, per (token, channel group) for values.  This is that packed form, for one
 * layer of a [batch][heads][capacity][head_dim] cache:
 *   k_codes [B][H][capacity][D*bits/8]   k_scale, k_zero fp16 [B][H][capacity/gs][D]
 *   v_codes [B][H][capacity][D*bits/8]   v_scale, v_zero fp16 [B][H][capacity][D/gs]
 * zero = the group minimum (an fp16 value), scale = fp16(max((max - min) / levels, eps)) with
 * levels = 2^bits - 1, code = clamp(rint((x - zero) / scale), 0, levels) (0 when the fp16 scale
 * is 0), stored LSB-first along the head dimension.  Its size is exactly the page's estimate.
 * All arrays 16-byte aligned; bits in {2, 4, 8}; group_size in {8, 16, 32, 64}; head_dim a
 * multiple of group_size, at most 256; capacity a multiple of group_size.
 */
typedef struct kivi_packed {
  int32_t bits;
  int32_t group_size;
  int32_t batch;
  int32_t num_heads;
  int32_t capacity;
  int32_t head_dim;
  uint8_t* k_codes;
  uint16_t* k_scale;
  uint16_t* k_zero;
  uint8_t* v_codes;
  uint16_t* v_scale;
  uint16_t* v_zero;
} kivi_packed;

/*
 * Pack tokens [lo, hi) of every layer's fp16 K and V (k[l], v[l]: device fp16 [B][H][capacity]
 * [D], 16-byte aligned; the same layout the in-place KIVI cache uses) into caches[l].  lo and hi
 * are multiples of group_size (the residual boundary of kivi_boundary always is).  eps is the
 * page's 1e-8.  Errors: KVQ_ERR_BITS, KVQ_ERR_SHAPE, KVQ_ERR_NULL, KVQ_ERR_ALIGN, KVQ_ERR_RANGE,
 * KVQ_ERR_CUDA.
 */
KVQ_API kvq_status kivi_pack(const kivi_packed* caches, const uint16_t* const* k,
                             const uint16_t* const* v, int n_layers, int lo, int hi, float eps,
                             kvq_stream_t stream);

/*
 * Decode attention of one query per batch row over a KIVI cache whose tokens [0, n_packed) are
 * packed in caches[l] and tokens [n_packed, offset) are still fp16 in k[l], v[l] (the residual
 * window).  q device fp16 [n_layers][B][num_q_heads][D]; out device float32, same shape; query
 * head j uses KV head j / (num_q_heads / H); the reconstruction of a packed element is
 * c * scale + zero in fp16 (one fused rounding), accumulation in float32.  Supports bits 2,
 * head_dim 64, group_size 16/32/64, at most 8 query heads per KV head; n_packed a multiple of
 * group_size; 0 <= n_packed <= offset <= capacity.  workspace: kivi_decode_attn_workspace(...)
 * bytes, 16-byte aligned, no initialisation needed.  dev_err (device int32, may be NULL) gets
 * KVQ_DEVERR_TIMEOUT OR-ed in if a staged copy never completed (the affected split then counts
 * no tokens).  Errors: KVQ_ERR_BITS, KVQ_ERR_SHAPE (bits, head_dim, group_size, num_q_heads),
 * KVQ_ERR_NULL, KVQ_ERR_ALIGN, KVQ_ERR_RANGE (n_packed, offset, grid limits), KVQ_ERR_WORKSPACE,
 * KVQ_ERR_CUDA.
 */
KVQ_API size_t kivi_decode_attn_workspace(int n_layers, int batch, int num_heads, int num_q_heads,
                                          int head_dim, int offset);

KVQ_API kvq_status kivi_decode_attn(const kivi_packed* caches, const uint16_t* const* k,
                                    const uint16_t* const* v, int n_layers, const uint16_t* q,
                                    int num_q_heads, int n_packed, int offset,
                                    float softmax_scale, float* out, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_err,
                                    kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * The KIVI cache protocol: update (append + flush) and trim (frontier rollback)
 * ------------------------------------------------------------------------------------------ */

/*
 * VeloxQuant-MLX source page "veloxquant_mlx.cache.kivi_cache": KIVIKVCache.update_and_fetch,
 * _quantization_boundary, trim and _rollback_frontier.  A kivi_state (host memory, owned by the
 * caller) tracks one cache of n_layers layers that append and trim together: `offset` tokens
 * held in [B][H][capacity][D] fp16 K and V caches, the first `n_quantized` of them quantized.
 * bits 2/4/8 give levels 2^bits - 1; eps is the page's 1e-8.  Fill it with kivi_state_init
 * (offset 0); the calls below advance it only when they succeed.
 */
typedef struct kivi_state {
  int32_t batch;
  int32_t num_heads;
  int32_t head_dim;         /* multiple of 8, <= 256 */
  int32_t capacity;
  int32_t bits;             /* 2, 4 or 8 */
  int32_t group_size;
  int32_t residual_length;  /* the page's residual window R (128 by default) */
  float eps;
  int32_t offset;           /* tokens held */
  int32_t n_quantized;      /* the quantization frontier */
} kivi_state;

KVQ_API kvq_status kivi_state_init(kivi_state* st, int batch, int num_heads, int head_dim,
                                   int capacity, int bits, int group_size, int residual_length);

/*
 * update_and_fetch for the page's in-place cache: copy the n_new new tokens of every layer
 * (k_new[l], v_new[l]: device fp16 [B][H][n_new][D], 16-byte aligned) into k_cache[l],
 * v_cache[l] at st->offset (one launch for all layers), then round-trip the tokens
 * [n_quantized, kivi_boundary(offset + n_new)) in place (kivi_quant_dequant, one launch), and
 * advance the state.  n_layers <= 32.  Errors: those of kivi_quant_dequant, KVQ_ERR_RANGE if the
 * tokens do not fit.  The "fetch" is the caches' first st->offset tokens.
 */
KVQ_API kvq_status kivi_update(kivi_state* st, uint16_t* const* k_cache, uint16_t* const* v_cache,
                               const uint16_t* const* k_new, const uint16_t* const* v_new,
                               int n_layers, int n_new, kvq_stream_t stream);

/*
 * trim for the page's in-place cache: drop the last n tokens (at most offset) and pull the
 * frontier down to min(n_quantized, (offset / group_size) * group_size).  Host only: the rows
 * between the new frontier and the new offset keep their round-tripped values in the cache and
 * are quantized again by the next flush (the double rounding the page bounds by one step).
 * Returns the number of tokens dropped.
 */
KVQ_API int kivi_trim(kivi_state* st, int n);

/*
 * update_and_fetch with the quantized region packed (kivi_packed, one per layer, matching the
 * state): append as kivi_update, then kivi_pack tokens [n_quantized, boundary) from the fp16
 * caches.  Attention: kivi_decode_attn(n_packed = st->n_quantized, offset = st->offset).
 */
KVQ_API kvq_status kivi_packed_update(kivi_state* st, const kivi_packed* caches,
                                      uint16_t* const* k_cache, uint16_t* const* v_cache,
                                      const uint16_t* const* k_new, const uint16_t* const* v_new,
                                      int n_layers, int n_new, kvq_stream_t stream);

/*
 * trim with the quantized region packed: as kivi_trim, and the rows that leave the packed region
 * ([new frontier, min(old frontier, new offset))) get their round-tripped values written into
 * the fp16 caches (kivi_unpack), as the page's in-place cache holds them.  *trimmed (may be
 * NULL) receives the number of tokens dropped.
 */
KVQ_API kvq_status kivi_packed_trim(kivi_state* st, const kivi_packed* caches,
                                    uint16_t* const* k_cache, uint16_t* const* v_cache,
                                    int n_layers, int n, int* trimmed, kvq_stream_t stream);

/*
 * Write the reconstruction fp16(float32(c * scale) + zero) of packed tokens [lo, hi) of every
 * layer into k[l], v[l] (device fp16 [B][H][capacity][D]).  Errors: KVQ_ERR_BITS, KVQ_ERR_SHAPE,
 * KVQ_ERR_NULL, KVQ_ERR_ALIGN, KVQ_ERR_RANGE, KVQ_ERR_CUDA.
 */
KVQ_API kvq_status kivi_unpack(const kivi_packed* caches, uint16_t* const* k, uint16_t* const* v,
                               int n_layers, int lo, int hi, kvq_stream_t stream);

/*
 * Decode attention for callers that cannot allocate device memory (no counterpart on the pages:
 * it is an addition of this library).  Same arguments, semantics and errors as kvq_decode_attn,
 * minus the workspace: the split partials go to a scratch array of 32 MiB that the library owns
 * in device memory, which every GPU that loads the library holds until the process exits.
 * Meant for code that cannot call cudaMalloc where it runs attention -- for example inside a
 * runtime whose allocator owns all device memory, or a serving loop that must not allocate
 * (cudaMalloc may synchronize the device) once it is running.  It calls no allocation routine.
 *   - The first call on a device looks up the scratch array's device address (cached per
 *     device); make that first call before any stream capture.
 *   - All calls share the one array: calls whose kernels overlap on the GPU (other streams,
 *     other threads) race on it and must be serialized by the caller.  Nothing in it needs to be
 *     cleared between calls: every partial a call reads was written earlier by that same call.
 *   - To fit the array, the number of splits over tokens is capped (each split of each
 *     (layer, sequence, KV head) unit takes 8,320 bytes), so a split may then cover more than
 *     the usual 256 tiles (4,096 tokens); a problem with more than 4,032
 *     n_layers * nseq * num_kv_heads units does not fit even with one split each and returns
 *     KVQ_ERR_RANGE with the byte counts in kvq_last_error().
 */
KVQ_API kvq_status kvq_decode_attn_noalloc(const kvq_pool* k_pools, const kvq_pool* v_pools,
                                           int n_layers, const uint16_t* q, int num_q_heads,
                                           const int32_t* page_table, int max_pages,
                                           const int32_t* seq_lens, int nseq, int max_seq_len,
                                           float softmax_scale, float* out, int32_t* dev_err,
                                           kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Norms of queries and keys with the position rotation
 * ------------------------------------------------------------------------------------------ */

/* Element type of the tensors below (16-bit ones are passed as their bit patterns).  KVQ_F32 is for the
 * entries that name it. */
typedef enum kvq_dtype { KVQ_F16 = 0, KVQ_BF16 = 1, KVQ_F32 = 2 } kvq_dtype;

/*
 * Host: the rotation frequencies inv_freq[i] (radians per position, finite, >= 0) as
 * kvq_qk_norm_rope reads them, phases[i] = round(frac(inv_freq[i] / 2 pi) * 2^64) mod 2^64: turns
 * per position in units of 2^-64.  A position times a phase, modulo 2^64, is the angle without
 * any loss for far positions.  Errors: KVQ_ERR_NULL, KVQ_ERR_RANGE.
 */
KVQ_API kvq_status kvq_rope_phases(const double* inv_freq, int n, uint64_t* phases);

/*
 * What stands between the projections and the cache: for every token t and head, the row x (D
 * values) becomes
 *   y_d = x_d / sqrt(mean_d x_d^2 + eps) * w_d                  (w NULL: y = x, no norm)
 * and then its first rotary_dim values are rotated in pairs (a, b), pair i by the angle
 * positions[t] * inv_freq[i]:  a' = a cos - b sin,  b' = b cos + a sin, with (a, b) =
 * (y_i, y_{i + rotary_dim / 2}), or (y_{2i}, y_{2i+1}) if interleaved.  Computed in float32 from
 * the inputs, rounded once to the output type.  A row whose sum of squares leaves float32's
 * range (bf16 values of 1e19 and more) gives 0 or NaN, a row of zeros with eps 0 NaN.
 * q, k           device, `dtype`, [num_tokens][heads][D], a token's heads contiguous, tokens
 *                q_stride / k_stride elements apart (a multiple of 8, >= heads * D): views into a
 *                fused projection's output are fine.  num_tokens may be 0.
 * q_out, k_out   the same with their own strides; q_out == q (k_out == k) with equal strides runs
 *                in place, any other overlap is a caller error.
 * positions      device int32 [num_tokens]; phases device uint64 [rotary_dim / 2] (may be NULL if
 *                rotary_dim is 0).
 * q_weight, k_weight  device float32 [D], 16-byte aligned, or NULL.
 * head_dim a multiple of 8 in [8, 256]; rotary_dim a multiple of 16 in [0, head_dim].
 * Errors: KVQ_ERR_SHAPE (dtype, heads < 1, head_dim, rotary_dim, strides), KVQ_ERR_NULL,
 * KVQ_ERR_ALIGN (16 bytes; phases 8), KVQ_ERR_RANGE (num_tokens < 0, eps not finite or < 0),
 * KVQ_ERR_CUDA.
 */
KVQ_API kvq_status kvq_qk_norm_rope(kvq_dtype dtype, const uint16_t* q, int64_t q_stride,
                                    const uint16_t* k, int64_t k_stride, uint16_t* q_out,
                                    int64_t q_out_stride, uint16_t* k_out, int64_t k_out_stride,
                                    int num_tokens, int num_q_heads, int num_kv_heads,
                                    int head_dim, int rotary_dim, int interleaved,
                                    const int32_t* positions, const uint64_t* phases,
                                    const float* q_weight, const float* k_weight, float eps,
                                    kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Attention over whole prompts
 * ------------------------------------------------------------------------------------------ */

/*
 * Causal attention of many query rows per sequence, the prompt's counterpart of kvq_decode_attn:
 * sequence s has new tokens cu_q[s] .. cu_q[s+1]-1 of q and keys cu_k[s] .. cu_k[s+1]-1 of k, v,
 * of which the last belong to the new tokens, so that new token i of Lq sees keys
 * 0 .. i + Lk - Lq (Lk == Lq: a whole prompt; Lk > Lq: its next chunk, or with Lq == 1 one decode
 * step, over keys held in 16 bits, e.g. by kvq_dequant_paged):
 *   out[i][j][:] = sum_t softmax(softmax_scale * q[i][j] . k[t][h])_t v[t][h][:],  h = j / (Hq/H)
 * with the softmax's sums in float32 and its weights rounded to the input type for the product
 * with v.  A row that sees no key gets 0 (and lse -inf).  Values of keys and of v that a row does
 * not see (infinities and NaN too) do not reach it.
 * q, k, v    device, `dtype`, [total_q][Hq][D] and [total_k][H][D], a token's heads contiguous,
 *            tokens *_stride elements apart (a multiple of 8, >= heads * D).
 * cu_q, cu_k device int32 [nseq+1], non-decreasing, at most total_q / total_k.  Rows of out (and
 *            lse) that belong to no sequence are left as they were.
 * max_q, max_k  host upper bounds on a sequence's new tokens and keys.  A sequence that exceeds
 *            them, or whose offsets are out of range, is skipped (KVQ_DEVERR_INDEX).
 * out        `dtype` [total_q][Hq][D]; lse float32 [total_q][Hq] or NULL: the natural logarithm of
 *            each row's sum of exponentials, by which results over different keys are joined.
 * workspace  device scratch of at least kvq_prompt_attn_workspace(...) bytes, 16-byte aligned, no
 *            initialisation needed; two calls that may overlap need one each.  The size for some
 *            nseq, total_q, max_q and max_k suffices for every call of the same heads and head_dim
 *            with none of the four larger (20.6 MB at most).
 * dev_err    may be NULL; also gets KVQ_DEVERR_TIMEOUT: a wait inside the kernel ran out, and the
 *            rows of out and lse that belong to a sequence hold unspecified values.  (No copy or
 *            product is in flight any more when a block that gave up ends.)
 * All pointers are device memory (not a host view: tiles are read by the tensor copy engine).
 * head_dim 64, 128 or 256; any Hq that is a multiple of H, at most 128 query heads per KV head.
 * Two calls with the same arguments give the same bits.  A weight below 2^-35 of its row's largest
 * may be rounded to 0, so that an infinite value that a row sees with such a weight gives NaN.
 * Errors: KVQ_ERR_SHAPE (dtype, heads, head_dim, strides), KVQ_ERR_NULL, KVQ_ERR_ALIGN,
 * KVQ_ERR_RANGE (counts, total_k above 2^31 - 129, more than 2^31 - 1 tiles of 128 rows;
 * softmax_scale not in (0, 2.3e38]), KVQ_ERR_WORKSPACE, KVQ_ERR_CUDA.
 */
KVQ_API size_t kvq_prompt_attn_workspace(int nseq, int total_q, int num_q_heads, int num_kv_heads,
                                         int head_dim, int max_q, int max_k);

KVQ_API kvq_status kvq_prompt_attn(kvq_dtype dtype, const uint16_t* q, int64_t q_stride,
                                   const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                   int64_t v_stride, int num_q_heads, int num_kv_heads,
                                   int head_dim, const int32_t* cu_q, const int32_t* cu_k,
                                   int nseq, int total_q, int total_k, int max_q, int max_k,
                                   float softmax_scale, uint16_t* out, float* lse,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                   kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Trees of drafted tokens over the packed pages
 * ------------------------------------------------------------------------------------------ */

#define KVQ_MAX_NODES 64  /* drafted tokens per sequence */

/*
 * Attention of a tree of drafted tokens: sequence s holds seq_lens[s] tokens, and its drafts,
 * nodes 0 .. n-1 (n = cu_nodes[s+1] - cu_nodes[s], at most max_nodes), have been appended behind
 * them with kvq_quant_pack_paged (start_pos = seq_lens, cu_new_tokens = cu_nodes), so that node i
 * is token seq_lens[s] + i of the pages.  parents[cu_nodes[s] + i] is the node that node i follows
 * (in [0, i)), or -1 if it follows the cached text.  Node i sees every cached token, its ancestors
 * and itself; otherwise the arithmetic is that of kvq_decode_attn, with the softmax weights
 * rounded to fp16 for the product with v_hat and the result rounded to fp16.  A chain (parents
 * i - 1) attends like n decode steps.
 * q, out     device fp16 [n_layers][total_nodes][num_q_heads][D], 16-byte aligned.  Rows of out
 *            that belong to no sequence are left as they were.
 * page_table, seq_lens, max_pages, k_pools, v_pools, dev_err  as for kvq_decode_attn; cu_nodes
 *            device int32 [nseq+1], non-decreasing, at most total_nodes; parents device int32
 *            [total_nodes].
 * max_nodes  host upper bound on a sequence's drafts, in [1, KVQ_MAX_NODES]; max_seq_len host
 *            upper bound on seq_lens[s] plus its drafts.  A sequence that exceeds them is skipped
 *            (KVQ_DEVERR_INDEX), and all of them are if offsets that fall give the same drafts to more
 *            sequences than the bounds have row tiles for; a parent outside [-1, i) counts as -1
 *            (KVQ_DEVERR_INDEX).  Tokens
 *            whose page id is out of range are not attended (KVQ_DEVERR_PAGE_RANGE).
 * workspace  kvq_tree_attn_workspace(...) bytes, 16-byte aligned, no initialisation needed; two
 *            calls that may overlap need one each.
 * dev_err    also gets KVQ_DEVERR_TIMEOUT, as for kvq_prompt_attn: the rows of out that belong to a
 *            sequence then hold unspecified values.
 * Values of drafts that a node does not see (infinities and NaN too) do not reach it.
 * head_dim 256; page_size a multiple of 16; at most 16 query heads per KV head; the plain pages only
 * (not those with sinks and outliers of kvq_decode_attn_side, nor packed KIVI).  One call's upper
 * bounds may make 2^30 tiles of 64 tokens at most (layers x KV heads x tiles of 128 rows x
 * max_seq_len / 64), and max_seq_len may be 2^31 - 65.
 * Errors: KVQ_ERR_SHAPE, KVQ_ERR_BITS, KVQ_ERR_NULL, KVQ_ERR_ALIGN, KVQ_ERR_RANGE (also
 * softmax_scale not in (0, 2.3e38]), KVQ_ERR_WORKSPACE, KVQ_ERR_CUDA.
 */
KVQ_API size_t kvq_tree_attn_workspace(int n_layers, int nseq, int total_nodes, int num_kv_heads,
                                       int num_q_heads, int head_dim, int max_nodes,
                                       int max_seq_len);

KVQ_API kvq_status kvq_tree_attn(const kvq_pool* k_pools, const kvq_pool* v_pools, int n_layers,
                                 const uint16_t* q, int num_q_heads, const int32_t* page_table,
                                 int max_pages, const int32_t* seq_lens, const int32_t* cu_nodes,
                                 const int32_t* parents, int nseq, int total_nodes, int max_nodes,
                                 int max_seq_len, float softmax_scale, uint16_t* out,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                 kvq_stream_t stream);

/*
 * Keep the accepted drafts: for sequence s and i = 0, 1, ..., the packed row (codes and scale, of
 * every head, in every pool) of token seq_lens[s] + accept[cu_accept[s] + i] is copied to token
 * seq_lens[s] + i.  All of a sequence's rows are read before any is written, so any order of node
 * numbers, repeated ones too, is fine.  seq_lens is not advanced: the caller adds the count.
 * pools      host array [n_tensors] (all with the same bits, num_heads, head_dim, page_size): the
 *            K and V pools of every layer, each once; no two sequences may share the pages that hold
 *            the drafts.
 * cu_accept  device int32 [nseq+1], non-decreasing, at most total_accept; accept device int32
 *            [total_accept], node numbers in [0, KVQ_MAX_NODES).  A sequence with more than
 *            KVQ_MAX_NODES of them, or offsets out of range, is skipped, and a row whose node
 *            number is out of range is (KVQ_DEVERR_INDEX); a row whose page id is out of range is
 *            skipped too (KVQ_DEVERR_PAGE_RANGE).
 * Errors: those of kvq_quant_pack_paged.
 */
KVQ_API kvq_status kvq_tree_commit(const kvq_pool* pools, int n_tensors, const int32_t* page_table,
                                   int max_pages, const int32_t* seq_lens,
                                   const int32_t* cu_accept, const int32_t* accept, int nseq,
                                   int total_accept, int32_t* dev_err, kvq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Beam search over the pages: selection, tables that share pages, attention over shared prefixes
 * ------------------------------------------------------------------------------------------ */

#define KVQ_MAX_BEAMS 64      /* beams per sequence */
#define KVQ_MAX_BEAM_OUT 64   /* candidates kvq_beam_select returns per sequence */
#define KVQ_MAX_SEQS 65536    /* rows of logits, sequences of attention per call */
#define KVQ_MAX_TABLE_SEQS 2048   /* old, and new, sequences per table update; rows per compaction */

/*
 * The step that decides which beams go on.  With x[b][v] the logits behind beam b of a sequence and
 *   t[b][v] = scores[b] + x[b][v] - log sum_w exp x[b][w]
 * the num_out candidates of largest t, in falling order, equal ones by beam and then token (those of one
 * beam that only float64 makes equal, behind a far score or near logits, by logit first):
 *   out_scores  float32 [nseq][num_out]   t
 *   out_parents int32 [nseq][num_out]     the candidate's row s * beams + b
 *   out_tokens  int32 [nseq][num_out]     v
 * Candidates of t = -inf (a token of logit -inf, all of a beam whose score is not finite) and of
 * t = NaN (all of a beam with a logit of NaN or +inf) are never chosen; where too few are left, the
 * rest is -inf, -1, -1.  With num_out = beams, out_parents is what kvq_table_update takes; a caller
 * that ends beams at a token asks for more and drops some.  A first step has one beam of score 0, the
 * others -inf (their logits are not read).
 * Within a beam the order is exactly that of the logits; between beams it is that of t up to what the rows'
 * log-sums are off: 2e-7 in the worst rows tried, 6e-8 in ordinary ones, below 2^-16 for any logits of up to
 * 2^17 tokens (the exponentials are float32's: 2^-22, and 2^-23 of their argument).  Two calls with the same
 * arguments give the same bits.
 * logits     device, `dtype` (KVQ_F16, KVQ_BF16 or KVQ_F32), nseq * beams rows of vocab elements,
 *            row_stride >= vocab elements apart; any alignment.
 * scores     device float32 [nseq][beams].
 * workspace  kvq_beam_select_workspace(...) bytes, 16-byte aligned, no initialisation needed; two calls
 *            that may overlap need one each.  The size for some nseq * beams, vocab and num_out suffices for
 *            every call with none of the three larger.
 * Errors: KVQ_ERR_SHAPE (dtype, beams, num_out, vocab, row_stride), KVQ_ERR_RANGE (nseq), KVQ_ERR_NULL,
 * KVQ_ERR_ALIGN, KVQ_ERR_WORKSPACE, KVQ_ERR_CUDA.
 */
KVQ_API size_t kvq_beam_select_workspace(int nseq, int beams, int vocab, int num_out);

KVQ_API kvq_status kvq_beam_select(kvq_dtype dtype, const void* logits, int64_t row_stride,
                                   const float* scores, int nseq, int beams, int vocab, int num_out,
                                   float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                                   void* workspace, size_t workspace_bytes, kvq_stream_t stream);

/*
 * The device's counterpart of the page allocator, for tables whose sequences share pages.  Its state
 * is the number of owners of each page, refs (device int32 [num_pages]): a page is free where it is 0.
 * Every entry of a sequence's row that it holds counts as one owner; a caller that keeps pages of its
 * own (a prefix cache, the host allocator's other users) counts itself there too.
 *
 * One call takes a step from the sequences of `table` (n_in rows, lens[p] tokens in the first
 * ceil(lens[p] / page_size) of held[p] pages) to those of `table_out` (n_out rows):
 *   - sequence s continues sequence parents[s] (-1: it starts empty).  It takes over the pages that
 *     hold its parent's tokens; several may (a fork), or none (the sequence ends);
 *   - room[s] > 0 maps the pages that the next room[s] tokens need.  A page that they begin in the
 *     middle of must then be the sequence's alone: of the sequences about to write into one page the
 *     first keeps it unless anybody else holds it, and the others get a copy of the rows in use, in
 *     every pool;
 *   - pages behind a parent's tokens, and those of sequences that nobody continues, lose an owner;
 *   - new pages are the free ones of lowest number, in the order of s and then of position.
 * The outputs: table_out's first held_out[s] entries of row s (those behind are left as they were),
 * lens_out[s] = the parent's length (the caller adds what it appends, at most room[s]),
 * held_out[s] = ceil((lens_out[s] + room[s]) / page_size) and refs_out, whole.  Nothing of the inputs is
 * changed, so outputs must not overlap them: a program keeps two of each and swaps them.  Sequences that
 * are in no row of the call keep their pages, so more than KVQ_MAX_TABLE_SEQS of them go through calls of
 * some each (refs_out of one is refs of the next).
 *
 * pools      host array [n_tensors]: the K and V pools of every layer, each once (all with the same
 *            bits, num_heads, head_dim, page_size and num_pages).
 * table, table_out  device int32, max_pages entries per row; lens, held [n_in], parents, room [n_out]
 *            device int32.
 * workspace  kvq_table_workspace(num_pages, max(n_in, n_out)) bytes, 16-byte aligned, no initialisation
 *            needed, or more; two calls that may overlap need one each.
 * dev_err    KVQ_DEVERR_NO_PAGES: fewer free pages than needed.  The inputs and the pools are as they
 *            were, the outputs are unspecified.  KVQ_DEVERR_INDEX: a row whose lengths contradict each
 *            other or max_pages counts as empty (its pages keep their owners), a parent out of range as
 *            -1, a room that is negative or does not fit as 0, counts below 0 are found.
 *            KVQ_DEVERR_PAGE_RANGE: an entry out of range is passed on and counted nowhere.
 *            KVQ_DEVERR_TIMEOUT: the blocks did not meet; the outputs are unspecified, the inputs and the
 *            pools as they were.
 * Errors: those of kvq_quant_pack_paged, KVQ_ERR_SHAPE (num_pages differ), KVQ_ERR_RANGE (more than
 * KVQ_MAX_TABLE_SEQS sequences; an output that is its input), KVQ_ERR_WORKSPACE.
 */
KVQ_API size_t kvq_table_workspace(int64_t num_pages, int nseq);

KVQ_API kvq_status kvq_table_update(const kvq_pool* pools, int n_tensors, const int32_t* table,
                                    int max_pages, const int32_t* lens, const int32_t* held, int n_in,
                                    const int32_t* refs, const int32_t* parents, const int32_t* room,
                                    int n_out, int32_t* table_out, int32_t* lens_out, int32_t* held_out,
                                    int32_t* refs_out, void* workspace, size_t workspace_bytes,
                                    int32_t* dev_err, kvq_stream_t stream);

/*
 * Moves the pages in use together: with n pages of refs != 0, those at n and above move, in their
 * order, to the free places below n, in every pool, and table_out (the first held[s] entries of each
 * row) and refs_out follow; *live (device int32) gets n.  The pages from n on are then free, e.g. to be
 * given back.  All sequences that hold pages have to be in the one call; other owners (see above) must not
 * remember page numbers.  Outputs must not overlap inputs.
 * dev_err    KVQ_DEVERR_INDEX: a held[s] outside [0, max_pages] counts as 0, an entry whose page has no
 *            owners keeps its number; KVQ_DEVERR_PAGE_RANGE: so does an entry out of range.
 * Other arguments and errors as for kvq_table_update.
 */
KVQ_API kvq_status kvq_table_compact(const kvq_pool* pools, int n_tensors, const int32_t* table,
                                     int max_pages, const int32_t* held, int nseq, const int32_t* refs,
                                     int32_t* table_out, int32_t* refs_out, int32_t* live,
                                     void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                     kvq_stream_t stream);

/*
 * Decode attention over pages of 4 bits, of one query per sequence, for groups of `beams` sequences
 * (s / beams is the group) that have their first shared_lens[group] tokens in common: these are read
 * once, from the pages of the group's first sequence, the others from each sequence's own.  beams = 1
 * with shared_lens NULL is the plain decode step: of 4-bit pages at 256 channels it is the faster one from
 * some 2,000 tokens on, or with many sequences (1.2 to 2.1 times); kvq_decode_attn has float32 results and
 * values rounded to fp16, takes 6 and 8 bits, too, and a few hundred tokens of one sequence sooner.
 *   out[l][s][j][:] = sum_t softmax(softmax_scale q[l][s][j] . k_t)_t v_t[:],   t in [0, seq_lens[s])
 * with k_t = code * scale, v_t likewise, not rounded (kvq_decode_attn's are, to fp16); softmax weights
 * times v's scale are rounded to 11 bits for the product with v's codes (where one is below 2^-24 of the
 * row's largest weight times its largest scale of V, to 2^-35 of that), sums are float32.
 * q, out     device, `dtype` (KVQ_F16 or KVQ_BF16), [n_layers][nseq][num_q_heads][D], 16-byte aligned; a
 *            sequence of length 0 gets 0.
 * k_pools, v_pools, page_table, seq_lens, dev_err  as for kvq_decode_attn; shared_lens device int32
 *            [nseq / beams] or NULL (all 0), at most the group's lengths.
 * max_shared, max_own  host upper bounds on shared_lens and on seq_lens - shared_lens.  Their sum must fit a
 *            row of the table (max_pages * page_size tokens, 2^31 - 65 at most), unless max_own is all
 *            that a row holds: for batches whose longest prefix and longest own part are of different
 *            groups, and where nothing tighter is known.  A bound of at most 113 own tokens lets one warp
 *            take a sequence's own tokens where there are many sequences (1.4 times as fast there); else
 *            loose bounds cost nothing.  A group whose lengths contradict the bounds or exceed the row
 *            gets 0 (KVQ_DEVERR_INDEX).  Tokens whose page id is out of range are not
 *            attended (KVQ_DEVERR_PAGE_RANGE).
 * workspace  kvq_beam_attn_workspace(...) bytes, 16-byte aligned, no initialisation needed; two calls that
 *            may overlap need one each.  The size for some n_layers, nseq and bounds suffices for every call
 *            of the same beams, heads and head_dim with none of these larger.
 * head_dim 64, 128 or 256; page_size a multiple of 16; at most 64 query heads per KV head.  Two calls
 * with the same arguments give the same bits.  Queries of 2^100 and more in magnitude, and scores that (times
 * log2 e) leave float32's range, may give NaN or 0.
 * Errors: KVQ_ERR_SHAPE, KVQ_ERR_BITS (other than 4), KVQ_ERR_NULL, KVQ_ERR_ALIGN, KVQ_ERR_RANGE (nseq not
 * a multiple of beams; bounds beyond a row of the table, see above; softmax_scale not in (0, 2.3e38]),
 * KVQ_ERR_WORKSPACE, KVQ_ERR_CUDA.
 */
KVQ_API size_t kvq_beam_attn_workspace(int n_layers, int nseq, int beams, int num_kv_heads,
                                       int num_q_heads, int head_dim, int max_shared, int max_own);

KVQ_API kvq_status kvq_beam_attn(kvq_dtype dtype, const kvq_pool* k_pools, const kvq_pool* v_pools,
                                 int n_layers, const uint16_t* q, int num_q_heads,
                                 const int32_t* page_table, int max_pages, const int32_t* seq_lens,
                                 const int32_t* shared_lens, int nseq, int beams, int max_shared,
                                 int max_own, float softmax_scale, uint16_t* out, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_err, kvq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
