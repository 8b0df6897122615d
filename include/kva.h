/*
 * kva.h - C ABI of the attention side of the paged key-value cache.
 *
 * The calls here stand next to those of kvw.h, are exported by the same
 * library (libkvw.so) and share its conventions, types and status codes:
 *   kva_append_qkv_paged     split a fused QKV projection, normalise and
 *                            rotate queries and keys per head, append keys
 *                            and values to the paged cache
 *   kva_gqa_decode_paged     attention of each new token's query heads over
 *                            its request's paged keys and values
 *   kva_mla_decode_paged     the same over the paged latent cache (absorbed
 *                            queries, one 576-wide row for all heads)
 * One step of a layer is append (GQA) or kvw_mla_rope_rmsnorm_quant (MLA)
 * followed by the decode call, on one stream.
 *
 * Conventions: those of kvw.h (asynchronous, caller-owned pointers, host
 * argument errors returned before any launch, device data errors reported as
 * KVW_ERR_* bits in *err_flags, ragged batches through input_row_offsets),
 * and for the two attention calls:
 * - They enqueue two kernels on `stream`: the attention, split over the
 *   contexts of all tokens so that every CTA reads the same amount of cache,
 *   and a join of the pieces.  The split depends only on the lengths, the
 *   sizes and the device, so equal calls give equal bits.
 * - `workspace` (device, 16-byte aligned) holds the pieces between the two
 *   kernels.  Its size depends on the sizes alone (the *_workspace calls),
 *   not on the batch or the lengths.  Its contents need no preparation and
 *   mean nothing after the call.  Calls that may run at the same time (two
 *   streams, two graphs replayed together) need a workspace each; calls
 *   that follow one another on a stream may share one.
 * - New token i of request b sits at slot position p = cache_lengths[b] + i
 *   and attends to the positions max(0, p - window + 1) .. p, its own
 *   included: its key and value (its latent row) are in the cache already.
 *   Any mix of new tokens per request is right; the split is made for few
 *   (neighbouring tokens of a request share a GQA pass over their contexts
 *   where their rows fit 16 to a key-value head, and read them one by one
 *   otherwise; shared reads meet in L2).
 * - A page table reaches max_pages_per_seq * page_size positions, at most
 *   2^32 - 256.  A position past that has no valid page.
 * - A position whose slot has no valid page takes no part in the softmax,
 *   as if masked, and sets KVW_ERR_PAGE.  A token left with no position at
 *   all, or whose every score is -infinity, gets a row of zeros and lse =
 *   -infinity.
 * - Malformed offsets set KVW_ERR_OFFSETS; out and lse are left as they were.
 * - The cache is read by the copy engine, whose stages complete through
 *   bounded waits: KVW_ERR_TIMEOUT as in kvw.h, out and lse are then partly
 *   written.  It takes strides that are positive, multiples of 16 bytes and
 *   below 2^40 bytes in every dimension of more than one index (pages,
 *   planes, tokens, heads; the layer stride is free): KVW_EINVAL for others,
 *   and at most 2^31 pages and rows of a page: KVW_EUNSUPPORTED beyond.
 * - The attention calls only read the cache: page tables may share pages.
 * - Cache rows behind a token's last position are never used, whatever they
 *   hold (NaN included).  A NaN or an infinity in a used row or in a query
 *   propagates as the formula has it.  The sums of weights times values are
 *   fp32 before their division: bf16 values above 2^100 may overflow them.
 * - out and lse must not overlap any input.
 */
#ifndef KVA_H
#define KVA_H

#include "kvw.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Appending keys and values.  Row t of `qkv` holds num_q_heads query heads,
 * then num_heads key heads, then num_heads value heads of head_size values
 * (num_heads, head_size of the cache).  For every new token t at slot
 * position pos:
 *   x = qkv head; for query and key heads with a gamma:
 *     x_j = x_j * rsqrt(mean(x^2) + epsilon) * (gamma_j + weight_offset)
 *   the first rope_dim columns of query and key heads are rotated by
 *     freqs_cis[p] (pairs (2k, 2k+1) when interleaved != 0, else
 *     (k, k + rope_dim/2); p as in kvw_qk_rope_paged_ragged: the slot
 *     position, position_ids[t], or the mrope section's row)
 *   q_out[t, h, :] = bf16(query head h)
 *   cache[page(pos), K, layer_idx, pos % page_size, g, :] = quant(key head g)
 *   cache[page(pos), V, ...] = quant(value head g)
 * Everything between the bf16 input and the stored value is fp32, rounded
 * once (quant: bf16, or E4M3 satfinite(y / scale), with the descriptor's
 * scale for keys and v_scale for values).  The sum of squares is added up in
 * an order of the kernel's choosing.
 *
 *   q_out          device, bf16, row t at q_out + t*q_out_row_stride elements
 *                  (>= num_q_heads*head_size, multiple of 8); may be qkv
 *                  itself with the same row stride (rotated in place)
 *   qkv            device, bf16, row stride qkv_row_stride elements
 *                  (>= (num_q_heads + 2*num_heads)*head_size, multiple of 8)
 *   q_gamma, k_gamma  device, bf16 [head_size], each NULL for no norm
 *   freqs_cis      device, f32 [freqs_rows, rope_dim], (cos, sin) interleaved;
 *                  may be NULL when rope_dim is 0
 *   rope_dim       0 or a multiple of 16, <= head_size
 *   position_ids, mrope_section   as kvw_qk_rope_paged_ragged (sections
 *                  counted in pairs, summing to rope_dim / 2)
 *   cache          host pointer: bf16 or E4M3, head_size a multiple of 16 and
 *                  <= 512; both planes (K, V) are written
 * num_q_heads may be 0 (cache write only, q_out NULL); num_q_heads +
 * 2*num_heads <= 4096 and tot_seq_len * (num_q_heads + 2*num_heads) <= 2^31.
 * A position >= freqs_rows (rope_dim > 0): nothing of that token is written.
 * An invalid page: its cache rows are skipped, the query rows are written.
 */
int kva_append_qkv_paged(void* q_out, int64_t q_out_row_stride, const void* qkv,
                         int64_t qkv_row_stride, const uint32_t* input_row_offsets,
                         uint32_t num_batches, uint32_t tot_seq_len, uint32_t num_q_heads,
                         const void* q_gamma, const void* k_gamma, float epsilon,
                         float weight_offset, const void* freqs_cis, uint32_t freqs_rows,
                         uint32_t rope_dim, const uint32_t* position_ids, int interleaved,
                         const uint32_t* mrope_section, const kvw_paged_cache_t* cache,
                         float v_scale, uint32_t layer_idx, uint32_t* err_flags,
                         cudaStream_t stream);

/*
 * Attention of new tokens over a paged GQA cache.  With G = num_q_heads /
 * num_heads (must divide), for token t at position p and query head h:
 *   s_j = sm_scale * dot(q[t, h], K[j, h / G])         (K: code * scale)
 *   s_j = softcap * tanh(s_j / softcap)                 if softcap > 0
 *   s_j = s_j - alibi_slopes[h] * (p - j)               if alibi_slopes
 *   out[t, h] = bf16(sum_j e^s_j V[j, h / G] / sum_j e^s_j)
 *   lse[t, h] = log(sum_j e^s_j)
 * over the positions j named above (window = 0: from 0).  Scores, softmax
 * statistics and sums are fp32; the products take bf16 operands with a bf16
 * cache and fp16 operands with an E4M3 cache (codes are exact in fp16; each
 * query row is brought into fp16's range by a power of two, which loses only
 * what is below 2^-39 of the row's largest value), and the weights e^s are
 * rounded to that type: by 2^-8 (bf16) or 2^-11 (fp16) of each at most, or, for
 * fp16 ones below 2^-23 of the row's largest, by 2^-34 of that.
 *
 *   out            device, bf16 [tot_seq_len, num_q_heads, head_size]
 *   lse            device, f32 [tot_seq_len, num_q_heads], or NULL
 *   q              device, bf16, row t at q + t*q_row_stride elements
 *                  (>= num_q_heads*head_size, multiple of 8)
 *   cache          host pointer: bf16 or E4M3 (scale > 0, v_scale > 0),
 *                  head_size a multiple of 16 and <= 256
 *   sm_scale       finite, > 0;  softcap finite, >= 0 (0: none, and so is one
 *                  above 2^64); a capped score is off by 2^-19 of itself
 *   window         0: none; else the number of positions seen, own included
 *   alibi_slopes   device, f32 [num_q_heads], or NULL
 *   workspace      device, kva_gqa_decode_workspace(...) bytes
 * tot_seq_len <= 2^20 and num_q_heads <= 4096.
 */
int kva_gqa_decode_paged(void* out, float* lse, const void* q, int64_t q_row_stride,
                         const uint32_t* input_row_offsets, uint32_t num_batches,
                         uint32_t tot_seq_len, uint32_t num_q_heads,
                         const kvw_paged_cache_t* cache, float v_scale, uint32_t layer_idx,
                         float sm_scale, float softcap, uint32_t window,
                         const float* alibi_slopes, void* workspace, uint64_t workspace_bytes,
                         uint32_t* err_flags, cudaStream_t stream);

/* Bytes of workspace for kva_gqa_decode_paged, into *bytes (host). */
int kva_gqa_decode_workspace(uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_size,
                             uint64_t* bytes);

/*
 * Attention of new tokens over the paged MLA latent cache, with queries
 * absorbed into the latent space.  For token t at position p and head h,
 * with row_j the 576-wide cache row of position j (code * scale for E4M3):
 *   s_j = sm_scale * (dot(q_latent[t, h], row_j[0:512])
 *                     + dot(q_rope[t, h], row_j[512:576]))
 *   out[t, h] = bf16(sum_j e^s_j row_j[0:512] / sum_j e^s_j)
 *   lse[t, h] = log(sum_j e^s_j)
 * over positions 0 .. p.  Precision as kva_gqa_decode_paged, except that the
 * scores of an E4M3 cache come from its codes and each query row as two E4M3
 * parts (the row's values to within 2^-21 of its largest, or 2^-133); a row
 * that holds an infinity or a NaN gives NaN.
 * An E4M3 cache halves the memory, not the time: the values are converted to
 * fp16 on the way, and a decode step takes about a tenth longer than over a
 * bf16 cache (256 contexts of up to 8192 positions: 128 heads 455 and 407 us,
 * 16 heads 219 and 204).
 *
 *   out            device, bf16 [tot_seq_len, num_heads, 512]
 *   lse            device, f32 [tot_seq_len, num_heads], or NULL
 *   q_latent       device, bf16, token t at q_latent + t*q_latent_row_stride
 *                  elements, its heads 512 apart (stride >= num_heads*512,
 *                  multiple of 8)
 *   q_rope         device, bf16, the same with 64 (the q_rope_out of
 *                  kvw_mla_rope_rmsnorm_quant has stride num_heads*64)
 *   cache          host pointer: bf16 or E4M3, num_heads 1, head_size 576
 *   workspace      device, kva_mla_decode_workspace(...) bytes
 * 1 <= num_heads <= 1024, tot_seq_len <= 2^20, query row strides below 2^39.
 */
int kva_mla_decode_paged(void* out, float* lse, const void* q_latent,
                         int64_t q_latent_row_stride, const void* q_rope,
                         int64_t q_rope_row_stride, const uint32_t* input_row_offsets,
                         uint32_t num_batches, uint32_t tot_seq_len, uint32_t num_heads,
                         const kvw_paged_cache_t* cache, uint32_t layer_idx, float sm_scale,
                         void* workspace, uint64_t workspace_bytes, uint32_t* err_flags,
                         cudaStream_t stream);

/* Bytes of workspace for kva_mla_decode_paged, into *bytes (host). */
int kva_mla_decode_workspace(uint32_t num_heads, uint64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* KVA_H */
