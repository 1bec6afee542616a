/*
 * bitlinear_attn.h -- C ABI of libbitlinear.so: the attention between the
 * q, k, v projections of a decoder layer and its o projection, and the paged
 * key-value cache it reads, on NVIDIA B200 (sm_100a).
 *
 * Defined by: "Distillix" README and "SLM750-Edge" section 2.2 (grouped
 * query heads, 12 Q / 4 KV; rotary positions; sliding window of 1024).
 *
 * The conventions of bitlinear.h hold (device pointers on the current
 * device, caller-owned memory, asynchronous on `stream`, bl_status, finite
 * inputs).  In addition:
 *   - Heads: Hq query heads share Hkv key / value heads, Hq % Hkv == 0; query
 *     head h reads key head h / (Hq / Hkv).  Head size D: 16 <= D <= 128,
 *     D % 16 == 0.
 *   - scale: positive.
 *   - Rows: q, k, v hold one row of heads per token; row t of q starts at
 *     q + t * q_stride elements (q_stride >= Hq * D, and a row must start on
 *     a 16-byte boundary), its heads are contiguous.  The q, k, v columns of
 *     one fused projection output are such rows.
 *   - Cache: pages of page_size tokens (a power of two, 8 <= page_size <=
 *     1024).  k_pages, v_pages [num_pages, Hkv, page_size, D]; row s of
 *     tables [max_seqs, max_pages] int32 lists the pages of sequence s, -1
 *     behind them; lengths [max_seqs] int32 its tokens.  What lies behind a
 *     sequence's last token in its last page is never used (it may be NaN).
 *     max_pages * page_size < 2^31.
 *   - Indexes that live on the device (sequence ids, lengths, table entries,
 *     positions) are checked by the kernels: an access that would leave its
 *     array is skipped, and bl_check_device_error then returns
 *     BL_ERR_INDEX.  A negative sequence id marks a padded entry of a batch:
 *     it is skipped, its outputs are left as they were, and it is no error.
 */
#ifndef BITLINEAR_ATTN_H
#define BITLINEAR_ATTN_H

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Paged cache of one layer, as the kernels see it. */
typedef struct {
    void *k_pages;         /* [num_pages, Hkv, page_size, D] */
    void *v_pages;         /* same */
    const int32_t *tables; /* [max_seqs, max_pages] */
    const int32_t *lengths; /* [max_seqs] */
    int64_t num_pages;
    int64_t page_size;
    int64_t max_seqs;
    int64_t max_pages;
    bl_dtype dtype;        /* of the pages: BL_F32 or BL_BF16 */
} bl_kv_cache;

/* ------------------------------------------------------------------------ */
/* Rotary positions on q and k, rounding, and the new rows into the cache.   */
/*                                                                           */
/*   (y_i, y_i+D/2) = (x_i c_i - x_i+D/2 s_i, x_i+D/2 c_i + x_i s_i)         */
/*   with (c, s) = row `position` of rope, i < D/2; in float32, rounded once */
/*                                                                           */
/* q [T, Hq, D], k, v [T, Hkv, D] of xdt (rows strided, see above).          */
/* rope [rope_len, D] float32: cos of D/2 angles, then sin; NULL: no         */
/* rotation.  inverse != 0 rotates back (the gradient of the rotation).      */
/* cu_seqlens [B + 1] int32: tokens of batch entry b are rows cu[b] ..       */
/* cu[b + 1] - 1 (rows behind cu[B] are left as they were); NULL: T == B,    */
/* one token each.  seq_ids [B] int32 the entry's sequence, NULL: b itself.  */
/* Positions: entry b's tokens are the last ones of its sequence, i.e.       */
/* position lengths[seq] - (cu[b + 1] - cu[b]) + i; without lengths (cache   */
/* and lengths NULL) position i.                                             */
/* q_out [T, Hq, D], k_out, v_out [T, Hkv, D] of odt, contiguous; any of     */
/* them NULL: not written.  cache NULL: no pages are written; otherwise      */
/* k and v go to their position's page (cache->lengths is used for the       */
/* positions; `lengths` must then be NULL).  q may be NULL with q_out NULL,  */
/* k and v may both be NULL with k_out, v_out and cache NULL.  An output may */
/* be the input it comes from (same type, contiguous), not overlap it        */
/* otherwise; with a cache a sequence is listed once per call.               */
/* ------------------------------------------------------------------------ */
bl_status bl_rope_append(const void *q, const void *k, const void *v, bl_dtype xdt, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                         const float *rope, int64_t rope_len, int inverse, const int32_t *cu_seqlens, int64_t B,
                         const int32_t *seq_ids, const int32_t *lengths, int64_t max_seqs, const bl_kv_cache *cache,
                         void *q_out, void *k_out, void *v_out, bl_dtype odt, bl_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Attention of one new token per sequence over the paged cache.             */
/*                                                                           */
/*   out[b, h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q[b, h] . k_j)  */
/*   over the visible keys j < lengths[seq_ids[b]]: all of them (window 0),  */
/*   or j >= length - window and the first `sinks` ones.                     */
/*   lse[b, h] = log(sum_j p_j)  (optional)                                  */
/*                                                                           */
/* The new token itself is in the cache already (bl_rope_append).  Products, */
/* statistics and sums in float32.  A sequence of length 0 gives out = 0,    */
/* lse = -inf.  q [B, Hq, D] of xdt, out [B, Hq, D] contiguous of xdt, lse   */
/* [B, Hq] float32 or NULL; seq_ids [B] int32 or NULL (entry b: sequence b;  */
/* B <= max_seqs).  B <= 65535.  The same inputs on the same GPU give the    */
/* same bits.                                                                */
/* ------------------------------------------------------------------------ */
size_t bl_attn_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D);
bl_status bl_attn_decode(const void *q, bl_dtype xdt, int64_t q_stride, int64_t B, int64_t Hq, int64_t Hkv,
                         int64_t D, const bl_kv_cache *cache, const int32_t *seq_ids, int64_t window,
                         int64_t sinks, float scale, void *workspace, size_t workspace_bytes, void *out,
                         float *lse, bl_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Page tables of a cache, kept on the device.                               */
/*                                                                           */
/* refs [num_pages] int32 counts the sequences that hold a page; 0 = free.   */
/* New pages are the free ones with the lowest numbers, in the order of the  */
/* call's entries, so the same calls give the same tables.  status [1] int32 */
/* (device) tells how a call ended; unless it is 0 nothing was changed:      */
/*   1  too few free pages        2  a sequence would outgrow its table row  */
/*   3  a bad entry: an id outside [0, max_seqs), one listed twice, a        */
/*      negative count or length, a fork onto a sequence that is not empty   */
/*      or that is a source too                                              */
/* Negative ids are padding (skipped).  num_pages <= 2^20, max_seqs <= 2^17, */
/* n <= 8192.                                                                */
/*                                                                           */
/* bl_kv_extend  entry i's sequence grows by counts[i] tokens: pages for     */
/*               them, lengths += counts; active [n] int32 (or NULL) = the   */
/*               ids, or -1 for each when the call failed: used as the       */
/*               seq_ids of bl_rope_append and bl_attn_decode it keeps a     */
/*               step that got no pages from writing anything                */
/* bl_kv_free    the sequences end: each of their pages' refs -= 1, table    */
/*               rows -1, lengths 0; an id listed twice, or of an empty      */
/*               sequence, does nothing more; ids >= max_seqs are skipped    */
/*               with BL_ERR_INDEX                                           */
/* bl_kv_fork    sequence dst[i] becomes a copy of src[i] of its own future: */
/*               full pages are shared (refs += 1), a last partial page is   */
/*               copied, in every plane of the pool                          */
/* bl_kv_compact the pages in use move to the lowest numbers: the k-th used  */
/*               page >= n_live goes to the k-th free page < n_live, n_live  */
/*               [1] int32 (out) = pages in use; tables and refs follow      */
/*                                                                           */
/* pool: `planes` arrays of num_pages pages of page_bytes each, plane p at   */
/* pool + p * num_pages * page_bytes (e.g. K and V of every layer);          */
/* page_bytes % 16 == 0.                                                     */
/* ------------------------------------------------------------------------ */
bl_status bl_kv_extend(int32_t *tables, int32_t *lengths, int32_t *refs, int64_t num_pages, int64_t page_size,
                       int64_t max_seqs, int64_t max_pages, const int32_t *seq_ids, const int32_t *counts,
                       int64_t n, int32_t *status, int32_t *active, bl_stream_t stream);
bl_status bl_kv_free(int32_t *tables, int32_t *lengths, int32_t *refs, int64_t num_pages, int64_t page_size,
                     int64_t max_seqs, int64_t max_pages, const int32_t *seq_ids, int64_t n, bl_stream_t stream);
size_t bl_kv_fork_workspace_bytes(int64_t n);
bl_status bl_kv_fork(void *pool, int64_t planes, int64_t page_bytes, int32_t *tables, int32_t *lengths,
                     int32_t *refs, int64_t num_pages, int64_t page_size, int64_t max_seqs, int64_t max_pages,
                     const int32_t *src, const int32_t *dst, int64_t n, void *workspace, size_t workspace_bytes,
                     int32_t *status, bl_stream_t stream);
size_t bl_kv_compact_workspace_bytes(int64_t num_pages);
bl_status bl_kv_compact(void *pool, int64_t planes, int64_t page_bytes, int32_t *tables, int32_t *refs,
                        int64_t num_pages, int64_t max_seqs, int64_t max_pages, void *workspace,
                        size_t workspace_bytes, int32_t *n_live, bl_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Causal attention over a ragged batch (prefill, training), with a sliding  */
/* window and first tokens that stay visible, and its gradients.             */
/*                                                                           */
/* Batch entry b: queries cu_q[b] .. cu_q[b + 1] - 1, keys cu_k[b] ..        */
/* cu_k[b + 1] - 1.  Its last query stands at its last key: query i has      */
/* position p = nk - nq + i and sees key j when j <= p and (window == 0 or   */
/* p - j < window or j < sinks).  A query that sees nothing (p < 0) gives    */
/* o = 0, lse = -inf and no gradient.                                        */
/*   s = scale q . k;  lse = log sum_j exp(s_j);  P = exp(s - lse);  o = P v */
/*   dv = P^T do;  dS = P o (do v^T - rowsum(do o o));                       */
/*   dq = scale dS k;  dk = scale dS^T q                                     */
/* dk and dv sum over the query heads of a shared head.  P and dS are        */
/* rounded to bfloat16 (half a step, 2^-8 relative, per term) where they     */
/* enter the tensor cores; everything else is float32 until the outputs are  */
/* rounded once.  No atomics: the same inputs give the same bits.            */
/*                                                                           */
/* q, do_ [Tq, Hq, D], k, v [Tk, Hkv, D] bfloat16, rows strided; o, dq       */
/* [Tq, Hq, D], dk, dv [Tk, Hkv, D] bfloat16, contiguous; lse [Hq, Tq]       */
/* float32.  cu_q, cu_k [B + 1] int32, increasing, from 0, ending at or      */
/* before Tq, Tk (rows behind the end are left as they were); max_q, max_k:  */
/* at least every entry's query and key count (an entry with more gives      */
/* BL_ERR_INDEX; the gradients leave its queries from max_q on out, and      */
/* neither o, dq from max_q on nor dk, dv from max_k on are written).        */
/* Tq, Tk, B >= 1, Tq * Hq and Tk * Hkv < 2^31, max_q, max_k < 2^24.         */
/* The gradients' workspace is Tq * Hq floats, and with a window and sinks   */
/* at most 4 * Tq * Hkv * D more.                                            */
/* ------------------------------------------------------------------------ */
bl_status bl_attn_forward(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                          int64_t v_stride, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                          const int32_t *cu_q, const int32_t *cu_k, int64_t B, int64_t max_q, int64_t max_k,
                          int64_t window, int64_t sinks, float scale, void *o, float *lse, bl_stream_t stream);
size_t bl_attn_backward_workspace_bytes(int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D, int64_t B,
                                        int64_t max_q, int64_t max_k, int64_t window, int64_t sinks);
bl_status bl_attn_backward(const void *do_, const void *q, const void *k, const void *v, const void *o,
                           const float *lse, int64_t do_stride, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                           const int32_t *cu_q, const int32_t *cu_k, int64_t B, int64_t max_q, int64_t max_k,
                           int64_t window, int64_t sinks, float scale, void *workspace, size_t workspace_bytes,
                           void *dq, void *dk, void *dv, bl_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_ATTN_H */
