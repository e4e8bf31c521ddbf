/*
 * specverify_serving.h -- what a serving loop needs around the verification of
 * drafts on AMD Instinct MI355X (gfx950), as a C ABI beside specverify.h and
 * specverify_tree.h (same library, same conventions: device pointers,
 * caller-owned buffers, no allocation and no synchronisation, host checks before
 * anything is enqueued, bit-deterministic results).
 *
 *   specverify_pages_resize     pages for the tokens of every request, taken from
 *                               the free list or given back to it; positions and
 *                               slots of new tokens
 *   specverify_rotate           norms and position rotation of queries and keys,
 *                               keys and values into their slots
 *   specverify_chunk_attention  a chunk of new tokens against all that is cached
 *                               up to each of them (a prompt, a part of one, a
 *                               single token)
 *   specverify_pages_fork       a request's cache for further requests: full pages
 *                               shared, the last one copied
 *   specverify_penalize         penalties for repeated tokens, biases and grammar
 *                               masks on the logits of drafted nodes
 *
 * Chunks
 * ------
 * - The new tokens of all requests are packed: request b owns rows
 *   chunk_start[b] .. chunk_start[b + 1] - 1 of every [T, ...] array, its tokens
 *   prefix_len[b], prefix_len[b] + 1, ... Lengths may differ, and be 0 or 1.
 *   Unlike drafted nodes they are committed at once: their keys and values go
 *   into the pages before they attend.
 *
 * Pages
 * -----
 * - The cache and the block table are those of specverify_tree.h.
 * - The free list is free_pages[*free_head ..]: pages are taken from its head, and
 *   come back in front of it.
 * - shares[p] is the number of requests that hold page p beside the first (0 for a
 *   free page and for one that a single request holds). Only full pages are
 *   shared, so what a request writes behind its prefix is its own.
 *
 * Every call has to be made with the device of its pointers and stream current.
 */
#ifndef SPECVERIFY_SERVING_H
#define SPECVERIFY_SERVING_H

#include "specverify_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Size limits checked on the host. */
#define SV_MAX_PAGE_BATCH (1 << 16)  /* requests or forks of a pages call */
#define SV_MAX_CACHE_PAGES (1 << 26) /* pages of a cache, in pages calls  */

/* Bits OR-ed into the device error word, beside those of the other headers. */
#define SV_ERR_REQUEST 128 /* a fork's source or target that it may not have */
#define SV_ERR_PENALTY 256 /* a repetition penalty that is not > 0           */

/*
 * Bytes of workspace of specverify_pages_resize (256-byte aligned, any contents;
 * calls that overlap in time need one each). Pure host function; 0 for sizes the
 * library rejects.
 */
size_t specverify_pages_resize_workspace_size(int64_t B, int64_t num_pages);

/*
 * Pages for what every request is to hold: its prefix_len[b] cached tokens and
 * the n_b new ones of its chunk. One that owns fewer takes them from the free
 * list, in request order; one that owns more gives the rest back (all of them
 * with prefix_len 0 and no new tokens: the request has ended). What is given back
 * comes first, so that others can take it.
 *   prefix_len  [B] int32, pages_in [B] int32: tokens cached, pages owned
 *   chunk_start [B+1] int32 or NULL (no new tokens)
 *   block_table [B, max_pages] int32, rows table_stride apart, updated in place:
 *               entries from pages_in[b] on are filled with the pages taken;
 *               entries of pages given back stay as they are
 *   free_pages  [num_free] int32, num_free >= num_pages, updated in place: the
 *               pages that came free, in order of their ids, in front of
 *               *free_head_in
 *   shares_in   [num_pages] int32 or NULL (no page is shared); shares_out
 *               [num_pages] int32 out, NULL when shares_in is
 *   pages_out   [B] int32 out; free_head_out [1] int32 out
 *   position    [T] int32 out: prefix_len + the token's index in the chunk
 *   slots       [T] int64 out: page * page_size + offset of that position
 * A page comes free when as many requests give it back as hold it. A request that
 * needs pages takes none when the list does not reach for it and all before it
 * (SV_ERR_PAGE, slots -1). One with wrong lengths (negative, longer than its pages
 * or than the block table: SV_ERR_LENGTH) or a wrong chunk (SV_ERR_TREE) keeps
 * what it owns and gets position and slots -1. An entry outside [0, num_pages)
 * that is given back is passed by; one that is taken or that a slot needs gives
 * entry and slot -1 (SV_ERR_PAGE). Rows outside every chunk get position and slots -1;
 * a row that a wrong chunk_start gives to several requests is the last one's. A
 * *free_head_in outside [0, num_free] is taken as num_free (SV_ERR_PAGE).
 * The _out arrays must not be the _in arrays.
 * Status: SV_EINVAL (null pointer but chunk_start, shares, device_error or, with
 * T = 0, position and slots; chunk_start NULL with T > 0; B outside [1, 2^16], T < 0
 * or >= 2^31, page_size no power of two, max_pages < 1, max_pages * page_size >=
 * 2^31, B * max_pages >= 2^40, num_pages outside [1, 2^26], num_free < num_pages or >= 2^31,
 * table_stride < max_pages or no stride, one of shares_in and shares_out alone, an
 * _out that is an _in), SV_EWORKSPACE, SV_EALIGN (workspace), SV_EHIP.
 */
int specverify_pages_resize(const int32_t* prefix_len, const int32_t* chunk_start,
                            const int32_t* pages_in, int32_t* block_table, int32_t* free_pages,
                            const int32_t* free_head_in, const int32_t* shares_in, int64_t B,
                            int64_t T, int64_t page_size, int64_t max_pages, int64_t table_stride,
                            int64_t num_pages, int64_t num_free, int32_t* pages_out,
                            int32_t* free_head_out, int32_t* shares_out, int32_t* position,
                            int64_t* slots, int32_t* device_error, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace of specverify_pages_fork (256-byte aligned, any contents;
 * calls that overlap in time need one each). Pure host function; 0 for sizes the
 * library rejects.
 */
size_t specverify_pages_fork_workspace_size(int64_t B, int64_t forks);

/*
 * The cache of request source[i] for request target[i], i < forks: the target's
 * table gets the source's full pages, which both hold from now on, and a page of
 * its own, from the free list in order of forks, with the tokens of the source's
 * last page if that is not full (of every layer).
 *   source, target [forks] int32: rows of the block table. A target owns no pages
 *                  and is named once; a source may have several targets
 *   prefix_len_in, pages_in [B] int32; prefix_len_out, pages_out [B] int32 out:
 *                  a target's are its source's tokens and the pages of those;
 *                  others' as they were
 *   block_table    [B, max_pages] int32, updated in place (the targets' rows)
 *   free_pages     [num_free] int32; free_head_in, free_head_out [1] int32
 *   shares_in, shares_out [num_pages] int32
 *   k_cache, v_cache [layers, num_pages, page_size, H, D] of 2- or 4-byte
 *                  elements (dtype), both with strides c_stride_l, c_stride_page,
 *                  c_stride_token, c_stride_h; in some order each axis steps over
 *                  all that those before span
 * A fork whose source or target is outside [0, B) or the same, whose target owns
 * pages or tokens, or is that of an earlier fork, is passed by (SV_ERR_REQUEST);
 * so is one whose source has wrong lengths (SV_ERR_LENGTH) and one that the free
 * list does not reach for (SV_ERR_PAGE). An entry of the source or the free list
 * outside [0, num_pages) becomes -1 in the target's table (SV_ERR_PAGE).
 * The _out arrays must not be the _in arrays.
 * Status: SV_EINVAL (null pointer but device_error or, with forks = 0, source and
 * target; B outside [1, 2^16], forks outside [0, 2^16], layers, H < 1, H >= 2^16, layers *
 * forks >= 2^31, D no multiple of 8 or outside [8, 256], page_size no power of two, max_pages
 * < 1, max_pages * page_size >= 2^31, num_pages outside [1, 2^26], num_free < 0 or >=
 * 2^31, table_stride < max_pages or no stride, a stride below 0 or from 2^48 on,
 * tokens of the cache that overlap, an _out that is an _in), SV_EDTYPE, SV_EALIGN
 * (cache pointers or strides not multiples of 16 bytes, workspace), SV_EWORKSPACE,
 * SV_EHIP.
 */
int specverify_pages_fork(const int32_t* source, const int32_t* target,
                          const int32_t* prefix_len_in, const int32_t* pages_in,
                          int32_t* block_table, const int32_t* free_pages,
                          const int32_t* free_head_in, const int32_t* shares_in, void* k_cache,
                          void* v_cache, int dtype, int64_t forks, int64_t B, int64_t layers,
                          int64_t H, int64_t D, int64_t c_stride_l, int64_t c_stride_page,
                          int64_t c_stride_token, int64_t c_stride_h, int64_t page_size,
                          int64_t max_pages, int64_t table_stride, int64_t num_pages,
                          int64_t num_free, int32_t* prefix_len_out, int32_t* pages_out,
                          int32_t* free_head_out, int32_t* shares_out, int32_t* device_error,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Queries and keys as attention takes them: x (1 / sqrt(mean x^2 + eps)) w for
 * each head where a weight is given, then the rotation by position. Of the first R
 * elements of a head, element i and element i + R / 2 (interleaved: 2 i and 2 i + 1)
 * become
 *   a' = a cos t - b sin t,  b' = b cos t + a sin t,  t = position * inv_freq[i],
 * the others stay. t is taken in float64, the rest in float32, and results are
 * rounded once.
 *   q         [T, Hq, D], k and v [T, Hkv, D]: strides q_stride_t, q_stride_h and,
 *             for k and v, k_stride_t, k_stride_h; v may be NULL without a cache
 *   q_weight, k_weight [D] float32 or of dtype (weight_dtype), each NULL for none
 *   position  [T] int32; a row whose position is negative is passed by: its
 *             outputs are left as they were
 *   inv_freq  [R / 2] float32
 *   q_out     [T, Hq, D], k_out [T, Hkv, D] out or NULL (with a cache): either may be
 *             its own input
 *   slots     [T] int64 and k_cache, v_cache [num_pages, page_size, Hkv, D], or all
 *             NULL: keys as in k_out and values go to these slots, which differ; a
 *             slot of -1 stores nothing, another one outside the cache neither
 *             (SV_ERR_PAGE)
 *   dtype     SV_F32, SV_BF16 or SV_F16, of all but weights, position, inv_freq
 * Status: SV_EINVAL (null pointer but the above and device_error or, with T = 0,
 * the [T, ...] arrays; k_out NULL without a cache; v NULL with one; slots and caches not
 * given together; T < 0, Hq, Hkv < 1, T * (Hq + Hkv) >= 2^31, D no multiple of 8 or outside
 * [8, 256], R odd or outside [2, D], eps negative, infinite or NaN, num_pages < 1, page_size
 * no power of two, num_pages * page_size >= 2^40, a stride below 0 or from 2^48 on, rows
 * of an output or tokens of the cache that overlap), SV_EDTYPE, SV_EALIGN (pointers or strides
 * of q, k, v, outputs or cache not multiples of 16 bytes), SV_EHIP.
 */
int specverify_rotate(const void* q, const void* k, const void* v, int dtype, int64_t T, int64_t Hq,
                      int64_t Hkv, int64_t D, int64_t R, int interleaved, int64_t q_stride_t,
                      int64_t q_stride_h, int64_t k_stride_t, int64_t k_stride_h,
                      const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                      const int32_t* position, const float* inv_freq, void* q_out,
                      int64_t qo_stride_t, int64_t qo_stride_h, void* k_out, int64_t ko_stride_t,
                      int64_t ko_stride_h, const int64_t* slots, void* k_cache, void* v_cache,
                      int64_t c_stride_page, int64_t c_stride_token, int64_t c_stride_h,
                      int64_t num_pages, int64_t page_size, int32_t* device_error, void* stream);

/*
 * Bytes of workspace of specverify_chunk_attention (256-byte aligned, any
 * contents; calls that overlap in time need one each). Pure host function; 0 for
 * sizes the library rejects.
 */
size_t specverify_chunk_attention_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                                                 int64_t D, int64_t max_chunk);

/*
 * Attention of chunks of new tokens over a paged cache that holds their keys and
 * values already:
 *   out[i, h] = sum_j softmax_j(scale * q[i, h] . k_j) v_j,
 * j over the request's positions 0 .. prefix_len[b] + (i - chunk_start[b]);
 * query head h reads key head h / (Hq / Hkv). Products and sums in float32; the
 * softmax weights are rounded to the storage type for the product with the
 * values, the output once.
 *   q           [T, Hq, D], strides q_stride_t, q_stride_h
 *   k_cache, v_cache, block_table: as specverify_tree_attention takes them
 *   dtype       SV_BF16 or SV_F16, of all of them and out
 *   prefix_len  [B] int32: tokens in front of the chunk; chunk_start [B+1] int32
 *   max_chunk   the longest chunk at most
 *   scale       > 0, scale / ln 2 finite
 *   out         [T, Hq, D], strides o_stride_t, o_stride_h, one axis stepping over
 *               all that the other spans; must not overlap an input
 *   lse         [T, Hq] float32 out or NULL: ln of the softmax's denominator
 * Values that a row does not see (of later tokens, in slots behind the chunk) do
 * not reach it, also when they are infinite or NaN; one that it sees makes its
 * column infinite or NaN. A page outside [0, num_pages) counts as zero keys and values
 * (SV_ERR_PAGE); a prefix_len below 0 or too long for the block table with the
 * chunk behind it is clamped to what fits (SV_ERR_LENGTH). The rows of a request
 * with a wrong chunk_start, a chunk longer than max_chunk (SV_ERR_TREE) or than the
 * block table (SV_ERR_LENGTH) are left as they were, and so are those outside
 * every chunk.
 * Status: SV_EINVAL (null pointer but lse, device_error or, with T = 0, q and out;
 * B, Hq, Hkv < 1, Hq not a multiple of Hkv, Hq / Hkv > 2^16, B * Hkv > 2^24, T < 0, T * Hq >=
 * 2^31, D no multiple of 8 or outside [8, 256], max_chunk outside [1, 2^31), page_size no
 * power of two, max_pages < 1 or max_pages * page_size > 2^31 - 2^14, num_pages < 1, a
 * stride below 0 or from 2^48 on, rows of out that overlap, table_stride < max_pages,
 * scale), SV_EDTYPE, SV_EALIGN (q, cache or out pointers or strides not multiples of 16
 * bytes), SV_EWORKSPACE, SV_EHIP.
 */
int specverify_chunk_attention(const void* q, const void* k_cache, const void* v_cache, int dtype,
                               int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                               int64_t max_chunk, int64_t q_stride_t, int64_t q_stride_h,
                               int64_t c_stride_page, int64_t c_stride_token, int64_t c_stride_h,
                               int64_t num_pages, int64_t page_size, const int32_t* block_table,
                               int64_t max_pages, int64_t table_stride, const int32_t* prefix_len,
                               const int32_t* chunk_start, float scale, void* out,
                               int64_t o_stride_t, int64_t o_stride_h, float* lse,
                               int32_t* device_error, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * The logits that tokens are drawn from, with what a request asks of them. For
 * row i of request b (drafted node i of its tree) and id v, let c be the number of
 * times that v was emitted: in history[b, prompt_len[b] .. prefix_len[b]) and among
 * the tokens of node i and its ancestors; s whether v occurs in history[b, 0 ..
 * prefix_len[b]) or among those nodes at all. Then, in float32 and in this order,
 *   x = s ? (x > 0 ? x / repetition[b] : x * repetition[b]) : x
 *   x = c > 0 ? x - (frequency[b] * c + presence[b]) : x
 *   x = x + the sum of the request's biases of v, in their order (if it has any)
 *   x = -inf where bit v % 32 of mask[i, v / 32] is 0
 * and is rounded to the output's type.
 *   logits      [T, V], rows stride apart; out [T, V], rows out_stride apart, may be
 *               logits itself (same type and stride)
 *   dtype, out_dtype  SV_F32 or SV_BF16 each
 *   tokens      [T] int32: the nodes' tokens, the roots' among them
 *   node_start  [B+1] int32, and ancestors [T, ceil(max_nodes / 64)] uint64 or NULL
 *               (chains): as specverify_tree_attention takes them. A step of
 *               gamma drafted tokens has gamma + 1 rows a request; a single token one
 *   history     [B, max_history] int32, rows history_stride apart: the tokens in the
 *               cache; prefix_len, prompt_len [B] int32
 *   repetition, presence, frequency [B] float32 (1, 0, 0: none)
 *   bias_start  [B+1] int32, bias_token [num_bias] int32, bias [num_bias] float32, or all
 *               NULL: request b's are those from bias_start[b] on
 *   mask        [T, ceil(V / 32)] int32, rows mask_stride apart, or NULL
 * Tokens outside [0, V) count for nothing (SV_ERR_TOKEN). A prefix_len or
 * prompt_len outside [0, max_history] is clamped to it (SV_ERR_LENGTH). A request
 * whose repetition is not > 0 (SV_ERR_PENALTY) or whose bias_start is wrong
 * (SV_ERR_LENGTH) gets rows of NaN, which every later step finds (SV_ERR_ROW). The
 * rows of a request with a wrong node_start (SV_ERR_TREE), and those outside every
 * request, are left as they were.
 * Status: SV_EINVAL (null pointer but ancestors, biases, mask, device_error or, with T = 0,
 * the [T, ...] arrays; biases not given together; B outside [1, 2^20], T < 0 or >= 2^31, V outside
 * [1, 2^22], max_nodes outside [1, 128], max_history < 1 or >= 2^31, num_bias < 0 or >= 2^31,
 * out_stride < V, history_stride < max_history, mask_stride < ceil(V / 32), a stride
 * below 0 or from 2^48 on, out that begins where logits does but differs in type or
 * stride), SV_EDTYPE, SV_EHIP.
 */
int specverify_penalize(const void* logits, int dtype, const int32_t* tokens,
                        const int32_t* node_start, const uint64_t* ancestors,
                        const int32_t* history, const int32_t* prefix_len,
                        const int32_t* prompt_len, const float* repetition, const float* presence,
                        const float* frequency, const int32_t* bias_start,
                        const int32_t* bias_token, const float* bias, const int32_t* mask,
                        int64_t B, int64_t T, int64_t V, int64_t max_nodes, int64_t max_history,
                        int64_t num_bias, int64_t stride, int64_t out_stride,
                        int64_t history_stride, int64_t mask_stride, void* out, int out_dtype,
                        int32_t* device_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_SERVING_H */
