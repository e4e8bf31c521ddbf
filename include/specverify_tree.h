/*
 * specverify_tree.h -- the verification step of a drafted token TREE on AMD
 * Instinct MI355X (gfx950), as a C ABI beside specverify.h (same library, same
 * conventions: device pointers, caller-owned buffers, no allocation and no
 * synchronisation, host checks before anything is enqueued, bit-deterministic
 * results).
 *
 * A serving loop calls, per decoding step of B requests,
 *   specverify_tree_plan       ancestor masks, positions, pages and slots
 *   specverify_tree_attention  the nodes' attention over the paged cache and
 *                              their ancestors (once per layer)
 *   specverify_tree_verify     the accepted path and the emitted token, from
 *                              probabilities and given uniforms
 *   specverify_tree_commit     the accepted nodes' keys and values into the pages
 *
 * Trees
 * -----
 * - The nodes of all requests are packed: request b owns rows
 *   node_start[b] .. node_start[b + 1] - 1 of every [T, ...] array, n_b of them
 *   (0 <= n_b <= max_nodes). Rows of [T, ...] outputs behind node_start[B] are
 *   left as they were.
 * - Row 0 of a request is its root: the last emitted token, whose keys and
 *   values are not in the cache yet. parents[i] is an index within the request,
 *   -1 for the root and 0 <= parents[i] < i for every other node. The children
 *   of a node are ordered by their index.
 * - A chain of gamma drafted tokens is the tree parents[i] = i - 1 with
 *   n = gamma + 1; a single decoded token is a tree of one node.
 * - The drafted nodes' keys and values stay OUTSIDE the cache, dense per node,
 *   until they are committed: a rejected node never takes a slot.
 *
 * Pages
 * -----
 * - The cache of a layer is [num_pages, page_size, heads, D] with D contiguous
 *   and any other strides; page_size is a power of two. Strides are in elements
 *   here and everywhere, 0 <= stride < 2^48.
 *   Position i of request b is at slot block_table[b, i / page_size] *
 *   page_size + i % page_size.
 *
 * Errors in device data never touch memory out of range: they set bits of the
 * optional device error word (only set, never cleared) and give the outputs
 * that each entry point names.
 *
 * Every call has to be made with the device of its pointers and stream current.
 */
#ifndef SPECVERIFY_TREE_H
#define SPECVERIFY_TREE_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Storage type beside SV_F32 and SV_BF16: IEEE half precision. */
#define SV_F16 2

/* Size limits checked on the host. */
#define SV_MAX_TREE_NODES 128            /* nodes of one request             */
#define SV_MAX_TREE_VOCAB (1 << 22)      /* vocabulary of tree_verify        */
#define SV_MAX_HEAD_DIM 256              /* width of a head, a multiple of 8 */

/* Bits OR-ed into the device error word, beside SV_ERR_TOKEN and SV_ERR_ROW. */
#define SV_ERR_TREE 8     /* node_start or parents are no tree, or it is deeper
                             than max_path - 1                               */
#define SV_ERR_PAGE 16    /* a page or slot outside the cache, or no free page */
#define SV_ERR_UNIFORM 32 /* a given uniform outside [0, 1) or NaN           */
#define SV_ERR_LENGTH 64  /* a prefix that is negative, longer than its pages
                             or than the block table                         */

/* How the drafted children of a node were drawn (specverify_tree_verify). */
#define SV_DRAFT_FIXED 0    /* given tokens, no draft probabilities            */
#define SV_DRAFT_IID 1      /* independent draws from the node's draft row     */
#define SV_DRAFT_DISTINCT 2 /* draws without replacement from the draft row    */

/*
 * Plan of a step: topology of the trees, and room in the cache for what may be
 * committed, in one launch.
 *   parents     [T] int32, node_start [B+1] int32: the trees
 *   prefix_len  [B] int32: tokens in the cache
 *   pages_in    [B] int32: pages that the request owns; block_table[b, 0 ..
 *               pages_in[b]) are valid
 *   block_table [B, max_pages] int32, rows table_stride apart, updated in place:
 *               entries from pages_in[b] on are filled with the pages taken
 *   free_pages  [num_free] int32, of which those from *free_head_in on are free
 *   max_path    longest path including its root (1 <= max_path <= max_nodes)
 *   ancestors   [T, W] uint64 out, W = ceil(max_nodes / 64): bit m % 64 of word
 *               m / 64 is set when node m is an ancestor of the row's node or
 *               the node itself
 *   depth       [T] int32 out: 0 for the root
 *   position    [T] int32 out: prefix_len + depth
 *   slots       [B, max_path] int64 out: where the i-th token of the committed
 *               path goes, for i < min(n_b, max_path); -1 elsewhere
 *   pages_out   [B] int32 out: pages_in + the pages taken
 *   free_head_out [1] int32 out: *free_head_in + all pages taken
 * A request takes the pages that prefix_len + min(n_b, max_path) tokens need
 * beyond those it owns, in request order from the free list and whatever its
 * parents are; one that needs pages takes none when the list does not reach for
 * it and all before it (SV_ERR_PAGE, slots -1).
 * A request whose tree is wrong (SV_ERR_TREE) gets ancestors 0, depth and
 * position -1 and slots -1; one with wrong lengths (SV_ERR_LENGTH) takes no
 * page and gets positions and slots -1. An entry of free_pages or block_table
 * outside [0, num_pages) that a slot needs gives slot -1 (SV_ERR_PAGE).
 * pages_out and free_head_out must not be pages_in and free_head_in.
 * Status: SV_EINVAL (null pointer but device_error, parents, ancestors, depth
 * or position with T = 0; B < 1, T < 0, max_nodes outside [1, 128], max_path
 * outside [1, max_nodes], page_size no power of two, max_pages, num_pages < 1
 * or num_free < 0 or any of them >= 2^31, B * max_pages or max_pages * page_size
 * + max_nodes >= 2^31, table_stride < max_pages or no stride, pages_out or free_head_out that
 * is pages_in or free_head_in), SV_EHIP.
 */
int specverify_tree_plan(const int32_t* parents, const int32_t* node_start,
                         const int32_t* prefix_len, const int32_t* pages_in, int32_t* block_table,
                         const int32_t* free_pages, const int32_t* free_head_in, int64_t B,
                         int64_t T, int64_t max_nodes, int64_t max_path, int64_t page_size,
                         int64_t max_pages, int64_t table_stride, int64_t num_pages,
                         int64_t num_free, uint64_t* ancestors, int32_t* depth, int32_t* position,
                         int64_t* slots, int32_t* pages_out, int32_t* free_head_out,
                         int32_t* device_error, void* stream);

/*
 * Bytes of workspace of specverify_tree_attention (256-byte aligned, any
 * contents; calls that overlap in time need one each). Pure host function;
 * 0 for sizes the library rejects.
 */
size_t specverify_tree_attention_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                                                int64_t D, int64_t max_nodes);

/*
 * Attention of drafted nodes over a paged prefix and their ancestors:
 *   out[i, h] = sum_j softmax_j(scale * q[i, h] . k_j) v_j
 * over all prefix_len[b] cached positions of the node's request and the nodes m
 * of the request whose bit is set in ancestors[i]; query head h reads key head
 * h / (Hq / Hkv). Products and sums in float32; the softmax weights are rounded
 * to the storage type for the product with the values, the output once.
 *   q           [T, Hq, D], strides q_stride_t, q_stride_h
 *   k_tree, v_tree [T, Hkv, D], both with strides n_stride_t, n_stride_h
 *   k_cache, v_cache [num_pages, page_size, Hkv, D], both with strides
 *               c_stride_page, c_stride_token, c_stride_h
 *   dtype       SV_BF16 or SV_F16, of all of them and out
 *   block_table [B, max_pages] int32, rows table_stride apart
 *   prefix_len  [B] int32, node_start [B+1] int32
 *   ancestors   [T, ceil(max_nodes / 64)] uint64 as specverify_tree_plan
 *               writes it, or any other mask over the request's nodes (bits
 *               from n_b on are ignored); NULL: node i sees nodes 0 .. i
 *   scale       > 0, scale / ln 2 finite
 *   out         [T, Hq, D], strides o_stride_t, o_stride_h, one axis stepping over
 *               all that the other spans; must not overlap an input
 *   lse         [T, Hq] float32 out or NULL: ln of the softmax's denominator
 * A row that sees nothing (empty prefix and mask) gives zeros and lse = -inf.
 * Values in masked places (nodes a row does not see, slots behind prefix_len)
 * do not reach it, also when they are infinite or NaN. An infinite or NaN value
 * of a node that a row sees becomes that row's in its column, whatever its
 * weight; one in the cache makes the column of every row of its request and head
 * infinite or NaN. A page outside
 * [0, num_pages) counts as zero keys and values (SV_ERR_PAGE); a prefix_len
 * outside [0, max_pages * page_size] is clamped to it (SV_ERR_LENGTH); the rows
 * of a request with a wrong node_start are left as they were (SV_ERR_TREE).
 * Status: SV_EINVAL (null pointer but ancestors, lse, device_error or, with
 * T = 0, the [T, ...] arrays; B, Hq, Hkv < 1, Hq not a multiple of Hkv, T < 0,
 * D no multiple of 8 or outside [8, 256], max_nodes outside [1, 128],
 * max_nodes * Hq / Hkv > 2^16, B * Hkv > 2^24, page_size no power of two,
 * max_pages < 1 or max_pages * page_size + max_nodes > 2^31 - 2^14, T * Hq >= 2^31,
 * num_pages < 1, a stride below 0 or from 2^48 on, rows of out that overlap,
 * table_stride < max_pages, scale), SV_EDTYPE, SV_EALIGN (q, k, v, cache or out pointers or
 * strides not multiples of 16 bytes), SV_EWORKSPACE, SV_EHIP.
 */
int specverify_tree_attention(
    const void* q, const void* k_tree, const void* v_tree, const void* k_cache,
    const void* v_cache, int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
    int64_t max_nodes, int64_t q_stride_t, int64_t q_stride_h, int64_t n_stride_t,
    int64_t n_stride_h, int64_t c_stride_page, int64_t c_stride_token, int64_t c_stride_h,
    int64_t num_pages, int64_t page_size, const int32_t* block_table, int64_t max_pages,
    int64_t table_stride, const int32_t* prefix_len, const int32_t* node_start,
    const uint64_t* ancestors, float scale, void* out, int64_t o_stride_t, int64_t o_stride_h,
    float* lse, int32_t* device_error, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace of specverify_tree_verify (256-byte aligned, any contents;
 * calls that overlap in time need one each). Pure host function; 0 for sizes
 * the library rejects.
 */
size_t specverify_tree_verify_workspace_size(int64_t B, int64_t V, int64_t max_nodes);

/*
 * Verification of drafted trees against the target's probabilities from given
 * random numbers (recursive rejection sampling down the tree; with one chain
 * it is the step's accept test and residual draw).
 *   target_probs [T, V], rows t_stride apart: row i is the target's
 *                distribution after node i
 *   draft_probs  [T, V], rows d_stride apart: row i is the distribution that
 *                node i's children were drawn from (rows of leaves may hold
 *                anything); NULL for SV_DRAFT_FIXED
 *   dtype        SV_F32 or SV_BF16, of both
 *   tokens       [T] int32 (a root's is not read), parents, node_start: the trees
 *   u            [T] double in [0, 1): node i's accept uniform (a root's is not read)
 *   r            [B] double in [0, 1): draws the emitted token
 *   max_path     row length of path and emitted
 *   accept_len   [B] int32 out: accepted drafted nodes
 *   path         [B, max_path] int32 out: the root (0), then the accepted nodes
 *                (indices within the request), then -1
 *   emitted      [B, max_path] int32 out or NULL: the accepted nodes' tokens,
 *                then the drawn one, then -1
 *   out_token    [B] int32 out: the drawn token
 * The walk starts at the root. At a node with target row p and draft row q, let
 * w = p, S = 1, a = 0, Q = 1. Its children x are tried in order: x is accepted
 * iff u S q(x) / Q < w(x), and the walk goes on from it. A rejection sets
 * a += S / Q, w = max(p - a q, 0), S = sum w, and for SV_DRAFT_DISTINCT
 * Q -= q(x). (So w / S is the residual max(w / S - q, 0) of the distribution
 * before, normalised.) For SV_DRAFT_FIXED x is accepted iff u S < w(x), and a
 * rejection sets S -= w(x), w(x) = 0. When no child is left the token is the
 * least v with C(v) > r C(V - 1), C the running sum of w in id order; if w is
 * zero everywhere (by rounding) it is drawn from p. All in float64 on the
 * stored values; sums are taken in a fixed order.
 * A request with a wrong tree (SV_ERR_TREE; also an accepted path longer than
 * max_path), a tried token outside [0, V) (SV_ERR_TOKEN), a uniform that is
 * needed and wrong (SV_ERR_UNIFORM), or a negative, infinite or NaN
 * probability among those read or no mass at all in the row that the token is
 * drawn from (SV_ERR_ROW) gets -1 in every output. So does one with no nodes,
 * without an error bit. A node's target row is read whole when the walk ends
 * there, and with its draft row when a child of it is rejected (not for
 * SV_DRAFT_FIXED); else only at the tried children's tokens.
 * Status: SV_EINVAL (null pointer but emitted, device_error or, with T = 0, the
 * [T, ...] arrays; draft_probs missing or, for SV_DRAFT_FIXED, given; unknown
 * mode; B < 1, T < 0, V outside [1, 2^22], max_nodes outside [1, 128], max_path
 * outside [1, max_nodes], a stride below 0 or from 2^48 on), SV_EDTYPE, SV_EWORKSPACE,
 * SV_EALIGN (workspace), SV_EHIP.
 */
int specverify_tree_verify(const void* target_probs, const void* draft_probs, int dtype, int mode,
                           const int32_t* tokens, const int32_t* parents,
                           const int32_t* node_start, int64_t B, int64_t T, int64_t V,
                           int64_t max_nodes, int64_t max_path, int64_t t_stride, int64_t d_stride,
                           const double* u, const double* r, int32_t* accept_len, int32_t* path,
                           int32_t* emitted, int32_t* out_token, int32_t* device_error,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Commit of the accepted nodes: the keys and values of path[b, 0 ..
 * accept_len[b]] (root and accepted nodes) of every layer are written to
 * slots[b, 0 ..], and the lengths advance.
 *   k_tree, v_tree   [layers, T, H, D], both with strides n_stride_l, n_stride_t, n_stride_h
 *   k_cache, v_cache [layers, num_pages, page_size, H, D], both with strides
 *                    c_stride_l, c_stride_page, c_stride_token, c_stride_h; in
 *                    some order each axis steps over all that those before span
 *   dtype            SV_F32, SV_BF16 or SV_F16
 *   path, accept_len as specverify_tree_verify writes them; slots as
 *                    specverify_tree_plan does (slots of different requests differ)
 *   prefix_len_in    [B] int32; prefix_len_out [B] int32 out, may be prefix_len_in:
 *                    prefix_len_in + accept_len + 1
 * A request with accept_len < 0 is passed by (its length stays). One with
 * accept_len >= max_path or a path outside its nodes (SV_ERR_TREE) or a slot
 * outside the cache (SV_ERR_PAGE) is not committed at all: nothing is written
 * and its length stays. The nodes must not overlap the cache.
 * Status: SV_EINVAL (null pointer but device_error or, with T = 0, the nodes;
 * layers, B, H < 1, T < 0, D no multiple of 8 or outside [8, 256], max_nodes
 * outside [1, 128], max_path outside [1, max_nodes], num_pages < 1, page_size no
 * power of two, num_pages * page_size >= 2^40, layers * B >= 2^31, H >= 2^16,
 * a stride below 0 or from 2^48 on, tokens of the cache that overlap), SV_EDTYPE, SV_EALIGN
 * (pointers or strides of nodes or cache not multiples of 16 bytes), SV_EHIP.
 */
int specverify_tree_commit(const void* k_tree, const void* v_tree, void* k_cache, void* v_cache,
                           int dtype, int64_t layers, int64_t B, int64_t T, int64_t H, int64_t D,
                           int64_t max_nodes, int64_t max_path, int64_t n_stride_l,
                           int64_t n_stride_t, int64_t n_stride_h, int64_t c_stride_l,
                           int64_t c_stride_page, int64_t c_stride_token, int64_t c_stride_h,
                           int64_t num_pages, int64_t page_size, const int32_t* node_start,
                           const int32_t* path, const int32_t* accept_len, const int64_t* slots,
                           const int32_t* prefix_len_in, int32_t* prefix_len_out,
                           int32_t* device_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_TREE_H */
