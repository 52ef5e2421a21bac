/*
 * gdn_attention.h -- C ABI of the softmax-attention layers that stand between gated-delta-net
 * layers: a paged key-value cache, and what serving does with it.  Beside the calls of
 * gdn_tree.h and gdn_layer.h a step takes the same requests, draft trees and accepted paths:
 *
 *     prompts      gdn_kv_append, gdn_kv_attend          (gdn_prefill)
 *     one token    gdn_kv_append, gdn_kv_decode          (gdn_decode)
 *     draft trees  gdn_kv_append with the nodes' depths,
 *                  gdn_kv_attend under their ancestor masks  (gdn_tree_verify)
 *     acceptance   gdn_kv_commit                         (gdn_tree_commit)
 *
 * Conventions are those of gdn_layer.h (device pointers, the caller's stream, nothing allocated,
 * gdn_status returned, gdn_last_error, GDN_DEV_* bits in *dev_status, strided token rows), and:
 *   - Slots.  A request's tokens lie in slots 0, 1, ... of its cache: slot s of request b is
 *     row s % page_size of page page_table[b][s / page_size] of the pools k and v, each
 *     [n_pages][page_size][n_kv_heads][d] with any strides over the first three (given in
 *     elements, the same for k and v; d is contiguous), so that pools with heads before rows, or
 *     k and v in one tensor, are taken as they are.  Requests may share pages of tokens that
 *     are only read.  Pages behind a request's last slot are not looked at, and what lies in
 *     slots behind it, NaN among it, does not matter.
 *   - lens[b] is the number of committed tokens.  New tokens (a prompt, one token, a draft's
 *     nodes) go to the slots from lens[b] on and are seen there by gdn_kv_attend and
 *     gdn_kv_decode with the same lens; the caller, or gdn_kv_commit, advances it afterwards.  lens[b]
 *     = -1 marks a row that is not in use (a batch padded to its graph's size).
 *   - Query head h reads key-value head h / (n_q_heads / n_kv_heads).
 *   - A page outside the pool, or a slot past the table, sets GDN_DEV_BAD_PAGE.
 *   - Supported: d in {16, 32, 64, 128, 256}, n_q_heads a multiple of n_kv_heads, page sizes
 *     from 1 on, tokens and cache in fp32 or bf16 (alike), heads of a token up to 2^31 - 1 entries
 *     together.  Sums and softmax statistics are fp32.
 */
#ifndef GDN_ATTENTION_H_
#define GDN_ATTENTION_H_

#include "gdn_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* further bits OR-ed into *dev_status */
#define GDN_DEV_BAD_PAGE      256   /* a page outside the pool, or a slot past the page table */
#define GDN_DEV_BAD_POSITION  512   /* a position outside the rotation's table */

typedef struct {
    int32_t batch;
    int32_t n_pages, page_size;
    int32_t max_pages;          /* columns of page_table */
    int32_t n_kv_heads, d;
    int32_t dtype;              /* gdn_dtype of the pools, and of a call's tokens */
    int64_t page_stride, slot_stride, head_stride;  /* elements */
    void *k, *v;
    const int32_t *page_table;  /* [B][max_pages] */
    const int32_t *lens;        /* [B] */
    int32_t *dev_status;
} gdn_kv_cache;

typedef struct {
    gdn_kv_cache cache;
    int32_t total_tokens;       /* T: rows of q, k, v, q_out */
    int32_t n_q_heads;          /* ignored where q is NULL */
    int32_t rot_dim;            /* rotated entries at the head of each row, even; 0: none */
    int32_t interleaved;        /* pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2) */
    int32_t n_positions;        /* rows of cos_sin */
    int32_t weight_dtype;       /* gdn_dtype of q_weight and k_weight */
    float eps;
    int64_t q_stride, k_stride, v_stride;  /* elements between tokens, 0 = contiguous */
    const void *q;              /* [T][n_q_heads][d], or NULL: keys and values only */
    const void *k, *v;          /* [T][n_kv_heads][d] */
    const int32_t *token_offsets;  /* [B+1] ascending from 0, or NULL: token b is request b's only one */
    const int32_t *depth;       /* [T] as from gdn_tree_build_desc, or NULL */
    const float *cos_sin;       /* [n_positions][rot_dim]: cosines, then sines, of a position's angles */
    const void *q_weight, *k_weight;  /* [d], or NULL: no norm */
    void *q_out;                /* [T][n_q_heads][d]; may be q where that is contiguous */
} gdn_kv_append_args;

/*
 * gdn_kv_append -- what stands before attention: token i of request b, at position
 * p = lens[b] + i (with depths: lens[b] + depth - 1, so that a draft's nodes stand where their
 * path puts them), is normed per head where a weight is given,
 *     x <- x / sqrt(mean x^2 + eps) * weight                (queries by q_weight, keys by k_weight)
 * and rotated,
 *     (x_1, x_2) <- (x_1 cos - x_2 sin, x_2 cos + x_1 sin)  for each pair of the first rot_dim entries,
 * queries to q_out, keys to slot lens[b] + i of the cache, values as they are.  One rounding to
 * the output's type.  A row that is not in use is left out, its q_out unwritten, and so are tokens
 * behind the last request's.  Offsets that descend or pass T set GDN_DEV_BAD_DESC, a position
 * outside the table GDN_DEV_BAD_POSITION; such tokens are left out.  Two tokens of a call
 * must not share a slot.
 */
GDN_API int gdn_kv_append(const gdn_kv_append_args *args, void *stream);

typedef struct {
    gdn_kv_cache cache;
    int32_t total_tokens;       /* T: rows of q and o (gdn_kv_decode: the batch) */
    int32_t max_tokens;         /* upper bound on any request's new tokens (gdn_kv_decode: not read) */
    int32_t n_q_heads;
    int32_t mask_words;         /* words of a row of anc_mask */
    int32_t out_dtype;          /* gdn_dtype of o */
    float scale;                /* of the scores */
    int64_t q_stride;           /* elements between tokens, 0 = contiguous */
    const void *q;              /* [T][n_q_heads][d] */
    const int32_t *token_offsets;  /* [B+1] ascending from 0 (gdn_kv_decode: not read) */
    const uint32_t *anc_mask;   /* [T][mask_words], or NULL: causal (gdn_kv_decode: not read) */
    void *o;                    /* [T][n_q_heads][d], 16-byte aligned */
    void *workspace;            /* gdn_kv_attend_workspace() bytes, 256-byte aligned; NULL if that is 0 */
    int64_t workspace_bytes;
} gdn_kv_attend_args;

/*
 * gdn_kv_attend -- several new tokens of each request attend to its cache, in which their own keys and
 * values stand already: o_i = sum_s p_is v_s with p_i the softmax over the seen slots s of
 * scale q_i . k_s.  Token i sees every slot before lens[b], and of the new tokens j those
 * whose bit j is set in its row of anc_mask (that of gdn_tree_build_desc: its path in the draft tree),
 * or, without a mask, those up to itself (a prompt).  A token that sees nothing gets zeros, and so do
 * the tokens of a row that is not in use; rows of o behind the last request's are left as they were.
 * A request longer than max_tokens, or than the mask has bits, sets GDN_DEV_TOO_MANY, offsets that
 * descend or pass T GDN_DEV_BAD_DESC, slots past the page table GDN_DEV_BAD_PAGE; that request is left out,
 * its outputs are not written.  After a page outside the pool the request's outputs are unspecified.
 * A NaN or infinity in a key or value reaches the tokens that see it, and no others (the whole
 * rows of those, as NaN, where it stands in the value of a new token); a token all of whose scores are
 * -infinity is NaN.
 * The work is cut along the slots into equal parts, one for each running block, whatever the lengths
 * are; parts of one token's softmax are joined by a second kernel in a fixed order: the same call gives the
 * same bits.  Page tables with room for few slots (1024 for the warp products, 128 for the general kernel; the room
 * counts, not the lengths) are not cut.
 * bf16 rows that start on 16 bytes run on the tensor cores.  More than 16 rows (max_tokens x query heads of a key-value head)
 * take tcgen05, with d from 64 on, pages of a multiple of 8 slots, at most 128 query heads to a key-value head and a positive
 * scale: there probabilities are rounded to bf16 before they are multiplied by values (2^-8 of each; their sum is kept of the
 * unrounded ones).  Others, and every gdn_kv_decode, take warp products of 16 rows, with probabilities as two bf16 numbers (2^-16).
 * fp32, and rows that do not start on 16 bytes, run the general kernel in fp32 arithmetic.
 */
GDN_API int gdn_kv_attend(const gdn_kv_attend_args *args, void *stream);

/*
 * gdn_kv_decode -- one new token for each request, token b for request b: gdn_kv_attend with
 * lens[b] + 1 slots seen.  The cache is read once for every 16 query heads of a key-value head; with more of them gdn_kv_attend
 * with one token a request, which reads it once, takes less (64 tokens over 100 to 8000 slots, heads of 128, 32 to one: 66 us
 * where this takes 94, 128 to one: 48 and 163).
 */
GDN_API int gdn_kv_decode(const gdn_kv_attend_args *args, void *stream);

/* Bytes of workspace that gdn_kv_attend, or gdn_kv_decode (decode nonzero), needs for these sizes (only the sizes, types,
 * strides, the sign of scale and the alignment of q and the pools are read); -1 for sizes that it would refuse.  A call uses its workspace alone:
 * two calls that may run at the same time need two. */
GDN_API int64_t gdn_kv_attend_workspace(const gdn_kv_attend_args *args, int32_t decode);

typedef struct {
    gdn_kv_cache cache;
    const int32_t *node_offsets;   /* [B+1] as for gdn_tree_commit */
    const int32_t *path_offsets;   /* [B+1] */
    const int32_t *path_idx;       /* request-local node ids, ascending within a path */
    int32_t total_path;            /* entries of path_idx */
    int32_t *new_lens;             /* [B], or NULL; not lens itself */
} gdn_kv_commit_args;

/*
 * gdn_kv_commit -- the accepted path's tokens move to where committed ones stand: slot
 * lens[b] + path[i] to slot lens[b] + i, in place, and new_lens[b] = lens[b] + the path's length.
 * A path that does not ascend within its request's nodes, or has more than 2^20, sets GDN_DEV_BAD_PATH, offsets that descend
 * (or pass total_path) GDN_DEV_BAD_DESC, a slot past the page table or a page outside the
 * pool GDN_DEV_BAD_PAGE: that request's cache stays as it was, and new_lens[b] = lens[b].
 */
GDN_API int gdn_kv_commit(const gdn_kv_commit_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTENTION_H_ */
