// attn_api.cu -- host side of gdn_attention.h: argument checks and kernel choice.
#include <cmath>

#include "attn.cuh"

namespace {

using gdn::fail;

int done(cudaError_t e, const char *what) {
    return e == cudaSuccess ? GDN_OK : fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool valid_dtype(int t) { return t == GDN_F32 || t == GDN_BF16; }

// Limits that keep slots, rows, grids and places within a token's row within 32 bits: 2^30 slots a request, 2^30 rows of
// query heads a call, 2^30 (request, head)s, 2^31 - 1 entries of a token's heads.
constexpr int64_t kMost = 1 << 30;

int check_cache(const gdn_kv_cache &c) {
    if (c.batch < 0) return fail(GDN_ERR_INVALID_ARG, "batch %d < 0", c.batch);
    if (c.n_pages < 0 || c.max_pages < 0) return fail(GDN_ERR_INVALID_ARG, "n_pages %d, max_pages %d: must be >= 0", c.n_pages, c.max_pages);
    if (c.page_size < 1) return fail(GDN_ERR_INVALID_ARG, "page_size %d < 1", c.page_size);
    if ((int64_t)c.page_size * c.max_pages > kMost)
        return fail(GDN_ERR_UNSUPPORTED, "%d pages of %d slots a request: more than 2^30 slots", c.max_pages, c.page_size);
    if (c.n_kv_heads < 1) return fail(GDN_ERR_INVALID_ARG, "head counts must be >= 1");
    if ((int64_t)c.batch * c.n_kv_heads > kMost) return fail(GDN_ERR_UNSUPPORTED, "more than 2^30 key-value heads in a call");
    if (c.d != 16 && c.d != 32 && c.d != 64 && c.d != 128 && c.d != 256)
        return fail(GDN_ERR_UNSUPPORTED, "d=%d: supported sizes are 16, 32, 64, 128, 256", c.d);
    if (!valid_dtype(c.dtype)) return fail(GDN_ERR_UNSUPPORTED, "unknown dtype %d", c.dtype);
    if (c.page_stride < 0 || c.slot_stride < 0 || c.head_stride < 0)
        return fail(GDN_ERR_INVALID_ARG, "strides of the cache must be >= 0");
    return GDN_OK;
}

int check_cache_pointers(const gdn_kv_cache &c) {
    if (!c.lens || (c.max_pages > 0 && !c.page_table) || (c.n_pages > 0 && (!c.k || !c.v)))
        return fail(GDN_ERR_INVALID_ARG, "a required pointer of the cache is NULL");
    return GDN_OK;
}

int check_stride(const char *name, int64_t stride, int64_t row) {
    if (stride && stride < row)
        return fail(GDN_ERR_INVALID_ARG, "%s_stride %lld: rows of %lld elements would overlap", name, (long long)stride, (long long)row);
    return GDN_OK;
}

int check_heads(int hq, int hkv) {
    if (hq < 1) return fail(GDN_ERR_INVALID_ARG, "head counts must be >= 1");
    if (hq % hkv) return fail(GDN_ERR_INVALID_ARG, "n_q_heads %d not a multiple of n_kv_heads %d", hq, hkv);
    return GDN_OK;
}

int check_row(const char *name, int heads, int d) {
    if ((int64_t)heads * d > INT32_MAX) return fail(GDN_ERR_UNSUPPORTED, "%s %d of %d entries: a token's row has 2^31 or more", name, heads, d);
    return GDN_OK;
}

int check_attend(const gdn_kv_attend_args *a, bool decode) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    const gdn_kv_cache &c = a->cache;
    if (int st = check_cache(c)) return st;
    if (int st = check_heads(a->n_q_heads, c.n_kv_heads)) return st;
    if (int st = check_row("n_q_heads", a->n_q_heads, c.d)) return st;
    if (!valid_dtype(a->out_dtype)) return fail(GDN_ERR_UNSUPPORTED, "unknown dtype (out %d)", a->out_dtype);
    if (a->total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "total_tokens %d < 0", a->total_tokens);
    if (decode && a->total_tokens != c.batch)
        return fail(GDN_ERR_INVALID_ARG, "total_tokens %d is not the batch %d", a->total_tokens, c.batch);
    if (!decode && a->max_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "max_tokens %d < 0", a->max_tokens);
    if (!decode && a->anc_mask && a->mask_words < 1) return fail(GDN_ERR_INVALID_ARG, "mask_words %d < 1", a->mask_words);
    if (!decode && a->anc_mask && a->mask_words > 1 << 20) return fail(GDN_ERR_UNSUPPORTED, "mask_words %d > 2^20", a->mask_words);
    if ((int64_t)a->total_tokens * a->n_q_heads > kMost) return fail(GDN_ERR_UNSUPPORTED, "more than 2^30 rows of query heads in a call");
    if (!std::isfinite(a->scale * gdn::attn::kLog2e)) return fail(GDN_ERR_INVALID_ARG, "scale %g is not finite, or too large", a->scale);
    return check_stride("q", a->q_stride, (int64_t)a->n_q_heads * c.d);
}

bool nothing(const gdn_kv_attend_args &a, bool decode) {
    return a.cache.batch == 0 || a.total_tokens == 0 || (!decode && a.max_tokens == 0);
}

// The kernel for a call: the tensor cores where a key-value head has more rows than the 16 of a warp product (eight drafts of 6 to 16
// nodes, 4 query heads each: 72 us by 16 rows at a time, 43 in tiles), by warp products below that, and the general kernel
// for fp32 and rows that do not start on 16 bytes.
gdn::attn::Choice choose(const gdn_kv_attend_args &a, bool decode) {
    if (!decode && a.max_tokens * (int64_t)(a.n_q_heads / a.cache.n_kv_heads) > 16 && gdn::attend_tc_supported(a)) return gdn::attend_tc_choice(a);
    return gdn::attend_mma_supported(a) ? gdn::attend_mma_choice(a, decode) : gdn::attend_simt_choice(a, decode);
}

int attend(const gdn_kv_attend_args *a, bool decode, void *stream) {
    if (int st = check_attend(a, decode)) return st;
    if (nothing(*a, decode)) return GDN_OK;
    const gdn_kv_cache &c = a->cache;
    if (int st = check_cache_pointers(c)) return st;
    if (!a->q || !a->o || (!decode && !a->token_offsets)) return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    if (reinterpret_cast<uintptr_t>(a->o) & 15) return fail(GDN_ERR_INVALID_ARG, "o must be 16-byte aligned");
    const gdn::attn::Choice x = choose(*a, decode);
    if (x.workspace > 0 && (!a->workspace || a->workspace_bytes < x.workspace))
        return fail(GDN_ERR_INVALID_ARG, "workspace of %lld bytes: %lld are needed", (long long)(a->workspace ? a->workspace_bytes : 0),
                    (long long)x.workspace);
    if (x.workspace > 0 && reinterpret_cast<uintptr_t>(a->workspace) & 255) return fail(GDN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    gdn::attn::Params p = {};
    p.batch = c.batch; p.hkv = c.n_kv_heads; p.group = a->n_q_heads / c.n_kv_heads;
    p.page_size = c.page_size; p.n_pages = c.n_pages; p.max_pages = c.max_pages;
    p.page_bits = (c.page_size & (c.page_size - 1)) ? -1 : __builtin_ctz((unsigned)c.page_size);
    p.total = a->total_tokens; p.max_tokens = decode ? 1 : a->max_tokens;
    p.page_stride = c.page_stride; p.slot_stride = c.slot_stride; p.head_stride = c.head_stride;
    p.q_stride = a->q_stride ? a->q_stride : (int64_t)a->n_q_heads * c.d;
    p.scale_log2 = a->scale * gdn::attn::kLog2e;
    // (a pool without pages is not read, but an address of its own spares the kernels a case)
    p.k = c.n_pages > 0 ? c.k : a->q; p.v = c.n_pages > 0 ? c.v : a->q; p.q = a->q; p.table = c.page_table; p.lens = c.lens;
    p.offsets = decode ? nullptr : a->token_offsets;
    p.mask = decode ? nullptr : a->anc_mask;
    p.mask_words = a->mask_words;
    p.whole = x.whole;
    p.o = a->o; p.out_bf16 = a->out_dtype == GDN_BF16; p.ws = static_cast<float *>(a->workspace); p.status = c.dev_status;
    return done(x.launch(p, x.runs, (cudaStream_t)stream), decode ? "kv_decode launch" : "kv_attend launch");
}

}  // namespace

extern "C" {

int gdn_kv_append(const gdn_kv_append_args *a, void *stream) {
    gdn::clear_error();
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    const gdn_kv_cache &c = a->cache;
    if (int st = check_cache(c)) return st;
    if (a->total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "total_tokens %d < 0", a->total_tokens);
    if (a->q) {
        if (int st = check_heads(a->n_q_heads, c.n_kv_heads)) return st;
        if (int st = check_row("n_q_heads", a->n_q_heads, c.d)) return st;
        if ((int64_t)a->total_tokens * a->n_q_heads > kMost) return fail(GDN_ERR_UNSUPPORTED, "more than 2^30 rows of query heads in a call");
        if (int st = check_stride("q", a->q_stride, (int64_t)a->n_q_heads * c.d)) return st;
    }
    if (int st = check_row("n_kv_heads", c.n_kv_heads, c.d)) return st;
    if (a->rot_dim < 0 || a->rot_dim > c.d || a->rot_dim % 2)
        return fail(GDN_ERR_INVALID_ARG, "rot_dim %d: must be even, at most d=%d", a->rot_dim, c.d);
    if (a->n_positions < 0) return fail(GDN_ERR_INVALID_ARG, "n_positions %d < 0", a->n_positions);
    if ((a->q_weight || a->k_weight) && !valid_dtype(a->weight_dtype)) return fail(GDN_ERR_UNSUPPORTED, "unknown dtype (weight %d)", a->weight_dtype);
    if (!(std::isfinite(a->eps) && a->eps >= 0.f)) return fail(GDN_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (int st = check_stride("k", a->k_stride, (int64_t)c.n_kv_heads * c.d)) return st;
    if (int st = check_stride("v", a->v_stride, (int64_t)c.n_kv_heads * c.d)) return st;
    if (!a->token_offsets && a->total_tokens != c.batch)
        return fail(GDN_ERR_INVALID_ARG, "total_tokens %d is not the batch %d, and there are no token_offsets", a->total_tokens, c.batch);
    if (c.batch == 0 || a->total_tokens == 0) return GDN_OK;
    if (int st = check_cache_pointers(c)) return st;
    if (!a->k || !a->v || (a->q && !a->q_out) || (a->rot_dim && a->n_positions > 0 && !a->cos_sin))
        return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    return done(gdn::launch_kv_append(*a, (cudaStream_t)stream), "kv_append launch");
}

int64_t gdn_kv_attend_workspace(const gdn_kv_attend_args *a, int32_t decode) {
    gdn::clear_error();
    if (check_attend(a, decode != 0)) return -1;
    return nothing(*a, decode != 0) ? 0 : choose(*a, decode != 0).workspace;
}

int gdn_kv_attend(const gdn_kv_attend_args *a, void *stream) {
    gdn::clear_error();
    return attend(a, false, stream);
}

int gdn_kv_decode(const gdn_kv_attend_args *a, void *stream) {
    gdn::clear_error();
    return attend(a, true, stream);
}

int gdn_kv_commit(const gdn_kv_commit_args *a, void *stream) {
    gdn::clear_error();
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    const gdn_kv_cache &c = a->cache;
    if (int st = check_cache(c)) return st;
    if (a->total_path < 0) return fail(GDN_ERR_INVALID_ARG, "total_path %d < 0", a->total_path);
    if (c.batch == 0) return GDN_OK;
    if (int st = check_cache_pointers(c)) return st;
    if (!a->node_offsets || !a->path_offsets || (a->total_path > 0 && !a->path_idx)) return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    if (a->new_lens && a->new_lens == c.lens) return fail(GDN_ERR_INVALID_ARG, "new_lens must not be lens");
    return done(gdn::launch_kv_commit(*a, (cudaStream_t)stream), "kv_commit launch");
}

}  // extern "C"
