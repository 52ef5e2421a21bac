// layer_api.cu -- host side of gdn_layer.h: argument checks and kernel choice.
#include <cmath>

#include "internal.cuh"

namespace {

using gdn::fail;

int done(cudaError_t e, const char *what) {
    return e == cudaSuccess ? GDN_OK : fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool supported_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

bool valid_dtype(int t) { return t == GDN_F32 || t == GDN_BF16; }

int check_heads(int hk, int hv) {
    if (hk < 1 || hv < 1) return fail(GDN_ERR_INVALID_ARG, "head counts must be >= 1");
    if (hv % hk) return fail(GDN_ERR_INVALID_ARG, "n_v_heads %d not a multiple of n_k_heads %d", hv, hk);
    if (hv > 65536) return fail(GDN_ERR_UNSUPPORTED, "n_v_heads %d > 65536", hv);
    return GDN_OK;
}

// a stride of 0 stands for contiguous rows of `row` elements
int check_stride(const char *name, int64_t stride, int64_t row) {
    if (stride && stride < row)
        return fail(GDN_ERR_INVALID_ARG, "%s_stride %lld: rows of %lld elements would overlap", name, (long long)stride, (long long)row);
    return GDN_OK;
}

int check_rule(int batch, int hk, int hv, int dk, int dv, int n_states, float scale, int qkv_dtype, int out_dtype, int64_t qs,
               int64_t ks, int64_t vs) {
    if (batch < 0) return fail(GDN_ERR_INVALID_ARG, "batch %d < 0", batch);
    if (int st = check_heads(hk, hv)) return st;
    if (!supported_dim(dk) || !supported_dim(dv))
        return fail(GDN_ERR_UNSUPPORTED, "d_k=%d d_v=%d: supported sizes are 16, 32, 64, 128", dk, dv);
    if (!valid_dtype(qkv_dtype) || !valid_dtype(out_dtype))
        return fail(GDN_ERR_UNSUPPORTED, "unknown dtype (qkv %d, out %d)", qkv_dtype, out_dtype);
    if (n_states < 0) return fail(GDN_ERR_INVALID_ARG, "n_states %d < 0", n_states);
    if (!std::isfinite(scale)) return fail(GDN_ERR_INVALID_ARG, "scale is not finite");
    if (int st = check_stride("q", qs, (int64_t)hk * dk)) return st;
    if (int st = check_stride("k", ks, (int64_t)hk * dk)) return st;
    return check_stride("v", vs, (int64_t)hv * dv);
}

int check_eps(float eps) {
    return std::isfinite(eps) && eps >= 0.f ? GDN_OK : fail(GDN_ERR_INVALID_ARG, "eps must be finite and >= 0");
}

int check_prefill(const gdn_prefill_args *a) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    if (int st = check_rule(a->batch, a->n_k_heads, a->n_v_heads, a->d_k, a->d_v, a->n_states, a->scale, a->qkv_dtype,
                            a->out_dtype, a->q_stride, a->k_stride, a->v_stride))
        return st;
    if (a->total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "total_tokens %d < 0", a->total_tokens);
    if (a->max_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "max_tokens %d < 0", a->max_tokens);
    return GDN_OK;
}

// Whether the chunked kernel runs.  A chunk takes it 12 us whatever it holds.  The recurrent one takes four tokens in
// about 1.3 us while its blocks are spread over idle SMs (one prompt of 32 heads, 8 / 16 / 28 / 32 / 64 tokens: 5.5,
// 7.1, 11.2, 11.9, 21.6 us against 12), longer where there are more of them (four prompts of 1 / 4 / 8 / 16 tokens:
// 12.3, 12.5, 15.4, 20.7 against 12.3), and with a (prompt, head) for every SM the chunked one is ahead from one token
// on (eight prompts of 1 / 16 tokens: 20.5, 34.7 against 18).
bool chunked(const gdn_prefill_args &a) {
    const int64_t items = (int64_t)a.batch * a.n_v_heads;
    return gdn::prefill_tc_supported(a) && (a.max_tokens > 28 || items >= gdn::sm_count() || items * a.max_tokens > 28 * 32);
}

}  // namespace

extern "C" {

int64_t gdn_prefill_workspace(const gdn_prefill_args *a) {
    gdn::clear_error();
    if (check_prefill(a)) return -1;
    return a->batch > 0 && chunked(*a) ? gdn::prefill_tc_workspace(*a) : 0;
}

int gdn_prefill(const gdn_prefill_args *a, void *stream) {
    gdn::clear_error();
    if (int st = check_prefill(a)) return st;
    if (a->batch == 0) return GDN_OK;
    if (!a->token_offsets || !a->S_new) return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    if (a->total_tokens > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->o))
        return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    if ((reinterpret_cast<uintptr_t>(a->S0) | reinterpret_cast<uintptr_t>(a->S_new)) & 15)
        return fail(GDN_ERR_INVALID_ARG, "S0 and S_new must be 16-byte aligned");
    if (chunked(*a)) {
        const int64_t need = gdn::prefill_tc_workspace(*a);
        if (need > 0 && (!a->workspace || a->workspace_bytes < need))
            return fail(GDN_ERR_INVALID_ARG, "workspace of %lld bytes: %lld are needed", (long long)(a->workspace ? a->workspace_bytes : 0), (long long)need);
        if (need > 0 && (reinterpret_cast<uintptr_t>(a->workspace) & 255))
            return fail(GDN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
        return done(gdn::launch_prefill_tc(*a, (cudaStream_t)stream), "prefill launch");
    }
    return done(gdn::launch_prefill_simt(*a, (cudaStream_t)stream), "prefill launch");
}

int gdn_decode(const gdn_decode_args *a, void *stream) {
    gdn::clear_error();
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    if (int st = check_rule(a->batch, a->n_k_heads, a->n_v_heads, a->d_k, a->d_v, a->n_states, a->scale, a->qkv_dtype,
                            a->out_dtype, a->q_stride, a->k_stride, a->v_stride))
        return st;
    if (a->batch == 0) return GDN_OK;
    if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->S || !a->o)
        return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    if (reinterpret_cast<uintptr_t>(a->S) & 15) return fail(GDN_ERR_INVALID_ARG, "S must be 16-byte aligned");
    return done(gdn::launch_decode(*a, (cudaStream_t)stream), "decode launch");
}

int gdn_qk_gates(const gdn_qk_gates_args *a, void *stream) {
    gdn::clear_error();
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    if (a->total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "total_tokens %d < 0", a->total_tokens);
    if (int st = check_heads(a->n_k_heads, a->n_v_heads)) return st;
    if (!supported_dim(a->d_k)) return fail(GDN_ERR_UNSUPPORTED, "d_k=%d: supported sizes are 16, 32, 64, 128", a->d_k);
    if (!valid_dtype(a->dtype)) return fail(GDN_ERR_UNSUPPORTED, "unknown dtype %d", a->dtype);
    if (int st = check_eps(a->eps)) return st;
    const int64_t row = (int64_t)a->n_k_heads * a->d_k;
    if (int st = check_stride("q", a->q_stride, row)) return st;
    if (int st = check_stride("k", a->k_stride, row)) return st;
    if (int st = check_stride("a", a->a_stride, a->n_v_heads)) return st;
    if (int st = check_stride("b", a->b_stride, a->n_v_heads)) return st;
    if (a->total_tokens == 0) return GDN_OK;
    if (!a->q || !a->k || !a->a || !a->b || !a->A_log || !a->dt_bias || !a->q_out || !a->k_out || !a->g || !a->beta)
        return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    return done(gdn::launch_qk_gates(*a, (cudaStream_t)stream), "qk_gates launch");
}

int gdn_norm_gate(const gdn_norm_gate_args *a, void *stream) {
    gdn::clear_error();
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    if (a->total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "total_tokens %d < 0", a->total_tokens);
    if (int st = check_heads(a->n_v_heads, a->n_v_heads)) return st;
    if (!supported_dim(a->d_v)) return fail(GDN_ERR_UNSUPPORTED, "d_v=%d: supported sizes are 16, 32, 64, 128", a->d_v);
    if (!valid_dtype(a->dtype) || !valid_dtype(a->weight_dtype))
        return fail(GDN_ERR_UNSUPPORTED, "unknown dtype (%d, weight %d)", a->dtype, a->weight_dtype);
    if (a->act != GDN_ACT_SILU && a->act != GDN_ACT_SIGMOID) return fail(GDN_ERR_UNSUPPORTED, "unknown activation %d", a->act);
    if (int st = check_eps(a->eps)) return st;
    const int64_t row = (int64_t)a->n_v_heads * a->d_v;
    if (int st = check_stride("o", a->o_stride, row)) return st;
    if (int st = check_stride("z", a->z_stride, row)) return st;
    if (a->total_tokens == 0) return GDN_OK;
    if (!a->o || !a->z || !a->weight || !a->y) return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    return done(gdn::launch_norm_gate(*a, (cudaStream_t)stream), "norm_gate launch");
}

int gdn_residual_norm(const gdn_residual_norm_args *a, void *stream) {
    gdn::clear_error();
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    if (a->total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "total_tokens %d < 0", a->total_tokens);
    if (a->width < 1) return fail(GDN_ERR_INVALID_ARG, "width %d < 1", a->width);
    if (a->width > 65536) return fail(GDN_ERR_UNSUPPORTED, "width %d > 65536", a->width);
    if (!valid_dtype(a->dtype) || !valid_dtype(a->weight_dtype))
        return fail(GDN_ERR_UNSUPPORTED, "unknown dtype (%d, weight %d)", a->dtype, a->weight_dtype);
    if (!std::isfinite(a->scale)) return fail(GDN_ERR_INVALID_ARG, "scale is not finite");
    if (int st = check_eps(a->eps)) return st;
    if (int st = check_stride("x", a->x_stride, a->width)) return st;
    if (int st = check_stride("y", a->y_stride, a->width)) return st;
    if (a->total_tokens == 0) return GDN_OK;
    if (!a->x || !a->y || !a->weight || !a->h || !a->n) return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
    return done(gdn::launch_residual_norm(*a, (cudaStream_t)stream), "residual_norm launch");
}

}  // extern "C"
