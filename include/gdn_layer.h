/*
 * gdn_layer.h -- C ABI of the layer around the draft tree: prompts and single
 * tokens through the gated delta rule, and the norms and gates that stand before
 * and after it.  A serving loop makes the committed state of gdn_tree.h with
 * gdn_prefill, verifies and commits draft trees on it, and falls back to
 * gdn_decode for a request without a draft; gdn_qk_gates makes the inputs of all
 * of them from a layer's projections, gdn_norm_gate and gdn_residual_norm take
 * their outputs back to the residual stream.
 *
 * Conventions are those of gdn_tree.h (device pointers, the caller's stream,
 * nothing allocated, gdn_status returned, gdn_last_error, GDN_DEV_* bits in
 * *dev_status, S[d_v][d_k] in fp32), and:
 *   - Token rows.  q, k [T][Hk][d_k], v [T][Hv][d_v] and the other inputs marked
 *     "strided" are given with the distance between consecutive tokens in
 *     elements (0: contiguous), so a slice of a fused projection is read in place.
 *     Inside a token the heads are contiguous.  Every other array is contiguous.
 *   - States lie in a pool [n_states][Hv][d_v][d_k]; request b uses the state
 *     slots[b], or state b where slots is NULL.  Two requests of one call must not
 *     share a slot.  The pools are 16-byte aligned.
 *   - Supported: d_k, d_v in {16, 32, 64, 128}, Hv a multiple of Hk, tokens in fp32
 *     or bf16.  Sums, norms and states are fp32.
 */
#ifndef GDN_LAYER_H_
#define GDN_LAYER_H_

#include "gdn_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a further bit OR-ed into *dev_status: a slot outside the pool */
#define GDN_DEV_BAD_SLOT    128

typedef struct {
    int32_t batch, n_k_heads, n_v_heads, d_k, d_v;
    int32_t total_tokens;   /* T: rows of q, k, v, g, beta, o */
    int32_t max_tokens;     /* upper bound on any prompt's length */
    int32_t n_states;       /* states in S0 and S_new */
    float scale;            /* output scale */
    int32_t qkv_dtype;      /* gdn_dtype of q, k, v */
    int32_t out_dtype;      /* gdn_dtype of o */
    int64_t q_stride, k_stride, v_stride;  /* elements between tokens, 0 = contiguous */
    const int32_t *token_offsets;          /* [B+1] ascending, from 0 to at most T */
    const void *q, *k, *v;
    const float *g, *beta;  /* [T][Hv] log-decay and write strength */
    const float *S0;        /* pool of initial states; NULL: every prompt starts from zero */
    const int32_t *slots;   /* [B] or NULL */
    const int32_t *fresh;   /* [B] or NULL: a nonzero entry starts its prompt from zero */
    void *o;                /* [T][Hv][d_v] */
    float *S_new;           /* pool of final states; may be S0 (in place) */
    void *workspace;        /* gdn_prefill_workspace() bytes, 256-byte aligned; NULL if that is 0 */
    int64_t workspace_bytes;
    int32_t *dev_status;
} gdn_prefill_args;

/*
 * gdn_prefill -- prompts of different lengths, packed: the gated delta rule over
 * each prompt from its initial state,
 *     S <- e^g_t S;  u = beta_t (v_t - S k_t);  S <- S + u k_t^T;  o_t = scale S q_t,
 * every token's output and the final state.  A prompt of length zero copies its
 * initial state.  A prompt longer than max_tokens sets GDN_DEV_TOO_MANY, offsets
 * that descend or pass T set GDN_DEV_BAD_DESC, and a slot outside the pool sets
 * GDN_DEV_BAD_SLOT; that request is skipped, its outputs and state are not written.
 * g = -infinity forgets the state.  A NaN or infinity in q, k or v, or a NaN in g or beta,
 * may reach any output of its own 64-token chunk, and of the tokens after it.
 * bf16 q/k/v/o with d_k = d_v = 128, 16-byte aligned rows and 32-byte aligned pools
 * run the chunked tensor-core kernel, unless the prompts are few and short (max_tokens
 * at most 28); everything else runs the recurrent one.  Where few prompts are long, the
 * chunked kernel cuts them into segments and needs the workspace.
 * The recurrent kernel computes in fp32 whatever the types, a token after another: bf16 prompts
 * with fp32 outputs get that, and take about ten times the chunked kernel's time (one prompt of
 * 16384 tokens, 32 heads: 5.2 ms, 0.5 ms).
 * Errors, norm-wise: states about 4e-6 (chunked) or 3e-7 (recurrent), bf16 outputs 1.68e-3
 * (chunked) or 1.66e-3, which is their own rounding.
 */
GDN_API int gdn_prefill(const gdn_prefill_args *args, void *stream);

/* Bytes of workspace that gdn_prefill needs for these sizes (only the sizes and types of
 * args are read, and whether its rows are strided); -1 for sizes that it would refuse. */
GDN_API int64_t gdn_prefill_workspace(const gdn_prefill_args *args);

typedef struct {
    int32_t batch, n_k_heads, n_v_heads, d_k, d_v;
    int32_t n_states;       /* states in S */
    float scale;
    int32_t qkv_dtype, out_dtype;
    int64_t q_stride, k_stride, v_stride;  /* elements between requests, 0 = contiguous */
    const void *q, *k, *v;  /* [B][Hk][d_k], [B][Hk][d_k], [B][Hv][d_v] */
    const float *g, *beta;  /* [B][Hv] */
    float *S;               /* pool, updated in place */
    const int32_t *slots;   /* [B] or NULL; -1: the row is not in use */
    void *o;                /* [B][Hv][d_v] */
    int32_t *dev_status;
} gdn_decode_args;

/*
 * gdn_decode -- one token for each request: the step of gdn_prefill on a state in
 * the pool.  A row whose slot is -1 (a batch padded to its graph's size) gets zeros
 * in o and touches no state; any other slot outside the pool sets GDN_DEV_BAD_SLOT
 * and its row is skipped.
 */
GDN_API int gdn_decode(const gdn_decode_args *args, void *stream);

typedef struct {
    int32_t total_tokens, n_k_heads, n_v_heads, d_k;
    float eps;
    int32_t dtype;          /* gdn_dtype of q, k, a, b and of q_out, k_out */
    int64_t q_stride, k_stride, a_stride, b_stride;  /* elements between tokens, 0 = contiguous */
    const void *q, *k;      /* [T][Hk][d_k] */
    const void *a, *b;      /* [T][Hv] */
    const float *A_log, *dt_bias;  /* [Hv] */
    void *q_out, *k_out;    /* [T][Hk][d_k]; may be q, k where those are contiguous */
    float *g, *beta;        /* [T][Hv] */
} gdn_qk_gates_args;

/*
 * gdn_qk_gates -- what stands before the rule: q and k of unit length per head,
 *     q_out = q / sqrt(sum q^2 + eps)          (k alike)
 *     g     = -exp(A_log) * log(1 + exp(a + dt_bias))
 *     beta  = 1 / (1 + exp(-b))
 */
GDN_API int gdn_qk_gates(const gdn_qk_gates_args *args, void *stream);

typedef enum { GDN_ACT_SILU = 0, GDN_ACT_SIGMOID = 1 } gdn_act;

typedef struct {
    int32_t total_tokens, n_v_heads, d_v;
    float eps;
    int32_t act;            /* gdn_act */
    int32_t dtype;          /* gdn_dtype of o, z and y */
    int32_t weight_dtype;   /* gdn_dtype of weight */
    int64_t o_stride, z_stride;  /* elements between tokens, 0 = contiguous */
    const void *o, *z;      /* [T][Hv][d_v] */
    const void *weight;     /* [d_v] */
    void *y;                /* [T][Hv][d_v]; may be o or z where that is contiguous */
} gdn_norm_gate_args;

/*
 * gdn_norm_gate -- what stands after the rule: each head's output normed and gated,
 *     y = o / sqrt(mean o^2 + eps) * weight * act(z),
 * act(z) = z / (1 + exp(-z)) (silu) or 1 / (1 + exp(-z)) (sigmoid).
 */
GDN_API int gdn_norm_gate(const gdn_norm_gate_args *args, void *stream);

typedef struct {
    int32_t total_tokens, width;
    float scale, eps;
    int32_t dtype;          /* gdn_dtype of x, y, h and n */
    int32_t weight_dtype;   /* gdn_dtype of weight and post_weight */
    int64_t x_stride, y_stride;  /* elements between tokens, 0 = contiguous */
    const void *x, *y;      /* [T][width] residual stream, block output */
    const void *weight;     /* [width] */
    const void *post_weight;  /* [width], or NULL: the block's output is added as it is */
    void *h, *n;            /* [T][width]; h may be x, n may be y, where those are contiguous */
} gdn_residual_norm_args;

/*
 * gdn_residual_norm -- between two blocks: the block's output y (after its own norm
 * where post_weight is given) added to the residual stream, and the next block's norm,
 *     y' = y / sqrt(mean y^2 + eps) * post_weight,  or y
 *     h  = x + scale * y'
 *     n  = h / sqrt(mean h^2 + eps) * weight        (of the unrounded h)
 * Any width from 1 to 65536.
 */
GDN_API int gdn_residual_norm(const gdn_residual_norm_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H_ */
