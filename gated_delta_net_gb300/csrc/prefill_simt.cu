// prefill_simt.cu -- prompts through the gated delta rule, one token after another:
// the general kernel, any supported widths, types and strides.
//
// A block takes a slab of state rows of one (prompt, value head); rows of S do not
// meet, so slabs are independent.  A row's d_k entries lie in the registers of d_k / 16
// lanes for the whole prompt.  Per token, with the old state,
//     u = beta (v - e^g S k),  o = scale (e^g S q + u (k . q)),  S <- e^g S + u k^T,
// so that both products are reduced together and the step's chain is one reduction
// and one update.  Tokens come in tiles of 16 through shared memory: the next tile's
// values are loaded into registers before the present tile is worked off.  The chain
// over the tokens bounds it: about 0.1 us a token whatever the number of heads, until
// the heads' blocks fill the GPU.
#include "internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 16;  // tokens a tile

struct Params {
    int hk, hv, dv, total, max_tokens, n_states, slabs;
    int64_t qs, ks, vs;
    float scale;
    const int32_t *offsets, *slots, *fresh;
    const void *q, *k, *v;
    const float *g, *beta, *S0;
    void *o;
    float *S_new;
    int32_t *status;
};

template <typename T, typename O, int DK>
__global__ void __launch_bounds__(kThreads) prefill_simt_kernel(Params p) {
    constexpr int LPR = DK / 16, kRows = kThreads / LPR;  // rows a block
    constexpr int kLoadK = kTile * DK / kThreads, kLoadV = kTile * (kRows < 128 ? kRows : 128) / kThreads;
    static_assert(kTile * DK % kThreads == 0, "whole loads");
    constexpr int kCols = kRows < 128 ? kRows : 128;  // value columns a block can use
    __shared__ __align__(16) float sk[2][kTile][DK], sq[2][kTile][DK];
    __shared__ float sv[2][kTile][kCols], so[kTile][kCols], skq[kTile], salpha[kTile], sbeta[kTile];

    const int tid = threadIdx.x, sub = tid % LPR, warp = tid >> 5, lane = tid & 31;
    const int slab = blockIdx.x % p.slabs, item = blockIdx.x / p.slabs;
    const int h = item % p.hv, b = item / p.hv, hk = h / (p.hv / p.hk);
    const int lo = __ldg(p.offsets + b), n = __ldg(p.offsets + b + 1) - lo;
    const int slot = p.slots ? __ldg(p.slots + b) : b;
    int err = 0;
    if (n < 0 || lo < 0 || lo + n > p.total) err = GDN_DEV_BAD_DESC;
    else if (n > p.max_tokens) err = GDN_DEV_TOO_MANY;
    else if (slot < 0 || slot >= p.n_states) err = GDN_DEV_BAD_SLOT;
    if (err) {
        if (tid == 0) flag(p.status, err);
        return;
    }
    const int lrow = tid / LPR, row = slab * kRows + lrow;
    const bool live = row < p.dv;
    const int ncols = min(kCols, p.dv - slab * kRows);
    const int64_t state = ((int64_t)slot * p.hv + h) * p.dv * DK + (int64_t)row * DK;
    float s[4][4];
    const bool zero = !p.S0 || (p.fresh && __ldg(p.fresh + b) != 0) || !live;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[c][e] = zero ? 0.f : p.S0[state + (c * LPR + sub) * 4 + e];

    const T *qb = static_cast<const T *>(p.q) + (int64_t)lo * p.qs + hk * DK;
    const T *kb = static_cast<const T *>(p.k) + (int64_t)lo * p.ks + hk * DK;
    const T *vb = static_cast<const T *>(p.v) + (int64_t)lo * p.vs + h * p.dv + slab * kRows;
    float rk[kLoadK], rq[kLoadK], rv[kLoadV];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kLoadK; ++i) {
            const int x = tid + i * kThreads, t = x / DK, d = x % DK;
            const bool in = t0 + t < n;
            rk[i] = in ? load_f(kb, (int64_t)(t0 + t) * p.ks + d) : 0.f;
            rq[i] = in ? load_f(qb, (int64_t)(t0 + t) * p.qs + d) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kLoadV; ++i) {
            const int x = tid + i * kThreads, t = x / kCols, d = x % kCols;
            rv[i] = t0 + t < n && d < ncols ? load_f(vb, (int64_t)(t0 + t) * p.vs + d) : 0.f;
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kLoadK; ++i) {
            const int x = tid + i * kThreads;
            sk[buf][x / DK][x % DK] = rk[i];
            sq[buf][x / DK][x % DK] = rq[i];
        }
#pragma unroll
        for (int i = 0; i < kLoadV; ++i) {
            const int x = tid + i * kThreads;
            sv[buf][x / kCols][x % kCols] = rv[i];
        }
    };
    if (n > 0) {
        fetch(0);
        put(0);
    }
    __syncthreads();
    for (int t0 = 0, buf = 0; t0 < n; t0 += kTile, buf ^= 1) {
        const int nt = min(kTile, n - t0);
        for (int t = warp; t < nt; t += kThreads / 32) {
            float x = 0.f;
            for (int d = lane; d < DK; d += 32) x = fmaf(sk[buf][t][d], sq[buf][t][d], x);
            x = warp_sum(x);
            if (lane == 0) {
                const int64_t at = (int64_t)(lo + t0 + t) * p.hv + h;
                skq[t] = x;
                salpha[t] = expf(__ldg(p.g + at));
                sbeta[t] = __ldg(p.beta + at);
            }
        }
        if (t0 + kTile < n) fetch(t0 + kTile);
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            float4 k4[4], q4[4];
            float xk = 0.f, xq = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                k4[c] = *reinterpret_cast<const float4 *>(&sk[buf][t][(c * LPR + sub) * 4]);
                q4[c] = *reinterpret_cast<const float4 *>(&sq[buf][t][(c * LPR + sub) * 4]);
                xk = fmaf(s[c][0], k4[c].x, fmaf(s[c][1], k4[c].y, fmaf(s[c][2], k4[c].z, fmaf(s[c][3], k4[c].w, xk))));
                xq = fmaf(s[c][0], q4[c].x, fmaf(s[c][1], q4[c].y, fmaf(s[c][2], q4[c].z, fmaf(s[c][3], q4[c].w, xq))));
            }
#pragma unroll
            for (int w = LPR / 2; w > 0; w >>= 1) {
                xk += __shfl_xor_sync(0xffffffffu, xk, w);
                xq += __shfl_xor_sync(0xffffffffu, xq, w);
            }
            const float alpha = salpha[t];
            const float u = live ? sbeta[t] * (sv[buf][t][lrow % kCols] - alpha * xk) : 0.f;
            if (live && sub == 0) so[t][lrow] = p.scale * fmaf(u, skq[t], alpha * xq);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[c][0] = fmaf(u, k4[c].x, alpha * s[c][0]);
                s[c][1] = fmaf(u, k4[c].y, alpha * s[c][1]);
                s[c][2] = fmaf(u, k4[c].z, alpha * s[c][2]);
                s[c][3] = fmaf(u, k4[c].w, alpha * s[c][3]);
            }
        }
        if (t0 + kTile < n) put(buf ^ 1);
        __syncthreads();
        for (int x = tid; x < nt * kCols; x += kThreads) {
            const int t = x / kCols, d = x % kCols;
            if (d < ncols)
                store_f(static_cast<O *>(p.o), ((int64_t)(lo + t0 + t) * p.hv + h) * p.dv + slab * kRows + d, so[t][d]);
        }
        // the next tile's first __syncthreads() stands between these reads and its writes of so
    }
    if (live) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) p.S_new[state + (c * LPR + sub) * 4 + e] = s[c][e];
    }
}

template <typename T, typename O, int DK>
cudaError_t run(Params p, int batch, cudaStream_t stream) {
    constexpr int rows = kThreads / (DK / 16);
    p.slabs = (p.dv + rows - 1) / rows;
    const int64_t blocks = (int64_t)batch * p.hv * p.slabs;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    prefill_simt_kernel<T, O, DK><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t pick(const Params &p, int dk, int batch, cudaStream_t stream) {
    switch (dk) {
        case 16: return run<T, O, 16>(p, batch, stream);
        case 32: return run<T, O, 32>(p, batch, stream);
        case 64: return run<T, O, 64>(p, batch, stream);
        case 128: return run<T, O, 128>(p, batch, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_prefill_simt(const gdn_prefill_args &a, cudaStream_t stream) {
    Params p = {};
    p.hk = a.n_k_heads; p.hv = a.n_v_heads; p.dv = a.d_v; p.total = a.total_tokens;
    p.max_tokens = a.max_tokens; p.n_states = a.n_states;
    p.qs = a.q_stride ? a.q_stride : (int64_t)a.n_k_heads * a.d_k;
    p.ks = a.k_stride ? a.k_stride : (int64_t)a.n_k_heads * a.d_k;
    p.vs = a.v_stride ? a.v_stride : (int64_t)a.n_v_heads * a.d_v;
    p.scale = a.scale;
    p.offsets = a.token_offsets; p.slots = a.slots; p.fresh = a.fresh;
    p.q = a.q; p.k = a.k; p.v = a.v; p.g = a.g; p.beta = a.beta; p.S0 = a.S0; p.o = a.o; p.S_new = a.S_new;
    p.status = a.dev_status;
    const bool ob = a.out_dtype == GDN_BF16;
    if (a.qkv_dtype == GDN_BF16)
        return ob ? pick<__nv_bfloat16, __nv_bfloat16>(p, a.d_k, a.batch, stream)
                  : pick<__nv_bfloat16, float>(p, a.d_k, a.batch, stream);
    return ob ? pick<float, __nv_bfloat16>(p, a.d_k, a.batch, stream) : pick<float, float>(p, a.d_k, a.batch, stream);
}

}  // namespace gdn
