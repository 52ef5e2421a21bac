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

constexpr int kThreads = 128;
constexpr int kTile = 16;  // tokens a tile
constexpr int kRpt = 1;    // rows a thread has part of

// two fp32 values in a register pair, for the packed fp32 instructions
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float sum(f2 x) {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
    return a + b;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

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
    constexpr int LPR = DK / 16, kGroups = kThreads / LPR, kRows = kGroups * kRpt;  // rows a block
    constexpr int kLoadK = kTile * DK / kThreads, kLoadV = kTile * (kRows < 128 ? kRows : 128) / kThreads;
    static_assert(kTile * DK % kThreads == 0, "whole loads");
    constexpr int kCols = kRows < 128 ? kRows : 128;  // value columns a block can use
    __shared__ __align__(16) float sk[2][kTile][DK], sq[2][kTile][DK];
    __shared__ float sv[2][kTile][kCols], so[kTile][kCols], skq[kTile], salpha[2][kTile], sbeta[2][kTile];

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
    const int lrow = tid / LPR;  // and kGroups further on
    const int ncols = min(kCols, p.dv - slab * kRows);
    const int64_t state = (((int64_t)slot * p.hv + h) * p.dv + slab * kRows + lrow) * DK + sub * 4;
    const bool zero = !p.S0 || (p.fresh && __ldg(p.fresh + b) != 0);
    bool live[kRpt];
    f2 s[kRpt][8];
#pragma unroll
    for (int i = 0; i < kRpt; ++i) {
        live[i] = lrow + i * kGroups < ncols;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float *from = p.S0 + state + i * kGroups * DK + c * LPR * 4;
            const bool z = zero || !live[i];
            s[i][2 * c] = z ? 0 : pair(from[0], from[1]);
            s[i][2 * c + 1] = z ? 0 : pair(from[2], from[3]);
        }
    }

    const T *qb = static_cast<const T *>(p.q) + (int64_t)lo * p.qs + hk * DK;
    const T *kb = static_cast<const T *>(p.k) + (int64_t)lo * p.ks + hk * DK;
    const T *vb = static_cast<const T *>(p.v) + (int64_t)lo * p.vs + h * p.dv + slab * kRows;
    float rk[kLoadK], rq[kLoadK], rv[kLoadV], rg = 0.f, rb = 0.f;
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
        if (tid < kTile && t0 + tid < n) {
            rg = __ldg(p.g + (int64_t)(lo + t0 + tid) * p.hv + h);
            rb = __ldg(p.beta + (int64_t)(lo + t0 + tid) * p.hv + h);
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
        if (tid < kTile) {
            salpha[buf][tid] = expf(rg);
            sbeta[buf][tid] = rb;
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
            if (lane == 0) skq[t] = x;
        }
        if (t0 + kTile < n) fetch(t0 + kTile);
        __syncthreads();
        // a token's k and q are read while the one before it is reduced
        f2 k0[8], q0[8];
        auto read = [&](int t, f2 (&k)[8], f2 (&q)[8]) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(&sk[buf][t][(c * LPR + sub) * 4]);
                const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(&sq[buf][t][(c * LPR + sub) * 4]);
                k[2 * c] = a.x;
                k[2 * c + 1] = a.y;
                q[2 * c] = b.x;
                q[2 * c + 1] = b.y;
            }
        };
        auto step = [&](int t, const f2 (&k)[8], const f2 (&q)[8]) {
            float xk[kRpt], xq[kRpt];
#pragma unroll
            for (int i = 0; i < kRpt; ++i) {
                f2 a0 = mul2(s[i][0], k[0]), a1 = mul2(s[i][1], k[1]), b0 = mul2(s[i][0], q[0]), b1 = mul2(s[i][1], q[1]);
#pragma unroll
                for (int e = 2; e < 8; e += 2) {
                    a0 = fma2(s[i][e], k[e], a0);
                    a1 = fma2(s[i][e + 1], k[e + 1], a1);
                    b0 = fma2(s[i][e], q[e], b0);
                    b1 = fma2(s[i][e + 1], q[e + 1], b1);
                }
                xk[i] = sum(a0) + sum(a1);
                xq[i] = sum(b0) + sum(b1);
            }
#pragma unroll
            for (int w = LPR / 2; w > 0; w >>= 1) {
#pragma unroll
                for (int i = 0; i < kRpt; ++i) {
                    xk[i] += __shfl_xor_sync(0xffffffffu, xk[i], w);
                    xq[i] += __shfl_xor_sync(0xffffffffu, xq[i], w);
                }
            }
            const float alpha = salpha[buf][t], beta = sbeta[buf][t], kq = skq[t];
            const f2 alpha2 = pair(alpha, alpha);
#pragma unroll
            for (int i = 0; i < kRpt; ++i) {
                const float u = live[i] ? beta * (sv[buf][t][(lrow + i * kGroups) % kCols] - alpha * xk[i]) : 0.f;
                if (live[i] && sub == 0) so[t][lrow + i * kGroups] = p.scale * fmaf(u, kq, alpha * xq[i]);
                const f2 u2 = pair(u, u);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[i][e] = fma2(u2, k[e], mul2(alpha2, s[i][e]));
            }
        };
        read(0, k0, q0);
#pragma unroll 1
        for (int t = 0; t < nt; t += 2) {
            f2 k1[8], q1[8];
            const bool second = t + 1 < nt;
            if (second) read(t + 1, k1, q1);
            step(t, k0, q0);
            if (t + 2 < nt) read(t + 2, k0, q0);
            if (second) step(t + 1, k1, q1);
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
#pragma unroll
    for (int i = 0; i < kRpt; ++i) {
        if (!live[i]) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            f2 *to = reinterpret_cast<f2 *>(p.S_new + state + i * kGroups * DK + c * LPR * 4);
            to[0] = s[i][2 * c];
            to[1] = s[i][2 * c + 1];
        }
    }
}

template <typename T, typename O, int DK>
cudaError_t run(Params p, int batch, cudaStream_t stream) {
    constexpr int rows = kThreads / (DK / 16) * kRpt;
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
