// prefill_simt.cu -- prompts through the gated delta rule, four tokens at a time: the
// general kernel, any supported widths, types and strides.
//
// A block takes a slab of state rows of one (prompt, value head); rows of S do not
// meet, so slabs are independent.  A row's d_k entries lie in the registers of d_k / 16
// lanes for the whole prompt.  For four tokens with the state S before them, a_i the
// decay from there to token i and e_ij that from token j to token i,
//     u_i = beta_i (v_i - a_i S k_i - sum_{j < i} e_ij (k_i.k_j) u_j)
//     o_i = scale (a_i S q_i + sum_{j <= i} e_ij (q_i.k_j) u_j)
//     S  <- a_3 S + sum_j e_3j u_j k_j^T,
// so that eight products with S are reduced together and the chain over the tokens is one
// reduction and one update for four of them.  The token products, which all rows share,
// are made by a warp for each four.  Tokens come in tiles of 16 through shared memory:
// the next tile's values are loaded into registers before the present tile is worked off.
// The chain over the steps bounds it, at 0.22 us a token (300 tokens of 16 heads in fp32:
// 68 us; one warp a scheduler), until the heads' blocks fill the GPU: 16865 tokens of 32
// heads take 3540 us, three blocks an SM, bound by what they issue.
#include "internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 16;  // tokens a tile
constexpr int kStep = 4;   // tokens a step
constexpr int kCoefA = 8, kCoefQ = 20, kCoef = 36;  // a step's coefficients
static_assert(kThreads / 32 * kStep == kTile, "a warp for each step's token products");

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
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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

// 16 bytes of a row as they are (vec: 16-byte aligned), and as floats in shared memory
template <typename T>
__device__ __forceinline__ uint4 raw16(const T *p, bool vec) {
    if (vec) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            r[i] = __float_as_uint(p[i]);
        } else {
            const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
            r[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
template <typename T>
__device__ __forceinline__ void put16(float *to, const uint4 &w) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<uint4 *>(to) = w;
    } else {
        *reinterpret_cast<uint4 *>(to) = make_uint4(w.x << 16, w.x & 0xFFFF0000u, w.y << 16, w.y & 0xFFFF0000u);
        *reinterpret_cast<uint4 *>(to + 4) = make_uint4(w.z << 16, w.z & 0xFFFF0000u, w.w << 16, w.w & 0xFFFF0000u);
    }
}

struct Params {
    bool vec;  // rows of q, k and v start on 16 bytes
    int hk, hv, dv, total, max_tokens, n_states, slabs, batch;
    bool sorted;  // prompts longest first
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
    constexpr int kCols = kRows < 128 ? kRows : 128;  // value columns a block can use
    constexpr int VE = 16 / sizeof(T), kPer = kThreads * VE;  // entries of 16 bytes, of one load of the block
    constexpr int kLoadK = (kTile * DK + kPer - 1) / kPer, kLoadV = (kTile * kCols + kPer - 1) / kPer;
    __shared__ __align__(16) float sk[2][kTile][DK], sq[2][kTile][DK];
    __shared__ __align__(16) float sv[2][kTile][kCols];
    __shared__ float so[kTile][kCols], salpha[2][kTile], sbeta[2][kTile];
    // of each step: beta_i e_ij k_i.k_j (10, 20, 21, 30, 31, 32), two of padding, a_i, beta_i, e_3i, and e_ij q_i.k_j in
    // rows i of four, zero above the diagonal
    __shared__ __align__(16) float scoef[kTile / kStep][kCoef];

    const int tid = threadIdx.x, sub = tid % LPR, warp = tid >> 5, lane = tid & 31;
    const int slab = blockIdx.x % p.slabs, item = blockIdx.x / p.slabs;
    const int h = item % p.hv, hk = h / (p.hv / p.hk);
    int b = item / p.hv;
    if (p.sorted) {
        __shared__ int slen[kThreads], pick;
        if (tid < p.batch) slen[tid] = prompt_length(p.offsets, tid);
        __syncthreads();
        if (tid < p.batch && length_rank(slen, p.batch, tid) == b) pick = tid;
        __syncthreads();
        b = pick;
    }
    const int lo = __ldg(p.offsets + b), hi = __ldg(p.offsets + b + 1);
    const bool inside = lo >= 0 && hi >= lo && hi <= p.total;
    const unsigned n = inside ? hi - lo : 0;  // with the tokens up to a tile past it more than an int can hold
    const int slot = p.slots ? __ldg(p.slots + b) : b;
    int err = 0;
    if (!inside) err = GDN_DEV_BAD_DESC;
    else if (n > (unsigned)p.max_tokens) err = GDN_DEV_TOO_MANY;
    else if (slot < 0 || slot >= p.n_states) err = GDN_DEV_BAD_SLOT;
    if (err) {
        if (tid == 0) flag(p.status, err);
        return;
    }
    const int lrow = tid / LPR;
    const int ncols = min(kCols, p.dv - slab * kRows);
    const bool live = lrow < ncols;
    // of the eight sums of a step (S k_i, S q_i) each lane of a row ends with kHeld; S q_i of tokens out0 on lies in its
    // entries from kFirst on, in the upper half of the lanes
    constexpr int kHeld = 2 * kStep / LPR, kFirst = LPR > 1 ? 0 : kStep;
    const int out0 = (sub * kHeld + kFirst) & (kStep - 1);
    const bool writes = live && sub * kHeld + kFirst >= kStep;
    const int64_t state = (((int64_t)slot * p.hv + h) * p.dv + slab * kRows + lrow) * DK + sub * 4;
    const bool zero = !p.S0 || (p.fresh && __ldg(p.fresh + b) != 0) || !live;
    f2 s[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float *from = p.S0 + state + c * LPR * 4;
        s[2 * c] = zero ? 0 : pair(from[0], from[1]);
        s[2 * c + 1] = zero ? 0 : pair(from[2], from[3]);
    }

    const T *qb = static_cast<const T *>(p.q) + (int64_t)lo * p.qs + hk * DK;
    const T *kb = static_cast<const T *>(p.k) + (int64_t)lo * p.ks + hk * DK;
    const T *vb = static_cast<const T *>(p.v) + (int64_t)lo * p.vs + h * p.dv + slab * kRows;
    uint4 rk[kLoadK], rq[kLoadK], rv[kLoadV];
    float rg = 0.f, rb = 0.f;
    auto fetch = [&](unsigned t0) {
#pragma unroll
        for (int i = 0; i < kLoadK; ++i) {
            const int x = (tid + i * kThreads) * VE, t = x / DK, d = x % DK;
            rk[i] = rq[i] = make_uint4(0u, 0u, 0u, 0u);
            if (t < kTile && t0 + t < n) {
                rk[i] = raw16(kb + (int64_t)(t0 + t) * p.ks + d, p.vec);
                rq[i] = raw16(qb + (int64_t)(t0 + t) * p.qs + d, p.vec);
            }
        }
#pragma unroll
        for (int i = 0; i < kLoadV; ++i) {
            const int x = (tid + i * kThreads) * VE, t = x / kCols, d = x % kCols;
            rv[i] = make_uint4(0u, 0u, 0u, 0u);
            if (t < kTile && t0 + t < n && d < ncols) rv[i] = raw16(vb + (int64_t)(t0 + t) * p.vs + d, p.vec);
        }
        rg = rb = 0.f;  // tokens past the end: no decay, nothing written
        if (tid < kTile && t0 + tid < n) {
            rg = __ldg(p.g + (int64_t)(lo + t0 + tid) * p.hv + h);
            rb = __ldg(p.beta + (int64_t)(lo + t0 + tid) * p.hv + h);
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kLoadK; ++i) {
            const int x = (tid + i * kThreads) * VE;
            if (x / DK < kTile) {
                put16<T>(&sk[buf][x / DK][x % DK], rk[i]);
                put16<T>(&sq[buf][x / DK][x % DK], rq[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kLoadV; ++i) {
            const int x = (tid + i * kThreads) * VE;
            if (x / kCols < kTile) put16<T>(&sv[buf][x / kCols][x % kCols], rv[i]);
        }
        if (tid < kTile) {
            salpha[buf][tid] = expf(rg);
            sbeta[buf][tid] = rb;
        }
    };
    if (n > 0) {
        fetch(0);
        put(0);
        scoef[warp][lane] = 0.f;
        if (lane < kCoef - 32) scoef[warp][32 + lane] = 0.f;
        __syncwarp();
    }
    __syncthreads();
    int buf = 0;
    for (unsigned t0 = 0; t0 < n; t0 += kTile, buf ^= 1) {
        const int nt = min((unsigned)kTile, n - t0);
        {
            // step number `warp`: its 16 token products, summed over the warp by halves so that lane 2 m ends with
            // number m
            const int g0 = warp * kStep;
            float x[16];
#pragma unroll
            for (int m = 0; m < 16; ++m) x[m] = 0.f;
            if (lane * 4 < DK) {
                float4 k[kStep], q[kStep];
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    k[i] = *reinterpret_cast<const float4 *>(&sk[buf][g0 + i][lane * 4]);
                    q[i] = *reinterpret_cast<const float4 *>(&sq[buf][g0 + i][lane * 4]);
                }
                auto dot = [](const float4 &a, const float4 &b) { return fmaf(a.x, b.x, a.y * b.y) + fmaf(a.z, b.z, a.w * b.w); };
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
#pragma unroll
                    for (int j = 0; j <= i; ++j) {
                        if (j < i) x[i * (i - 1) / 2 + j] = dot(k[i], k[j]);
                        x[6 + i * (i + 1) / 2 + j] = dot(q[i], k[j]);
                    }
                }
            }
#pragma unroll
            for (int w = 16, m = 8; w >= 2; w >>= 1, m >>= 1) {
#pragma unroll
                for (int e = 0; e < m; ++e) {
                    const bool up = lane & w;
                    const float send = up ? x[e] : x[e + m], keep = up ? x[e + m] : x[e];
                    x[e] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                }
            }
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
            const int m = lane >> 1;
            int i = 0, j = 0;  // of product number m
            if (m < 6) {
                i = m < 1 ? 1 : m < 3 ? 2 : 3;
                j = m - i * (i - 1) / 2;
            } else {
                i = m < 7 ? 0 : m < 9 ? 1 : m < 12 ? 2 : 3;
                j = m - 6 - i * (i + 1) / 2;
            }
            float e = 1.f;
            for (int t = j + 1; t <= i; ++t) e *= salpha[buf][g0 + t];
            if (!(lane & 1)) {
                scoef[warp][m < 6 ? m : kCoefQ + 4 * i + j] = e * x[0] * (m < 6 ? sbeta[buf][g0 + i] : 1.f);
            } else if (m < 12) {  // a_i, beta_i, e_3i
                const int t0i = m & 3;
                float y = 1.f;
                if (m < 4) for (int t = 0; t <= t0i; ++t) y *= salpha[buf][g0 + t];
                else if (m < 8) y = sbeta[buf][g0 + t0i];
                else for (int t = t0i + 1; t < kStep; ++t) y *= salpha[buf][g0 + t];
                scoef[warp][kCoefA + m] = y;
            }
        }
        if (t0 + kTile < n) fetch(t0 + kTile);
        __syncthreads();
#pragma unroll 1
        for (int t = 0; t < nt; t += kStep) {
            const float *coef = scoef[t / kStep];
            float cf[kCoefQ];
#pragma unroll
            for (int c = 0; c < kCoefQ; c += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(coef + c);
                cf[c] = v.x; cf[c + 1] = v.y; cf[c + 2] = v.z; cf[c + 3] = v.w;
            }
            float4 qc[kHeld - kFirst];
            float qa[kHeld - kFirst];
#pragma unroll
            for (int e = 0; e < kHeld - kFirst; ++e) {
                qc[e] = *reinterpret_cast<const float4 *>(coef + kCoefQ + 4 * (out0 + e));
                qa[e] = coef[kCoefA + out0 + e];
            }
            f2 k[kStep][8];
            float x[2 * kStep];  // S k_i, S q_i
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                f2 a0, a1, b0, b1;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(&sk[buf][t + i][(c * LPR + sub) * 4]);
                    const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(&sq[buf][t + i][(c * LPR + sub) * 4]);
                    k[i][2 * c] = a.x;
                    k[i][2 * c + 1] = a.y;
                    a0 = c ? fma2(s[2 * c], a.x, a0) : mul2(s[0], a.x);
                    a1 = c ? fma2(s[2 * c + 1], a.y, a1) : mul2(s[1], a.y);
                    b0 = c ? fma2(s[2 * c], q.x, b0) : mul2(s[0], q.x);
                    b1 = c ? fma2(s[2 * c + 1], q.y, b1) : mul2(s[1], q.y);
                }
                x[i] = sum(add2(a0, a1));
                x[kStep + i] = sum(add2(b0, b1));
            }
            // summed over the row's lanes by halves, lane `sub` ends with number sub kHeld on; S k_i then goes to all of
            // them, S q_i stays where it makes token i's output
#pragma unroll
            for (int w = LPR / 2, m = 4; w > 0; w >>= 1, m >>= 1) {
                const bool up = sub & w;
#pragma unroll
                for (int e = 0; e < m; ++e) {
                    const float send = up ? x[e] : x[e + m], keep = up ? x[e + m] : x[e];
                    x[e] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                }
            }
            float u[kStep];
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                const float *a = cf + kCoefA, *beta = a + kStep;
                const float xk = LPR > 1 ? __shfl_sync(0xffffffffu, x[i % kHeld], i / kHeld, LPR) : x[i];
                u[i] = beta[i] * (sv[buf][t + i][lrow % kCols] - a[i] * xk);
#pragma unroll
                for (int j = 0; j < i; ++j) u[i] = fmaf(-cf[i * (i - 1) / 2 + j], u[j], u[i]);
            }
#pragma unroll
            for (int e = kFirst; e < kHeld; ++e) {
                const float4 c = qc[e - kFirst];
                const int i = out0 + e - kFirst;
                float o = fmaf(c.x, u[0], qa[e - kFirst] * x[e]);
                if constexpr (LPR <= 2) {  // i is known
                    if (i >= 1) o = fmaf(c.y, u[1], o);
                    if (i >= 2) o = fmaf(c.z, u[2], o);
                    if (i >= 3) o = fmaf(c.w, u[3], o);
                } else {  // a later token's NaN is not this one's
                    o = fmaf(c.y, i >= 1 ? u[1] : 0.f, o);
                    o = fmaf(c.z, i >= 2 ? u[2] : 0.f, o);
                    o = fmaf(c.w, i >= 3 ? u[3] : 0.f, o);
                }
                if (writes) so[t + i][lrow] = p.scale * o;
            }
            const f2 a3 = pair(cf[kCoefA + 3], cf[kCoefA + 3]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = mul2(a3, s[e]);
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                const float w = cf[kCoefA + 8 + j] * u[j];
                const f2 w2 = pair(w, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = fma2(w2, k[j][e], s[e]);
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
        for (int c = 0; c < 4; ++c) {
            f2 *to = reinterpret_cast<f2 *>(p.S_new + state + c * LPR * 4);
            to[0] = s[2 * c];
            to[1] = s[2 * c + 1];
        }
    }
}

// Prompts are taken longest first where not all blocks are resident at once (about three an SM) and a block has a
// thread for each prompt: 24 prompts of 1 to 400 tokens of 32 heads 1020 us, in their own order 1063.
template <typename T, typename O, int DK>
cudaError_t run(Params p, int batch, cudaStream_t stream) {
    constexpr int rows = kThreads / (DK / 16);
    p.slabs = (p.dv + rows - 1) / rows;
    const int64_t blocks = (int64_t)batch * p.hv * p.slabs;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    p.batch = batch;
    p.sorted = batch > 1 && batch <= kThreads && blocks > 3 * sm_count();
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
    const int e = a.qkv_dtype == GDN_BF16 ? 2 : 4;
    p.vec = ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) == 0 &&
            p.qs * e % 16 == 0 && p.ks * e % 16 == 0 && p.vs * e % 16 == 0;
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
