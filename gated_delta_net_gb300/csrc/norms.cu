// norms.cu -- the norms and gates around the rule: unit q/k with decay and write
// strength, the gated norm of each head's output, and the residual stream's norms.
//
// All three are bound by memory: every input is read once and every output written
// once, a row stays in registers between its sum of squares and its result.  Heads
// are narrow (d <= 128), so a row takes 16 bytes a lane and as few lanes as that
// needs (a half-warp for 128 bf16 values).  16384 tokens of 16 key and 32 value heads of 128 in bf16
// take 43.7 us (qk_gates, 6.3 TB/s) and 59.5 us (norm_gate, 6.8 TB/s), 8192 rows of 5120 with the post norm
// 53.8 us (residual_norm, 6.2 TB/s), 2 us less each than without the early launch.
#include <algorithm>

#include "internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kAnyThreads = 256;  // a row of any width

// 16 bytes of a row as floats, from any address (vec: 16-byte aligned)
template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);
    static __device__ __forceinline__ void load(const T *p, bool vec, float (&x)[N]) {
        if (vec) {
            const uint4 w = *reinterpret_cast<const uint4 *>(p);
            unpack(w, x);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = load_f(p, i);
        }
    }
    static __device__ __forceinline__ void store(T *p, bool vec, const float (&x)[N]) {
        if (vec) {
            *reinterpret_cast<uint4 *>(p) = pack(x);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) store_f(p, i, x[i]);
        }
    }
    // the 16 bytes as they are
    static __device__ __forceinline__ uint4 raw(const T *p, bool vec) {
        if (vec) return *reinterpret_cast<const uint4 *>(p);
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (N == 4) {
                r[i] = __float_as_uint(p[i]);
            } else {
                const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
                r[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
            }
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[N]) {
        const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (N == 4) {
                x[i] = __uint_as_float(r[i]);
            } else {
                x[2 * i] = __uint_as_float(r[i] << 16);
                x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[N]) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (N == 4) {
                r[i] = __float_as_uint(x[i]);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                r[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
};

// N weights as floats (vec: the weights start on 16 bytes, i a multiple of N)
template <typename W, int N>
__device__ __forceinline__ void load_weights(const void *w, int64_t i, bool vec, float (&x)[N]) {
    constexpr int M = Vec<W>::N;
    const W *p = static_cast<const W *>(w) + i;
    if constexpr (N >= M) {
#pragma unroll
        for (int j = 0; j < N; j += M) {
            float part[M];
            Vec<W>::load(p + j, vec, part);
#pragma unroll
            for (int e = 0; e < M; ++e) x[j + e] = part[e];
        }
    } else {  // four bf16 weights beside four fp32 values
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = load_f(p, j);
    }
}

// n / d for 0 <= n < 2^31 by a product (64-bit quotients cost more than the rest of a row)
struct Quotient {
    uint32_t d, m, s;
    explicit Quotient(uint32_t by = 1) : d(by), m(0), s(0) {
        while ((1ull << s) < d) ++s;
        m = (uint32_t)((((1ull << s) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + expf(-x)); }

// x times its gate.  What is rounded to bf16 takes the fast exponential and quotient (a few 2^-21 for the
// gates that are not negligible); with the exact ones the kernel is bound by arithmetic: 77 us for 16384
// tokens of 32 heads of 128, against 59.5.  In fp32, with twice the bytes, they fit beside them: 113 us.
template <typename T>
__device__ __forceinline__ float gated(float x, float z, int act) {
    const float num = act == GDN_ACT_SILU ? x * z : x;
    if constexpr (sizeof(T) == 2) return __fdividef(num, 1.f + __expf(-z));
    else return num / (1.f + expf(-z));
}

// ---------------------------------------------------------------------------
// qk_gates
// ---------------------------------------------------------------------------
struct QkGates {
    int rows, cells;      // q rows = k rows = T Hk; gate cells = T Hv
    int64_t qs, ks, as, bs;
    int hk, hv, row_blocks;  // row_blocks: blocks over the q and k rows; the others take the gates
    Quotient by_hk, by_hv;
    float eps;
    bool vec;
    const void *q, *k, *a, *b;
    const float *A_log, *dt_bias;
    void *qo, *ko;
    float *g, *beta;
};

template <typename T, int LPR, int NR>
__global__ void __launch_bounds__(kThreads, 16) qk_gates_kernel(QkGates p) {
    after_previous();
    constexpr int N = Vec<T>::N, D = N * LPR, kRowsPerBlock = kThreads / LPR;
    if ((int)blockIdx.x < p.row_blocks) {
        const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
        const int first = blockIdx.x * (kRowsPerBlock * NR) + group;
        float x[NR][N];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = first + r * kRowsPerBlock;
            const bool is_k = row >= p.rows;
            const int i = is_k ? row - p.rows : row, t = p.by_hk.of(i), h = i - t * p.hk;
            if (row < 2 * p.rows) {
                const T *src = is_k ? static_cast<const T *>(p.k) + t * p.ks : static_cast<const T *>(p.q) + t * p.qs;
                Vec<T>::load(src + h * D + lane * N, p.vec, x[r]);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) x[r][j] = 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) s = fmaf(x[r][j], x[r][j], s);
            const float inv = rsqrtf(group_sum<LPR>(s) + p.eps);
#pragma unroll
            for (int j = 0; j < N; ++j) x[r][j] *= inv;
            const int row = first + r * kRowsPerBlock;
            const bool is_k = row >= p.rows;
            const int64_t i = is_k ? row - p.rows : row;
            if (row < 2 * p.rows)
                Vec<T>::store(static_cast<T *>(is_k ? p.ko : p.qo) + i * D + lane * N, p.vec, x[r]);
        }
        return;
    }
    const int stride = (gridDim.x - p.row_blocks) * kThreads;
    for (int64_t c = (int)(blockIdx.x - p.row_blocks) * kThreads + threadIdx.x; c < p.cells; c += stride) {
        const int t = p.by_hv.of((uint32_t)c), h = (int)c - t * p.hv;
        const float x = load_f(static_cast<const T *>(p.a), t * p.as + h) + p.dt_bias[h];
        p.g[c] = -expf(p.A_log[h]) * (fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))));
        p.beta[c] = sigmoid_f(load_f(static_cast<const T *>(p.b), t * p.bs + h));
    }
}

// ---------------------------------------------------------------------------
// norm_gate
// ---------------------------------------------------------------------------
struct NormGate {
    int rows, hv, act;
    int64_t os, zs;
    Quotient by_hv;
    float eps;
    bool vec, wvec;
    const void *o, *z, *w;
    void *y;
};

template <typename T, typename W, int LPR, int NR>
__global__ void __launch_bounds__(kThreads, 12) norm_gate_kernel(NormGate p) {
    after_previous();
    constexpr int N = Vec<T>::N, D = N * LPR, kRowsPerBlock = kThreads / LPR;
    const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int first = blockIdx.x * (kRowsPerBlock * NR) + group;
    uint4 ro[NR], rz[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = first + r * kRowsPerBlock, t = p.by_hv.of(row), h = row - t * p.hv;
        ro[r] = rz[r] = make_uint4(0u, 0u, 0u, 0u);
        if (row < p.rows) {
            ro[r] = Vec<T>::raw(static_cast<const T *>(p.o) + t * p.os + h * D + lane * N, p.vec);
            rz[r] = Vec<T>::raw(static_cast<const T *>(p.z) + t * p.zs + h * D + lane * N, p.vec);
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        float x[N], z[N], w[N], s = 0.f;
        Vec<T>::unpack(ro[r], x);
#pragma unroll
        for (int j = 0; j < N; ++j) s = fmaf(x[j], x[j], s);
        const float inv = rsqrtf(group_sum<LPR>(s) * (1.f / D) + p.eps);
        Vec<T>::unpack(rz[r], z);
        load_weights<W>(p.w, lane * N, p.wvec, w);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = gated<T>(x[j] * (inv * w[j]), z[j], p.act);
        const int64_t row = first + r * kRowsPerBlock;
        if (row < p.rows) Vec<T>::store(static_cast<T *>(p.y) + row * D + lane * N, p.vec, x);
    }
}

// ---------------------------------------------------------------------------
// residual_norm
// ---------------------------------------------------------------------------
struct ResidualNorm {
    int64_t xs, ys;
    int width;
    float scale, eps;
    bool wvec;
    const void *x, *y, *w, *pw;
    void *h, *n;
};

// the block's sum of x, in every thread; `red` holds 33 floats
__device__ __forceinline__ float block_sum(float x, float *red) {
    x = warp_sum(x);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return x;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = (int)(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
    return warp_sum(x);
}

// a block takes rows a grid apart, NV 16-byte pieces a thread: the weights stay in registers (there is
// room for them up to NV = 2), and the next row is on its way while a row is summed
template <typename T, typename W, int NV, bool POST>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) residual_norm_kernel(ResidualNorm p, int rows) {
    after_previous();
    constexpr int N = Vec<T>::N;
    __shared__ float red[32];
    const int pieces = p.width / N;
    const T *x = static_cast<const T *>(p.x), *y = static_cast<const T *>(p.y);
    uint4 nx[NV], ny[NV];
    auto fetch = [&](int row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            nx[i] = ny[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c < pieces) {
                nx[i] = load_streaming(x + row * p.xs + c * N);
                ny[i] = load_streaming(y + row * p.ys + c * N);
            }
        }
    };
    fetch(blockIdx.x);
    constexpr bool KEEP = NV <= 2;
    float kw[KEEP ? NV : 1][N], kpw[KEEP && POST ? NV : 1][N];
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < pieces) {
                load_weights<W>(p.w, c * N, p.wvec, kw[i]);
                if constexpr (POST) load_weights<W>(p.pw, c * N, p.wvec, kpw[i]);
            }
        }
    }
    auto weights = [&](const void *from, const float (&kept)[N], int c, float (&w)[N]) {
        if constexpr (KEEP) {
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = kept[j];
        } else {
            load_weights<W>(from, c * N, p.wvec, w);
        }
    };
    for (int row = blockIdx.x; row < rows; row += gridDim.x) {
        float h[NV][N], b[NV][N];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec<T>::unpack(nx[i], h[i]);
            Vec<T>::unpack(ny[i], b[i]);
        }
        if (row + (int)gridDim.x < rows) fetch(row + gridDim.x);
        float inv = p.scale;
        if constexpr (POST) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) s = fmaf(b[i][j], b[i][j], s);
            inv *= rsqrtf(block_sum(s, red) / (float)p.width + p.eps);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < pieces) {
                float pw[N];
                if constexpr (POST) weights(p.pw, kpw[KEEP ? i : 0], c, pw);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    h[i][j] = fmaf(POST ? inv * pw[j] : inv, b[i][j], h[i][j]);
                    s = fmaf(h[i][j], h[i][j], s);
                }
                Vec<T>::store(static_cast<T *>(p.h) + (int64_t)row * p.width + c * N, true, h[i]);
            }
        }
        inv = rsqrtf(block_sum(s, red) / (float)p.width + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < pieces) {
                float w[N];
                weights(p.w, kw[KEEP ? i : 0], c, w);
#pragma unroll
                for (int j = 0; j < N; ++j) h[i][j] *= inv * w[j];
                Vec<T>::store(static_cast<T *>(p.n) + (int64_t)row * p.width + c * N, true, h[i]);
            }
        }
    }
}

// any width and alignment: the row is read again for each of the three steps (from L1
// and L2); the last one writes h and n together, as either may lie on an input
template <typename T, typename W>
__global__ void __launch_bounds__(kAnyThreads) residual_norm_any_kernel(ResidualNorm p) {
    after_previous();
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.xs, *y = static_cast<const T *>(p.y) + row * p.ys;
    const W *w = static_cast<const W *>(p.w), *pw = static_cast<const W *>(p.pw);
    float inv = 1.f;
    if (pw) {
        float s = 0.f;
        for (int c = threadIdx.x; c < p.width; c += kAnyThreads) {
            const float v = load_f(y, c);
            s = fmaf(v, v, s);
        }
        inv = rsqrtf(block_sum(s, red) / (float)p.width + p.eps);
    }
    auto at = [&](int c) {
        float v = load_f(y, c);
        if (pw) v *= inv * load_f(pw, c);
        return fmaf(p.scale, v, load_f(x, c));
    };
    float s = 0.f;
    for (int c = threadIdx.x; c < p.width; c += kAnyThreads) {
        const float v = at(c);
        s = fmaf(v, v, s);
    }
    const float inv_h = rsqrtf(block_sum(s, red) / (float)p.width + p.eps);
    for (int c = threadIdx.x; c < p.width; c += kAnyThreads) {
        const float v = at(c);
        store_f(static_cast<T *>(p.h), row * p.width + c, v);
        store_f(static_cast<T *>(p.n), row * p.width + c, v * inv_h * load_f(w, c));
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// whether rows `stride` elements apart, from base, all start on 16 bytes
bool vec_rows(const void *base, int64_t stride, int elem) { return aligned16(base) && stride * elem % 16 == 0; }

// Rows a thread has in flight: two, or one where two would leave SMs without a block.  Small blocks that
// fill the SM's registers keep the most bytes on their way (16384 tokens of 32 heads of 128, qk_gates:
// 128 threads x 2 rows 45.6 us, 256 x 2 47, 256 x 4 56; norm_gate 73, 83 and 125, and 62 with the rows
// waiting as the bytes they came as).
template <int PER>
int rows_in_flight(int64_t rows) { return rows >= (int64_t)PER * 2 * sm_count() ? 2 : 1; }

template <typename T, int LPR>
cudaError_t run_qk_gates(QkGates p, cudaStream_t stream) {
    constexpr int per = kThreads / LPR;
    const int nr = rows_in_flight<per>(2ll * p.rows);
    p.row_blocks = (2 * p.rows + per * nr - 1) / (per * nr);
    const int gate_blocks = std::min((p.cells + kThreads - 1) / kThreads, 2048);
    const unsigned grid = p.row_blocks + gate_blocks;
    return launch_early(nr == 2 ? qk_gates_kernel<T, LPR, 2> : qk_gates_kernel<T, LPR, 1>, grid, kThreads, stream, p);
}

template <typename T>
cudaError_t pick_qk_gates(const QkGates &p, int d, cudaStream_t stream) {
    switch (d / Vec<T>::N) {
        case 2: return run_qk_gates<T, 2>(p, stream);
        case 4: return run_qk_gates<T, 4>(p, stream);
        case 8: return run_qk_gates<T, 8>(p, stream);
        case 16: return run_qk_gates<T, 16>(p, stream);
        case 32: return run_qk_gates<T, 32>(p, stream);
    }
    return cudaErrorInvalidValue;
}

template <typename T, typename W, int LPR>
cudaError_t run_norm_gate(const NormGate &p, cudaStream_t stream) {
    constexpr int per = kThreads / LPR;
    if (rows_in_flight<per>(p.rows) == 2)
        return launch_early(norm_gate_kernel<T, W, LPR, 2>, (p.rows + per * 2 - 1) / (per * 2), kThreads, stream, p);
    return launch_early(norm_gate_kernel<T, W, LPR, 1>, (p.rows + per - 1) / per, kThreads, stream, p);
}

template <typename T, typename W>
cudaError_t pick_norm_gate(const NormGate &p, int d, cudaStream_t stream) {
    switch (d / Vec<T>::N) {
        case 2: return run_norm_gate<T, W, 2>(p, stream);
        case 4: return run_norm_gate<T, W, 4>(p, stream);
        case 8: return run_norm_gate<T, W, 8>(p, stream);
        case 16: return run_norm_gate<T, W, 16>(p, stream);
        case 32: return run_norm_gate<T, W, 32>(p, stream);
    }
    return cudaErrorInvalidValue;
}

template <typename T, typename W>
cudaError_t pick_residual_norm(const ResidualNorm &p, int tokens, bool vec, cudaStream_t stream) {
    constexpr int N = Vec<T>::N;
    const int pieces = p.width / N;
    if (!vec || p.width % N || pieces > 2048) {
        return launch_early(residual_norm_any_kernel<T, W>, (unsigned)tokens, kAnyThreads, stream, p);
    }
    // few rows: as many threads a row as there are pieces; many: two pieces a thread (four past 1024 pieces),
    // and as many blocks as stay resident
    const int nv = tokens <= 2 * sm_count() && pieces <= 1024 ? 1 : pieces <= 1024 ? 2 : 4;
    const int threads = ((pieces + nv - 1) / nv + 31) / 32 * 32;
    const unsigned grid = (unsigned)std::min<int64_t>(tokens, (int64_t)sm_count() * std::max(1, 768 / threads));
    auto go = [&](auto kernel) { return launch_early(kernel, grid, threads, stream, p, tokens); };
    if (p.pw) return nv == 1 ? go(residual_norm_kernel<T, W, 1, true>) : nv == 2 ? go(residual_norm_kernel<T, W, 2, true>) : go(residual_norm_kernel<T, W, 4, true>);
    return nv == 1 ? go(residual_norm_kernel<T, W, 1, false>) : nv == 2 ? go(residual_norm_kernel<T, W, 2, false>) : go(residual_norm_kernel<T, W, 4, false>);
}

}  // namespace

// Row numbers stay below 2^30: more tokens than that go in several launches.
cudaError_t launch_qk_gates(const gdn_qk_gates_args &a, cudaStream_t stream) {
    const int e = a.dtype == GDN_BF16 ? 2 : 4;
    QkGates p;
    p.hk = a.n_k_heads;
    p.hv = a.n_v_heads;
    p.by_hk = Quotient(p.hk);
    p.by_hv = Quotient(p.hv);
    const int64_t qk_row = (int64_t)p.hk * a.d_k;
    p.qs = a.q_stride ? a.q_stride : qk_row;
    p.ks = a.k_stride ? a.k_stride : qk_row;
    p.as = a.a_stride ? a.a_stride : p.hv;
    p.bs = a.b_stride ? a.b_stride : p.hv;
    p.eps = a.eps;
    p.vec = vec_rows(a.q, p.qs, e) && vec_rows(a.k, p.ks, e) && aligned16(a.q_out) && aligned16(a.k_out);
    p.A_log = a.A_log;
    p.dt_bias = a.dt_bias;
    const int64_t most = std::max<int64_t>(1, (1ll << 29) / p.hv);  // tokens a launch (Hk <= Hv)
    for (int64_t t = 0; t < a.total_tokens; t += most) {
        const int64_t n = std::min(most, a.total_tokens - t);
        p.rows = (int)(n * p.hk);
        p.cells = (int)(n * p.hv);
        p.q = static_cast<const char *>(a.q) + t * p.qs * e;
        p.k = static_cast<const char *>(a.k) + t * p.ks * e;
        p.a = static_cast<const char *>(a.a) + t * p.as * e;
        p.b = static_cast<const char *>(a.b) + t * p.bs * e;
        p.qo = static_cast<char *>(a.q_out) + t * qk_row * e;
        p.ko = static_cast<char *>(a.k_out) + t * qk_row * e;
        p.g = a.g + t * p.hv;
        p.beta = a.beta + t * p.hv;
        const cudaError_t err = a.dtype == GDN_BF16 ? pick_qk_gates<__nv_bfloat16>(p, a.d_k, stream) : pick_qk_gates<float>(p, a.d_k, stream);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

cudaError_t launch_norm_gate(const gdn_norm_gate_args &a, cudaStream_t stream) {
    const int e = a.dtype == GDN_BF16 ? 2 : 4;
    NormGate p;
    p.hv = a.n_v_heads;
    p.by_hv = Quotient(p.hv);
    const int64_t row = (int64_t)p.hv * a.d_v;
    p.os = a.o_stride ? a.o_stride : row;
    p.zs = a.z_stride ? a.z_stride : row;
    p.act = a.act;
    p.eps = a.eps;
    p.vec = vec_rows(a.o, p.os, e) && vec_rows(a.z, p.zs, e) && aligned16(a.y);
    p.wvec = aligned16(a.weight);
    p.w = a.weight;
    const bool wb = a.weight_dtype == GDN_BF16;
    const int64_t most = std::max<int64_t>(1, (1ll << 30) / p.hv);
    for (int64_t t = 0; t < a.total_tokens; t += most) {
        p.rows = (int)(std::min(most, a.total_tokens - t) * p.hv);
        p.o = static_cast<const char *>(a.o) + t * p.os * e;
        p.z = static_cast<const char *>(a.z) + t * p.zs * e;
        p.y = static_cast<char *>(a.y) + t * row * e;
        const cudaError_t err =
            a.dtype == GDN_BF16
                ? (wb ? pick_norm_gate<__nv_bfloat16, __nv_bfloat16>(p, a.d_v, stream) : pick_norm_gate<__nv_bfloat16, float>(p, a.d_v, stream))
                : (wb ? pick_norm_gate<float, __nv_bfloat16>(p, a.d_v, stream) : pick_norm_gate<float, float>(p, a.d_v, stream));
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

cudaError_t launch_residual_norm(const gdn_residual_norm_args &a, cudaStream_t stream) {
    const int e = a.dtype == GDN_BF16 ? 2 : 4;
    ResidualNorm p = {};
    p.width = a.width;
    p.xs = a.x_stride ? a.x_stride : a.width;
    p.ys = a.y_stride ? a.y_stride : a.width;
    p.scale = a.scale;
    p.eps = a.eps;
    p.wvec = aligned16(a.weight) && (!a.post_weight || aligned16(a.post_weight));
    p.w = a.weight; p.pw = a.post_weight;
    const bool vec = vec_rows(a.x, p.xs, e) && vec_rows(a.y, p.ys, e) && vec_rows(a.h, a.width, e) && vec_rows(a.n, a.width, e);
    const bool wb = a.weight_dtype == GDN_BF16;
    const int64_t most = 1ll << 30;
    for (int64_t t = 0; t < a.total_tokens; t += most) {
        const int n = (int)std::min(most, a.total_tokens - t);
        p.x = static_cast<const char *>(a.x) + t * p.xs * e;
        p.y = static_cast<const char *>(a.y) + t * p.ys * e;
        p.h = static_cast<char *>(a.h) + t * a.width * e;
        p.n = static_cast<char *>(a.n) + t * a.width * e;
        const cudaError_t err =
            a.dtype == GDN_BF16
                ? (wb ? pick_residual_norm<__nv_bfloat16, __nv_bfloat16>(p, n, vec, stream) : pick_residual_norm<__nv_bfloat16, float>(p, n, vec, stream))
                : (wb ? pick_residual_norm<float, __nv_bfloat16>(p, n, vec, stream) : pick_residual_norm<float, float>(p, n, vec, stream));
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace gdn
