// norms.cu -- the norms and gates around the rule: unit q/k with decay and write
// strength, the gated norm of each head's output, and the residual stream's norms.
//
// All three are bound by memory: every input is read once and every output written
// once, a row stays in registers between its sum of squares and its result.  Heads
// are narrow (d <= 128), so a row takes 16 bytes a lane and as few lanes as that
// needs (a half-warp for 128 bf16 values), and a lane has several rows in flight.
#include "internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

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

template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + expf(-x)); }

// ---------------------------------------------------------------------------
// qk_gates
// ---------------------------------------------------------------------------
struct QkGates {
    int64_t rows, cells;  // q rows = k rows = T Hk; gate cells = T Hv
    int64_t qs, ks, as, bs;
    int hk, hv, row_blocks;  // row_blocks: blocks over the q and k rows; the others take the gates
    float eps;
    bool vec;
    const void *q, *k, *a, *b;
    const float *A_log, *dt_bias;
    void *qo, *ko;
    float *g, *beta;
};

template <typename T, int LPR, int NR>
__global__ void __launch_bounds__(kThreads) qk_gates_kernel(QkGates p) {
    constexpr int N = Vec<T>::N, D = N * LPR, kRowsPerBlock = kThreads / LPR;
    if ((int)blockIdx.x < p.row_blocks) {
        const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
        const int64_t first = (int64_t)blockIdx.x * (kRowsPerBlock * NR) + group;
        float x[NR][N];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int64_t row = first + r * kRowsPerBlock;
            const bool is_k = row >= p.rows;
            const int64_t i = is_k ? row - p.rows : row, t = i / p.hk;
            const int h = (int)(i - t * p.hk);
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
            const int64_t row = first + r * kRowsPerBlock;
            const bool is_k = row >= p.rows;
            const int64_t i = is_k ? row - p.rows : row;
            if (row < 2 * p.rows)
                Vec<T>::store(static_cast<T *>(is_k ? p.ko : p.qo) + i * D + lane * N, p.vec, x[r]);
        }
        return;
    }
    const int64_t stride = (int64_t)(gridDim.x - p.row_blocks) * kThreads;
    for (int64_t c = (int64_t)(blockIdx.x - p.row_blocks) * kThreads + threadIdx.x; c < p.cells; c += stride) {
        const int64_t t = c / p.hv;
        const int h = (int)(c - t * p.hv);
        const float x = load_f(static_cast<const T *>(p.a), t * p.as + h) + __ldg(p.dt_bias + h);
        p.g[c] = -expf(__ldg(p.A_log + h)) * (fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))));
        p.beta[c] = sigmoid_f(load_f(static_cast<const T *>(p.b), t * p.bs + h));
    }
}

// ---------------------------------------------------------------------------
// norm_gate
// ---------------------------------------------------------------------------
struct NormGate {
    int64_t rows, os, zs;
    int hv, act;
    float eps;
    bool vec, wvec;
    const void *o, *z, *w;
    void *y;
};

template <typename T, typename W, int LPR, int NR>
__global__ void __launch_bounds__(kThreads) norm_gate_kernel(NormGate p) {
    constexpr int N = Vec<T>::N, D = N * LPR, kRowsPerBlock = kThreads / LPR;
    const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int64_t first = (int64_t)blockIdx.x * (kRowsPerBlock * NR) + group;
    float w[N];
    load_weights<W>(p.w, lane * N, p.wvec, w);
    float x[NR][N], z[NR][N];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int64_t row = first + r * kRowsPerBlock, t = row / p.hv;
        const int h = (int)(row - t * p.hv);
        if (row < p.rows) {
            Vec<T>::load(static_cast<const T *>(p.o) + t * p.os + h * D + lane * N, p.vec, x[r]);
            Vec<T>::load(static_cast<const T *>(p.z) + t * p.zs + h * D + lane * N, p.vec, z[r]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[r][j] = z[r][j] = 0.f;
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) s = fmaf(x[r][j], x[r][j], s);
        const float inv = rsqrtf(group_sum<LPR>(s) * (1.f / D) + p.eps);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float gate = sigmoid_f(z[r][j]);
            if (p.act == GDN_ACT_SILU) gate *= z[r][j];
            x[r][j] *= inv * w[j] * gate;
        }
        const int64_t row = first + r * kRowsPerBlock;
        if (row < p.rows) Vec<T>::store(static_cast<T *>(p.y) + row * D + lane * N, p.vec, x[r]);
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

// one block a row, NV 16-byte pieces a thread, all of the row in registers
template <typename T, typename W, int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) residual_norm_kernel(ResidualNorm p) {
    constexpr int N = Vec<T>::N;
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.xs, *y = static_cast<const T *>(p.y) + row * p.ys;
    const int pieces = p.width / N;
    float h[NV][N], b[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < pieces) {
            Vec<T>::load(x + c * N, true, h[i]);
            Vec<T>::load(y + c * N, true, b[i]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) h[i][j] = b[i][j] = 0.f;
        }
    }
    float inv = 1.f;
    if (p.pw) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) s = fmaf(b[i][j], b[i][j], s);
        inv = rsqrtf(block_sum(s, red) / (float)p.width + p.eps);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < pieces) {
            if (p.pw) {
                float w[N];
                load_weights<W>(p.pw, c * N, p.wvec, w);
#pragma unroll
                for (int j = 0; j < N; ++j) b[i][j] *= inv * w[j];
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                h[i][j] = fmaf(p.scale, b[i][j], h[i][j]);
                s = fmaf(h[i][j], h[i][j], s);
            }
            Vec<T>::store(static_cast<T *>(p.h) + row * p.width + c * N, true, h[i]);
        }
    }
    inv = rsqrtf(block_sum(s, red) / (float)p.width + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < pieces) {
            float w[N];
            load_weights<W>(p.w, c * N, p.wvec, w);
#pragma unroll
            for (int j = 0; j < N; ++j) h[i][j] *= inv * w[j];
            Vec<T>::store(static_cast<T *>(p.n) + row * p.width + c * N, true, h[i]);
        }
    }
}

// any width and alignment: the row is read again for each of the three steps (from L1
// and L2); the last one writes h and n together, as either may lie on an input
template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) residual_norm_any_kernel(ResidualNorm p) {
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.xs, *y = static_cast<const T *>(p.y) + row * p.ys;
    const W *w = static_cast<const W *>(p.w), *pw = static_cast<const W *>(p.pw);
    float inv = 1.f;
    if (pw) {
        float s = 0.f;
        for (int c = threadIdx.x; c < p.width; c += kThreads) {
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
    for (int c = threadIdx.x; c < p.width; c += kThreads) {
        const float v = at(c);
        s = fmaf(v, v, s);
    }
    const float inv_h = rsqrtf(block_sum(s, red) / (float)p.width + p.eps);
    for (int c = threadIdx.x; c < p.width; c += kThreads) {
        const float v = at(c);
        store_f(static_cast<T *>(p.h), row * p.width + c, v);
        store_f(static_cast<T *>(p.n), row * p.width + c, v * inv_h * load_f(w, c));
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// whether rows `stride` elements apart, from base, all start on 16 bytes
bool vec_rows(const void *base, int64_t stride, int elem) { return aligned16(base) && stride * elem % 16 == 0; }

template <typename T, int LPR>
cudaError_t run_qk_gates(QkGates p, cudaStream_t stream) {
    constexpr int NR = 4, per = kThreads / LPR * NR;
    const int64_t row_blocks = (2 * p.rows + per - 1) / per;
    int64_t gate_blocks = (p.cells + kThreads - 1) / kThreads;
    if (gate_blocks > 2048) gate_blocks = 2048;
    if (row_blocks + gate_blocks > 0x7fffffff) return cudaErrorInvalidValue;
    p.row_blocks = (int)row_blocks;
    qk_gates_kernel<T, LPR, NR><<<(unsigned)(row_blocks + gate_blocks), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
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
    constexpr int NR = 4, per = kThreads / LPR * NR;
    const int64_t blocks = (p.rows + per - 1) / per;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    norm_gate_kernel<T, W, LPR, NR><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
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
    if (!vec || p.width % N || pieces > 4 * 512) {
        residual_norm_any_kernel<T, W><<<(unsigned)tokens, kThreads, 0, stream>>>(p);
    } else if (pieces <= 1024 && tokens <= 2 * sm_count()) {
        residual_norm_kernel<T, W, 1><<<(unsigned)tokens, (pieces + 31) / 32 * 32, 0, stream>>>(p);
    } else {
        residual_norm_kernel<T, W, 4><<<(unsigned)tokens, ((pieces + 3) / 4 + 31) / 32 * 32, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_gates(const gdn_qk_gates_args &a, cudaStream_t stream) {
    const int e = a.dtype == GDN_BF16 ? 2 : 4;
    QkGates p = {};
    p.rows = (int64_t)a.total_tokens * a.n_k_heads;
    p.cells = (int64_t)a.total_tokens * a.n_v_heads;
    p.hk = a.n_k_heads;
    p.hv = a.n_v_heads;
    p.qs = a.q_stride ? a.q_stride : (int64_t)a.n_k_heads * a.d_k;
    p.ks = a.k_stride ? a.k_stride : (int64_t)a.n_k_heads * a.d_k;
    p.as = a.a_stride ? a.a_stride : a.n_v_heads;
    p.bs = a.b_stride ? a.b_stride : a.n_v_heads;
    p.eps = a.eps;
    p.vec = vec_rows(a.q, p.qs, e) && vec_rows(a.k, p.ks, e) && aligned16(a.q_out) && aligned16(a.k_out);
    p.q = a.q; p.k = a.k; p.a = a.a; p.b = a.b;
    p.A_log = a.A_log; p.dt_bias = a.dt_bias;
    p.qo = a.q_out; p.ko = a.k_out; p.g = a.g; p.beta = a.beta;
    return a.dtype == GDN_BF16 ? pick_qk_gates<__nv_bfloat16>(p, a.d_k, stream) : pick_qk_gates<float>(p, a.d_k, stream);
}

cudaError_t launch_norm_gate(const gdn_norm_gate_args &a, cudaStream_t stream) {
    const int e = a.dtype == GDN_BF16 ? 2 : 4;
    NormGate p = {};
    p.rows = (int64_t)a.total_tokens * a.n_v_heads;
    p.hv = a.n_v_heads;
    p.os = a.o_stride ? a.o_stride : (int64_t)a.n_v_heads * a.d_v;
    p.zs = a.z_stride ? a.z_stride : (int64_t)a.n_v_heads * a.d_v;
    p.act = a.act;
    p.eps = a.eps;
    p.vec = vec_rows(a.o, p.os, e) && vec_rows(a.z, p.zs, e) && aligned16(a.y);
    p.wvec = aligned16(a.weight);
    p.o = a.o; p.z = a.z; p.w = a.weight; p.y = a.y;
    const bool wb = a.weight_dtype == GDN_BF16;
    if (a.dtype == GDN_BF16)
        return wb ? pick_norm_gate<__nv_bfloat16, __nv_bfloat16>(p, a.d_v, stream)
                  : pick_norm_gate<__nv_bfloat16, float>(p, a.d_v, stream);
    return wb ? pick_norm_gate<float, __nv_bfloat16>(p, a.d_v, stream) : pick_norm_gate<float, float>(p, a.d_v, stream);
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
    p.x = a.x; p.y = a.y; p.w = a.weight; p.pw = a.post_weight; p.h = a.h; p.n = a.n;
    const bool vec = vec_rows(a.x, p.xs, e) && vec_rows(a.y, p.ys, e) && vec_rows(a.h, a.width, e) && vec_rows(a.n, a.width, e);
    const bool wb = a.weight_dtype == GDN_BF16;
    if (a.dtype == GDN_BF16)
        return wb ? pick_residual_norm<__nv_bfloat16, __nv_bfloat16>(p, a.total_tokens, vec, stream)
                  : pick_residual_norm<__nv_bfloat16, float>(p, a.total_tokens, vec, stream);
    return wb ? pick_residual_norm<float, __nv_bfloat16>(p, a.total_tokens, vec, stream)
              : pick_residual_norm<float, float>(p, a.total_tokens, vec, stream);
}

}  // namespace gdn
