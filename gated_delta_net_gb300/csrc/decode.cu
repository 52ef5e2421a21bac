// decode.cu -- one token a request through the gated delta rule, states in a pool.
//
// Per (request, value head), with the state S[d_v][d_k]:
//     u = beta (v - e^g S k),  S <- e^g S + u k^T,  o = scale (e^g S q + u (k . q))
// S k and S q are taken of the old state in one pass, so a state is read once, held
// in registers and written once: 8 bytes an entry and about 7 operations, bound by
// memory.  A row of S takes d_k / 16 lanes with four 16-byte pieces each (128
// contiguous bytes an instruction for d_k = 128); a warp has two sets of rows in
// flight, and a block takes an eighth of the heads' rows or more, so that a single
// request still spreads over the GPU.  A head's blocks are neighbours, so that its state is
// read and written in one run, and it passes the cache as something not needed again soon:
// 256 requests of 32 heads take 152 us, 6.9 TB/s (155 without the early launch, 169 with none of
// this).
#include "internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kSets = 2;  // row sets a warp has in flight

struct DecodeParams {
    int hk, hv, dv, n_states, slab_bits;  // blocks a head takes, a power of two
    int64_t qs, ks, vs;
    float scale;
    bool vec;  // q and k rows start on 16 bytes
    const void *q, *k, *v;
    const float *g, *beta;
    float *S;
    const int32_t *slots;
    void *o;
    int32_t *status;
};

template <typename T>
__device__ __forceinline__ void load4(const T *p, bool vec, float (&x)[4]) {
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            const float4 w = *reinterpret_cast<const float4 *>(p);
            x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xFFFF0000u);
            x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = load_f(p, i);
    }
}

template <typename T, typename O, int DK>
__global__ void __launch_bounds__(kThreads) decode_kernel(DecodeParams p) {
    after_previous();
    constexpr int LPR = DK / 16, kRowsPerSet = 32 / LPR, kRowsPerBlock = kThreads / 32 * kSets * kRowsPerSet;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LPR;
    const int item = blockIdx.x >> p.slab_bits, slab = blockIdx.x & ((1 << p.slab_bits) - 1);
    const int b = item / p.hv, h = item % p.hv, hk = h / (p.hv / p.hk);
    const int row0 = slab * kRowsPerBlock + warp * (kSets * kRowsPerSet) + lane / LPR;
    const int slot = p.slots ? p.slots[b] : b;
    O *o = static_cast<O *>(p.o) + ((int64_t)b * p.hv + h) * p.dv;
    if (slot < 0 || slot >= p.n_states) {
        if (slot == -1) {
#pragma unroll
            for (int i = 0; i < kSets; ++i)
                if (sub == 0 && row0 + i * kRowsPerSet < p.dv) store_f(o, row0 + i * kRowsPerSet, 0.f);
        } else if (threadIdx.x == 0) {
            flag(p.status, GDN_DEV_BAD_SLOT);
        }
        return;
    }
    float *S = p.S + ((int64_t)slot * p.hv + h) * p.dv * DK;
    float4 s[kSets][4];
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
        const int row = row0 + i * kRowsPerSet;
        if (row < p.dv) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint4 w = load_streaming(S + (int64_t)row * DK + (c * LPR + sub) * 4);
                s[i][c] = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) s[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    const T *qp = static_cast<const T *>(p.q) + b * p.qs + hk * DK, *kp = static_cast<const T *>(p.k) + b * p.ks + hk * DK;
    float q[4][4], k[4][4], kq = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        load4(kp + (c * LPR + sub) * 4, p.vec, k[c]);
        load4(qp + (c * LPR + sub) * 4, p.vec, q[c]);
    }
    const float alpha = expf(p.g[(int64_t)b * p.hv + h]), beta = p.beta[(int64_t)b * p.hv + h];
    float v[kSets];
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
        const int row = row0 + i * kRowsPerSet;
        v[i] = row < p.dv ? load_f(static_cast<const T *>(p.v) + b * p.vs + h * p.dv, row) : 0.f;
    }
    float sk[kSets] = {}, sq[kSets] = {};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) kq = fmaf(k[c][e], q[c][e], kq);
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            const float x[4] = {s[i][c].x, s[i][c].y, s[i][c].z, s[i][c].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sk[i] = fmaf(x[e], k[c][e], sk[i]);
                sq[i] = fmaf(x[e], q[c][e], sq[i]);
            }
        }
    }
#pragma unroll
    for (int w = LPR / 2; w > 0; w >>= 1) {
        kq += __shfl_xor_sync(0xffffffffu, kq, w);
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], w);
            sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], w);
        }
    }
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
        const int row = row0 + i * kRowsPerSet;
        if (row >= p.dv) continue;
        const float u = beta * (v[i] - alpha * sk[i]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float4 x = s[i][c];
            x.x = fmaf(u, k[c][0], alpha * x.x);
            x.y = fmaf(u, k[c][1], alpha * x.y);
            x.z = fmaf(u, k[c][2], alpha * x.z);
            x.w = fmaf(u, k[c][3], alpha * x.w);
            __stcs(reinterpret_cast<float4 *>(S + (int64_t)row * DK + (c * LPR + sub) * 4), x);
        }
        if (sub == 0) store_f(o, row, p.scale * fmaf(u, kq, alpha * sq[i]));
    }
}

template <typename T, typename O, int DK>
cudaError_t run(DecodeParams p, int batch, cudaStream_t stream) {
    constexpr int rows = kThreads / 32 * kSets * (32 / (DK / 16));
    const int64_t items = (int64_t)batch * p.hv;
    while (rows << p.slab_bits < p.dv) ++p.slab_bits;
    if (items << p.slab_bits > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_early(decode_kernel<T, O, DK>, (unsigned)(items << p.slab_bits), kThreads, stream, p);
}

template <typename T, typename O>
cudaError_t pick(const DecodeParams &p, int dk, int batch, cudaStream_t stream) {
    switch (dk) {
        case 16: return run<T, O, 16>(p, batch, stream);
        case 32: return run<T, O, 32>(p, batch, stream);
        case 64: return run<T, O, 64>(p, batch, stream);
        case 128: return run<T, O, 128>(p, batch, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode(const gdn_decode_args &a, cudaStream_t stream) {
    const int e = a.qkv_dtype == GDN_BF16 ? 2 : 4;
    DecodeParams p = {};
    p.hk = a.n_k_heads; p.hv = a.n_v_heads; p.dv = a.d_v; p.n_states = a.n_states;
    p.qs = a.q_stride ? a.q_stride : (int64_t)a.n_k_heads * a.d_k;
    p.ks = a.k_stride ? a.k_stride : (int64_t)a.n_k_heads * a.d_k;
    p.vs = a.v_stride ? a.v_stride : (int64_t)a.n_v_heads * a.d_v;
    p.scale = a.scale;
    p.vec = ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k)) & 15) == 0 && p.qs * e % 16 == 0 &&
            p.ks * e % 16 == 0;
    p.q = a.q; p.k = a.k; p.v = a.v; p.g = a.g; p.beta = a.beta; p.S = a.S; p.slots = a.slots; p.o = a.o;
    p.status = a.dev_status;
    const bool ob = a.out_dtype == GDN_BF16;
    if (a.qkv_dtype == GDN_BF16)
        return ob ? pick<__nv_bfloat16, __nv_bfloat16>(p, a.d_k, a.batch, stream)
                  : pick<__nv_bfloat16, float>(p, a.d_k, a.batch, stream);
    return ob ? pick<float, __nv_bfloat16>(p, a.d_k, a.batch, stream) : pick<float, float>(p, a.d_k, a.batch, stream);
}

}  // namespace gdn
