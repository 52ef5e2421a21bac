// kv_append.cu -- new tokens into the paged cache, norm and position rotation on the way.
//
// Per token: each query and key head's row x of d entries, x / sqrt(mean x^2 + eps) * w where there is a norm, the first
// rot_dim entries turned by the position's angles; values copied.  Every byte is read once and written once: bound
// by memory, or for a few tokens by the launch and one chain of loads (offsets, length, page, row).
// A block takes a token, with one warp or four; d / 8 lanes take a row with 8 entries each, one row after another, so that a token's cosines and
// sines are read once into registers.  The partner of an entry in a pair is 8 lanes or fewer away, or its neighbour.
// 16384 tokens of 16 + 2 heads of 256, a quarter turned, with norms: 72 us for 340 MB, 4.7 TB/s (50 at the copy's rate); what is left is
// latency (half the issue slots are free, waits for loads come first), with three rows of a lane on their way (one: 78 us).  In fp32 three
// do not fit the registers and 56 to 104 bytes spill.
// Where rows do not start on 16 bytes, or half the rotated width is no multiple of 8, entries and partners are read one by one.
#include "attn.cuh"

namespace gdn {
namespace {

using attn::launch_dependent;


struct AppendParams {
    int batch, hq, hkv, page_size, n_pages, max_pages, total, rot, n_positions;
    float eps;
    int64_t page_stride, slot_stride, head_stride, qs, ks, vs;
    const void *q, *k, *v, *q_weight, *k_weight;
    const int32_t *table, *lens, *offsets, *depth;
    const float *cos_sin;
    void *q_out, *k_cache, *v_cache;
    int32_t *status;
    bool weight_bf16;
};

// eight entries as they lie in memory
template <typename T, bool VEC>
struct Raw {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
        } else {
            T *x = reinterpret_cast<T *>(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = p[i];
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
        } else {
            const T *x = reinterpret_cast<const T *>(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = x[i];
        }
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        const T *y = reinterpret_cast<const T *>(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = load_f(y, i);
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    if constexpr (VEC && sizeof(T) == 2) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else if constexpr (VEC) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) store_f(p, i, x[i]);
    }
}

__device__ __forceinline__ float weight_at(const void *w, bool bf16, int i) {
    return bf16 ? load_f(static_cast<const __nv_bfloat16 *>(w), i) : load_f(static_cast<const float *>(w), i);
}

// VEC: 16-byte pieces (weights and angles too), and the partner of lane l's entries (halves) is another lane's; INTER: pairs of neighbours
template <typename T, int D, bool VEC, bool INTER, int kThreads>
__global__ void __launch_bounds__(kThreads, VEC ? 640 / kThreads : 1) append_kernel(AppendParams p) {
    after_previous();
    constexpr int L = D / 8, G = kThreads / L;  // lanes a row, rows a block has in flight
    const int t = blockIdx.x, tid = threadIdx.x, sub = tid % L, e0 = sub * 8, half = p.rot / 2, h0 = tid / L;
    // the first rows are on their way while the token's place is found, the later ones while those before them are worked on
    const T *q_from = static_cast<const T *>(p.q) + t * p.qs + e0, *k_from = static_cast<const T *>(p.k) + t * p.ks + e0,
            *v_from = static_cast<const T *>(p.v) + t * p.vs + e0;
    constexpr int kAhead = 3;  // rows of a lane on their way
    Raw<T, VEC> q_next[kAhead] = {}, k_next[1] = {}, v_next = {};
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (h0 + i * G < p.hq) q_next[i].load(q_from + (h0 + i * G) * D);
    if (h0 < p.hkv) k_next[0].load(k_from + h0 * D), v_next.load(v_from + h0 * D);
    int b = t, i = 0;
    if (p.offsets) {
        int upto = 0;
        for (int j = 0; j < p.batch; j += kThreads)
            upto += __syncthreads_count(j + tid < p.batch && p.offsets[j + tid + 1] <= t);
        if (t == 0) {  // looked at once
            bool bad = tid == 0 && p.offsets[0] != 0;
            for (int j = tid; j < p.batch; j += kThreads) bad = bad || p.offsets[j + 1] < p.offsets[j] || p.offsets[j + 1] > p.total;
            if (bad) flag(p.status, GDN_DEV_BAD_DESC);
        }
        if (upto >= p.batch) return;
        b = upto;
        i = t - p.offsets[b];
        if (i < 0 || p.offsets[b] < 0 || p.offsets[b + 1] > p.total || t >= p.offsets[b + 1]) return;
    }
    const int len = p.lens[b];
    if (len == -1) return;
    const int64_t slot = (int64_t)len + i;
    const int64_t position = p.depth ? (int64_t)len + p.depth[t] - 1 : slot;
    // (a table has at most 2^30 slots)
    const int page = slot < (1 << 30) ? (int)slot / p.page_size : p.max_pages;
    int bad = 0, id = 0;
    if (len < 0 || page >= p.max_pages) bad = GDN_DEV_BAD_PAGE;
    else if (id = p.table[(int64_t)b * p.max_pages + page]; id < 0 || id >= p.n_pages) bad = GDN_DEV_BAD_PAGE;
    else if (p.rot && (position < 0 || position >= p.n_positions)) bad = GDN_DEV_BAD_POSITION;
    if (bad) {
        if (tid == 0) flag(p.status, bad);
        return;
    }
    const int64_t at = id * p.page_stride + ((int)slot - page * p.page_size) * p.slot_stride;

    // this lane's angles: entry e0 + n turns with pair (e0 + n) % half, or (e0 + n) / 2 in neighbours; the first of a pair subtracts
    float cs[8], sn[8];
    const float *angles = p.cos_sin + position * p.rot;
    if (VEC && !INTER) {
        // (half is a multiple of 8: all eight are turned or none, and their angles lie side by side)
        const bool turned = e0 < p.rot;
        const float sign = e0 < half ? -1.f : 1.f;
#pragma unroll
        for (int n = 0; n < 8; ++n) cs[n] = 1.f, sn[n] = 0.f;
        if (turned) {
            const float *c = angles + (e0 < half ? e0 : e0 - half);
            Raw<float, true> raw;
            raw.load(c);
            raw.values(cs);
            raw.load(c + half);
            raw.values(sn);
#pragma unroll
            for (int n = 0; n < 8; ++n) sn[n] *= sign;
        }
    } else {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int e = e0 + n;
            const int pair = INTER ? e / 2 : e < half ? e : e - half;
            const bool turned = e < p.rot;
            cs[n] = turned ? angles[pair] : 1.f;
            sn[n] = turned ? angles[half + pair] * ((INTER ? (e & 1) == 0 : e < half) ? -1.f : 1.f) : 0.f;
        }
    }
    const unsigned mates = (L == 32 ? 0xffffffffu : (1u << (L & 31)) - 1) << ((tid & 31) / L * L);  // the lanes of a row
    // entry n of a row is r (x_n a_n + y_n b_n), y its partner and r the norm's factor: weights and angles make a and b once
    auto turn = [&](const T *from, int n_heads, auto &next, const void *w, T *to, int64_t pitch) {
        const bool turned = VEC && !INTER && e0 < p.rot;  // (otherwise each entry by itself)
        const int away = half / 8, mate = (e0 < half ? sub + away : sub - away) & (L - 1);
        float a[8], b[8];
        if (VEC && !INTER && w) {
            if (p.weight_bf16) {
                Raw<__nv_bfloat16, true> raw;
                raw.load(static_cast<const __nv_bfloat16 *>(w) + e0);
                raw.values(a);
            } else {
                Raw<float, true> raw;
                raw.load(static_cast<const float *>(w) + e0);
                raw.values(a);
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) b[n] = __shfl_sync(mates, a[n], mate, L);
        } else {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const int e = e0 + n, pe = INTER ? e ^ 1 : e < half ? e + half : e - half;
                a[n] = w ? weight_at(w, p.weight_bf16, e) : 1.f;
                b[n] = w && e < p.rot ? weight_at(w, p.weight_bf16, pe) : 1.f;
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) a[n] *= cs[n], b[n] *= sn[n];
        constexpr int N = sizeof(next) / sizeof(next[0]);
        auto one = [&](int h, Raw<T, VEC> &place) {
            const Raw<T, VEC> now = place;
            if (h + N * G < n_heads) place.load(from + (h + N * G) * D);
            float x[8], y[8], z[8], r = 1.f;
            now.values(x);
            if (w) {
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 8; ++n) sum = fmaf(x[n], x[n], sum);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mates, sum, o, L);
                r = rsqrtf(sum * (1.f / D) + p.eps);
            }
            if constexpr (INTER) {
#pragma unroll
                for (int n = 0; n < 8; ++n) y[n] = x[n ^ 1];
            } else if constexpr (VEC) {
#pragma unroll
                for (int n = 0; n < 8; ++n) y[n] = __shfl_sync(mates, x[n], mate, L);
            } else {
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const int e = e0 + n;
                    y[n] = e < p.rot ? load_f(from - e0 + h * D, e < half ? e + half : e - half) : 0.f;
                }
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                z[n] = x[n] * a[n];
                if (VEC && !INTER ? turned : e0 + n < p.rot) z[n] = fmaf(y[n], b[n], z[n]);
                if (w) z[n] *= r;
            }
            __syncwarp(mates);  // q_out may be q: partners have been read
            store8<T, VEC>(to + h * pitch, z);
        };
        for (int h = h0; h < n_heads; h += N * G) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (h + i * G < n_heads) one(h + i * G, next[i]);
        }
    };
    if (p.hq) turn(q_from, p.hq, q_next, p.q_weight, static_cast<T *>(p.q_out) + (int64_t)t * p.hq * D + e0, D);
    turn(k_from, p.hkv, k_next, p.k_weight, static_cast<T *>(p.k_cache) + at + e0, p.head_stride);
    T *v_to = static_cast<T *>(p.v_cache) + at + e0;
    for (int h = h0; h < p.hkv; h += G) {
        const Raw<T, VEC> now = v_next;
        if (h + G < p.hkv) v_next.load(v_from + (h + G) * D);
        now.store(v_to + h * p.head_stride);
    }
}

template <typename T, int D, int kThreads>
cudaError_t run_threads(const AppendParams &p, bool vec, bool inter, cudaStream_t stream) {
    auto kernel = vec ? (inter ? append_kernel<T, D, true, true, kThreads> : append_kernel<T, D, true, false, kThreads>)
                      : (inter ? append_kernel<T, D, false, true, kThreads> : append_kernel<T, D, false, false, kThreads>);
    return launch_dependent(kernel, dim3(p.total), kThreads, 0, stream, p);
}

// One warp a token where there are many: a token's place is found, and its factors made, by each warp that has a part of it
// (16384 tokens of 20 rows of 256: 86 us with four warps).  Few tokens are spread over more threads.
template <typename T, int D>
cudaError_t run(const AppendParams &p, bool vec, bool inter, cudaStream_t stream) {
    return p.total >= 16 * sm_count() ? run_threads<T, D, 32>(p, vec, inter, stream) : run_threads<T, D, 128>(p, vec, inter, stream);
}

template <typename T>
cudaError_t pick(const AppendParams &p, int d, bool vec, bool inter, cudaStream_t stream) {
    switch (d) {
        case 16: return run<T, 16>(p, vec, inter, stream);
        case 32: return run<T, 32>(p, vec, inter, stream);
        case 64: return run<T, 64>(p, vec, inter, stream);
        case 128: return run<T, 128>(p, vec, inter, stream);
        default: return run<T, 256>(p, vec, inter, stream);
    }
}

}  // namespace

cudaError_t launch_kv_append(const gdn_kv_append_args &a, cudaStream_t stream) {
    const gdn_kv_cache &c = a.cache;
    const int e = c.dtype == GDN_BF16 ? 2 : 4;
    AppendParams p = {};
    p.batch = c.batch; p.hq = a.q ? a.n_q_heads : 0; p.hkv = c.n_kv_heads;
    p.page_size = c.page_size; p.n_pages = c.n_pages; p.max_pages = c.max_pages; p.total = a.total_tokens;
    p.rot = a.rot_dim; p.n_positions = a.n_positions; p.eps = a.eps;
    p.page_stride = c.page_stride; p.slot_stride = c.slot_stride; p.head_stride = c.head_stride;
    p.qs = a.q_stride ? a.q_stride : (int64_t)a.n_q_heads * c.d;
    p.ks = a.k_stride ? a.k_stride : (int64_t)c.n_kv_heads * c.d;
    p.vs = a.v_stride ? a.v_stride : (int64_t)c.n_kv_heads * c.d;
    p.q = a.q; p.k = a.k; p.v = a.v; p.q_weight = a.q_weight; p.k_weight = a.k_weight;
    p.table = c.page_table; p.lens = c.lens; p.offsets = a.token_offsets; p.depth = a.depth; p.cos_sin = a.cos_sin;
    p.q_out = a.q_out; p.k_cache = c.k; p.v_cache = c.v; p.status = c.dev_status;
    p.weight_bf16 = a.weight_dtype == GDN_BF16;
    const uintptr_t pointers = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                               reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.q_weight) | reinterpret_cast<uintptr_t>(a.k_weight) |
                               reinterpret_cast<uintptr_t>(a.cos_sin) | reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v);
    const int64_t strides = (p.hq ? p.qs : 0) | p.ks | p.vs | p.page_stride | p.slot_stride | p.head_stride;
    const bool vec = (pointers & 15) == 0 && strides * e % 16 == 0 && (a.interleaved || a.rot_dim % 16 == 0);
    return c.dtype == GDN_BF16 ? pick<__nv_bfloat16>(p, c.d, vec, a.interleaved != 0, stream)
                               : pick<float>(p, c.d, vec, a.interleaved != 0, stream);
}

}  // namespace gdn
