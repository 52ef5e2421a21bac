// attend_simt.cu -- attention over a paged cache, general: fp32, and bf16 that the tensor-core kernels do not take.
//
// A block has 16 rows (or 8, or 4) and takes 32 slots at a time: keys and values to shared memory as fp32 (the next tile's are on their way in
// registers meanwhile, where rows start on 16 bytes), the scores one slot a
// lane, a quarter of the rows a warp, the running maximum and sum of a row in its warp, then the outputs with a column (or two) a thread.
// fp32 arithmetic throughout.  What bounds it is shared-memory reads beside the multiplications (five 16-byte
// reads for 16 of them in the scores): 6 single tokens over 100 to 23617 slots, 8 heads of 128, 167 us for 582 MB (86); 71
// over 100 to 7194, 8 query heads to one of 128, 100 us for 236 MB (35); 3 trees of 100 nodes behind 1000 slots, 16 heads
// of 128 to 4, 212 us; 8 trees of 128 nodes behind 200 to 2200 slots, the same heads, 817 us, 12.6 TFLOP/s.
#include "attn.cuh"

namespace gdn {
namespace {

using namespace attn;

constexpr int kKT = 32, kThreads = 128, kMostWhole = 4, kCost = 1;

// R: rows of a block
template <int D, int R>
struct Shared {
    float q[R][D + 4], k[kKT][D + 4], v[kKT][D], p[kKT][R + 4], m[R], f[R], l[R];
    int64_t at[kKT];
    Scratch find;
};

// Rows of D entries from elements `at` of x, as fp32 (VEC: that is what they are); zeros where at < 0.
template <typename T, int D, bool VEC>
__device__ __forceinline__ void load_rows(const void *x, const int64_t *at, int rows, float *to, int ld) {
    const T *src = static_cast<const T *>(x);
    if constexpr (VEC) {
        for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
            const int row = i / (D / 4), c = i % (D / 4) * 4;
            const float4 y = at[row] >= 0 ? *reinterpret_cast<const float4 *>(src + at[row] + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(to + row * ld + c) = y;
        }
    } else {
        for (int i = threadIdx.x; i < rows * D; i += kThreads) {
            const int row = i / D, c = i % D;
            to[row * ld + c] = at[row] >= 0 ? load_f(src, at[row] + c) : 0.f;
        }
    }
}

// A thread's share of a tile's keys and values in fp32, on its way while the tile before it is worked on.
template <int D>
struct Ahead {
    static constexpr int N = kKT * (D / 4) / kThreads;
    float4 k[N], v[N];
    __device__ __forceinline__ void load(const Params &p, const Place &at, int slot0, int seen) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int n = i * kThreads + threadIdx.x, slot = slot0 + n / (D / 4);
            const int64_t off = slot < seen ? slot_offset(p, at.b, at.h, slot) : -1;
            k[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (off >= 0) {
                k[i] = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.k) + off + n % (D / 4) * 4);
                v[i] = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.v) + off + n % (D / 4) * 4);
            }
        }
    }
    __device__ __forceinline__ void store(float *k_to, int k_ld, float *v_to, int v_ld) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int n = i * kThreads + threadIdx.x, row = n / (D / 4), c = n % (D / 4) * 4;
            *reinterpret_cast<float4 *>(k_to + row * k_ld + c) = k[i];
            *reinterpret_cast<float4 *>(v_to + row * v_ld + c) = v[i];
        }
    }
};

template <typename T, int D, bool VEC, int R>
__global__ void __launch_bounds__(kThreads) attend_simt_kernel(Params p, int runs) {
    after_previous();
    extern __shared__ __align__(16) uint8_t raw[];
    using S = Shared<D, R>;
    S &s = *reinterpret_cast<S *>(raw);
    // for the outputs: columns of a thread, groups of threads that share the rows (threads past them have none), rows of each
    constexpr int kCols = D > kThreads ? D / kThreads : 1, kGroups = D >= kThreads ? 1 : kThreads / D < R ? kThreads / D : R, kMine = R / kGroups;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, run = blockIdx.x;
    int64_t per, t, end;
    Place at;
    if (p.whole) {
        item_of<kKT>(p, run, (p.max_tokens * p.group + R - 1) / R, t, end, at);
    } else {
        find<kKT>(p, runs, run, run == 0 ? p.status : nullptr, s.find, per, t, end, at);
        if (tid == 0) tell_cut<kKT>(p, R, D, runs, run, per, t, end, at);
    }
    if (t >= end) return;
    Request r = request(p, at.b, nullptr);
    while (t < end) {
        const Span span = span_of<kKT>(p, r, at, end - t);
        const int tiles = span.tiles, first = span.first, last = span.last, seen = seen_slots(p, r, at.qt), common = common_slots(p, r, at.qt);
        if (last <= first) break;
        const int64_t row0 = (int64_t)at.qt * R, rows = (int64_t)r.n * p.group;
        if (tid < R) {
            const int64_t q = row0 + tid;
            s.at[tid] = q < rows ? (r.first + q / p.group) * p.q_stride + (at.h * p.group + q % p.group) * D : -1;
        }
        if (tid < R) s.m[tid] = -INFINITY, s.l[tid] = 0.f;
        __syncthreads();
        load_rows<T, D, VEC>(p.q, s.at, R, &s.q[0][0], D + 4);
        float acc[kMine][kCols] = {};
        Ahead<D> ahead;
        if constexpr (VEC) ahead.load(p, at, first * kKT, seen);
        for (int tile = first; tile < last; ++tile) {
            const int slot0 = tile * kKT;
            __syncthreads();
            if constexpr (VEC) {
                ahead.store(&s.k[0][0], D + 4, &s.v[0][0], D);
                __syncthreads();
                if (tile + 1 < last) ahead.load(p, at, slot0 + kKT, seen);
            } else {
                if (tid < kKT) s.at[tid] = slot0 + tid < seen ? slot_offset(p, at.b, at.h, slot0 + tid) : -1;
                __syncthreads();
                load_rows<T, D, VEC>(p.k, s.at, kKT, &s.k[0][0], D + 4);
                load_rows<T, D, VEC>(p.v, s.at, kKT, &s.v[0][0], D);
                __syncthreads();
            }
            float x[R / 4] = {};
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const float4 k = *reinterpret_cast<const float4 *>(&s.k[lane][c]);
#pragma unroll
                for (int i = 0; i < R / 4; ++i) {
                    const float4 q = *reinterpret_cast<const float4 *>(&s.q[warp + 4 * i][c]);
                    x[i] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, x[i]))));
                }
            }
            const int slot = slot0 + lane;
#pragma unroll
            for (int i = 0; i < R / 4; ++i) {
                const int row = warp + 4 * i;
                const int64_t q = row0 + row;
                float y = slot < seen && q < rows && sees(p, r, (int)(q / p.group), slot) ? x[i] * p.scale_log2 : -INFINITY;
                float m = y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const float z = __shfl_xor_sync(0xffffffffu, m, o);
                    m = fmaxf(m, z);
                }
                const float old = s.m[row];
                m = fmaxf(m, old);
                const float base = m == -INFINITY ? 0.f : m;
                // a NaN score has no place in the maximum, and makes the sum NaN
                const float e = exp2f(y - base), f = exp2f(old - base);
                const float sum = warp_sum(e);
                __syncwarp();
                s.p[lane][row] = e;
                if (lane == 0) s.m[row] = m, s.f[row] = f, s.l[row] = fmaf(s.l[row], f, sum);
            }
            __syncthreads();
            const int g = min(tid / D, kGroups - 1);
            const bool masked = slot0 + kKT > common;  // what is not seen there may be anything
#pragma unroll
            for (int i = 0; i < kMine; ++i)
#pragma unroll
                for (int c = 0; c < kCols; ++c) acc[i][c] *= s.f[g * kMine + i];
#pragma unroll 8
            for (int j = 0; j < kKT; ++j) {
                float v[kCols];
#pragma unroll
                for (int c = 0; c < kCols; ++c) v[c] = s.v[j][(tid + c * kThreads) % D];
                float e[kMine];
                if constexpr (kMine % 4 == 0) {
#pragma unroll
                    for (int i = 0; i < kMine; i += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(&s.p[j][g * kMine + i]);
                        e[i] = x.x, e[i + 1] = x.y, e[i + 2] = x.z, e[i + 3] = x.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kMine; ++i) e[i] = s.p[j][g * kMine + i];
                }
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    if (!masked || e[i] != 0.f) {
#pragma unroll
                        for (int c = 0; c < kCols; ++c) acc[i][c] = fmaf(e[i], v[c], acc[i][c]);
                    }
                }
            }
        }
        __syncthreads();
        const bool whole = first == 0 && last == tiles;
        const int which = first == 0, g = tid / D;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int row = g * kMine + i;
            const int64_t q = row0 + row;
            if (g >= kGroups || q >= rows) continue;
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const int col = (tid + c * kThreads) % D;
                if (whole) {
                    const float y = s.l[row] == 0.f ? inverse(p, r, (int)(q / p.group), 0.f) : acc[i][c] / s.l[row];
                    const int64_t to = ((int64_t)(r.first + q / p.group) * p.hkv * p.group + at.h * p.group + q % p.group) * D + col;
                    if (p.out_bf16) store_f(static_cast<__nv_bfloat16 *>(p.o), to, y);
                    else store_f(static_cast<float *>(p.o), to, y);
                } else {
                    part_out(p, R, D, run, which)[row * D + col] = acc[i][c];
                }
            }
        }
        if (!whole && tid < R) {
            float *st = part_stat(p, R, D, runs, run, which) + tid * 2;
            st[0] = s.m[tid], st[1] = s.l[tid];
        }
        t += span.units;
        if (t < end) next_item(p, at, r);
        __syncthreads();
    }
}

template <typename T, int D, bool VEC, int R>
cudaError_t run(Params p, int runs, cudaStream_t stream) {
    static int have[16];
    p.rows = R, p.cost = kCost;
    const cudaError_t e = ensure_smem(attend_simt_kernel<T, D, VEC, R>, (int)sizeof(Shared<D, R>), have);
    if (e != cudaSuccess) return e;
    const cudaError_t f = launch_dependent(attend_simt_kernel<T, D, VEC, R>, dim3(runs), kThreads, sizeof(Shared<D, R>), stream, p, runs);
    return f != cudaSuccess || p.whole ? f : launch_join<D, R>(p, runs, stream);
}

template <typename T, bool VEC, int R>
cudaError_t (*pick(int d))(Params, int, cudaStream_t) {
    switch (d) {
        case 16: return run<T, 16, VEC, R>;
        case 32: return run<T, 32, VEC, R>;
        case 64: return run<T, 64, VEC, R>;
        case 128: return run<T, 128, VEC, R>;
        default: return run<T, 256, VEC, R>;
    }
}

}  // namespace

attn::Choice attend_simt_choice(const gdn_kv_attend_args &a, bool decode) {
    const gdn_kv_cache &c = a.cache;
    // fp32 rows on 16 bytes: four (or eight) rows a block where a request has no more (16 would compute four times what one head needs: 6 single
    // tokens over 100..23617 slots, 8 heads of 128, 373 us)
    const bool vec = c.dtype == GDN_F32 && aligned16(a), few = vec && (decode ? 1 : (int64_t)a.max_tokens) * (a.n_q_heads / c.n_kv_heads) <= 4;
    const bool some = vec && !few && (decode ? 1 : (int64_t)a.max_tokens) * (a.n_q_heads / c.n_kv_heads) <= 8;
    const int R = few ? 4 : some ? 8 : 16;
    Choice x;
    x.whole = whole_items(a, decode, R, kKT, kMostWhole, x.runs);
    if (!x.whole) x.runs = most_runs(a, decode, R, kKT, c.d == 256 ? 2 : 3);  // (what their registers leave room for)
    x.workspace = x.whole ? 0 : 4 * workspace_floats(R, c.d, x.runs);
    // (bf16 rows on 16 bytes are the tensor cores')
    x.launch = c.dtype == GDN_BF16 ? pick<__nv_bfloat16, false, 16>(c.d)
               : few               ? pick<float, true, 4>(c.d)
               : some              ? pick<float, true, 8>(c.d)
               : vec               ? pick<float, true, 16>(c.d)
                                   : pick<float, false, 16>(c.d);
    return x;
}

}  // namespace gdn
