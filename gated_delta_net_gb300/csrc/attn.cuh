// attn.cuh -- what the attention kernels share (gdn_attention.h): slots of the paged cache, and how the work is cut.
//
// An item is a request's key-value head with one tile of R = Params::rows rows (row r: token r / group, query head r % group of
// those that share the head); its work is the tiles of KT slots that any of its rows sees, and what beginning and ending it
// costs (Params::cost, in tiles).  All items' work, one
// item after another, are cut into equal runs, one for each block.  A run that has all of an item writes its
// outputs; the others write the sum, the maximum and the unscaled output of what they had to the workspace, at most
// two of them a block (the item it ends, the item it begins), and join_kernel adds an item's parts in order.
// So every block has the same work whatever the lengths are, nothing depends on the host knowing them, and the result
// does not depend on timing.
#pragma once

#include "internal.cuh"

namespace gdn {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    int batch, hkv, group, page_size, n_pages, max_pages, total, max_tokens, mask_words;
    int rows, cost;                         // R: rows of an item; what an item costs besides its tiles, in tiles
    int64_t page_stride, slot_stride, head_stride, q_stride;
    float scale_log2;
    const void *k, *v, *q;
    const int32_t *table, *lens, *offsets;  // offsets NULL: token b is request b's only one
    const uint32_t *mask;                   // NULL: causal
    void *o;
    float *ws;                              // for R <= CAP rows: [blocks][2][CAP][d] outputs, [blocks][2][CAP][2] maxima (base 2) and sums, [blocks] Cut
    int32_t *status;
    int page_bits;                          // log2 of page_size, or -1
    bool out_bf16;
    bool whole;                             // a run for each item, none cut
};

// The tokens of request b: the first one's row, how many (0: the request is left out), the committed ones
// (-1: not in use).
struct Request {
    int first, n, len;
};
__device__ __forceinline__ Request request(const Params &p, int b, int32_t *status) {
    Request r = {b, 1, p.lens[b]};
    int bad = 0;
    if (p.offsets) {
        const int lo = p.offsets[b], hi = p.offsets[b + 1];
        r.first = lo;
        r.n = hi - lo;
        if (lo < 0 || hi < lo || hi > p.total) bad = GDN_DEV_BAD_DESC;
        else if (r.n > p.max_tokens || (p.mask && r.n > 32 * p.mask_words)) bad = GDN_DEV_TOO_MANY;
    }
    if (!bad && r.n > 0 && (r.len < -1 || (r.len >= 0 && (int64_t)r.len + r.n > (int64_t)p.max_pages * p.page_size))) bad = GDN_DEV_BAD_PAGE;
    if (bad) {
        r.n = 0;
        if (status) flag(status, bad);
    }
    return r;
}

// Slots that some row of tile qt sees (0: none), and the tiles they make (one at least, which writes the zeros).
__device__ __forceinline__ int seen_slots(const Params &p, const Request &r, int qt) {
    if (r.len < 0) return 0;
    return r.len + (p.mask ? r.n : min(r.n, ((qt + 1) * p.rows + p.group - 1) / p.group));
}
// Slots from the first on that all of its rows see.
__device__ __forceinline__ int common_slots(const Params &p, const Request &r, int qt) {
    return r.len < 0 ? 0 : r.len + (p.mask ? 0 : qt * p.rows / p.group + 1);
}
template <int KT>
__device__ __forceinline__ int item_tiles(const Params &p, const Request &r, int qt) {
    return max(1, (seen_slots(p, r, qt) + KT - 1) / KT);
}
__device__ __forceinline__ int row_tiles(const Params &p, const Request &r) {
    return (int)((uint32_t)(r.n * p.group + p.rows - 1) / (uint32_t)p.rows);  // (n group is at most 2^30)
}
// sum of floor((a i + b) / m) for i = 0 .. n - 1 (a, b >= 0), by turning the lattice points under the line over as in Euclid's algorithm
// (the reciprocity of such sums: Graham, Knuth, Patashnik, Concrete Mathematics, section 3.5)
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    int64_t sum = 0;
#pragma unroll 1
    while (n > 0) {
        if (a >= m) sum += n * (n - 1) / 2 * (a / m), a %= m;
        if (b >= m) sum += n * (b / m), b %= m;
        const int64_t top = a * n + b;
        if (top < m) break;
        n = top / m, b = top % m;
        const int64_t old = m;
        m = a, a = old;
    }
    return sum;
}
// all tiles of one head of a request: tile qt ends at floor((R (qt + 1) + group - 1) / group) of the new tokens
template <int KT>
__device__ __forceinline__ int64_t head_tiles(const Params &p, const Request &r) {
    const int nq = row_tiles(p, r);
    if (nq == 0) return 0;
    const int last = item_tiles<KT>(p, r, nq - 1) + p.cost;
    if (p.mask || r.len < 0 || nq == 1) return (int64_t)nq * last;
    return last + (int64_t)(nq - 1) * p.cost + floor_sum(nq - 1, (int64_t)p.group * KT, p.rows, p.rows + p.group - 1 + p.group * ((int64_t)r.len + KT - 1));
}

// A place in the work: unit `off` of an item, whose tiles come after `cost` units.
struct Place {
    int b, h, qt, off;
};

// What find() shares between the threads of a block.
struct Scratch {
    int64_t warp_sum[32];
    int64_t rest;
    Place at;
};

__device__ __forceinline__ int64_t div_up(int64_t a, int64_t b) {
    return (a | b) >> 31 ? (a + b - 1) / b : (int64_t)(((uint32_t)a + (uint32_t)b - 1) / (uint32_t)b);
}

// Sum of `mine` over the block's threads before this one, and over all.  Every thread of the block calls this.
__device__ __forceinline__ int64_t scan(int64_t mine, Scratch &s, int64_t &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) s.warp_sum[warp] = upto;
    __syncthreads();
    int64_t before = upto - mine;
    total = 0;
#pragma unroll 1
    for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        const int64_t x = s.warp_sum[w];
        if (w < warp) before += x;
        total += x;
    }
    return before;
}

// How many tiles a run has, and where run number `run` of `runs` begins and ends (begin == end: nothing to do); `at`
// is the place where it begins.  Every thread of the block calls this.
template <int KT>
static __device__ __noinline__ void find(const Params &p, int runs, int run, int32_t *status, Scratch &s, int64_t &per, int64_t &begin,
                                     int64_t &end, Place &at) {
    const int nt = blockDim.x, tid = threadIdx.x;
    const int each = (p.batch + nt - 1) / nt, b0 = min(p.batch, tid * each), b1 = min(p.batch, b0 + each);
    int64_t mine = 0, total;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += p.hkv * head_tiles<KT>(p, request(p, b, status));
    const int64_t before = scan(mine, s, total);
    per = div_up(total, runs);
    begin = min(total, per * run);
    end = min(total, begin + per);
    if (begin >= end) return;
    if (before <= begin && begin < before + mine) {
        int64_t rest = begin - before;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const Request r = request(p, b, nullptr);
            const int64_t ht = head_tiles<KT>(p, r);
            if (rest >= ht * p.hkv) {
                rest -= ht * p.hkv;
                continue;
            }
            const int h = (int)(div_up(rest + 1, ht) - 1);
            rest -= h * ht;
            int qt = 0;
            if (p.mask || r.len < 0 || r.n == 1) {
                const int t = item_tiles<KT>(p, r, 0) + p.cost;
                qt = (int)(div_up(rest + 1, t) - 1);
                rest -= (int64_t)qt * t;
            }
            s.at = Place{b, h, qt, 0};
            s.rest = rest;
            break;
        }
    }
    __syncthreads();
    at = s.at;
    const Request r = request(p, at.b, nullptr);
    if (p.mask || r.len < 0 || r.n == 1) {
        at.off = (int)s.rest;
        return;
    }
    // a prompt's tiles differ: the threads share its rows
    const int nq = row_tiles(p, r), share = (nq + nt - 1) / nt, q0 = min(nq, tid * share), q1 = min(nq, q0 + share);
    mine = 0;
#pragma unroll 1
    for (int q = q0; q < q1; ++q) mine += item_tiles<KT>(p, r, q) + p.cost;
    int64_t rest = s.rest - scan(mine, s, total);
    if (rest >= 0 && rest < mine) {
        int q = q0;
#pragma unroll 1
        for (int t; rest >= (t = item_tiles<KT>(p, r, q) + p.cost); ++q) rest -= t;
        s.at.qt = q;
        s.at.off = (int)rest;
    }
    __syncthreads();
    at = s.at;
}

// the item after `at`'s
__device__ __forceinline__ void next_item(const Params &p, Place &at, Request &r) {
    at.off = 0;
    if (++at.qt < row_tiles(p, r)) return;
    at.qt = 0;
    if (++at.h < p.hkv) return;
    at.h = 0;
    do {
        if (++at.b >= p.batch) return;
        r = request(p, at.b, nullptr);
    } while (r.n == 0);
}

// What a run with `left` units of work has of the item it is at: tiles first .. last - 1 (none where it ends before them), and
// how many units that takes.
struct Span {
    int tiles, first, last, units;
};
template <int KT>
__device__ __forceinline__ Span span_of(const Params &p, const Request &r, const Place &at, int64_t left) {
    Span s;
    s.tiles = item_tiles<KT>(p, r, at.qt);
    s.first = max(0, at.off - p.cost);
    s.last = (int)min((int64_t)s.tiles, at.off + left - p.cost);
    s.units = p.cost + s.tiles - at.off;
    return s;
}

// The offset of slot s of request b, head h, in the pools; -1 where its page is outside the pool.
__device__ __forceinline__ int64_t slot_offset(const Params &p, int b, int h, int s) {
    const int page = p.page_bits >= 0 ? s >> p.page_bits : s / p.page_size;
    const int row = s - page * p.page_size;
    const int id = p.table[(int64_t)b * p.max_pages + page];
    if (id < 0 || id >= p.n_pages) {
        flag(p.status, GDN_DEV_BAD_PAGE);
        return -1;
    }
    return id * p.page_stride + row * p.slot_stride + h * p.head_stride;
}

// Whether token i of a request sees slot s.
__device__ __forceinline__ bool sees(const Params &p, const Request &r, int i, int s) {
    if (s < r.len) return true;
    const int j = s - r.len;
    if (j >= r.n) return false;
    return p.mask ? (p.mask[(int64_t)(r.first + i) * p.mask_words + (j >> 5)] >> (j & 31)) & 1 : j <= i;
}

// Whether a new token sees any slot (row: its words of the mask, NULL: causal).  Only then is a row whose sum is zero one whose
// scores are all -infinity: their softmax is NaN, where nothing is seen outputs are zeros.
__device__ __forceinline__ bool sees_any(int len, int n, const uint32_t *row) {
    if (len != 0 || !row) return len >= 0;
#pragma unroll 1
    for (int j = 0; j < n; j += 32)
        if (row[j >> 5] & (n - j < 32 ? (1u << (n - j)) - 1 : 0xffffffffu)) return true;
    return false;
}
// the factor of token i's outputs, whose sum is l
__device__ __forceinline__ float inverse(const Params &p, const Request &r, int i, float l) {
    if (l != 0.f) return 1.f / l;
    return sees_any(r.len, r.n, p.mask ? p.mask + (int64_t)(r.first + i) * p.mask_words : nullptr) ? __int_as_float(0x7fc00000) : 0.f;
}

__device__ __forceinline__ float *part_out(const Params &p, int cap, int d, int run, int which) {
    return p.ws + ((int64_t)run * 2 + which) * cap * d;
}
__device__ __forceinline__ float *part_stat(const Params &p, int cap, int d, int runs, int run, int which) {
    return p.ws + (int64_t)runs * 2 * cap * d + ((int64_t)run * 2 + which) * cap * 2;
}

// The same where every item has a run of its own (the first rows of a head, the others, the next head, ..): begin is 0.
template <int KT>
__device__ __forceinline__ void item_of(const Params &p, int run, int tiles_of_rows, int64_t &begin, int64_t &end, Place &at) {
    const int item = run / tiles_of_rows;
    at = Place{item / p.hkv, item % p.hkv, run % tiles_of_rows, 0};
    const Request r = request(p, at.b, at.h == 0 && at.qt == 0 && threadIdx.x == 0 ? p.status : nullptr);
    begin = 0;
    end = at.qt < row_tiles(p, r) ? p.cost + item_tiles<KT>(p, r, at.qt) : 0;
}

// What joins an item that is cut at the start of a run, told by that run's block: rows 0 where there is nothing to join, because
// the run begins with an item, or the item was cut earlier already.
struct Cut {
    int rows, last;    // the item's rows, and the last run that has a part of it
    int row, first, head;  // its first row in the request, the request's first token, the key-value head
    int request;
    int pad[2];
};
__device__ __forceinline__ Cut *cut_of(const Params &p, int cap, int d, int runs, int run) {
    return reinterpret_cast<Cut *>(p.ws + (int64_t)runs * 2 * cap * (d + 2)) + run;
}
template <int KT>
__device__ __forceinline__ void tell_cut(const Params &p, int cap, int d, int runs, int run, int64_t per, int64_t begin, int64_t end, const Place &at) {
    Cut c = {};
    if (begin < end && at.off > p.cost && at.off - p.cost <= per) {
        const Request r = request(p, at.b, nullptr);
        c.rows = min(p.rows, r.n * p.group - at.qt * p.rows);
        c.last = (int)(div_up(begin - at.off + p.cost + item_tiles<KT>(p, r, at.qt), per) - 1);
        c.row = at.qt * p.rows, c.first = r.first, c.head = at.h, c.request = at.b;
    }
    *cut_of(p, cap, d, runs, run) = c;
}
inline int64_t workspace_floats(int cap, int d, int runs) { return (int64_t)runs * (2 * cap * (d + 2) + (int)sizeof(Cut) / 4); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four consecutive entries of row `row` of o (in elements).
__device__ __forceinline__ void store4(const Params &p, int64_t at, float4 x) {
    if (p.out_bf16) {
        __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        uint2 w = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + at) = w;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at) = x;
    }
}

// Joins the parts of the item that is cut first at the start of run blockIdx.x + 1: with the parts' maxima m_c, sums l_c
// and unscaled outputs o_c, o = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c.  What it takes is the latency of its loads: a warp has
// two rows at once; where there are many parts (one long cache has them by the dozen) a block's warps have one row together, and
// every eighth part each.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinRows = 2, kJoinFew = 8;

// V consecutive entries of a lane, N times 128 apart
template <int V, int N>
__device__ __forceinline__ void add_part(const float *x, float f, float (&o)[N][V]) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if constexpr (V == 4) {
            const float4 y = *reinterpret_cast<const float4 *>(x + n * 128);
            o[n][0] = fmaf(f, y.x, o[n][0]), o[n][1] = fmaf(f, y.y, o[n][1]), o[n][2] = fmaf(f, y.z, o[n][2]), o[n][3] = fmaf(f, y.w, o[n][3]);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) o[n][k] = fmaf(f, x[k], o[n][k]);
        }
    }
}
template <int D, int V, int N>
__device__ __forceinline__ void put_row(const Params &p, const Cut &cut, int row, int lane, float l, const float (&o)[N][V]) {
    const int q = cut.row + row;
    const float inv = l != 0.f ? 1.f / l : inverse(p, request(p, cut.request, nullptr), q / p.group, l);
    const int token = cut.first + q / p.group, head = cut.head * p.group + q % p.group;
    const int64_t to = ((int64_t)token * p.hkv * p.group + head) * D + lane * V;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if constexpr (V == 4) {
            store4(p, to + n * 128, make_float4(o[n][0] * inv, o[n][1] * inv, o[n][2] * inv, o[n][3] * inv));
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (p.out_bf16) store_f(static_cast<__nv_bfloat16 *>(p.o), to + k, o[n][k] * inv);
                else store_f(static_cast<float *>(p.o), to + k, o[n][k] * inv);
            }
        }
    }
}

template <int D, int CAP>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(Params p, int runs) {
    after_previous();
    constexpr int V = D >= 128 ? 4 : D / 32 ? D / 32 : 1, N = D > 128 ? D / 128 : 1;
    __shared__ float sums[kJoinWarps][D];
    const int run = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cut cut = *cut_of(p, CAP, D, runs, run);
    const int parts = cut.last - run + 2;
    const float *stat = part_stat(p, CAP, D, runs, run, 0) - 2 * CAP * 2, *out = part_out(p, CAP, D, run, 0) - 2 * CAP * D + lane * V;
    // part 0 is the second of the run before, the others the first of theirs
    auto which = [&](int c) { return (int64_t)(c * 2 + (c == 0)) * CAP; };
    const bool mine = lane * V < D;
    if (parts <= kJoinFew) {
#pragma unroll 1
        for (int row = (blockIdx.y * kJoinWarps + warp) * kJoinRows; row < cut.rows; row += gridDim.y * kJoinWarps * kJoinRows) {
            float m[kJoinRows], l[kJoinRows] = {}, o[kJoinRows][N][V] = {};
            float2 st[kJoinFew][kJoinRows];
#pragma unroll
            for (int c = 0; c < kJoinFew; ++c)
#pragma unroll
                for (int i = 0; i < kJoinRows; ++i)
                    st[c][i] = c < parts && row + i < cut.rows ? *reinterpret_cast<const float2 *>(stat + (which(c) + row + i) * 2) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < kJoinRows; ++i) {
                m[i] = -INFINITY;
#pragma unroll
                for (int c = 0; c < kJoinFew; ++c) m[i] = fmaxf(m[i], st[c][i].x);
                if (m[i] == -INFINITY) m[i] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < kJoinFew; ++c) {
                if (c < parts) {
#pragma unroll
                    for (int i = 0; i < kJoinRows; ++i) {
                        const float f = exp2_fast(st[c][i].x - m[i]);
                        l[i] = fmaf(f, st[c][i].y, l[i]);
                        if (mine && row + i < cut.rows) add_part<V, N>(out + (which(c) + row + i) * D, f, o[i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kJoinRows; ++i)
                if (mine && row + i < cut.rows) put_row<D, V, N>(p, cut, row + i, lane, l[i], o[i]);
        }
        return;
    }
#pragma unroll 1
    for (int row = blockIdx.y; row < cut.rows; row += gridDim.y) {
        float m = -INFINITY, l = 0.f, o[N][V] = {};
        for (int c = lane; c < parts; c += 32) m = fmaxf(m, stat[(which(c) + row) * 2]);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
        if (m == -INFINITY) m = 0.f;
        for (int c = lane; c < parts; c += 32) {
            const float2 st = *reinterpret_cast<const float2 *>(stat + (which(c) + row) * 2);
            l = fmaf(exp2_fast(st.x - m), st.y, l);
        }
        l = warp_sum(l);
        if (mine) {
#pragma unroll 8
            for (int c = warp; c < parts; c += kJoinWarps) add_part<V, N>(out + (which(c) + row) * D, exp2_fast(stat[(which(c) + row) * 2] - m), o);
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int k = 0; k < V; ++k) sums[warp][n * 128 + lane * V + k] = o[n][k];
        }
        __syncthreads();
        if (warp == 0 && mine) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int col = n * 128 + lane * V + k;
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kJoinWarps; ++w) sum += sums[w][col];
                    o[n][k] = sum;
                }
            put_row<D, V, N>(p, cut, row, lane, l, o);
        }
        __syncthreads();
    }
}

// A launch that may take its place while the kernel before it ends; the kernel calls after_previous() first.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int CAP>
cudaError_t launch_join(const Params &p, int runs, cudaStream_t stream) {
    if (runs < 2) return cudaSuccess;
    return launch_dependent(join_kernel<D, CAP>, dim3(runs - 1, p.rows < 16 ? p.rows : 16), kJoinThreads, 0, stream, p, runs);
}

// A kernel of this family for some sizes: how many blocks, their workspace, and the launch.
struct Choice {
    int runs;
    int64_t workspace;
    cudaError_t (*launch)(Params p, int runs, cudaStream_t stream);
    bool whole;
};

// blocks_an_sm runs for each SM, and no more than there can be tiles
inline int most_runs(const gdn_kv_attend_args &a, bool decode, int R, int KT, int blocks_an_sm) {
    const int64_t room = (int64_t)blocks_an_sm * sm_count();
    const int64_t group = a.n_q_heads / a.cache.n_kv_heads, slots = (int64_t)a.cache.max_pages * a.cache.page_size;
    const int64_t factors[4] = {a.cache.batch, a.cache.n_kv_heads, ((decode ? 1 : (int64_t)a.max_tokens) * group + R - 1) / R, (slots + KT - 1) / KT};
    int64_t n = 1;
    for (int64_t f : factors) {
        n *= f < 1 ? 1 : f < room ? f : room;
        if (n > room) n = room;
    }
    return (int)n;
}

// Whether each item gets a block of its own, and how many there are: where no request can have more than `most` tiles of slots, and
// a call's items fit into a few waves.  (Sizes are looked at, not lengths, which the host does not know.)
inline bool whole_items(const gdn_kv_attend_args &a, bool decode, int R, int KT, int most, int &items) {
    const int64_t group = a.n_q_heads / a.cache.n_kv_heads, slots = (int64_t)a.cache.max_pages * a.cache.page_size;
    const int64_t n = (int64_t)a.cache.batch * a.cache.n_kv_heads * (((decode ? 1 : (int64_t)a.max_tokens) * group + R - 1) / R);
    items = (int)(n < 1 << 30 ? n : 1 << 30);
    return slots <= (int64_t)most * KT && n <= 1 << 20;
}

// whether every row of the queries and of the cache starts on 16 bytes
inline bool aligned16(const gdn_kv_attend_args &a) {
    const gdn_kv_cache &c = a.cache;
    const int e = c.dtype == GDN_BF16 ? 2 : 4;
    const int64_t qs = a.q_stride ? a.q_stride : (int64_t)a.n_q_heads * c.d;
    return ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) & 15) == 0 &&
           (qs | c.page_stride | c.slot_stride | c.head_stride) * e % 16 == 0;
}

}  // namespace attn

// kernels for the sizes of a call (the general one always; d is one of the supported widths)
attn::Choice attend_simt_choice(const gdn_kv_attend_args &a, bool decode);
// few rows a key-value head: bf16, rows on 16 bytes
bool attend_mma_supported(const gdn_kv_attend_args &a);
attn::Choice attend_mma_choice(const gdn_kv_attend_args &a, bool decode);
// many rows: bf16, d from 64 on, pages of whole groups of 8 slots, a positive scale
bool attend_tc_supported(const gdn_kv_attend_args &a);
attn::Choice attend_tc_choice(const gdn_kv_attend_args &a);

}  // namespace gdn
