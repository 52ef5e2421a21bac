// attend_mma.cu -- attention over a paged cache for few rows a key-value head (single tokens, small drafts), bf16.
//
// 16 rows share what is read of the cache, so that its bytes bound it: 4 d bytes a slot and head, 44 bytes a ns and SM.
// A block has four warps; of a tile of 64 slots each takes 16, through a ring of its own in shared memory (cp.async, 16-byte
// pieces, swizzled for ldmatrix), and keeps its own running maximum, sum and outputs, so that nothing in the loop waits
// for another warp.  The products are m16n8k16 warp products: with 16 rows a tcgen05 tile of 128 would be seven eighths
// empty, and what they cost here is a tenth of the time the bytes take.  The ring runs ahead over the ends of items,
// with the page of the tile after the next looked up one tile earlier.  At an item's end the warps' parts are joined in
// shared memory.
// 128 single tokens over 10 to 6000 slots, 32 heads of 128 to 8: 237 us for 1.47 GB, 6.2 TB/s; one over 131072, 4 heads: 55 us for
// 268 MB, of which 40 are the bytes, the rest the start (finding the work, the first loads) and the join.  Heads of 256 have one block
// an SM and a ring of two tiles: 64 tokens over 100 to 8000 slots, 16 heads to 2, 114 us, 4.7 TB/s.
// Probabilities are two bf16 numbers for their product with the values, the second what rounding leaves of the first (2^-16 of each
// together): outputs lose no more than their own rounding.  With one (2^-8), widths to 128 take as long within 2 %, 64 tokens over 100
// to 8000 slots, 16 heads of 256 to 2, 109 us where this takes 114.
// A new token's value that is not finite is replaced by zeros and makes the sums of the rows that see it NaN: a
// probability of zero times it would reach the others.
#include "attn.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace attn;
using sm100::smem_u32;

// kMostWhole: a request's tiles up to which its items are not cut (700 slots, 8 heads: 16 us so, 26 cut and joined, of which the second
// launch is the most).  kCost: what an item costs besides its tiles (128 tokens over 10 to 6000 slots with 1, 2, 3, 4: 241, 229, 230, 231 us).
constexpr int kR = 16, kWarps = 4, kThreads = kWarps * 32, kKeys = 16, kKT = kWarps * kKeys, kMostWhole = 16, kCost = 2;

template <int D>
struct Ring {
    static constexpr int kRow = D * 2, kTile = kKeys * kRow;    // bytes of a slot's keys, of a warp's 16 slots
    static constexpr int kStages = D == 256 ? 2 : D == 128 ? 3 : D == 64 ? 6 : 8;
    static constexpr int kWarp = kStages * 2 * kTile;
    static constexpr int kJoin = kR * D * 4;                    // a warp's outputs, where it joins the others
    static constexpr int kQ = D == 256 ? kR * kRow : 0;         // queries that do not fit into registers
    static constexpr int kBytes = kWarps * kWarp + 2 * kJoin + kQ;
    static constexpr int kBlocks = kBytes > 113 * 1024 ? 1 : 2; // an SM
};

// byte offset of 16-byte piece c of row `row` in a tile: eight rows of one column of pieces lie in different banks
template <int D>
__device__ __forceinline__ uint32_t piece(int row, int c) {
    constexpr int C = D / 8;
    return row * (D * 2) + ((C >= 8 ? c ^ (row & 7) : c ^ ((row / (8 / C)) & (C - 1))) << 4);
}

__device__ __forceinline__ void ldmatrix4(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int D>
__global__ void __launch_bounds__(kThreads) attend_mma_kernel(Params p, int runs) {
    after_previous();
    using S = Ring<D>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ Scratch scratch;
    __shared__ float stat[kWarps][kR][2];
    constexpr int C = D / 8, kN = D / 8;  // 16-byte pieces of a row; output tiles of 8 columns
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, run = blockIdx.x;
    const int g = lane >> 2, t4 = lane & 3;
    int64_t per, t, end;
    Place at;
    if (p.whole) {
        item_of<kKT>(p, run, (p.max_tokens * p.group + kR - 1) / kR, t, end, at);
    } else {
        find<kKT>(p, runs, run, run == 0 ? p.status : nullptr, scratch, per, t, end, at);
        if (tid == 0) tell_cut<kKT>(p, kR, D, runs, run, per, t, end, at);
    }
    if (t >= end) return;
    uint8_t *ring = sm + warp * S::kWarp;
    float *mine = reinterpret_cast<float *>(sm + kWarps * S::kWarp + (warp & 1) * S::kJoin);
    const uint32_t ring_at = smem_u32(ring);
    const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(p.k), *V = static_cast<const __nv_bfloat16 *>(p.v);

    // ---- the ring: tiles from `l_tile` on are on their way, and where the next one lies is known
    Place load = at;
    Request lr = request(p, load.b, nullptr);
    int64_t l_left = end - t, l_off = -1;
    Span ls = span_of<kKT>(p, lr, load, l_left);
    int l_seen = seen_slots(p, lr, load.qt), l_tile = ls.first, l_ids = 0, l_ids_at = ls.first - 32;
    bool l_more = ls.first < ls.last;
    const bool aligned_pages = p.page_size % kKeys == 0;  // a warp's 16 slots lie in one page: lanes look up 32 tiles' at once
    auto look_up = [&]() {
        if (aligned_pages) {
            if (l_tile - l_ids_at >= 32) {
                l_ids_at = l_tile;
                const int slot = (l_tile + lane) * kKT + warp * kKeys;
                l_ids = l_tile + lane < ls.last && slot < l_seen ? p.table[(int64_t)load.b * p.max_pages + (p.page_bits >= 0 ? slot >> p.page_bits : slot / p.page_size)] : 0;
            }
        } else {
            const int slot = l_tile * kKT + warp * kKeys + (lane & 15);
            l_off = slot < l_seen ? slot_offset(p, load.b, load.h, slot) : -1;
        }
    };
    auto issue = [&](int stage) {
        if (l_more) {
            const int slot0 = l_tile * kKT + warp * kKeys;
            int there = l_seen - slot0;  // slots of these 16 that are seen
            const uint32_t to = ring_at + stage * 2 * S::kTile;
            int64_t base = 0;
            if (aligned_pages) {
                const int id = __shfl_sync(0xffffffffu, l_ids, l_tile - l_ids_at);
                base = id * p.page_stride + (p.page_bits >= 0 ? slot0 & (p.page_size - 1) : slot0 % p.page_size) * p.slot_stride + load.h * p.head_stride;
                if (there > 0 && (id < 0 || id >= p.n_pages)) {
                    there = 0;
                    if (lane == 0) flag(p.status, GDN_DEV_BAD_PAGE);
                }
            }
#pragma unroll
            for (int i = 0; i < (kKeys * C + 31) / 32; ++i) {
                const int n = i * 32 + lane, row = n / C, c = n % C;
                int64_t from = base + row * p.slot_stride;
                bool ok = row < there;
                if (!aligned_pages) {
                    from = __shfl_sync(0xffffffffu, l_off, row & 15);
                    ok = ok && from >= 0;
                }
                from = ok ? from + c * 8 : 0;
                copy16(to + piece<D>(row, c), K + from, ok);
                copy16(to + S::kTile + piece<D>(row, c), V + from, ok);
            }
            if (++l_tile == ls.last) {
                l_left -= ls.units;
                l_more = l_left > 0;
                if (l_more) {
                    next_item(p, load, lr);
                    ls = span_of<kKT>(p, lr, load, l_left);
                    l_seen = seen_slots(p, lr, load.qt);
                    l_tile = ls.first, l_ids_at = ls.first - 32;
                    l_more = ls.first < ls.last;
                }
            }
            if (l_more) look_up();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (!l_more) return;
    look_up();
#pragma unroll 1
    for (int s = 0; s < S::kStages - 1; ++s) issue(s);

    Request r = request(p, at.b, nullptr);
    int stage = 0, free_stage = S::kStages - 1;
    while (t < end) {
        const Span span = span_of<kKT>(p, r, at, end - t);
        const int tiles = span.tiles, first = span.first, last = span.last, seen = seen_slots(p, r, at.qt), common = common_slots(p, r, at.qt);
        if (last <= first) break;
        const int row0 = at.qt * kR, rows = r.n * p.group;
        // ---- this lane's rows: g and g + 8
        const __nv_bfloat16 *q[2];
        int token[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = row0 + g + 8 * i;
            token[i] = n / p.group;
            q[i] = n < rows ? static_cast<const __nv_bfloat16 *>(p.q) + (int64_t)(r.first + token[i]) * p.q_stride + (at.h * p.group + n % p.group) * D
                            : nullptr;
            if (n >= rows) token[i] = -1;
        }
        uint32_t qf[D == 256 ? 1 : D / 16][4];
        const uint32_t q_at = smem_u32(sm + kWarps * S::kWarp + 2 * S::kJoin);
        if constexpr (D == 256) {
            for (int i = tid; i < kR * C; i += kThreads) {
                const int row = i / C, c = i % C, n = row0 + row;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (n < rows)
                    x = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + (int64_t)(r.first + n / p.group) * p.q_stride +
                                                         (at.h * p.group + n % p.group) * D + c * 8);
                *reinterpret_cast<uint4 *>(sm + kWarps * S::kWarp + 2 * S::kJoin + piece<D>(row, c)) = x;
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qf[ks][i] = q[i & 1] ? *reinterpret_cast<const uint32_t *>(q[i & 1] + ks * 16 + (i >> 1) * 8 + t4 * 2) : 0u;
        }
        float o[kN][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 1
        for (int tile = first; tile < last; ++tile) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
            __syncwarp();
            issue(free_stage);
            free_stage = stage;
            const uint32_t kt = ring_at + stage * 2 * S::kTile, vt = kt + S::kTile;
            uint8_t *v_rows = ring + stage * 2 * S::kTile + S::kTile;
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
            // ---- scores of 16 slots
            float s[2][4] = {};
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b[4], a[4];
                // matrices: slots 0-7 and 8-15, each with the lower and the upper 8 of 16 entries
                ldmatrix4(kt + piece<D>((lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)), b);
                if constexpr (D == 256) ldmatrix4(q_at + piece<D>((lane & 7) + (((lane >> 3) & 1) << 3), ks * 2 + (lane >> 4)), a);
                else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = qf[ks][i];
                }
                mma(s[0], a, b[0], b[1]);
                mma(s[1], a, b[2], b[3]);
            }
            const int slot0 = tile * kKT + warp * kKeys;
            bool poisoned[2] = {false, false};
            if (slot0 + kKeys > common) {
                uint32_t spoilt = 0;  // new tokens' values that are not finite
                if ((r.n > 1 || p.mask) && slot0 < seen) {  // (a single token sees itself, unless a mask leaves it out)
                    const int row = lane & 15;
                    bool finite = true;
                    for (int c = lane >> 4; c < C; c += 2) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(v_rows + piece<D>(row, c));
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) finite = finite && (w[i] & 0x7F80u) != 0x7F80u && (w[i] & 0x7F800000u) != 0x7F800000u;
                    }
                    spoilt = __ballot_sync(0xffffffffu, !finite && slot0 + row >= r.len);
                    spoilt = (spoilt | spoilt >> 16) & 0xFFFFu;
                    if (spoilt >> row & 1)
                        for (int c = lane >> 4; c < C; c += 2) *reinterpret_cast<uint4 *>(v_rows + piece<D>(row, c)) = make_uint4(0, 0, 0, 0);
                    __syncwarp();
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = n * 8 + t4 * 2 + (i & 1), slot = slot0 + key, tk = token[i >> 1];
                        const bool see = slot < seen && tk >= 0 && sees(p, r, tk, slot);
                        s[n][i] = see ? s[n][i] * p.scale_log2 : -INFINITY;
                        poisoned[i >> 1] = poisoned[i >> 1] || (see && (spoilt >> key & 1));
                    }
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[n][i] *= p.scale_log2;
            }
            // ---- running maximum and sum (this lane's part of it)
            uint32_t a[4], rest[4];
            float f[2];
            bool moved = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                x = fmaxf(x, m[i]);
                const float base = x == -INFINITY ? 0.f : x;
                f[i] = exp2_fast(m[i] - base);
                moved = moved || x != m[i];
                m[i] = x;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    s[n][2 * i] = exp2_fast(s[n][2 * i] - base);
                    s[n][2 * i + 1] = exp2_fast(s[n][2 * i + 1] - base);
                }
                l[i] = fmaf(l[i], f[i], (s[0][2 * i] + s[0][2 * i + 1]) + (s[1][2 * i] + s[1][2 * i + 1]));
                if (poisoned[i]) l[i] = __int_as_float(0x7fc00000);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w = a[2 * n + i] = pack(s[n][2 * i], s[n][2 * i + 1]);
                    rest[2 * n + i] = pack(s[n][2 * i] - __uint_as_float(w << 16), s[n][2 * i + 1] - __uint_as_float(w & 0xffff0000u));
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < kN; ++n) o[n][0] *= f[0], o[n][1] *= f[0], o[n][2] *= f[1], o[n][3] *= f[1];
            }
            // ---- outputs
#pragma unroll
            for (int n = 0; n < kN; n += 2) {
                uint32_t b[4];
                ldmatrix4_t(vt + piece<D>(lane & 15, n + (lane >> 4)), b);
                mma(o[n], a, b[0], b[1]);
                mma(o[n + 1], a, b[2], b[3]);
                mma(o[n], rest, b[0], b[1]);
                mma(o[n + 1], rest, b[2], b[3]);
            }
            __syncwarp();  // the tile may be overwritten
        }
        // ---- the four warps' parts: the third and fourth to the first and second, those to the block
        auto place = [&](int i, int n) { return reinterpret_cast<float2 *>(mine + (g + 8 * i) * D + ((n * 8 + t4 * 2) ^ ((g & 3) << 3) % D)); };
        auto put = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (t4 == 0) stat[warp][g + 8 * i][0] = m[i], stat[warp][g + 8 * i][1] = l[i];
#pragma unroll
                for (int n = 0; n < kN; ++n) *place(i, n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
            }
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        if (warp >= 2) put();
        __syncthreads();
        if (warp < 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float other = stat[warp + 2][g + 8 * i][0], x = fmaxf(m[i], other), base = x == -INFINITY ? 0.f : x;
                const float e = exp2_fast(m[i] - base), f = exp2_fast(other - base);
                m[i] = x;
                l[i] = fmaf(e, l[i], f * stat[warp + 2][g + 8 * i][1]);
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const float2 y = *place(i, n);
                    o[n][2 * i] = fmaf(e, o[n][2 * i], f * y.x), o[n][2 * i + 1] = fmaf(e, o[n][2 * i + 1], f * y.y);
                }
            }
            put();
        }
        __syncthreads();
        const bool whole = first == 0 && last == tiles;
        const int which = first == 0;
        const float *parts = reinterpret_cast<const float *>(sm + kWarps * S::kWarp);
        for (int i = tid; i < kR * (D / 4); i += kThreads) {
            const int row = i / (D / 4), col = i % (D / 4) * 4, n = row0 + row;
            if (n >= rows) continue;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int w = 0; w < 2; ++w) mm = fmaxf(mm, stat[w][row][0]);
            const float base = mm == -INFINITY ? 0.f : mm;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const float e = exp2_fast(stat[w][row][0] - base);
                const float4 x = *reinterpret_cast<const float4 *>(parts + w * (S::kJoin / 4) + row * D + (col ^ ((row & 3) << 3) % D));
                ll = fmaf(e, stat[w][row][1], ll);
                y.x = fmaf(e, x.x, y.x), y.y = fmaf(e, x.y, y.y), y.z = fmaf(e, x.z, y.z), y.w = fmaf(e, x.w, y.w);
            }
            if (whole) {
                const float inv = inverse(p, r, n / p.group, ll);
                const int64_t to = ((int64_t)(r.first + n / p.group) * p.hkv * p.group + at.h * p.group + n % p.group) * D + col;
                store4(p, to, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
            } else {
                *reinterpret_cast<float4 *>(part_out(p, kR, D, run, which) + row * D + col) = y;
                if (col == 0) *reinterpret_cast<float2 *>(part_stat(p, kR, D, runs, run, which) + row * 2) = make_float2(mm, ll);
            }
        }
        __syncthreads();
        t += span.units;
        if (t < end) next_item(p, at, r);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D>
cudaError_t run(Params p, int runs, cudaStream_t stream) {
    static int have[16];
    p.rows = kR, p.cost = kCost;
    const cudaError_t e = ensure_smem(attend_mma_kernel<D>, Ring<D>::kBytes, have);
    if (e != cudaSuccess) return e;
    const cudaError_t f = launch_dependent(attend_mma_kernel<D>, dim3(runs), kThreads, Ring<D>::kBytes, stream, p, runs);
    return f != cudaSuccess || p.whole ? f : launch_join<D, kR>(p, runs, stream);
}

template <int D>
Choice choice(const gdn_kv_attend_args &a, bool decode) {
    Choice x = {0, 0, run<D>, false};
    x.whole = whole_items(a, decode, kR, kKT, kMostWhole, x.runs);
    if (!x.whole) x.runs = most_runs(a, decode, kR, kKT, Ring<D>::kBlocks);
    return x;
}

}  // namespace

bool attend_mma_supported(const gdn_kv_attend_args &a) { return a.cache.dtype == GDN_BF16 && attn::aligned16(a); }

attn::Choice attend_mma_choice(const gdn_kv_attend_args &a, bool decode) {
    Choice x;
    switch (a.cache.d) {
        case 16: x = choice<16>(a, decode); break;
        case 32: x = choice<32>(a, decode); break;
        case 64: x = choice<64>(a, decode); break;
        case 128: x = choice<128>(a, decode); break;
        default: x = choice<256>(a, decode);
    }
    x.workspace = x.whole ? 0 : 4 * workspace_floats(kR, a.cache.d, x.runs);
    return x;
}

}  // namespace gdn
