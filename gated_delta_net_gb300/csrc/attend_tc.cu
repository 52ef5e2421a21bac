// attend_tc.cu -- attention over a paged cache on the tensor cores: bf16, d = 64, 128 or 256 (sm_103a).
//
// For draft trees and prompts the two products bound it: 4 d operations a row and slot.  A block (one an SM) has an item of two
// tiles of up to 128 rows (whole tokens: 128 / group of them, their query heads side by side; one tile for
// d = 256), whose queries stay in shared memory, and takes its part of the cache in tiles of 128 slots (64 for d = 256):
//     S = Q K^T      tcgen05, both from shared memory, to tensor memory
//     P = 2^(S scale - m)   scores from tensor memory, probabilities as bf16 back over them
//     O += P V       tcgen05, P from tensor memory, V as it lies in shared memory (MN-major)
// While one tile's scores are in registers, the other tile's products run.  Where there is one tile of rows (they fit into it,
// or d = 256, whose outputs take half of the tensor memory), its scores are a tile of slots ahead in a second buffer.
//
// The maximum that outputs are scaled by is moved, and they are multiplied, only where a row's maximum grew by more than 2^8: then
// probabilities are up to 2^8, which neither bf16 nor the fp32 sums lose anything by.
// P is rounded to bf16 (2^-8 of each) as the operand beside V; their sum is kept of the unrounded ones.  As two bf16 numbers
// (2^-16) it takes a third longer: the prompt below 635 us, the trees 250.
//
// 12 warps (8 for one tile of rows):
//     4 for each tile of rows, a thread a row.  The first half of a tile's probabilities is multiplied while the second is made.
//       (Two threads a row, which swap their maxima, are slower: 744 us against 684 for 8192 tokens, 32 heads of 128.)
//     1 issues the products
//     1 loads: keys and values with a TMA box for each page's rows, 128-byte swizzled (pages behind the last seen
//       slot, or outside the pool, are read past the pool's end, as zeros), queries (64 entries of the group's
//       heads of 128 / group tokens); and walks the items, which the other roles learn from it
//     1 sends outputs
//     1 looks at values before they are multiplied: rows behind the last seen slot become zeros (their
//       probability is zero, but they may be anything), and so do new tokens' that are not finite, whose
//       readers' sums become NaN instead
// Every wait is bounded; one that runs out sets GDN_DEV_TIMEOUT.
//
// One prompt of 8192 tokens behind 777, 32 heads of 128 to 8: 450 us, 1454 TFLOP/s; 64 trees of 128 nodes behind 200 to 2200 slots:
// 185 us.  A tile of 128 slots takes two tiles of rows about 2450 cycles, of which their products need 2048, at which shared memory is
// busy as well (operands 192 KB, loads 64 KB, at 128 bytes a cycle); an item's end and beginning take 7000, and an item's
// masked tiles 1000 more each.  The first product of a block starts 10 us after its launch.  Heads of 256: a tile of 64 slots has 1024
// cycles of products and 1536 of shared memory, and the prompt with 16 heads to 2 takes 610 us, 1073 TFLOP/s.
#include "attn.cuh"
#include "sm100.cuh"
#include "tc_tiles.cuh"

namespace gdn {
namespace {

using namespace attn;
using namespace sm100;
using tiles::pack_bf16;

constexpr int kTileRows = 128;
constexpr float kGrow = 8.f;  // log2 of what a probability may grow to before the maximum moves

// stands for the length of a row that is not in use: slots lie 2^30 tokens behind it, where neither causally (a request has at most
// 2^30) nor by the mask (2^25) a token sees them
constexpr int kNotInUse = -(1 << 30);

// An item, or the part of it that is this block's, as the other roles see it: with all that they need at its end, for reading
// the kernel's parameters there, out of a cache that nobody else keeps them in, takes over a thousand cycles.
struct __align__(16) Job {
    int n;              // tiles; 0: no more
    int tile;           // the first one
    int seen, common;
    int len, tokens;    // the request's
    int token;          // the item's first one
    int mask_words;
    const uint32_t *mask;  // the request's rows, or NULL: causal
    uint8_t *to;        // where the item's first row goes
    float2 *stat;       // a part's maxima and sums; NULL: the item is whole
    int64_t token_pitch;  // bytes between outputs
    int head_pitch;
    int first, head;    // the request's first row; key-value head
    int bf16;           // outputs are
    int boxes;          // tiles of rows that go out as TMA boxes
};
constexpr int kJobs = 3;  // an item is told while the one before it begins and the one before that may be read

// U: tiles of rows
template <int D, int U>
struct Shape {
    static constexpr int kRowWarps = U * 4, kThreads = kRowWarps * 32 + 128;
    static constexpr int NB = U == 1 ? 2 : 1;       // buffers of scores for each
    static constexpr int KT = D == 256 ? 64 : 128;    // slots of a tile
    static constexpr int H = D / 64;                  // halves (64 entries, 128 bytes) of a row
    static constexpr int kQTile = kTileRows * 128;    // bytes of one half of a tile of queries
    static constexpr int kHalf = KT * 128;            // of one half of a tile of keys or values
    static constexpr int kStage = H * kHalf;
    static constexpr int kQ = U * H * kQTile;
    static constexpr int KS = D == 64 ? 5 : D == 128 && U == 1 ? 3 : 2, VS = D == 64 ? 5 : 2;  // tiles of keys, of values held at a time
    static constexpr int CAP = U * kTileRows;
    static constexpr uint32_t kScores = 0, kOut = U * NB * KT;  // tensor-memory columns
    // words of a tile's rows that were not finite.  They are read after the tile's probabilities have been handed over, so there is
    // room for twice the tiles: those of tile c + 2 VS are written when tile c + VS has been multiplied
    static constexpr int kSpoilt = KT / 32;
    // barriers
    static constexpr int KFULL = 0, KEMPTY = KFULL + KS, VFULL = KEMPTY + KS, VEMPTY = VFULL + VS, READY = VEMPTY + VS, SCORES = READY + VS,
                         PROBS = SCORES + U * NB, DONE = PROBS + U * NB * 2, FREE = DONE + U, QFULL = FREE + U, QEMPTY = QFULL + 1, JFULL = QEMPTY + 1, JEMPTY = JFULL + kJobs, OUT = JEMPTY + kJobs, TAKEN = OUT + U, DRAIN = TAKEN + U, PROBE = DRAIN + 1, COUNT = PROBE + 1;
    static constexpr int OFF_K = kQ, OFF_V = OFF_K + KS * kStage, OFF_OUT = OFF_V + VS * kStage, OFF_SPOILT = OFF_OUT + kRowWarps * 4096, OFF_JOB = (OFF_SPOILT + 2 * VS * kSpoilt * 4 + 15) / 16 * 16,
                         OFF_SCRATCH = OFF_JOB + kJobs * (int)sizeof(Job), OFF_BAR = OFF_SCRATCH + (int)sizeof(Scratch);
    static constexpr int kBytes = OFF_BAR + COUNT * 8 + 8;
    static_assert(kOut + U * D <= 512, "tensor memory");
    static_assert(kBytes <= 232448, "shared memory");
};

struct TcParams {
    Params p;
    int tile_tokens;  // tokens of a tile of rows
    int box;          // slots of a TMA box
    int probe;        // polls of a wait that runs out, for tests (0: none)
};

// after a wait that ran out the others look once
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, bool &ok) {
    if (!mbar_wait(bar, parity, ok ? 1u << 20 : 1u)) ok = false;
    return ok;
}
// the same by a whole warp, which goes on or gives up together
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, bool &ok) {
    wait(bar, parity, ok);
    return ok = __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Products are issued by a whole converged warp, of which the elected lane (lead) issues.  Low word of a descriptor: start
// address and, for MN-major operands, the distance between halves; the rest is the same for all 128-byte-swizzled tiles.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t at, int lbo_bytes) { return ((at >> 4) & 0x3FFFu) | ((uint32_t)(lbo_bytes >> 4) << 16); }
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead), "r"(kDescHi) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "mov.b64 db, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead), "r"(kDescHi) : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t *bar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 ::"r"(smem_u32(bar)), "r"(lead) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(uint32_t a, uint32_t b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 parts(f2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// What a row with maximum m multiplies its scores by.  m times sc is rounded, past 2^30 by so much that the largest score's power may
// not be finite.  There fp32 scores that differ at all have weights 2^64 or more apart, 2^32 or more with the power of two below sc,
// whose product is exact: the largest has all the weight either way.  (Subtracting the maximum before the product, in a
// branch that such rows take, cost others 1 to 3 %; this 0 at d = 128, 1 to 2 % at 64 and 256.)
__device__ __forceinline__ float scale_of(float m, float sc) {
    return fabsf(m * sc) > 1073741824.f ? __uint_as_float(max(__float_as_uint(sc) & 0x7F800000u, 0x00800000u)) : sc;
}

// Bits 0..31: whether token i of the request sees slots from .. from + 31.
__device__ __forceinline__ uint32_t seen_word(const Job &w, int i, int from) {
    const int j = from - w.len;  // the first one's number among the new tokens
    auto below = [](int n) { return n <= 0 ? 0u : n < 32 ? (1u << n) - 1 : 0xffffffffu; };
    if (!w.mask) return below(i - j + 1);
    const uint32_t *row = w.mask + (int64_t)i * w.mask_words;
    const int at = j >> 5;
    const uint32_t lo = at >= 0 && at < w.mask_words ? row[at] : 0u, hi = at >= -1 && at + 1 < w.mask_words ? row[at + 1] : 0u;
    return (__funnelshift_r(lo, hi, j & 31) & below(w.tokens - j)) | below(-j);  // committed slots
}

// The walk over a run's items, alike in every role.
struct Walk {
    Place at;
    Request r;
    int64_t left;
    int first, last, tiles, units, seen, common;
    template <int KT>
    __device__ __forceinline__ void item(const Params &p) {
        const Span s = span_of<KT>(p, r, at, left);
        tiles = s.tiles, first = s.first, last = s.last, units = s.units;
        seen = seen_slots(p, r, at.qt);
        common = common_slots(p, r, at.qt);
    }
    template <int KT>
    __device__ __forceinline__ bool next(const Params &p) {
        left -= units;
        if (left <= 0) return false;
        next_item(p, at, r);
        item<KT>(p);
        return first < last;
    }
};

template <int D, int U>
__global__ void __launch_bounds__(Shape<D, U>::kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap o_map, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                     const __grid_constant__ TcParams tp, int runs) {
    after_previous();
    using S = Shape<D, U>;
    constexpr int KT = S::KT, NB = S::NB;
    extern __shared__ __align__(1024) uint8_t sm[];
    const Params &p = tp.p;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + S::OFF_BAR);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + S::OFF_BAR + S::COUNT * 8);
    Scratch &scratch = *reinterpret_cast<Scratch *>(sm + S::OFF_SCRATCH);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, run = blockIdx.x;
    int64_t per, begin, end;
    Place start;
    find<KT>(p, runs, run, run == 0 ? p.status : nullptr, scratch, per, begin, end, start);
    if (tid == 0) tell_cut<KT>(p, S::CAP, D, runs, run, per, begin, end, start);
    if (begin >= end) return;
    if (smem_u32(sm) & 1023) {  // what the swizzled tiles need
        flag(p.status, GDN_DEV_INTERNAL);
        return;
    }
    if (warp == S::kRowWarps) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < S::COUNT; ++i) {
            const bool rows = (i >= S::PROBS && i < S::DONE) || (i >= S::FREE && i < S::QFULL) || (i >= S::OUT && i < S::TAKEN);
            mbar_init(bar + i, rows ? kTileRows : i >= S::JEMPTY && i < S::OUT ? S::kRowWarps + 3 : 1);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = uniform(*slot);
    const uint32_t base = smem_u32(sm);
    bool ok = true;
    int item = 0;
    // the next item, or NULL after the last one; and the end of reading it
    auto take = [&]() -> const Job * {
        const int i = item % kJobs;
        if (!warp_wait(&bar[S::JFULL + i], (item / kJobs) & 1, ok)) return nullptr;
        ++item;
        const Job *w = reinterpret_cast<const Job *>(sm + S::OFF_JOB) + i;
        return w->n > 0 ? w : nullptr;
    };
    auto drop = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[S::JEMPTY + (item - 1) % kJobs]);
    };

    if (warp < S::kRowWarps) {
        // ------------------------------------------------------------------ a row
        const int u = warp >> 2, x = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t o_at = tm + S::kOut + u * D + lanes;
        const int own_token = u * tp.tile_tokens + x / p.group, own_head = x % p.group;
        const int own_row = own_token * p.group + own_head;
        const bool own = x < tp.tile_tokens * p.group;
        const float sc = p.scale_log2, grow = kGrow / sc;
        int c = 0, rounds = 0;
        while (const Job *wp = take()) {
            const Job &w = *wp;
            const int token = w.token + own_token;
            const bool live = own && token < w.tokens;
            float m = -INFINITY;
            f2 l2 = pair(0u, 0u);
#pragma unroll 1
            for (int j = 0; j < w.n; ++j, ++c) {
                const int buf = u * NB + c % NB;
                const uint32_t s_at = tm + S::kScores + buf * KT + lanes;
                constexpr int N = KT / 32;
                const int slot0 = (w.tile + j) * KT;
                uint32_t s[N][32];
                if (!warp_wait(&bar[S::SCORES + buf], (c / NB) & 1, ok)) break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < N; ++i) tmem_ld32_nowait(s_at + i * 32, s[i]);
                const bool masked = slot0 + KT > w.common;
#pragma unroll
                for (int i = 0; i < N; ++i) tmem_wait_ld_into(s[i]);
                if (masked) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const uint32_t see = live ? seen_word(w, token, slot0 + i * 32) : 0u;
#pragma unroll
                        for (int n = 0; n < 32; ++n) s[i][n] = see & 1u << n ? s[i][n] : 0xff800000u;  // -infinity
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int n = 0; n < 32; n += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(s[i][n + 2 * k])), __uint_as_float(s[i][n + 2 * k + 1]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool move = top > m + grow || m == -INFINITY;
                // the products before are done: with one buffer these scores came after them
                if (NB == 2 && c > 0 && !warp_wait(&bar[S::DONE + u], (c - 1) & 1, ok)) break;
                if (j == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, move)) {
                    tc_fence_after();
                    const float now = move ? fmaxf(top, m) : m;
                    // (from the products as they are rounded beside the scores, or the difference, which is exact, where those are exact)
                    const float f = m == -INFINITY ? 0.f : exp2_fast(scale_of(now, sc) == sc ? __fsub_rn(__fmul_rn(m, sc), __fmul_rn(now, sc)) : (m - now) * sc);
                    m = now;
                    l2 = fma2(l2, pair(__float_as_uint(f), __float_as_uint(f)), pair(0x80000000u, 0x80000000u));
#pragma unroll 1
                    for (int i = 0; i < D; i += 16) {
                        uint32_t o[16];
                        tmem_ld16_nowait(o_at + i, o);
                        tmem_wait_ld_into(o);
#pragma unroll
                        for (int n = 0; n < 16; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f);
                        tmem_st16(o_at + i, o);
                    }
                }
                const float by = scale_of(m, sc), off = m == -INFINITY ? 0.f : -m * by;
                const f2 sc2 = pair(__float_as_uint(by), __float_as_uint(by)), off2 = pair(__float_as_uint(off), __float_as_uint(off));
                // the first half of the probabilities is multiplied while the second is made
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    // a masked tile's values are waited for before the last hand-over, behind which nothing keeps their barrier from
                    // a phase more (behind the last of the probabilities, with as much certainty, this took more registers: 88
                    // bytes spilled, not 16; a prompt of 8192 tokens 497 us, not 447)
                    if (masked && i == N / 2) warp_wait(&bar[S::READY + c % S::VS], (c / S::VS) & 1, ok);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t packed[8];
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            float2 z = parts(fma2(pair(s[i][h * 16 + 2 * n], s[i][h * 16 + 2 * n + 1]), sc2, off2));
                            z.x = exp2_fast(z.x), z.y = exp2_fast(z.y);
                            l2 = add2(l2, pair(__float_as_uint(z.x), __float_as_uint(z.y)));
                            packed[n] = pack_bf16(z.x, z.y);
                        }
                        tmem_st8(s_at + i * 16 + h * 8, packed);
                    }
                    if (i == N / 2 - 1 || i == N - 1) {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(&bar[S::PROBS + buf * 2 + (i == N - 1)]);
                    }
                }
                if (masked) {
                    if (!ok) break;
                    const uint32_t *sp = reinterpret_cast<const uint32_t *>(sm + S::OFF_SPOILT) + c % (2 * S::VS) * S::kSpoilt;
                    uint32_t hit = 0;
#pragma unroll 1
                    for (int i = 0; i < N; ++i)
                        if (sp[i] && live) hit |= sp[i] & seen_word(w, token, slot0 + i * 32);
                    if (hit) l2 = pair(0x7fc00000u, 0x7fc00000u);  // and stays NaN
                }
            }
            if (!ok) break;
            // ---- outputs
            if (!warp_wait(&bar[S::DONE + u], (c - 1) & 1, ok)) break;
            tc_fence_after();
            const float2 ll = parts(l2);
            const float l = ll.x + ll.y;
            float inv = w.stat ? 1.f : l == 0.f ? 0.f : 1.f / l;
            // (scores that are all -infinity)
            if (l == 0.f && !w.stat && live && sees_any(w.len, w.tokens, w.mask ? w.mask + (int64_t)token * w.mask_words : nullptr)) inv = __int_as_float(0x7fc00000);
            if (w.stat && live) w.stat[own_row] = make_float2(m * sc, l);
            // 64 columns at a time to shared memory, from where another warp sends them as TMA boxes.  (Stores by these warps
            // keep the memory pipe, and what stands behind it in the block, for 4000 cycles an item, whole rows or 16 bytes a
            // lane.)  Parts, and a request's last tokens where they do not fill a tile, go out from here, four rows at a time.
            const bool boxed = u < w.boxes;
            uint8_t *out = sm + S::OFF_OUT + warp * 4096;
            const int64_t mine = live ? own_token * w.token_pitch + own_head * w.head_pitch : -1;
            auto rows_out = [&](int at) {  // the 128 bytes from `at` on
                __syncwarp();
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const int k = n * 4 + (lane >> 3);
                    const int64_t row = __shfl_sync(0xffffffffu, mine, k);
                    if (row >= 0)
                        *reinterpret_cast<uint4 *>(w.to + row + at + (lane & 7) * 16) = *reinterpret_cast<const uint4 *>(out + k * 128 + ((lane & 7) ^ (k & 7)) * 16);
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int i = 0; i < D; i += 64) {
                uint32_t o[64];
                tmem_ld32_nowait(o_at + i, reinterpret_cast<uint32_t(&)[32]>(o[0]));
                tmem_ld32_nowait(o_at + i + 32, reinterpret_cast<uint32_t(&)[32]>(o[32]));
                tmem_wait_ld_into(reinterpret_cast<uint32_t(&)[32]>(o[0]));
                tmem_wait_ld_into(reinterpret_cast<uint32_t(&)[32]>(o[32]));
                if (i + 64 == D) {
                    tc_fence_before();
                    mbar_arrive(&bar[S::FREE + u]);
                }
#pragma unroll
                for (int n = 0; n < 64; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * inv);
                auto put = [&](int n, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
                    *reinterpret_cast<uint4 *>(out + lane * 128 + (n ^ (lane & 7)) * 16) = make_uint4(a, b, c, d);
                };
                if (rounds > 0 && !warp_wait(&bar[S::TAKEN + u], (rounds - 1) & 1, ok)) break;  // the place is free
                if (w.bf16) {
#pragma unroll
                    for (int n = 0; n < 32; ++n) o[n] = pack_bf16(__uint_as_float(o[2 * n]), __uint_as_float(o[2 * n + 1]));
#pragma unroll
                    for (int n = 0; n < 8; ++n) put(n, o[4 * n], o[4 * n + 1], o[4 * n + 2], o[4 * n + 3]);
                    if (boxed) {
                        fence_proxy_async_smem();
                        mbar_arrive(&bar[S::OUT + u]);
                        ++rounds;
                    } else {
                        rows_out(i * 2);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int n = 0; n < 8; ++n) put(n, o[h * 32 + 4 * n], o[h * 32 + 4 * n + 1], o[h * 32 + 4 * n + 2], o[h * 32 + 4 * n + 3]);
                        rows_out(i * 4 + h * 128);
                    }
                }
            }
            if (!ok) break;
            drop();
        }
    } else if (warp == S::kRowWarps) {
        // ------------------------------------------------------------------ products
        const uint32_t lead = elect();
        const uint32_t id_s = idesc_bf16_f32(128, KT), id_o = idesc_bf16_f32(128, D) | (1u << 16);  // V is MN-major
        const uint32_t d_q = uniform(desc_lo(base, 0));
        auto scores = [&](int u, int c) {  // S of tile number c
            const uint32_t d_k = uniform(desc_lo(base + S::OFF_K + c % S::KS * S::kStage, 0));
            const int buf = u * NB + c % NB;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_ss(lead, tm + S::kScores + buf * KT, d_q + (((u * S::H + (ks >> 2)) * S::kQTile + (ks & 3) * 32) >> 4),
                       d_k + (((ks >> 2) * S::kHalf + (ks & 3) * 32) >> 4), id_s, ks > 0);
            commit(lead, &bar[S::SCORES + buf]);
        };
        auto keys = [&](int c) {
            warp_wait(&bar[S::KFULL + c % S::KS], (c / S::KS) & 1, ok);
            tc_fence_after();
            return ok;
        };
        int c0 = 0;
        while (const Job *wp = take()) {
            const Job &w = *wp;
            const int n = w.n;
            if (!warp_wait(&bar[S::QFULL], (item - 1) & 1, ok) || !keys(c0)) break;
#pragma unroll 1
            for (int u = 0; u < U; ++u) scores(u, c0);
            commit(lead, &bar[S::KEMPTY + c0 % S::KS]);
            if (n == 1) commit(lead, &bar[S::QEMPTY]);
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const int c = c0 + j;
                const bool more = j + 1 < n;
                if (NB == 2 && more) {
                    if (!keys(c + 1)) break;
                    scores(0, c + 1);
                    commit(lead, &bar[S::KEMPTY + (c + 1) % S::KS]);
                    if (j + 2 == n) commit(lead, &bar[S::QEMPTY]);
                }
                if (!warp_wait(&bar[S::READY + c % S::VS], (c / S::VS) & 1, ok)) break;
                const uint32_t d_v = uniform(desc_lo(base + S::OFF_V + c % S::VS * S::kStage, S::kHalf));
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int buf = u * NB + c % NB;
                    if (!warp_wait(&bar[S::PROBS + buf * 2], (c / NB) & 1, ok)) break;
                    if (j == 0 && item > 1 && !warp_wait(&bar[S::FREE + u], item & 1, ok)) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < KT / 16; ++ks) {
                        if (ks == KT / 32) {
                            if (!warp_wait(&bar[S::PROBS + buf * 2 + 1], (c / NB) & 1, ok)) break;
                            tc_fence_after();
                        }
                        mma_ts(lead, tm + S::kOut + u * D, tm + S::kScores + buf * KT + ks * 8, d_v + ((ks * 2048) >> 4), id_o, j + ks > 0);
                    }
                    if (!ok) break;
                    commit(lead, &bar[S::DONE + u]);
                    if (NB == 1 && more) {
                        if (u == 0 && !keys(c + 1)) break;
                        scores(u, c + 1);
                    }
                }
                if (!ok) break;
                commit(lead, &bar[S::VEMPTY + c % S::VS]);
                if (NB == 1 && more) {
                    commit(lead, &bar[S::KEMPTY + (c + 1) % S::KS]);
                    if (j + 2 == n) commit(lead, &bar[S::QEMPTY]);
                }
            }
            if (!ok) break;
            c0 += n;
            drop();
        }
        // no product is under way when the block ends
        commit(lead, &bar[S::DRAIN]);
        bool done = true;
        if (!wait(&bar[S::DRAIN], 0, done)) ok = false;
    } else if (warp == S::kRowWarps + 1) {
        // ------------------------------------------------------------------ keys, values, queries
        const int boxes = KT / tp.box;  // of one half; lane: half lane / boxes, box lane % boxes
        const bool mine = lane < boxes * S::H;
        const int half = lane / boxes, at_slot = lane % boxes * tp.box;
        auto page_of = [&](const Walk &v, int tile) {
            const int s = tile * KT + at_slot;
            if (!mine || s >= v.seen) return p.n_pages;
            const int id = p.table[(int64_t)v.at.b * p.max_pages + s / p.page_size];
            if (id >= 0 && id < p.n_pages) return id;
            flag(p.status, GDN_DEV_BAD_PAGE);
            return p.n_pages;
        };
        Walk v;
        v.at = start;
        v.r = request(p, start.b, nullptr);
        v.left = end - begin;
        v.item<KT>(p);
        int c = 0, id = page_of(v, v.first), k_sent = 0, v_sent = 0, q_sent = 0;
        auto load = [&](int kv, int at, uint64_t *full, int page, int row, int h) {
            if (lane == 0) mbar_arrive_expect_tx(full, S::kStage);
            __syncwarp();
            if (mine)
                tma_load_4d(base + at + half * S::kHalf + at_slot * 128, kv ? &v_map : &k_map, full, half * 64, page == p.n_pages ? 0 : row, h, page);
        };
        auto load_queries = [&](int first, int h) {
            if (q_sent > 0 && !warp_wait(&bar[S::QEMPTY], (q_sent - 1) & 1, ok)) return;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar[S::QFULL], U * S::H * 128 * tp.tile_tokens * p.group);
#pragma unroll 1
                for (int i = 0; i < U * S::H; ++i)
                    tma_load_3d(sm + i * S::kQTile, &q_map, &bar[S::QFULL], i % S::H * 64, h * p.group, first + i / S::H * tp.tile_tokens);
            }
            ++q_sent;
        };
        auto tell = [&](bool more) {
            const int i = item % kJobs;
            if (item >= kJobs && !warp_wait(&bar[S::JEMPTY + i], (item / kJobs - 1) & 1, ok)) return;
            if (lane == 0) {
                Job j = {};
                if (more) {
                    const bool whole = v.last - v.first == v.tiles;
                    const int token = v.at.qt * U * tp.tile_tokens, e = whole && p.out_bf16 ? 2 : 4;
                    j.n = v.last - v.first, j.tile = v.first, j.seen = v.seen, j.common = v.common;
                    j.len = v.r.len < 0 ? kNotInUse : v.r.len, j.tokens = v.r.n, j.token = token, j.first = v.r.first, j.head = v.at.h;
                    j.mask_words = p.mask_words;
                    j.mask = p.mask ? p.mask + (int64_t)v.r.first * p.mask_words : nullptr;
                    j.bf16 = e == 2;
                    j.boxes = e == 2 ? min(U, (v.r.n - token) / tp.tile_tokens) : 0;
                    j.head_pitch = D * e;
                    j.token_pitch = (int64_t)D * e * (whole ? p.hkv * p.group : p.group);
                    if (whole) {
                        j.to = static_cast<uint8_t *>(p.o) + ((int64_t)(v.r.first + token) * p.hkv * p.group + v.at.h * p.group) * (D * e);
                    } else {
                        j.to = reinterpret_cast<uint8_t *>(part_out(p, S::CAP, D, run, v.first == 0));
                        j.stat = reinterpret_cast<float2 *>(part_stat(p, S::CAP, D, runs, run, v.first == 0));
                    }
                }
                *reinterpret_cast<Job *>(sm + S::OFF_JOB + i * sizeof(Job)) = j;
                mbar_arrive(&bar[S::JFULL + i]);
            }
            ++item;
        };
        bool more = v.first < v.last;
        tell(more);
        while (more && ok) {
            // this item's loads, the next one's place worked out behind the first of them
            const int first = v.first, last = v.last, h = v.at.h, q_first = v.r.first + v.at.qt * U * tp.tile_tokens;
            Walk now = v;
            for (int t = first; t < last; ++t, ++c) {
                const int page = id, row = (t * KT + at_slot) % p.page_size;
                if (t + 1 < last) id = page_of(now, t + 1);  // a tile ahead
                if (c == 0) load_queries(q_first, h);
                if (c >= S::KS && !warp_wait(&bar[S::KEMPTY + c % S::KS], (c / S::KS - 1) & 1, ok)) break;
                load(0, S::OFF_K + c % S::KS * S::kStage, &bar[S::KFULL + c % S::KS], page, row, h);
                k_sent = c + 1;
                if (c >= S::VS && !warp_wait(&bar[S::VEMPTY + c % S::VS], (c / S::VS - 1) & 1, ok)) break;
                load(1, S::OFF_V + c % S::VS * S::kStage, &bar[S::VFULL + c % S::VS], page, row, h);
                v_sent = c + 1;
                if (t == first) {
                    // queries once the item's before are done with: behind the first keys and values
                    if (c > 0) load_queries(q_first, h);
                    if (!ok) break;
                    more = v.next<KT>(p);
                    tell(more);
                    if (!ok) break;
                }
            }
            if (more) id = page_of(v, v.first);
        }
        // no copy is under way when the block ends
        bool done = true;
        for (int n = max(0, k_sent - S::KS); n < k_sent; ++n) wait(&bar[S::KFULL + n % S::KS], (n / S::KS) & 1, done);
        for (int n = max(0, v_sent - S::VS); n < v_sent; ++n) wait(&bar[S::VFULL + n % S::VS], (n / S::VS) & 1, done);
        if (q_sent > 0) wait(&bar[S::QFULL], (q_sent - 1) & 1, done);
        ok = ok && done;
    } else if (warp == S::kRowWarps + 3) {
        // ------------------------------------------------------------------ outputs
        int rounds[U] = {};
        if (tp.probe > 0 && !mbar_wait(&bar[S::PROBE], 0, (uint32_t)tp.probe) && lane == 0) flag(p.status, GDN_DEV_TIMEOUT);
        while (const Job *wp = ok ? take() : nullptr) {
            const Job &w = *wp;
            for (int n = 0; n < w.boxes * S::H && ok; ++n) {
                // the tiles take turns, as their outputs come
                const int u = n % w.boxes, x = n / w.boxes * 64;
                const int k = u ? rounds[U - 1] : rounds[0];
                if (!warp_wait(&bar[S::OUT + u], k & 1, ok)) break;
                if (lane == 0) {
                    tma_store_3d(&o_map, sm + S::OFF_OUT + u * kTileRows * 128, x, w.head * p.group, w.first + w.token + u * tp.tile_tokens);
                    bulk_commit();
                    bulk_wait_read();
                    mbar_arrive(&bar[S::TAKEN + u]);
                }
                __syncwarp();
                if (u) ++rounds[U - 1];
                else ++rounds[0];
            }
            if (ok) drop();
        }
    } else {
        // ------------------------------------------------------------------ values
        int c = 0;
        while (const Job *wp = ok ? take() : nullptr) {
            const Job &w = *wp;
            for (int j = 0; j < w.n; ++j, ++c) {
                const int st = c % S::VS, slot0 = (w.tile + j) * KT;
                if (!warp_wait(&bar[S::VFULL + st], (c / S::VS) & 1, ok)) break;
                if (slot0 + KT > w.common) {
                    uint32_t *spoilt = reinterpret_cast<uint32_t *>(sm + S::OFF_SPOILT) + c % (2 * S::VS) * S::kSpoilt;
                    uint8_t *v = sm + S::OFF_V + st * S::kStage;
#pragma unroll 1
                    for (int i = 0; i < KT / 32; ++i) {
                        const int row = i * 32 + lane, s = slot0 + row;
                        bool bad = false;
                        if ((w.tokens > 1 || w.mask) && s >= w.len && s < w.seen) {  // (a single token sees itself, unless a mask leaves it out)
                            uint32_t over = 0;  // bf16 entries with all exponent bits set carry into their sign bit
#pragma unroll 8
                            for (int k = 0; k < S::H * 8; ++k) {
                                const uint4 y = *reinterpret_cast<const uint4 *>(v + (k >> 3) * S::kHalf + row * 128 + ((k & 7) ^ (row & 7)) * 16);
                                over |= (y.x & 0x7F807F80u) + 0x00800080u, over |= (y.y & 0x7F807F80u) + 0x00800080u;
                                over |= (y.z & 0x7F807F80u) + 0x00800080u, over |= (y.w & 0x7F807F80u) + 0x00800080u;
                            }
                            bad = over & 0x80008000u;
                        }
                        if (bad || s >= w.seen)
#pragma unroll 8
                            for (int k = 0; k < S::H * 8; ++k)
                                *reinterpret_cast<uint4 *>(v + (k >> 3) * S::kHalf + row * 128 + ((k & 7) ^ (row & 7)) * 16) = make_uint4(0, 0, 0, 0);
                        const uint32_t word = __ballot_sync(0xffffffffu, bad);
                        if (lane == 0) spoilt[i] = word;
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[S::READY + st]);
            }
            drop();
        }
    }
    if (!ok) flag(p.status, GDN_DEV_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == S::kRowWarps) tmem_dealloc(tm, 512);
}

// [n_pages][page_size][hkv][d] with the cache's strides as (d, row, head, page); boxes of 64 x box x 1 x 1
bool encode_pool(CUtensorMap *map, const void *pool, const Params &p, int d, int box) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)p.page_size, (cuuint64_t)p.hkv, (cuuint64_t)p.n_pages};
    // (a stride that is never taken may be anything)
    cuuint64_t strides[3] = {p.page_size > 1 ? (cuuint64_t)p.slot_stride * 2 : 16, p.hkv > 1 ? (cuuint64_t)p.head_stride * 2 : 16,
                             p.n_pages > 1 ? (cuuint64_t)p.page_stride * 2 : 16};
    cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pool), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T][heads][d] as (d, head, token); boxes of a tile of rows
bool encode_tokens(CUtensorMap *map, const void *rows, int64_t stride, const Params &p, int d, int tile_tokens) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)p.hkv * p.group, (cuuint64_t)p.total};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    cuuint32_t boxes[3] = {64, (cuuint32_t)p.group, (cuuint32_t)tile_tokens}, estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(rows), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int U>
cudaError_t run(Params p, int runs, cudaStream_t stream) {
    using S = Shape<D, U>;
    static int have[16];
    const cudaError_t e = ensure_smem(attend_tc_kernel<D, U>, S::kBytes, have);
    if (e != cudaSuccess) return e;
    TcParams tp;
    tp.tile_tokens = kTileRows / p.group;
    tp.probe = wait_probe_polls();
    tp.box = p.page_size & -p.page_size;
    if (tp.box > S::KT) tp.box = S::KT;
    p.rows = U * tp.tile_tokens * p.group, p.cost = U == 2 ? 3 : 2;
    tp.p = p;
    CUtensorMap q, o, k, v;
    if (!encode_tokens(&q, p.q, p.q_stride, p, D, tp.tile_tokens) || !encode_tokens(&o, p.o, (int64_t)p.hkv * p.group * D, p, D, tp.tile_tokens) || !encode_pool(&k, p.k, p, D, tp.box) || !encode_pool(&v, p.v, p, D, tp.box))
        return cudaErrorInvalidValue;
    const cudaError_t f = launch_dependent(attend_tc_kernel<D, U>, dim3(runs), S::kThreads, S::kBytes, stream, q, o, k, v, tp, runs);
    return f != cudaSuccess ? f : launch_join<D, S::CAP>(p, runs, stream);
}

template <int D, int U>
Choice choice(const gdn_kv_attend_args &a) {
    using S = Shape<D, U>;
    const int group = a.n_q_heads / a.cache.n_kv_heads;
    Choice x = {};
    x.runs = most_runs(a, false, U * (kTileRows / group) * group, S::KT, 1);
    x.workspace = 4 * workspace_floats(S::CAP, D, x.runs);
    x.launch = run<D, U>;
    return x;
}

}  // namespace

bool attend_tc_supported(const gdn_kv_attend_args &a) {
    const gdn_kv_cache &c = a.cache;
    // (strides of a tensor map: above 0 where they are taken, below 2^40 bytes)
    auto fits = [](int64_t stride, int64_t n) { return n <= 1 || (stride > 0 && stride < (int64_t)1 << 39); };
    return c.dtype == GDN_BF16 && (c.d == 64 || c.d == 128 || c.d == 256) && c.page_size % 8 == 0 && c.n_pages > 0 && a.scale > 0.f &&
           a.n_q_heads / c.n_kv_heads <= kTileRows && attn::aligned16(a) && fits(c.slot_stride, c.page_size) && fits(c.head_stride, c.n_kv_heads) &&
           fits(c.page_stride, c.n_pages) && a.q_stride < (int64_t)1 << 39;
}

attn::Choice attend_tc_choice(const gdn_kv_attend_args &a) {
    // one tile of rows where all of a request's fit
    const int group = a.n_q_heads / a.cache.n_kv_heads;
    const bool one = a.max_tokens <= kTileRows / group;
    if (a.cache.d == 64) return one ? choice<64, 1>(a) : choice<64, 2>(a);
    if (a.cache.d == 128) return one ? choice<128, 1>(a) : choice<128, 2>(a);
    return choice<256, 1>(a);
}

}  // namespace gdn
