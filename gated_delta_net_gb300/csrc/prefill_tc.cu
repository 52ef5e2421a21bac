// prefill_tc.cu -- prompts through the gated delta rule in chunks of 64 tokens on the
// tensor cores: bf16 q/k/v/o, d_k = d_v = 128 (sm_103a).
//
// For a chunk with the state S before it and gamma_i the sum of g over tokens 0..i,
//     A_ij = beta_i e^(gamma_i - gamma_j) k_i.k_j   (j < i),   T = (I + A)^-1
//     U    = T' V - W S^T,   T'_ij = T_ij beta_j,   W = T'' K,   T''_ij = T'_ij e^gamma_j
//     o_i  = scale e^gamma_i S q_i + sum_{j <= i} scale e^(gamma_i - gamma_j) (q_i.k_j) u_j
//     S   <- e^gamma_63 S + sum_t e^(gamma_63 - gamma_t) u_t k_t^T.
// Everything but the last three lines is free of S, so it runs ahead of the chain over the
// chunks.  Products run on tcgen05 transposed, so that the 128 rows of d_v (or d_k) are the
// MMA's rows and the 64 tokens its columns:
//     [K;Q] K^T    128 x 64     Gram and q.k at once
//     W^T = K^T T''^T, U^T = V^T T'^T - S W^T, O^T = S Q^T and U^T Y^T, dS = U'^T K.
//
// Precision: the state's chain keeps fp32 sums, and its operands that are not bf16 already
// (T', T'', W, S, U') enter as pairs hi + lo of bf16, x = hi + lo to 2^-18; lo x lo is left
// out (2^-18).  The state comes out about 4e-6 (norm-wise) from exact: bf16 is what the tensor
// core takes beside the bf16 tokens, and a third part of each operand would not fit.  The output
// takes the same pairs of S, and Y and U as tf32 (2^-12): 1.68e-3 from exact, of which 1.66e-3
// are its own rounding to bf16.
//
// T and Y are lower triangles: they lie in shared memory, and are multiplied, by strips of 16
// columns without the rows above them, which is what makes room for Y in 32 bits.
//
// One block an SM (all 512 tensor-memory columns), 28 warps:
//     warp 0        issues W
//     warp 1        issues [K;Q] K^T
//     warp 2        issues U, O and dS: the chain
//     warp 3        walks the items, loads K and Q of three chunks, the chunk's gates: gamma by a scan, and its exponentials
//     warps 4-7, 9, 11  A and Y; T = (I + A)^-1 is then found in blocks of 16:
//     warps 8, 10   T's diagonal blocks
//     warps 12-15   T's other blocks, T', T''
//     warps 16-19   load V, W to shared memory, S Q^T's factors, the outputs to global memory
//     warps 20-27   the state's hi + lo operand and its decay, U' hi + lo
// The state stays in tensor memory as the sum that dS is added to.  The chain for a chunk is
// S split -> S W^T -> U split -> dS.
//
// The roles run different code at the same time, and what it costs to fetch bounds them as much as
// what they compute: loops stay rolled where their steps are alike.
//
// 64 prompts of 16 to 512 tokens, 32 value heads, states gathered from a pool: 262 us for 597 MB that have
// to move (88 us); one prompt of 16384 tokens in four segments, 32 heads: 504 us.  (With S, U and Y rounded to bf16 for
// the outputs 255 and 497, and the outputs 2.8e-3 from exact.)  What bounds it is the latency of the chain, 3.3 us a
// chunk alone and 4.2 beside the other roles: no pipe is busy for half of the time (issue 47 % of cycles with 7 warps
// a scheduler, tensor pipe a third).
#include <algorithm>

#include "internal.cuh"
#include "sm100.cuh"
#include "tc_tiles.cuh"

namespace gdn {
namespace {

using namespace sm100;
using tiles::bf16_hi;
using tiles::bf16_lo;
using tiles::kD;
using tiles::named_sync;
using tiles::pack_bf16;

constexpr int kC = 64;         // tokens a chunk
constexpr int kThreads = 896;  // 28 warps
constexpr int kKQ = 3;         // chunks of K and Q, of Y and of gates held at a time
constexpr int kDecays = 4;

// shared memory (bytes from a 1024-aligned base)
constexpr int kTile = kC * 128;              // 64 rows of 128 bytes: half of a token tile
constexpr int OFF_KQ = 0;                    // [kKQ][2 halves of d][K, Q] tiles
constexpr int OFF_V = OFF_KQ + kKQ * 4 * kTile;  // [2 halves] tiles
// Lower triangles, by strips of 16 columns without the rows above them: a strip's 16-byte columns one after the other,
// rows next to each other (strip s has 64 - 16 s rows, and strip_rows(s) lie in those before it)
__host__ __device__ constexpr int strip_rows(int s) { return 72 * s - 8 * s * s; }
constexpr int kTriT = strip_rows(4) * 32;    // T: bf16, two 16-byte columns a strip
constexpr int kTriY = strip_rows(4) * 64;    // Y: fp32, four
constexpr int OFF_T = OFF_V + 2 * kTile;     // T' hi, lo, T'' hi, lo (negated): rows i, columns j
constexpr int OFF_W = OFF_T + 4 * kTriT;     // W^T hi, lo: 128 rows of d_k, columns i
constexpr int OFF_Y = OFF_W + 4 * kTile;     // [kKQ] Y: rows i, columns j
constexpr int OFF_A = OFF_Y + kKQ * kTriY;   // [2] ten 16 x 16 blocks, bf16 hi and lo: A below the diagonal (6), T on
                                             // it (4; before T is known, A's diagonal blocks in fp32)
constexpr int kBlocks = 10 * 1024;
constexpr int OFF_SC = OFF_A + 2 * kBlocks;  // [kKQ] gates of a chunk, floats:
constexpr int SC_REL = 0, SC_BETA = 64, SC_BG = 128;  // (gamma_e - gamma_j) log2 e, e the last token of j's block of 16; beta;
                                             // -beta e^gamma
constexpr int SC_COL = 192;                  // e^(gamma_r - gamma_j) for r = 16, 32, 48 and j < r
constexpr int SC_EG = 288, SC_FD = 352;      // scale e^gamma, e^(gamma_63 - gamma)
constexpr int SC_JOB = 416;                  // the chunk itself (Job)
constexpr int kGates = 432 * 4;
constexpr int OFF_MASK = OFF_SC + kKQ * kGates;  // fp32 [17][16]: row n is 0 in its first n columns, -10^30 after them
constexpr int OFF_EL = OFF_MASK + 17 * 64;      // [kDecays] e^gamma_63
constexpr int OFF_SLOT = OFF_EL + kDecays * 4;
constexpr int OFF_NEXT = OFF_SLOT + 16;      // answer to a request for the next item
constexpr int kSorted = 256;  // prompts that can be put in order
constexpr int OFF_ORDER = OFF_NEXT + 16;
constexpr int OFF_BAR = OFF_ORDER + kSorted;
enum Bar {
    B_FULL = 0, B_EMPTY = B_FULL + kKQ, B_SCFREE = B_EMPTY + kKQ, B_GATES = B_SCFREE + kKQ, B_YFREE = B_GATES + kKQ,
    B_BLK = B_YFREE + kKQ, B_BLKFREE = B_BLK + 2, B_DIAG = B_BLKFREE + 2, B_VFULL = B_DIAG + 4,
    B_G, B_GFREE, B_T, B_TFREE, B_W, B_WRDY, B_S, B_U, B_SL, B_UST, B_SQ, B_SQRD, B_UPD, B_O, B_OFREE, B_MID, B_NEXT, B_DRAIN, B_PROBE = B_DRAIN + 3, B_COUNT
};
constexpr int kSmem = OFF_BAR + B_COUNT * 8;
static_assert(kSmem <= 232448, "one block an SM");

// tensor-memory columns
constexpr uint32_t TM_DS = 0, TM_S = 128, TM_U = 256, TM_O = 320, TM_G = 384, TM_W = 448;
constexpr uint32_t TM_SHI = TM_S, TM_SLO = TM_S + 64;
// U' hi, lo lie over S lo, which is free once S W^T and S lo Q^T are done.  U's sum is itself the left-hand operand of Y U
constexpr uint32_t TM_UHI = TM_SLO, TM_ULO = TM_SLO + 32;

struct Params {
    int hk_n, hv_n, total, max_tokens, n_states, batch, items, probe;
    bool sorted;                    // prompts longest first
    int seg0, seg, segs;            // tokens of the first segment and of the others, multiples of 64; segments a prompt can have
    uint32_t group_inv;             // ceil(2^32 / heads that share a key head), 0 for one
    float scale;
    const int32_t *offsets, *slots, *fresh;
    const float *g, *beta, *S0;
    __nv_bfloat16 *o;
    float *S_new, *ws;
    int32_t *status;
};

// Few prompts do not fill the GPU, so a prompt is cut into segments.  A first pass over all segments but the last
// finds, without outputs, each one's state from zero (from S0 for the first) and its effect on a state before it
// (the same from the identity and with v = 0: rows of the state do not meet, so S -> S M + L).  A small kernel
// joins them, and a second pass runs every segment from the state before it.  Workspace of a (request, head), in
// states: S before segments 0 .. segs - 1 (after the first pass: S0, L of segments 0 .. segs - 2), M of segments
// 1 .. segs - 2.
struct Item {
    int h, hk, lo, n, chunks, err;
    bool skip;          // has no such segment, or is refused
    bool unit;          // from the identity, without v
    const float *from;  // the state before it, null for zero
    float *to;          // where the one after it goes, null for nowhere
};

// Item number idx of the grid: (slice, request, head).  A slice is a segment, the first one last, as it may be
// shorter; in the first pass the slices are the inner segments, the same from the identity, and the first segment.
struct Walk {
    const uint8_t *order;  // of the prompts, null for their own
    int idx, h, b, s;
    __device__ __forceinline__ void set(const Params &p, int i) {
        idx = i;
        const int u = (unsigned)i / (unsigned)p.hv_n;
        h = i - u * p.hv_n;
        s = (unsigned)u / (unsigned)p.batch;
        b = u - s * p.batch;
        if (order) b = order[b];
    }
    // what an item's parameters are made of
    struct Raw {
        int lo, hi, slot, fresh;
    };
    __device__ __forceinline__ Raw raw(const Params &p) const {
        Raw r = {__ldg(p.offsets + b), __ldg(p.offsets + b + 1), b, 0};
        if (p.slots) r.slot = __ldg(p.slots + b);
        if (p.fresh) r.fresh = __ldg(p.fresh + b);
        return r;
    }
    template <bool OUT>
    __device__ __forceinline__ Item item(const Params &p, const Raw &raw) const {
        Item x;
        x.h = h;
        x.hk = p.group_inv ? __umulhi((uint32_t)h, p.group_inv) : h;
        x.lo = raw.lo;
        const bool inside = raw.lo >= 0 && raw.hi >= raw.lo && raw.hi <= p.total;
        x.n = inside ? raw.hi - raw.lo : 0;
        const int slot = raw.slot;
        x.err = 0;
        if (!inside) x.err = GDN_DEV_BAD_DESC;
        else if (x.n > p.max_tokens) x.err = GDN_DEV_TOO_MANY;
        else if (slot < 0 || slot >= p.n_states) x.err = GDN_DEV_BAD_SLOT;
        const int64_t state = ((int64_t)slot * p.hv_n + h) * (kD * kD);
        float *ws = p.ws + ((int64_t)b * p.hv_n + h) * (2 * p.segs - 2) * (kD * kD);
        x.unit = !OUT && s >= p.segs - 2 && s < 2 * p.segs - 4;
        const bool first = s == (OUT ? p.segs - 1 : 2 * p.segs - 4);
        const int seg = first ? 0 : x.unit ? s - (p.segs - 3) : s + 1;
        const int off = first ? 0 : p.seg0 + (seg - 1) * p.seg, len = first ? p.seg0 : p.seg;
        const bool last = x.n - off <= len, one = x.n <= p.seg0;
        x.skip = x.err || (seg > 0 && x.n <= off) || (!OUT && last);
        const bool zero = !p.S0 || raw.fresh != 0;
        if (OUT) {
            x.from = one ? (zero ? nullptr : p.S0 + state) : ws + seg * (kD * kD);
            x.to = last ? p.S_new + state : nullptr;
        } else {
            x.from = seg == 0 && !zero ? p.S0 + state : nullptr;
            x.to = ws + (x.unit ? p.segs + seg - 1 : seg + 1) * (kD * kD);
        }
        x.lo += off;
        x.n = min(x.n - off, len);
        x.chunks = x.skip ? 0 : (x.n + kC - 1) / kC;
        return x;
    }
};

// A chunk as the roles see it, put beside its gates by the warp that makes them.
struct Job {
    int tok, nv, h, flags;  // its first token; tokens of the segment from there on; value head; kFirst ..
    const float *from;      // state before the segment, null for zero
    float *to;              // place for the state after it, null for none
};
constexpr int kFirst = 1, kLast = 2, kUnit = 4, kEnd = 8;  // first, last chunk of a segment; from the identity; no more

// A chunk's number, its place in the rings of three, and the parity of their round.
struct Ring {
    int cc = 0, kq = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        ++cc;
        if (++kq == kKQ) {
            kq = 0;
            ph ^= 1;
        }
    }
};

// Bounded wait; after a first one that ran out the others only look once, and the role ends before its
// next chunk, so that a block whose pipeline broke still ends soon.  A phase is waited for before the
// one after it can complete, or the parity would alias: what runs two chunks ahead or behind has two
// barriers.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, bool &ok) {
    if (!mbar_wait(bar, parity, ok ? 1u << 20 : 1u)) ok = false;
}

// the same by a whole warp
__device__ __forceinline__ void wwait(uint64_t *bar, uint32_t parity, bool &ok) {
    wait(bar, parity, ok);
    __syncwarp();
}

// the warp's next chunk, or false after the last one (or a wait that ran out)
__device__ __forceinline__ bool take(const uint8_t *sm, uint64_t *bar, const Ring &r, Job &j, bool &ok) {
    wait(&bar[B_GATES + r.kq], r.ph, ok);
    if (!__all_sync(0xffffffffu, ok)) return false;
    j = *reinterpret_cast<const Job *>(sm + OFF_SC + r.kq * kGates + SC_JOB * 4);
    return !(j.flags & kEnd);
}

__device__ __forceinline__ uint32_t sw(int row, int chunk16) {  // byte offset in a tile of 128-byte rows
    return (uint32_t)(row * 128 + ((chunk16 ^ (row & 7)) << 4));
}

// MMA issue by a whole converged warp, one elected lane of which (lead) issues: descriptors stay in uniform
// registers, and an MMA takes 25 cycles to issue (52 in a branch of lane 0, as long as a 128 x 64 x 16 one runs).
// A descriptor is given by its low word (start address; the rest is the same for all 128-byte-swizzled tiles up
// to the distance between the 64-element halves of an MN-major operand).
__device__ __forceinline__ uint32_t desc_lo(const void *tile, int lbo_bytes) {
    return ((smem_u32(tile) >> 4) & 0x3FFFu) | ((uint32_t)(lbo_bytes >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// a strip of a triangle: not swizzled, groups of 8 rows after one another, its rows between 16-byte columns
constexpr uint32_t kStripHi = (128u >> 4) | (1u << 14);
// low word of columns 16-byte 2 half.. of strip s of a triangle at (smem address >> 4), `columns` of them a strip
__device__ __forceinline__ constexpr uint32_t strip_lo(uint32_t at, int columns, int s, int half) {
    return (at + strip_rows(s) * columns + half * 2 * (64 - 16 * s)) | (uint32_t)(64 - 16 * s) << 16;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
    return r;
}

// HI: the high word of b
template <uint32_t HI = kDescHi>
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %7};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead), "r"(kDescHi), "r"(HI) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "mov.b64 db, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead), "r"(kDescHi) : "memory");
}
// tf32 operands: A, 8 columns of tensor memory, times a strip
__device__ __forceinline__ void mma_ts_tf32(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "mov.b64 db, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], db, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead), "r"(kStripHi) : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t *bar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 ::"r"(smem_u32(bar)), "r"(lead) : "memory");
}

// two fp32 values in a register pair, for the packed fp32 instructions
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 pair(uint32_t a, uint32_t b) { return pair(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ float2 parts(f2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ void unpair(f2 x, uint32_t &a, uint32_t &b) { asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(x)); }
// 8 floats from and to global memory, 32-byte aligned (a null source reads as zero)
__device__ __forceinline__ void load8(const float *p, f2 (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = 0;
    if (p) asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]) : "l"(p) : "memory");
}
__device__ __forceinline__ void store8(float *p, const f2 (&v)[4]) {
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]) : "memory");
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
// A tf32 product cuts both its operands off behind 11 bits, each by 0.36 2^-10 on average (a mantissa from 1 to 2): made up
// for in one of them, it rounds them.
constexpr float kTf32Up = 1.f + 0.72f / 1024;
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// hi + lo bf16 pairs of two values: packed hi, packed lo
__device__ __forceinline__ void split2(f2 x, uint32_t &hi, uint32_t &lo) {
    const float2 v = parts(x);
    hi = pack_bf16(v.x, v.y);
    const float2 rest = parts(fma2(pair(bf16_lo(hi), bf16_hi(hi)), pair(-1.f, -1.f), x));
    lo = pack_bf16(rest.x, rest.y);
}

// byte offset of 8 columns from 8 c8 of row r in a 16 x 16 bf16 block (rows of 32 bytes, halves exchanged in
// every other group of four rows, so that eight rows cover all banks)
__device__ __forceinline__ uint32_t blk(int r, int c8) { return (uint32_t)(r * 32 + ((c8 ^ ((r >> 2) & 1)) << 4)); }

// float index of columns 4 c4.. of row i of A's diagonal blocks
__device__ __forceinline__ int diag_at(int i, int c4) { return i * 16 + ((c4 ^ ((i >> 1) & 3)) << 2); }

// warp-wide 16 x 16 products of bf16 fragments in registers (the small triangular solve; fp32 sums)
__device__ __forceinline__ void ldm(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stm(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d += (hi + lo of a) (hi + lo of the block at `addr`, this lane's row address)
__device__ __forceinline__ void mul_block(float (&d)[2][4], const uint32_t (&ahi)[4], const uint32_t (&alo)[4], uint32_t addr) {
    uint32_t bh[4], bl[4];
    ldm_t(addr, bh);
    ldm_t(addr + 512, bl);
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        mma16(d[nt], ahi, bh[2 * nt], bh[2 * nt + 1]);
        mma16(d[nt], alo, bh[2 * nt], bh[2 * nt + 1]);
        mma16(d[nt], ahi, bl[2 * nt], bl[2 * nt + 1]);
    }
}
struct Frag {  // a block as a left-hand operand
    uint32_t hi[4], lo[4];
};
__device__ __forceinline__ void load_left(uint32_t addr, Frag &f) {
    ldm(addr, f.hi);
    ldm(addr + 512, f.lo);
}

// -(accumulators) as the left-hand operand of the next product
__device__ __forceinline__ void to_left_neg(const float (&d)[2][4], Frag &f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(pair(-d[e >> 1][2 * (e & 1)], -d[e >> 1][2 * (e & 1) + 1]), f.hi[e], f.lo[e]);
}

// accumulators to a block in shared memory, `addr` this lane's row address
__device__ __forceinline__ void put_plain(uint32_t addr, const float (&d)[2][4]) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(pair(d[e >> 1][2 * (e & 1)], d[e >> 1][2 * (e & 1) + 1]), hi[e], lo[e]);
    stm(addr, hi);
    stm(addr + 512, lo);
}

// T's block (bi, bj) as T' and -T'', hi and lo, into the tiles the tensor cores read
__device__ __forceinline__ void put_block(uint32_t tt, const float *sc, int bi, int bj, int lane, const float (&v)[2][4]) {
    const int rows = 64 - 16 * bj;  // of strip bj
    const uint32_t addr = tt + strip_rows(bj) * 32 + ((lane >> 4) * rows + 16 * (bi - bj) + (lane & 15)) * 16;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f2 f = *reinterpret_cast<const f2 *>(sc + (w ? SC_BG : SC_BETA) + 16 * bj + 8 * (e >> 1) + (lane & 3) * 2);
            split2(mul2(pair(v[e >> 1][2 * (e & 1)], v[e >> 1][2 * (e & 1) + 1]), f), hi[e], lo[e]);
        }
        stm(addr + 2 * w * kTriT, hi);
        stm(addr + (2 * w + 1) * kTriT, lo);
    }
}
__device__ __forceinline__ void diag_block(uint32_t addr, float (&v)[2][4]) {
    Frag f;
    load_left(addr, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e >> 1][2 * (e & 1)] = bf16_lo(f.hi[e]) + bf16_lo(f.lo[e]);
        v[e >> 1][2 * (e & 1) + 1] = bf16_hi(f.hi[e]) + bf16_hi(f.lo[e]);
    }
}

// sum of two double-floats
__device__ __forceinline__ void dd_add(float &ah, float &al, float bh, float bl) {
    const float s = __fadd_rn(ah, bh), t = __fsub_rn(s, ah);
    float e = __fadd_rn(__fsub_rn(ah, __fsub_rn(s, t)), __fsub_rn(bh, t));
    e = __fadd_rn(e, __fadd_rn(al, bl));
    ah = __fadd_rn(s, e);
    al = __fsub_rn(e, __fsub_rn(ah, s));
}

// zeros in rows nv.. of a tile's two halves, `apart` bytes from each other, for the tensor core to read
__device__ __forceinline__ void zero_tail(uint8_t *tile, int apart, int nv, int lane) {
    if (nv >= kC) return;
#pragma unroll 1
    for (int i0 = nv * 8; i0 < kC * 8; i0 += 32) {  // the same steps in every lane: the warp issues products
        const int i = i0 + lane;
        if (i < kC * 8) {
            *reinterpret_cast<uint4 *>(tile + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(tile + apart + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// OUT: outputs and final states; otherwise the first pass over segments
template <bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
prefill_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, Params p) {
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + OFF_SLOT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3;
    if ((smem_u32(sm) & 1023u) != 0u) {
        if (tid == 0) flag(p.status, GDN_DEV_INTERNAL);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            const bool four = i == B_T || i == B_MID || i == B_WRDY || i == B_OFREE || i == B_SQRD || (i >= B_SCFREE && i < B_GATES) ||
                              (i >= B_BLKFREE && i < B_DIAG);
            const uint32_t n = four ? 4 : i == B_GFREE ? (OUT ? 6 : 3) : i >= B_BLK && i < B_BLKFREE ? (OUT ? 7 : 4)
                               : i == B_S || i == B_UST ? 8 : i == B_TFREE ? 2 : 1;
            mbar_init(&bar[i], n);
        }
        fence_mbar_init();
        // test hook: a wait that runs out, before the roles' own waits begin
        if (p.probe > 0 && !mbar_wait(&bar[B_PROBE], 0, (uint32_t)p.probe)) flag(p.status, GDN_DEV_TIMEOUT);
    }
    for (int i = tid; i < 17 * 16; i += kThreads)
        reinterpret_cast<float *>(sm + OFF_MASK)[diag_at(i >> 4, (i >> 2) & 3) + (i & 3)] = (i & 15) < (i >> 4) ? 0.f : -1e30f;
    fence_proxy_async_smem();
    if (warp == 2) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    if (p.sorted) {
        int *len = reinterpret_cast<int *>(sm + OFF_W);
        if (tid < p.batch) len[tid] = prompt_length(p.offsets, tid);
        __syncthreads();
        if (tid < p.batch) sm[OFF_ORDER + length_rank(len, p.batch, tid)] = (uint8_t)tid;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    bool ok = true;
    float *el = reinterpret_cast<float *>(sm + OFF_EL);
    Ring at;
    Job j;

    if (warp < 4) {
        const uint32_t lead = elect();
        const uint32_t tm = uniform(tmem);
        if (warp == 0) {
            // ---------------------------------------------------------------- W^T = K^T T''^T
            const uint32_t id = idesc_bf16_f32(128, 0) | (1u << 15);  // K^T is MN-major
            const uint32_t d_t = uniform(smem_u32(sm + OFF_T) >> 4);
            for (; take(sm, bar, at, j, ok); at.next()) {
                wwait(&bar[B_T], at.cc & 1, ok);
                if (at.cc > 0) wwait(&bar[B_WRDY], (at.cc - 1) & 1, ok);  // the W before it has been read
                tc_fence_after();
                const uint32_t d_k = uniform(desc_lo(sm + OFF_KQ + at.kq * 4 * kTile, 2 * kTile));
#pragma unroll 1
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_ss<kStripHi>(lead, tm + TM_W + 16 * ks, d_k + ks * 128, strip_lo(d_t + (2 + part) * (kTriT >> 4), 2, ks, 0),
                                         id | (uint32_t)(8 - 2 * ks) << 17, part + ks > 0);
                commit(lead, &bar[B_W]);
                commit(lead, &bar[B_TFREE]);
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------------- [K;Q] K^T
            const uint32_t id = idesc_bf16_f32(128, kC);
            for (; take(sm, bar, at, j, ok); at.next()) {
                uint8_t *kt = sm + OFF_KQ + at.kq * 4 * kTile;
                wwait(&bar[B_FULL + at.kq], at.ph, ok);
                if (at.cc > 0) wwait(&bar[B_GFREE], (at.cc - 1) & 1, ok);
                zero_tail(kt, 2 * kTile, j.nv, lane);  // keys past the prompt's end, whatever the next prompt holds
                tc_fence_after();
                const uint32_t d = uniform(desc_lo(kt, 0));
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t o = ((ks >> 2) * 2 * kTile + (ks & 3) * 32) >> 4;
                    mma_ss(lead, tm + TM_G, d + o, d + o, id, ks > 0);
                }
                commit(lead, &bar[B_G]);
            }
        } else if (warp == 2) {
            // ---------------------------------------------------------------- the chain's products
            const uint32_t id_u = idesc_bf16_f32(128, 0) | (1u << 15);  // V^T (MN-major) T'^T, by strips
            const uint32_t id_sw = idesc_bf16_f32(128, kC) | (1u << 16); // S (tensor memory) W^T, W MN-major
            const uint32_t id_k = idesc_bf16_f32(128, kC);               // K-major right-hand side
            const uint32_t id_ds = idesc_bf16_f32(128, kD) | (1u << 16); // U' K, K MN-major
            const uint32_t id_yu = (1u << 4) | (2u << 7) | (2u << 10) | ((128u >> 4) << 24);  // tf32 U^T Y^T, by strips
            const uint32_t d_v = uniform(desc_lo(sm + OFF_V, kTile)), d_t = uniform(smem_u32(sm + OFF_T) >> 4), d_w = uniform(desc_lo(sm + OFF_W, 0));
            for (; take(sm, bar, at, j, ok); at.next()) {
                    const int cc = at.cc, kq = at.kq;
                    const bool unit = !OUT && (j.flags & kUnit), zero = (j.flags & kFirst) && !j.from && !unit;
                    uint8_t *kt = sm + OFF_KQ + kq * 4 * kTile;
                    wwait(&bar[B_VFULL], cc & 1, ok);
                    zero_tail(sm + OFF_V, kTile, j.nv, lane);
                    // U^T = V^T T'^T, once the U before it has been read
                    wwait(&bar[B_T], cc & 1, ok);
                    if (OUT && cc > 0) wwait(&bar[B_O], (cc - 1) & 1, ok);
                    tc_fence_after();
                    if (!unit) {
#pragma unroll 1
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_ss<kStripHi>(lead, tm + TM_U + 16 * ks, d_v + ks * 128, strip_lo(d_t + part * (kTriT >> 4), 2, ks, 0),
                                                 id_u | (uint32_t)(8 - 2 * ks) << 17, part + ks > 0);
                    }
                    commit(lead, &bar[B_TFREE]);
                    // U^T += S (-W)^T: hi hi, lo hi, hi lo
                    wwait(&bar[B_WRDY], cc & 1, ok);
                    wwait(&bar[B_S], cc & 1, ok);
                    tc_fence_after();
                    if (!zero) {  // from zero, S W^T and S Q^T are left out
#pragma unroll 1
                        for (int part = 0; part < 3; ++part)
#pragma unroll 2
                            for (int ks = 0; ks < 8; ++ks)
                                mma_ts(lead, tm + TM_U, tm + TM_SHI + (part & 1) * (TM_SLO - TM_SHI) + ks * 8,
                                       d_w + (part >> 1) * (2 * kTile >> 4) + ks * 128, id_sw, !unit || part + ks > 0);
                    }
                    commit(lead, &bar[B_U]);
                    const uint32_t d_q = uniform(desc_lo(kt + kTile, 0)), d_k = uniform(desc_lo(kt, 2 * kTile));
                    if (OUT) {  // O^T = S Q^T
                        if (cc > 0) wwait(&bar[B_OFREE], (cc - 1) & 1, ok);
                        tc_fence_after();
                        // S lo first: U' takes its place
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            if (!zero) {
#pragma unroll 2
                                for (int ks = 0; ks < 8; ++ks)
                                    mma_ts(lead, tm + TM_O, tm + (part ? TM_SHI : TM_SLO) + ks * 8,
                                           d_q + (((ks >> 2) * 2 * kTile + (ks & 3) * 32) >> 4), id_k, part + ks > 0);
                            }
                            commit(lead, &bar[part ? B_SQ : B_SL]);
                        }
                    }
                    // S += U'^T K
                    wwait(&bar[B_UST], cc & 1, ok);
                    tc_fence_after();
#pragma unroll 1
                    for (int part = 0; part < 2; ++part)
#pragma unroll 2
                        for (int ks = 0; ks < 4; ++ks)
                            mma_ts(lead, tm + TM_DS, tm + TM_UHI + part * (TM_ULO - TM_UHI) + ks * 8, d_k + ks * 128, id_ds, !zero || part + ks > 0);
                    commit(lead, &bar[B_UPD]);
                    if (OUT) {  // O^T += U^T Y^T, once S Q^T has its factors
                        wwait(&bar[B_SQRD], cc & 1, ok);
                        tc_fence_after();
                        const uint32_t d_y = uniform(smem_u32(sm + OFF_Y + kq * kTriY) >> 4);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts_tf32(lead, tm + TM_O + 16 * (ks >> 1), tm + TM_U + 8 * ks, strip_lo(d_y, 4, ks >> 1, ks & 1),
                                        id_yu | (uint32_t)(8 - 2 * (ks >> 1)) << 17, !zero || ks > 0);
                        commit(lead, &bar[B_O]);
                        commit(lead, &bar[B_YFREE + kq]);
                    }
                    commit(lead, &bar[B_EMPTY + kq]);
            }
        } else if (warp == 3) {
            // ---------------------------------------------------------------- items, gates, K and Q
            // The grid has a block for each item; a running block takes the items of blocks that have not begun (they
            // are cancelled then), so that prompts of different lengths spread evenly
            Walk walk;
            walk.order = p.sorted ? sm + OFF_ORDER : nullptr;
            walk.set(p, blockIdx.x);
            uint32_t asked = 0;
            auto ask = [&]() {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bar[B_NEXT], 16);
                    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                                 ::"r"(smem_u32(sm + OFF_NEXT)), "r"(smem_u32(&bar[B_NEXT])) : "memory");
                }
                ++asked;
            };
            auto answer = [&]() {  // the next item's number, or -1
                wwait(&bar[B_NEXT], (asked - 1) & 1, ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return -1;
                uint32_t got, first;
                asm volatile("{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%2];\n\t"
                             "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\t"
                             "mov.u32 %1, 0;\n\t@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
                             : "=r"(got), "=r"(first) : "r"(smem_u32(sm + OFF_NEXT)) : "memory");
                fence_proxy_async_smem();  // read, before the next answer is written there
                __syncwarp();
                return got ? (int)first : -1;
            };
            // a place in the rings was last read by T and the chain of three chunks before
            auto place = [&]() {
                if (at.cc >= kKQ) {
                    wwait(&bar[B_SCFREE + at.kq], at.ph ^ 1, ok);
                    wwait(&bar[B_EMPTY + at.kq], at.ph ^ 1, ok);
                }
                ok = __all_sync(0xffffffffu, ok);
                return reinterpret_cast<float *>(sm + OFF_SC + at.kq * kGates);
            };
            while (ok && walk.idx >= 0) {
                const Item x = walk.template item<OUT>(p, walk.raw(p));
                if (x.chunks <= 0) ask();
                if (OUT && lane == 0 && x.err) flag(p.status, x.err);
                if (x.chunks == 0 && !x.skip && x.from != x.to) {  // no tokens: the state as it is
                    for (int i = lane; i < kD * kD / 4; i += 32)
                        reinterpret_cast<float4 *>(x.to)[i] = x.from ? reinterpret_cast<const float4 *>(x.from)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                float g[2], b[2];  // of tokens 2 lane, 2 lane + 1 of the next chunk
                auto fetch = [&](int c) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = c * kC + 2 * lane + e;
                        g[e] = b[e] = 0.f;
                        if (t < x.n) {
                            g[e] = __ldg(p.g + (int64_t)(x.lo + t) * p.hv_n + x.h);
                            b[e] = __ldg(p.beta + (int64_t)(x.lo + t) * p.hv_n + x.h);
                        }
                    }
                };
                if (x.chunks > 0) fetch(0);
                for (int c = 0; c < x.chunks && ok; ++c, at.next()) {
                    // gamma: a scan in pairs of floats, so that a decay that forgets everything leaves the
                    // differences between later tokens as they were.  e^-200 is zero, whatever lies below it
                    const float g0 = g[0] < -200.f ? -200.f : g[0], g1 = g[1] < -200.f ? -200.f : g[1];
                    const float b0 = b[0], b1 = b[1];
                    if (c + 1 < x.chunks) fetch(c + 1);
                    else ask();
                    float h = g0, l = 0.f;
                    dd_add(h, l, g1, 0.f);
#pragma unroll 1
                    for (int o = 1; o < 32; o <<= 1) {
                        float h2 = __shfl_up_sync(0xffffffffu, h, o), l2 = __shfl_up_sync(0xffffffffu, l, o);
                        if (lane >= o) {
                            dd_add(h2, l2, h, l);
                            h = h2;
                            l = l2;
                        }
                    }
                    float h0 = h, l0 = l;  // without the lane's second token
                    dd_add(h0, l0, -g1, 0.f);
                    const float hl = __shfl_sync(0xffffffffu, h, 31), ll = __shfl_sync(0xffffffffu, l, 31);
                    const float hh[2] = {h0, h}, lw[2] = {l0, l}, bb[2] = {b0, b1};
                    float rel[2], bg[2], eg[2], fd[2], rc[2][4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x0 = __expf(hh[e] + lw[e]);
                        bg[e] = -bb[e] * x0;
                        eg[e] = p.scale * x0;
                        fd[e] = __expf((hl - hh[e]) + (ll - lw[e]));
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // from the blocks' first tokens r = 16 q, held by lane 8 q
                        const float rh = __shfl_sync(0xffffffffu, h0, 8 * q), rl = __shfl_sync(0xffffffffu, l0, 8 * q);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            rc[e][q] = __expf((rh - hh[e]) + (rl - lw[e]));
                        }
                    }
                    // Within a block from its last token: a difference of two such is good to 2^-24 of the larger one, and
                    // where that is large, what lies there no longer counts at the block's end.  (From the first token, a
                    // strong decay early in the block cost all that came after it: 12 tokens that forget, 7e-5 of the state.)
                    const float eh = __shfl_sync(0xffffffffu, h, lane | 7), elo = __shfl_sync(0xffffffffu, l, lane | 7);
#pragma unroll
                    for (int e = 0; e < 2; ++e) rel[e] = 1.4426950408889634f * ((eh - hh[e]) + (elo - lw[e]));
                    const float last = __expf(hl + ll);
                    float *sc = place();
                    if (!ok) break;
                    if (lane == 0) {
                        uint8_t *dst = sm + OFF_KQ + at.kq * 4 * kTile;
                        mbar_arrive_expect_tx(&bar[B_FULL + at.kq], (OUT ? 4 : 2) * kTile);
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            tma_load_3d(dst + half * 2 * kTile, &tmK, &bar[B_FULL + at.kq], half * 64, x.hk, x.lo + c * kC);
                            if (OUT) tma_load_3d(dst + half * 2 * kTile + kTile, &tmQ, &bar[B_FULL + at.kq], half * 64, x.hk, x.lo + c * kC);
                        }
                        Job *job = reinterpret_cast<Job *>(sc + SC_JOB);
                        job->tok = x.lo + c * kC;
                        job->nv = x.n - c * kC;
                        job->h = x.h;
                        job->flags = (c == 0 ? kFirst : 0) | (c == x.chunks - 1 ? kLast : 0) | (x.unit ? kUnit : 0);
                        job->from = x.from;
                        job->to = x.to;
                        el[at.cc & (kDecays - 1)] = last;
                    }
                    __syncwarp();
                    auto put = [&](int to, float v0, float v1) { *reinterpret_cast<float2 *>(sc + to + 2 * lane) = make_float2(v0, v1); };
                    put(SC_REL, rel[0], rel[1]);
                    put(SC_BETA, b0, b1);
                    put(SC_BG, bg[0], bg[1]);
                    put(SC_EG, eg[0], eg[1]);
                    put(SC_FD, fd[0], fd[1]);
#pragma unroll
                    for (int q = 1; q < 4; ++q) {
                        if (lane < 8 * q) put(SC_COL + 8 * q * (q - 1), rc[0][q], rc[1][q]);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[B_GATES + at.kq]);
                }
                const int next = ok ? answer() : -1;
                if (next < 0) break;
                walk.set(p, next);
            }
            float *sc = place();
            if (ok) {
                if (lane == 0) {
                    reinterpret_cast<Job *>(sc + SC_JOB)->flags = kEnd;
                    mbar_arrive(&bar[B_GATES + at.kq]);
                }
            }
            // every load has landed before the block ends, whatever became of its reader
            for (int i = 0; i < kKQ && i < at.cc; ++i) mbar_wait(&bar[B_FULL + i], ((at.cc - 1 - i) / kKQ) & 1, 1u << 16);
            if (asked > 0) mbar_wait(&bar[B_NEXT], (asked - 1) & 1, 1u << 16);
        }
        if (warp < 3) {  // what this warp issued is done before the block ends, whatever became of its reader
            commit(lead, &bar[B_DRAIN + warp]);
            mbar_wait(&bar[B_DRAIN + warp], 0, 1u << 16);
        }
    } else if (warp < 12 && (warp < 8 || (quad & 1))) {
        // -------------------------------------------------------------------- A, Y: 32 rows, 32 columns a warp
        const int row = quad * 32 + lane, i = row & 63, own = i >> 4;  // own: the row's block of 16
        const int cb0 = warp < 8 ? 0 : 2;             // its first block of columns; rows 0..31 have two only
        const bool is_y = row >= 64;                  // of Y (none in a pass without outputs)
        const int last = (i & 15) + (is_y ? 1 : 0);  // columns of the own block that count
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const float *mask = reinterpret_cast<const float *>(sm + OFF_MASK);
        for (; (OUT || !is_y) && take(sm, bar, at, j, ok); at.next()) {
                const int cc = at.cc, kq = at.kq;
                const float *sc = reinterpret_cast<const float *>(sm + OFF_SC + kq * kGates);
                uint8_t *blocks = sm + OFF_A + (cc & 1) * kBlocks, *yt = sm + OFF_Y + kq * kTriY;
                float *diag = reinterpret_cast<float *>(blocks + 6 * 1024);
                const f2 rel = pair(-sc[SC_REL + i], -sc[SC_REL + i]);
                const float f = is_y ? kTf32Up * p.scale : sc[SC_BETA + i], fr = f * exp2_approx(sc[SC_REL + 16 * own] - sc[SC_REL + i]);
                if (cc >= 2) wwait(&bar[B_BLKFREE + (cc & 1)], (cc / 2 - 1) & 1, ok);
                if (is_y && cc >= kKQ) wwait(&bar[B_YFREE + kq], at.ph ^ 1, ok);
                wwait(&bar[B_G], cc & 1, ok);
                tc_fence_after();
                uint32_t nr[16];  // the next 16 columns
                tmem_ld16_nowait(tmem + lanes + TM_G + cb0 * 16, nr);
#pragma unroll 1
                for (int cb = cb0; cb < cb0 + 2; ++cb) {
                    {
                        uint32_t r[16];
                        f2 m[8];
                        tmem_wait_ld_into(nr);
#pragma unroll
                        for (int j = 0; j < 16; ++j) r[j] = nr[j];
                        if (cb == cb0) tmem_ld16_nowait(tmem + lanes + TM_G + (cb + 1) * 16, nr);
                        if (cb < own) {  // left of the own block: e^(gamma_i - gamma_r) e^(gamma_r - gamma_j)
                            const float *col = sc + SC_COL + 8 * own * (own - 1) + cb * 16;
                            const f2 F = pair(fr, fr);
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(col + j);
                                m[j / 2] = mul2(mul2(F, e.x), pair(r[j], r[j + 1]));
                                m[j / 2 + 1] = mul2(mul2(F, e.y), pair(r[j + 2], r[j + 3]));
                            }
                        } else if (cb == own) {
                            const f2 F = pair(f, f);
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(sc + SC_REL + cb * 16 + j);
                                const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(mask + diag_at(last, j >> 2));
                                const float2 d0 = parts(add2(add2(rel, x.x), k.x)), d1 = parts(add2(add2(rel, x.y), k.y));
                                m[j / 2] = mul2(pair(exp2_approx(d0.x), exp2_approx(d0.y)), mul2(F, pair(r[j], r[j + 1])));
                                m[j / 2 + 1] = mul2(pair(exp2_approx(d1.x), exp2_approx(d1.y)), mul2(F, pair(r[j + 2], r[j + 3])));
                            }
                        }
                        if (cb <= own) {
                            if (is_y) {
                                uint8_t *to = yt + strip_rows(cb) * 64 + (i - 16 * cb) * 16;
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    *reinterpret_cast<ulonglong2 *>(to + q * (64 - 16 * cb) * 16) = make_ulonglong2(m[2 * q], m[2 * q + 1]);
                                }
                            } else if (cb == own) {
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    *reinterpret_cast<ulonglong2 *>(diag + diag_at(i, q)) = make_ulonglong2(m[2 * q], m[2 * q + 1]);
                            } else {
                                uint8_t *to = blocks + (own * (own - 1) / 2 + cb) * 1024;
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    uint32_t hi[4], lo[4];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) split2(m[4 * q + e], hi[e], lo[e]);
                                    *reinterpret_cast<uint4 *>(to + blk(i & 15, q)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                                    *reinterpret_cast<uint4 *>(to + 512 + blk(i & 15, q)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                                }
                            }
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before();
                if (is_y) fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar[B_GFREE]);
                    // rows 0..31 hold the first two diagonal blocks, the right half of rows 32..63 the others
                    if (!is_y && (quad == 0 || cb0 == 2)) mbar_arrive(&bar[B_DIAG + quad * 2 + (cc & 1)]);
                    if (quad != 0) mbar_arrive(&bar[B_BLK + (cc & 1)]);
                }
        }
    } else if (warp < 12) {
        // -------------------------------------------------------------------- T's diagonal blocks, two a warp
        // Lane l row l mod 16 of one.  From T (I + A) = I, t_j = -A_rj - sum_{j < k < r} t_k A_kj, for falling k
        for (; take(sm, bar, at, j, ok); at.next()) {
                const int cc = at.cc;
                uint8_t *blocks = sm + OFF_A + (cc & 1) * kBlocks;
                const float *diag = reinterpret_cast<const float *>(blocks + 6 * 1024);
                wwait(&bar[B_DIAG + quad + (cc & 1)], (cc / 2) & 1, ok);
                {
                    const int r = lane & 15, b0 = quad * 16 + (lane & 16);
                    f2 t[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 v = *reinterpret_cast<const float4 *>(diag + diag_at(b0 + r, q));
                        t[2 * q] = pair(-v.x, -v.y);
                        t[2 * q + 1] = pair(-v.z, -v.w);
                    }
#pragma unroll
                    for (int k = 14; k >= 1; --k) {
                        const float2 v = parts(t[k >> 1]);
                        const float tk = k < r ? ((k & 1) ? -v.y : -v.x) : 0.f;
                        const f2 n = pair(tk, tk);
#pragma unroll
                        for (int q = 0; 4 * q < k; ++q) {  // row k of A is zero from column k on
                            const ulonglong2 v4 = *reinterpret_cast<const ulonglong2 *>(diag + diag_at(b0 + k, q));
                            t[2 * q] = fma2(n, v4.x, t[2 * q]);
                            if (4 * q + 2 < k) t[2 * q + 1] = fma2(n, v4.y, t[2 * q + 1]);
                        }
                    }
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 v = parts(t[j]);
                        split2(pair(2 * j < r ? v.x : 2 * j == r ? 1.f : 0.f, 2 * j + 1 < r ? v.y : 2 * j + 1 == r ? 1.f : 0.f), hi[j], lo[j]);
                    }
                    __syncwarp();  // the block has been read: T's takes its place
                    uint8_t *to = blocks + (6 + (b0 >> 4)) * 1024;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        *reinterpret_cast<uint4 *>(to + blk(r, q)) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                        *reinterpret_cast<uint4 *>(to + 512 + blk(r, q)) = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_BLK + (cc & 1)]);
        }
    } else if (warp < 16) {
        // -------------------------------------------------------------------- the rest of T, T', T''
        const uint32_t tt = smem_u32(sm + OFF_T);
        const uint32_t lane_at = blk((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
        for (; take(sm, bar, at, j, ok); at.next()) {
                const int cc = at.cc, kq = at.kq;
                const float *sc = reinterpret_cast<const float *>(sm + OFF_SC + kq * kGates);
                uint8_t *blocks = sm + OFF_A + (cc & 1) * kBlocks;
                const uint32_t base = smem_u32(blocks) + lane_at;
                // blocks: A10 0, A20 1, A21 2, A30 3, A31 4, A32 5, T00 6, T11 7, T22 8, T33 9.
                // By blocks of 32, T21 = -T22 A21 T11: two warps take the two inner blocks T10 and T32 (into the
                // places of A10 and A32) and the right half of T21, two its left half
                wwait(&bar[B_BLK + (cc & 1)], (cc / 2) & 1, ok);
                float t0[2][4] = {}, t1[2][4] = {};
                {
                    float a[2][4] = {}, b[2][4] = {};
                    Frag f, n;
                    load_left(base + (quad == 0 ? 7 : quad == 2 ? 8 : 9) * 1024, f);
                    mul_block(a, f.hi, f.lo, base + (quad == 0 ? 0 : quad == 1 ? 5 : quad == 2 ? 1 : 3) * 1024);
                    if (quad < 2) {
                        to_left_neg(a, n);
                        mul_block(t0, n.hi, n.lo, base + (quad == 0 ? 6 : 8) * 1024);  // T10 = -T11 A10 T00, T32 = -T33 A32 T22
                        put_plain(base + (quad == 0 ? 0 : 5) * 1024, t0);
                        if (quad == 0) load_left(base + 8 * 1024, f);
                        mul_block(b, f.hi, f.lo, base + (quad == 0 ? 2 : 4) * 1024);   // T22 A21; T33 A31 of T32 A21 + T33 A31
                    } else {
                        mul_block(b, f.hi, f.lo, base + (quad == 2 ? 2 : 4) * 1024);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[B_MID]);
                    wwait(&bar[B_MID], cc & 1, ok);
                    if (quad & 1) {
                        load_left(base + 5 * 1024, f);
                        mul_block(b, f.hi, f.lo, base + 2 * 1024);
                        if (quad == 3) mul_block(a, f.hi, f.lo, base + 1 * 1024);
                    }
                    to_left_neg(b, n);
                    mul_block(t1, n.hi, n.lo, base + (quad < 2 ? 7 : 0) * 1024);  // T21, T31: times T11; the left half's: T10
                    if (quad >= 2) {
                        to_left_neg(a, n);
                        mul_block(t1, n.hi, n.lo, base + 6 * 1024);
                        diag_block(base + (quad == 2 ? 8 : 9) * 1024, t0);
                    }
                }
                if (cc > 0) wwait(&bar[B_TFREE], (cc - 1) & 1, ok);
                // quad 0: T10, T21, T00; 1: T32, T31, T11; 2: T22, T20; 3: T33, T30
#pragma unroll 1
                for (int w = 0; w < (quad < 2 ? 3 : 2); ++w) {
                    const int bi = w == 0 ? (quad == 0 ? 1 : quad == 1 ? 3 : quad) : w == 1 ? 2 + (quad & 1) : quad;
                    const int bj = w == 0 ? (quad == 0 ? 0 : quad == 1 ? 2 : quad) : w == 1 ? (quad < 2 ? 1 : 0) : quad;
                    put_block(tt, sc, bi, bj, lane, t0);
                    if (w == 0) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) t0[e >> 2][e & 3] = t1[e >> 2][e & 3];
                    } else {
                        diag_block(base + (6 + quad) * 1024, t0);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar[B_T]);
                    mbar_arrive(&bar[B_SCFREE + kq]);
                    mbar_arrive(&bar[B_BLKFREE + (cc & 1)]);
                }
        }
    } else if (warp < 20) {
        // -------------------------------------------------------------------- W to shared memory, outputs
        const int row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        auto factors = [&](int cc, int kq) {  // S Q^T times scale e^gamma, in place, before U^T Y^T is added
            const float *eg = reinterpret_cast<const float *>(sm + OFF_SC + kq * kGates) + SC_EG;
            wwait(&bar[B_SQ], cc & 1, ok);
            tc_fence_after();
#pragma unroll 1
            for (int j0 = 0; j0 < 64; j0 += 16) {
                uint32_t r[16];
                tmem_ld16_nowait(tmem + lanes + TM_O + j0, r);
                tmem_wait_ld_into(r);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(eg + j0 + j);
                    unpair(mul2(e.x, pair(r[j], r[j + 1])), r[j], r[j + 1]);
                    unpair(mul2(e.y, pair(r[j + 2], r[j + 3])), r[j + 2], r[j + 3]);
                }
                tmem_st16(tmem + lanes + TM_O + j0, r);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B_SQRD]);
        };
        auto outputs = [&](int cc, int tok, int nv, int h) {
            wwait(&bar[B_O], cc & 1, ok);
            tc_fence_after();
            uint16_t *dst = reinterpret_cast<uint16_t *>(p.o) + ((int64_t)tok * p.hv_n + h) * kD + row;
            const int64_t step = (int64_t)p.hv_n * kD;
#pragma unroll 1
            for (int j0 = 0; j0 < 64; j0 += 16) {
                uint32_t r[16];
                tmem_ld16_nowait(tmem + lanes + TM_O + j0, r);
                tmem_wait_ld_into(r);
                if (j0 == 48) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[B_OFREE]);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const uint32_t w = pack_bf16(__uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                    if (j0 + j < nv) dst[0] = (uint16_t)w;
                    if (j0 + j + 1 < nv) dst[step] = (uint16_t)(w >> 16);
                    dst += 2 * step;
                }
            }
        };
        int loads = 0;
        int p_tok = 0, p_nv = 0, p_h = 0;  // the chunk before, whose outputs are still to come
        for (bool more = true; more; at.next()) {
            more = take(sm, bar, at, j, ok);
            if (!__all_sync(0xffffffffu, ok)) break;
            const int cc = at.cc;
            bool w_first = false;
            if (more) {
                if (cc > 0) wwait(&bar[B_U], (cc - 1) & 1, ok);  // the chunk before has its U: V and W have been read
                if (warp == 16 && lane == 0 && ok) {
                    ++loads;
                    mbar_arrive_expect_tx(&bar[B_VFULL], 2 * kTile);
                    for (int half = 0; half < 2; ++half)
                        tma_load_3d(sm + OFF_V + half * kTile, &tmV, &bar[B_VFULL], half * 64, j.h, j.tok);
                }
                __syncwarp();
                w_first = __shfl_sync(0xffffffffu, mbar_test_wait(&bar[B_W], cc & 1), 0);
            }
            // W of this chunk and the factors of the one before: what is there first
#pragma unroll 1
            for (int step = 0; step < 2; ++step) {
                if ((step == 0) != w_first) {
                    if (OUT && cc > 0) factors(cc - 1, at.kq == 0 ? kKQ - 1 : at.kq - 1);
                } else if (more) {
                    wwait(&bar[B_W], cc & 1, ok);
                    tc_fence_after();
                    uint8_t *wt = sm + OFF_W;
#pragma unroll 1
                    for (int j0 = 0; j0 < 64; j0 += 16) {
                        uint32_t r[16];
                        tmem_ld16_nowait(tmem + lanes + TM_W + j0, r);
                        tmem_wait_ld_into(r);
                        uint32_t hi[8], lw[8];
#pragma unroll
                        for (int j = 0; j < 16; j += 2) split2(pair(r[j], r[j + 1]), hi[j / 2], lw[j / 2]);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t off = sw(row, j0 / 8 + q);
                            *reinterpret_cast<uint4 *>(wt + off) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                            *reinterpret_cast<uint4 *>(wt + 2 * kTile + off) = make_uint4(lw[4 * q], lw[4 * q + 1], lw[4 * q + 2], lw[4 * q + 3]);
                        }
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[B_WRDY]);
                }
            }
            if (OUT && cc > 0) outputs(cc - 1, p_tok, p_nv, p_h);
            p_tok = j.tok;
            p_nv = j.nv;
            p_h = j.h;
        }
        if (loads > 0) mbar_wait(&bar[B_VFULL], (loads - 1) & 1, 1u << 16);  // landed, read or not
    } else {
        // -------------------------------------------------------------------- the state
        const int row = quad * 32 + lane, half = (warp - 20) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const int64_t mine = row * kD + half * 64;
        for (; take(sm, bar, at, j, ok); at.next()) {
            const int cc = at.cc, kq = at.kq;
            const bool zero = (j.flags & kFirst) && !j.from && (OUT || !(j.flags & kUnit));  // nothing to split, nor to add to
            if (zero) {
            } else if (j.flags & kFirst) {
                // S into tensor memory, whose last reader was this thread
#pragma unroll 1
                for (int i = 0; i < 64; i += 32) {
                    f2 v[4][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        load8(j.from ? j.from + mine + i + 8 * q : nullptr, v[q]);
                        if (!OUT && (j.flags & kUnit) && (row >> 3) == (half * 64 + i) / 8 + q) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (((row & 7) >> 1) == e) v[q][e] = (row & 1) ? pair(0.f, 1.f) : pair(1.f, 0.f);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t r[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) unpair(v[q][e], r[2 * e], r[2 * e + 1]);
                        tmem_st8(lanes + TM_DS + half * 64 + i + 8 * q, r);
                    }
                }
                tmem_wait_st();
            } else {
                wwait(&bar[B_UPD], (cc - 1) & 1, ok);  // the chunk before is in the sum, and U' has been read
            }
                const float *sc = reinterpret_cast<const float *>(sm + OFF_SC + kq * kGates) + half * 32;
                tc_fence_after();
                // S as hi + lo, and its sum times e^gamma_63, ready for dS
                const f2 decay = pair(el[cc & (kDecays - 1)], el[cc & (kDecays - 1)]);
#pragma unroll 1
                for (int j0 = 0; !zero && j0 < 64; j0 += 8) {
                    uint32_t r[8], hi[4], lw[4];
                    tmem_ld8_nowait(lanes + TM_DS + half * 64 + j0, r);
                    tmem_wait_ld_into(r);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const f2 v = pair(r[e], r[e + 1]);
                        split2(v, hi[e / 2], lw[e / 2]);
                        unpair(mul2(v, decay), r[e], r[e + 1]);
                    }
                    tmem_st4(lanes + TM_SHI + half * 32 + j0 / 2, hi);
                    tmem_st4(lanes + TM_SLO + half * 32 + j0 / 2, lw);
                    tmem_st8(lanes + TM_DS + half * 64 + j0, r);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_S]);

                wwait(&bar[B_U], cc & 1, ok);
                tc_fence_after();
#pragma unroll 1
                for (int j0 = 0; j0 < 32; j0 += 16) {
                    uint32_t r[16], hi[8], lw[8];
                    tmem_ld16_nowait(lanes + TM_U + half * 32 + j0, r);
                    tmem_wait_ld_into(r);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(sc + SC_FD + j0 + j);
                        split2(mul2(pair(r[j], r[j + 1]), f.x), hi[j / 2], lw[j / 2]);
                        split2(mul2(pair(r[j + 2], r[j + 3]), f.y), hi[j / 2 + 1], lw[j / 2 + 1]);
                    }
                    if (OUT && j0 == 0) {  // S lo has been read
                        wwait(&bar[B_SL], cc & 1, ok);
                        tc_fence_after();
                    }
                    tmem_st8(lanes + TM_UHI + half * 16 + j0 / 2, hi);
                    tmem_st8(lanes + TM_ULO + half * 16 + j0 / 2, lw);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_UST]);
            if (!(j.flags & kLast)) continue;
            wwait(&bar[B_UPD], cc & 1, ok);
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; j.to && i < 64; i += 16) {
                uint32_t r[16];
                tmem_ld16_nowait(lanes + TM_DS + half * 64 + i, r);
                tmem_wait_ld_into(r);
                f2 v[4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = pair(r[8 * q + 2 * e], r[8 * q + 2 * e + 1]);
                    store8(j.to + mine + i + 8 * q, v);
                }
            }
        }
    }
    if (!ok) flag(p.status, GDN_DEV_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, 512);
}

// The states before the segments of prompts that have several, in place of the first pass's: S before segment s + 1
// is S_s M_s + L_s, in fp32.  A block takes R rows of one (request, head).  M comes to shared memory a step ahead, as
// it does not depend on the chain; each of the eight warps takes 16 rows of M, so that M is read there once, and the
// warps' sums are added up over M's place.
constexpr int join_smem(int rows) { return (2 * kD * kD + rows * kD) * 4; }
template <int R>
__global__ void __launch_bounds__(256) prefill_join_kernel(Params p) {
    extern __shared__ __align__(16) float join[];
    float *S = join + 2 * kD * kD;  // [R][kD]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = blockIdx.x % (kD / R), item = blockIdx.x / (kD / R), h = item % p.hv_n, b = item / p.hv_n;
    const int lo = __ldg(p.offsets + b), hi = __ldg(p.offsets + b + 1), slot = p.slots ? __ldg(p.slots + b) : b;
    const int n = lo >= 0 && hi >= lo && hi <= p.total ? hi - lo : 0;
    if (n <= p.seg0 || n > p.max_tokens || slot < 0 || slot >= p.n_states) return;
    const int segs = 1 + (n - p.seg0 + p.seg - 1) / p.seg;
    float *ws = p.ws + (int64_t)item * (2 * p.segs - 2) * (kD * kD);
    auto fetch = [&](int s) {
        if (s < segs - 1) {
            const float *M = ws + (int64_t)(p.segs + s - 1) * (kD * kD);
            const uint32_t to = smem_u32(join + (s & 1) * kD * kD);
#pragma unroll
            for (int i = tid * 4; i < kD * kD; i += 1024)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 4), "l"(M + i) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(1);
    const bool zero = !p.S0 || (p.fresh && __ldg(p.fresh + b) != 0);
    const float *S0 = p.S0 + ((int64_t)slot * p.hv_n + h) * (kD * kD);
    const int64_t rows = (int64_t)part * R * kD;
#pragma unroll
    for (int i = tid * 4; i < R * kD; i += 1024) {
        // the final state may go to S0's place while segment 0 runs
        *reinterpret_cast<float4 *>(ws + rows + i) = zero ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4 *>(S0 + rows + i);
        *reinterpret_cast<float4 *>(S + i) = *reinterpret_cast<const float4 *>(ws + kD * kD + rows + i);
    }
    for (int s = 1; s < segs - 1; ++s) {
        float *L = ws + (int64_t)(s + 1) * (kD * kD) + rows, *M = join + (s & 1) * kD * kD;
        float4 x[R / 8];
#pragma unroll
        for (int i = 0; i < R / 8; ++i) x[i] = *reinterpret_cast<const float4 *>(L + tid * 4 + i * 1024);
        fetch(s + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        f2 acc[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = 0;
#pragma unroll 1
        for (int k = warp * 16; k < warp * 16 + 16; k += 4) {
            ulonglong2 m[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = *reinterpret_cast<const ulonglong2 *>(M + (k + e) * kD + lane * 4);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 v = *reinterpret_cast<const float4 *>(S + r * kD + k);
                const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[r][0] = fma2(pair(y[e], y[e]), m[e].x, acc[r][0]);
                    acc[r][1] = fma2(pair(y[e], y[e]), m[e].y, acc[r][1]);
                }
            }
        }
        __syncthreads();  // M has been read
#pragma unroll
        for (int r = 0; r < R; ++r) *reinterpret_cast<ulonglong2 *>(M + (warp * R + r) * kD + lane * 4) = make_ulonglong2(acc[r][0], acc[r][1]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < R / 8; ++i) {
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(M + w * R * kD + tid * 4 + i * 1024);
                x[i] = make_float4(x[i].x + y.x, x[i].y + y.y, x[i].z + y.z, x[i].w + y.w);
            }
            *reinterpret_cast<float4 *>(L + tid * 4 + i * 1024) = x[i];
            *reinterpret_cast<float4 *>(S + tid * 4 + i * 1024) = x[i];
        }
        __syncthreads();  // the sums have been read: the M after the next may come
    }
}


// [T][H][128] bf16 tokens `stride` elements apart as a 3-D tensor (d, head, token); boxes of 64 x 1 x 64,
// 128-byte swizzle
bool encode(CUtensorMap *map, const void *base, int heads, int total, int64_t stride) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)heads, (cuuint64_t)total};
    cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)kC};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

int64_t token_stride(int64_t given, int heads) { return given ? given : (int64_t)heads * kD; }

}  // namespace

bool prefill_tc_supported(const gdn_prefill_args &a) {
    const int64_t qs = token_stride(a.q_stride, a.n_k_heads), ks = token_stride(a.k_stride, a.n_k_heads),
                  vs = token_stride(a.v_stride, a.n_v_heads);
    return a.qkv_dtype == GDN_BF16 && a.out_dtype == GDN_BF16 && a.d_k == kD && a.d_v == kD && a.total_tokens > 0 &&
           tiles::aligned16(a.q) && tiles::aligned16(a.k) && tiles::aligned16(a.v) && aligned32(a.S0) &&
           aligned32(a.S_new) && qs % 8 == 0 && ks % 8 == 0 && vs % 8 == 0 && std::max(qs, std::max(ks, vs)) < (1ll << 38) &&
           (int64_t)a.batch * a.n_v_heads <= 0x7fffffff - 65536 && a.n_v_heads <= 65535 && tensor_map_encoder() != nullptr;
}

// How many segments a prompt is cut into (1: none), and their lengths.  In units of a chunk's time on a full GPU (4.2 us;
// with few blocks running it is down to 0.72 of that): a pass takes L + 3 for a wave of blocks with segments of L chunks,
// the first pass 0.7 of that; a join step takes 0.4, the launches 3.  The first pass has an item for each first segment
// and two for each inner one: where it would leave a few first segments over, these are made a half or a third as long,
// and two or three of them go one after the other beside the inner ones.  One prompt of 16384 tokens with 32 heads:
// 842 us in one piece, with 2, 3, 4, 6, 8, 16 equal segments 795, 571, 622, 643, 658, 790 (all at one build); 565 with
// three and 504 with four, the first of them of half the length (at a later one).
int plan_segments(const gdn_prefill_args &a, int &seg0, int &seg) {
    const int64_t sms = sm_count(), items = (int64_t)a.batch * a.n_v_heads;
    const int64_t chunks = std::max<int64_t>(1, ((int64_t)std::min(a.max_tokens, a.total_tokens) + kC - 1) / kC);
    // time of `count` items of `len`, then `count0` shorter ones of `len0`
    auto pass = [&](double count, double len, double count0, double len0) {
        const double full = std::floor(count / sms), rest = count - full * sms;
        double t = full * len;
        if (rest > 0) {
            count0 -= (sms - std::ceil(rest)) * std::floor(len / len0);
            t += len;
        }
        t += std::ceil(std::max(0.0, count0) / sms) * len0;
        return t;
    };
    auto speed = [&](double blocks) { return 0.715 + 0.285 * std::min(1.0, blocks / sms); };
    double best = 0.9 * pass((double)items, (double)chunks + 3, 0, 1) * speed((double)items);  // worth a tenth at least
    int segs = 1;
    seg0 = seg = (int)std::min<int64_t>(chunks * kC, 0x7fffffc0);
    for (int64_t s = 2; s <= std::min<int64_t>(chunks, 128) && items < sms && items * (2 * s - 3) <= 6 * sms; ++s) {
        for (int part = 1; part <= 3; ++part) {
            // len0 + 3 = (len + 3) / part and len0 + (s - 1) len = chunks, as far as whole chunks go
            const int64_t len = (part * (chunks + 3) - 3 + part * (s - 1)) / (part * (s - 1) + 1), len0 = chunks - (s - 1) * len;
            if (len0 < 1) continue;
            // segments that have tokens: those of every prompt, or as many as all the tokens fill
            const double pieces = std::min<double>((double)a.batch * s, (double)a.total_tokens / (len * kC) + a.batch) * a.n_v_heads;
            const double inner = std::max(0.0, pieces - 2 * items), more = std::max(0.0, pieces - items);
            const double firsts = std::min((double)items, more);
            const double cost = pass(more, (double)len + 3, (double)items, (double)len0 + 3) * speed(pieces) +
                                0.7 * pass(2 * inner, (double)len + 3, firsts, (double)len0 + 3) * speed(2 * inner + firsts) +
                                0.4 * (s - 2) + 3;
            if (cost < best) {
                best = cost;
                segs = (int)s;
                seg0 = (int)(len0 * kC);
                seg = (int)(len * kC);
            }
        }
    }
    return segs;
}

int64_t prefill_tc_workspace(const gdn_prefill_args &a) {
    int seg0, seg;
    const int segs = plan_segments(a, seg0, seg);
    return segs == 1 ? 0 : (int64_t)a.batch * a.n_v_heads * (2 * segs - 2) * (kD * kD * 4);
}

template <bool OUT>
cudaError_t launch_pass(const CUtensorMap &tmQ, const CUtensorMap &tmK, const CUtensorMap &tmV, Params p, int slices, cudaStream_t stream) {
    p.items = p.batch * p.hv_n * slices;
    // the longest first, so that the blocks end together: 256 us for 64 prompts of 16 to 512 tokens, in their own order 267 (at
    // one build)
    p.sorted = slices == 1 && p.batch > 1 && p.batch <= kSorted && p.items > sm_count();
    static int have[16];
    cudaError_t e = ensure_smem(prefill_tc_kernel<OUT>, kSmem, have);
    if (e != cudaSuccess) return e;
    prefill_tc_kernel<OUT><<<(unsigned)p.items, kThreads, kSmem, stream>>>(tmQ, tmK, tmV, p);
    return cudaGetLastError();
}

template <int R>
cudaError_t launch_join(const Params &p, cudaStream_t stream) {
    static int have[16];
    cudaError_t e = ensure_smem(prefill_join_kernel<R>, join_smem(R), have);
    if (e != cudaSuccess) return e;
    prefill_join_kernel<R><<<(unsigned)(p.batch * p.hv_n * (kD / R)), 256, join_smem(R), stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_prefill_tc(const gdn_prefill_args &a, cudaStream_t stream) {
    CUtensorMap tmQ, tmK, tmV;
    if (!encode(&tmQ, a.q, a.n_k_heads, a.total_tokens, token_stride(a.q_stride, a.n_k_heads)) ||
        !encode(&tmK, a.k, a.n_k_heads, a.total_tokens, token_stride(a.k_stride, a.n_k_heads)) ||
        !encode(&tmV, a.v, a.n_v_heads, a.total_tokens, token_stride(a.v_stride, a.n_v_heads)))
        return cudaErrorInvalidValue;
    Params p = {};
    p.hk_n = a.n_k_heads; p.hv_n = a.n_v_heads; p.total = a.total_tokens; p.max_tokens = a.max_tokens;
    p.n_states = a.n_states; p.batch = a.batch; p.probe = wait_probe_polls();
    const int group = a.n_v_heads / a.n_k_heads;
    p.group_inv = group == 1 ? 0u : (uint32_t)(((1ull << 32) + group - 1) / group);
    p.scale = a.scale;
    p.offsets = a.token_offsets; p.slots = a.slots; p.fresh = a.fresh;
    p.g = a.g; p.beta = a.beta; p.S0 = a.S0;
    p.o = static_cast<__nv_bfloat16 *>(a.o); p.S_new = a.S_new; p.ws = static_cast<float *>(a.workspace); p.status = a.dev_status;
    p.segs = plan_segments(a, p.seg0, p.seg);
    if (p.segs > 1) {
        cudaError_t e = launch_pass<false>(tmQ, tmK, tmV, p, 2 * p.segs - 3, stream);
        if (e != cudaSuccess) return e;
        e = p.batch * p.hv_n * 8 >= sm_count() ? launch_join<16>(p, stream) : launch_join<8>(p, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_pass<true>(tmQ, tmK, tmV, p, p.segs, stream);
}

}  // namespace gdn
