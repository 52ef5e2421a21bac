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
// (T', T'', W, S, U') enter as pairs hi + lo of bf16, x = hi + lo to 2^-17; lo x lo is left
// out (2^-18).  The state comes out about 5e-6 (norm-wise) from exact.  The output's own
// products take S, U and Y rounded once to bf16, like the output itself.
//
// One block an SM (all 512 tensor-memory columns), 20 warps:
//     warp 0        loads by TMA: K and Q of three chunks, V of two
//     warp 1        issues the Gram and W products, whichever is ready
//     warp 2        issues U, O and dS: the chain
//     warps 4-7     gates, A, T = (I + A)^-1 by blocks of 16, 32, 64 in fp32, T', T'', Y
//     warps 8-11    W to shared memory, the outputs to global memory
//     warps 12-19   the state in registers (a row of 64 entries each), its hi + lo operand in
//                   tensor memory, and U's
// The chain for a chunk is: S split -> S W^T -> U split -> dS -> S.
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
constexpr int kThreads = 640;  // 20 warps
constexpr int kKQ = 3, kV = 2, kRing = 3, kDecays = 8;

// shared memory (bytes from a 1024-aligned base)
constexpr int kTile = kC * 128;              // 64 rows of 128 bytes: half of a token tile
constexpr int OFF_KQ = 0;                    // [kKQ][2 halves of d][K, Q] tiles
constexpr int OFF_V = OFF_KQ + kKQ * 4 * kTile;  // [kV][2 halves] tiles
constexpr int OFF_T = OFF_V + kV * 2 * kTile;    // T' hi, lo, T'' hi, lo (negated): rows i, columns j
constexpr int OFF_W = OFF_T + 4 * kTile;     // W^T hi, lo: 128 rows of d_k, columns i
constexpr int OFF_Y = OFF_W + 4 * kTile;     // [2] Y: rows i, columns j
constexpr int OFF_A = OFF_Y + 2 * kTile;     // fp32 [64][64] A, then T
constexpr int OFF_SC = OFF_A + kC * kC * 4;  // fp32 gamma hi, lo, beta, beta e^gamma (of the chunk in work)
constexpr int OFF_RING = OFF_SC + 4 * kC * 4;    // [kRing] scale e^gamma, e^(gamma_63 - gamma)
constexpr int OFF_EL = OFF_RING + kRing * 2 * kC * 4;  // [kDecays] e^gamma_63
constexpr int OFF_SLOT = OFF_EL + kDecays * 4;
constexpr int OFF_BAR = OFF_SLOT + 16;
enum Bar {
    B_FULL = 0, B_EMPTY = B_FULL + kKQ, B_VFULL = B_EMPTY + kKQ, B_VEMPTY = B_VFULL + kV,
    B_G = B_VEMPTY + kV, B_GFREE, B_T, B_TFREE, B_W, B_WRDY, B_S, B_U, B_UST, B_UBF, B_SQ, B_SQRD, B_UPD, B_O, B_OFREE,
    B_PROBE, B_COUNT
};
constexpr int kSmem = OFF_BAR + B_COUNT * 8;
static_assert(kSmem <= 232448, "one block an SM");

// tensor-memory columns
constexpr uint32_t TM_DS = 0, TM_S = 128, TM_U = 256, TM_O = 320, TM_G = 384, TM_W = 448;
constexpr uint32_t TM_SHI = TM_S, TM_SLO = TM_S + 64;
// U' hi, lo lie over S lo (free once S W^T is done), U over S hi (free once S Q^T is done)
constexpr uint32_t TM_UHI = TM_SLO, TM_ULO = TM_SLO + 32, TM_UBF = TM_SHI;

struct Params {
    int hk_n, hv_n, total, max_tokens, n_states, items, probe;
    float scale;
    const int32_t *offsets, *slots, *fresh;
    const float *g, *beta, *S0;
    __nv_bfloat16 *o;
    float *S_new;
    int32_t *status;
};

struct Item {
    int h, hk, lo, n, chunks, err;
    int64_t state;  // first entry of its state in the pools
    bool zero;      // starts from zero
};

__device__ __forceinline__ Item item_of(const Params &p, int idx) {
    Item x;
    const int b = idx / p.hv_n;
    x.h = idx % p.hv_n;
    x.hk = x.h / (p.hv_n / p.hk_n);
    x.lo = __ldg(p.offsets + b);
    x.n = __ldg(p.offsets + b + 1) - x.lo;
    const int slot = p.slots ? __ldg(p.slots + b) : b;
    x.err = 0;
    if (x.n < 0 || x.lo < 0 || x.lo + x.n > p.total) x.err = GDN_DEV_BAD_DESC;
    else if (x.n > p.max_tokens) x.err = GDN_DEV_TOO_MANY;
    else if (slot < 0 || slot >= p.n_states) x.err = GDN_DEV_BAD_SLOT;
    x.zero = !p.S0 || (p.fresh && __ldg(p.fresh + b) != 0);
    x.state = ((int64_t)slot * p.hv_n + x.h) * (kD * kD);
    x.chunks = x.err ? 0 : (x.n + kC - 1) / kC;
    return x;
}

// Bounded wait; after a first one that ran out the others only look once, so that a block
// whose pipeline broke still ends soon.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, bool &ok) {
    if (!mbar_wait(bar, parity, ok ? (1u << 20) : 1u)) ok = false;
}

__device__ __forceinline__ uint32_t sw(int row, int chunk16) {  // byte offset in a tile of 128-byte rows
    return (uint32_t)(row * 128 + ((chunk16 ^ (row & 7)) << 4));
}

// hi + lo bf16 pairs of two values: packed hi, packed lo
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
}

// float index of (row, col) in the fp32 64 x 64 tile: 16-byte pieces permuted by the row, so that
// a piece of eight consecutive rows covers all banks
__device__ __forceinline__ int at(int row, int col) { return row * kC + ((((col >> 2) ^ (row & 7)) << 2) | (col & 3)); }

__device__ __forceinline__ float4 ld4(const float *a, int row, int col) {
    return *reinterpret_cast<const float4 *>(a + at(row, col));
}
__device__ __forceinline__ void st4(float *a, int row, int col, float4 v) { *reinterpret_cast<float4 *>(a + at(row, col)) = v; }

// sum of two double-floats
__device__ __forceinline__ void dd_add(float &ah, float &al, float bh, float bl) {
    const float s = __fadd_rn(ah, bh), t = __fsub_rn(s, ah);
    float e = __fadd_rn(__fsub_rn(ah, __fsub_rn(s, t)), __fsub_rn(bh, t));
    e = __fadd_rn(e, __fadd_rn(al, bl));
    ah = __fadd_rn(s, e);
    al = __fsub_rn(e, __fsub_rn(ah, s));
}

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
            const uint32_t n = i == B_GFREE || i == B_T || i == B_WRDY || i == B_SQRD || i == B_OFREE ? 4
                               : i == B_S || i == B_UST || i == B_UBF                               ? 8
                               : i == B_TFREE                                                       ? 2
                                                                                                    : 1;
            mbar_init(&bar[i], n);
        }
        fence_mbar_init();
    }
    // Y's tiles and A's upper blocks are zero above the diagonal blocks that are written
    for (int i = tid; i < (2 * kTile + kC * kC * 4) / 16; i += kThreads)
        *reinterpret_cast<uint4 *>(sm + OFF_Y + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    if (warp == 2) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    bool ok = true;

    if (warp < 4) {
        reg_dealloc<40>();
        if (warp == 0 && lane == 0) {
            // ---------------------------------------------------------------- loads
            if (p.probe > 0) ok = mbar_wait(&bar[B_PROBE], 0, (uint32_t)p.probe);
            bool go = true;  // the pipeline's own waits
            int cc = 0, kq = 0, n_kq = 0, n_v = 0;
            for (int idx = blockIdx.x; idx < p.items && go; idx += gridDim.x) {
                const Item x = item_of(p, idx);
                if (x.err) flag(p.status, x.err);
                for (int c = 0; c < x.chunks; ++c, ++cc, kq = kq + 1 == kKQ ? 0 : kq + 1) {
                    const int row = x.lo + c * kC, v = cc & 1;
                    uint8_t *dst = sm + OFF_KQ + kq * 4 * kTile;
                    if (cc >= kKQ) wait(&bar[B_EMPTY + kq], (cc / kKQ - 1) & 1, go);
                    if (!go) break;  // nothing is loaded over a stage that may be in use
                    ++n_kq;
                    mbar_arrive_expect_tx(&bar[B_FULL + kq], 4 * kTile);
                    for (int half = 0; half < 2; ++half) {
                        tma_load_3d(dst + half * 2 * kTile, &tmK, &bar[B_FULL + kq], half * 64, x.hk, row);
                        tma_load_3d(dst + half * 2 * kTile + kTile, &tmQ, &bar[B_FULL + kq], half * 64, x.hk, row);
                    }
                    if (cc >= kV) wait(&bar[B_VEMPTY + v], (cc / kV - 1) & 1, go);
                    if (!go) break;
                    ++n_v;
                    mbar_arrive_expect_tx(&bar[B_VFULL + v], 2 * kTile);
                    for (int half = 0; half < 2; ++half)
                        tma_load_3d(sm + OFF_V + (v * 2 + half) * kTile, &tmV, &bar[B_VFULL + v], half * 64, x.h, row);
                }
            }
            // every load has landed before the block ends, whatever became of its reader
            for (int i = 0; i < kKQ && i < n_kq; ++i) mbar_wait(&bar[B_FULL + i], ((n_kq - 1 - i) / kKQ) & 1, 1u << 16);
            for (int i = 0; i < kV && i < n_v; ++i) mbar_wait(&bar[B_VFULL + i], ((n_v - 1 - i) / kV) & 1, 1u << 16);
            ok = ok && go;
        } else if (warp == 1) {
            // ---------------------------------------------------------------- Gram and W products
            const uint32_t id_g = idesc_bf16_f32(128, kC), id_w = idesc_bf16_f32(128, kC) | (1u << 15);
            int idx = blockIdx.x, c = 0;  // the next Gram's item and chunk in it
            Item x;
            auto seek = [&]() {  // the first item from idx on that has chunks
                for (; idx < p.items; idx += gridDim.x) {
                    x = item_of(p, idx);
                    if (x.chunks > 0) break;
                }
            };
            seek();
            int gcc = 0, wcc = 0, gkq = 0, wkq = 0;
            for (uint32_t idle = 0; idx < p.items || wcc < gcc;) {
                bool g = false, w = false;
                if (lane == 0) {
                    g = idx < p.items && mbar_test_wait(&bar[B_FULL + gkq], (gcc / kKQ) & 1) &&
                        (gcc == 0 || mbar_test_wait(&bar[B_GFREE], (gcc - 1) & 1));
                    w = wcc < gcc && mbar_test_wait(&bar[B_T], wcc & 1) &&
                        (wcc == 0 || mbar_test_wait(&bar[B_WRDY], (wcc - 1) & 1));
                }
                g = __shfl_sync(0xffffffffu, g, 0);
                w = __shfl_sync(0xffffffffu, w, 0);
                if (w) {
                    if (lane == 0) {
                        tc_fence_after();
                        const uint8_t *kt = sm + OFF_KQ + wkq * 4 * kTile;
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_bf16(tmem + TM_W, smem_desc(smem_u32(kt + ks * 2048), 2 * kTile, 1024, 2),
                                         smem_desc(smem_u32(sm + OFF_T + (2 + part) * kTile + ks * 32), 16, 1024, 2), id_w,
                                         part > 0 || ks > 0);
                        mma_commit(&bar[B_W]);
                        mma_commit(&bar[B_TFREE]);
                    }
                    ++wcc;
                    wkq = wkq + 1 == kKQ ? 0 : wkq + 1;
                }
                if (g) {
                    wait(&bar[B_FULL + gkq], (gcc / kKQ) & 1, ok);  // complete: every lane sees the tile
                    uint8_t *kt = sm + OFF_KQ + gkq * 4 * kTile;
                    const int nv = x.n - c * kC;
                    if (nv < kC) {  // keys past the prompt's end: zero, whatever the next prompt holds
                        for (int half = 0; half < 2; ++half)
                            for (int i = nv * 8 + lane; i < kC * 8; i += 32)
                                *reinterpret_cast<uint4 *>(kt + half * 2 * kTile + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint64_t d = smem_desc(smem_u32(kt + (ks >> 2) * 2 * kTile + (ks & 3) * 32), 16, 1024, 2);
                            mma_bf16(tmem + TM_G, d, d, id_g, ks > 0);
                        }
                        mma_commit(&bar[B_G]);
                    }
                    ++gcc;
                    gkq = gkq + 1 == kKQ ? 0 : gkq + 1;
                    if (++c == x.chunks) {
                        c = 0;
                        idx += gridDim.x;
                        seek();
                    }
                }
                idle = g || w ? 0 : idle + 1;
                if (idle > (1u << 22)) {
                    ok = false;
                    break;
                }
            }
        } else if (warp == 2) {
            // ---------------------------------------------------------------- the chain's products
            const uint32_t id_u = idesc_bf16_f32(128, kC) | (1u << 15);  // V^T (MN-major) T'^T
            const uint32_t id_sw = idesc_bf16_f32(128, kC) | (1u << 16); // S (tensor memory) W^T, W MN-major
            const uint32_t id_k = idesc_bf16_f32(128, kC);               // K-major right-hand side
            const uint32_t id_ds = idesc_bf16_f32(128, kD) | (1u << 16); // U' K, K MN-major
            int cc = 0, kq = 0;
            for (int idx = blockIdx.x; idx < p.items; idx += gridDim.x) {
                const Item x = item_of(p, idx);
                for (int c = 0; c < x.chunks; ++c, ++cc, kq = kq + 1 == kKQ ? 0 : kq + 1) {
                    const int v = cc & 1;
                    uint8_t *kt = sm + OFF_KQ + kq * 4 * kTile, *vt = sm + OFF_V + v * 2 * kTile;
                    wait(&bar[B_VFULL + v], (cc / kV) & 1, ok);
                    const int nv = x.n - c * kC;
                    if (nv < kC) {
                        for (int half = 0; half < 2; ++half)
                            for (int i = nv * 8 + lane; i < kC * 8; i += 32)
                                *reinterpret_cast<uint4 *>(vt + half * kTile + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        // U^T = V^T T'^T
                        wait(&bar[B_T], cc & 1, ok);
                        tc_fence_after();
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_bf16(tmem + TM_U, smem_desc(smem_u32(vt + ks * 2048), kTile, 1024, 2),
                                         smem_desc(smem_u32(sm + OFF_T + part * kTile + ks * 32), 16, 1024, 2), id_u,
                                         part > 0 || ks > 0);
                        mma_commit(&bar[B_TFREE]);
                        mma_commit(&bar[B_VEMPTY + v]);
                        // U^T += S (-W)^T: hi hi, lo hi, hi lo
                        wait(&bar[B_WRDY], cc & 1, ok);
                        wait(&bar[B_S], cc & 1, ok);
                        tc_fence_after();
#pragma unroll
                        for (int part = 0; part < 3; ++part)
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)
                                mma_bf16_ts(tmem + TM_U, tmem + (part == 1 ? TM_SLO : TM_SHI) + ks * 8,
                                            smem_desc(smem_u32(sm + OFF_W + (part == 2 ? 2 * kTile : 0) + ks * 2048), kTile, 1024, 2),
                                            id_sw, true);
                        mma_commit(&bar[B_U]);
                        // O^T = S Q^T
                        if (cc > 0) wait(&bar[B_OFREE], (cc - 1) & 1, ok);
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_bf16_ts(tmem + TM_O, tmem + TM_SHI + ks * 8,
                                        smem_desc(smem_u32(kt + kTile + (ks >> 2) * 2 * kTile + (ks & 3) * 32), 16, 1024, 2), id_k, ks > 0);
                        mma_commit(&bar[B_SQ]);
                        // dS = U'^T K
                        wait(&bar[B_UST], cc & 1, ok);
                        tc_fence_after();
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_bf16_ts(tmem + TM_DS, tmem + (part ? TM_ULO : TM_UHI) + ks * 8,
                                            smem_desc(smem_u32(kt + ks * 2048), 2 * kTile, 1024, 2), id_ds, part > 0 || ks > 0);
                        mma_commit(&bar[B_UPD]);
                        // O^T of the chunk's own tokens = U^T Y^T, once S Q^T has been read
                        wait(&bar[B_UBF], cc & 1, ok);
                        wait(&bar[B_SQRD], cc & 1, ok);
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_bf16_ts(tmem + TM_O, tmem + TM_UBF + ks * 8,
                                        smem_desc(smem_u32(sm + OFF_Y + (cc & 1) * kTile + ks * 32), 16, 1024, 2), id_k, ks > 0);
                        mma_commit(&bar[B_O]);
                        mma_commit(&bar[B_EMPTY + kq]);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp < 8) {
        // -------------------------------------------------------------------- gates, A, T, T', T'', Y
        reg_dealloc<88>();
        float *A = reinterpret_cast<float *>(sm + OFF_A);
        float *ghi = reinterpret_cast<float *>(sm + OFF_SC), *glo = ghi + kC, *sbeta = ghi + 2 * kC, *sbg = ghi + 3 * kC;
        float *el = reinterpret_cast<float *>(sm + OFF_EL);
        const int t128 = tid - 128, row = quad * 32 + lane, i = row & 63;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        int cc = 0, ring = 0;
        for (int idx = blockIdx.x; idx < p.items; idx += gridDim.x) {
            const Item x = item_of(p, idx);
            float pg[2] = {0.f, 0.f}, pb[2] = {0.f, 0.f};  // g and beta of tokens 2 lane, 2 lane + 1 of the next chunk
            auto fetch = [&](int c) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = c * kC + 2 * lane + e;
                    pg[e] = pb[e] = 0.f;
                    if (t < x.n) {
                        pg[e] = __ldg(p.g + (int64_t)(x.lo + t) * p.hv_n + x.h);
                        pb[e] = __ldg(p.beta + (int64_t)(x.lo + t) * p.hv_n + x.h);
                    }
                }
            };
            if (quad == 0 && x.chunks > 0) fetch(0);
            for (int c = 0; c < x.chunks; ++c, ++cc, ring = ring + 1 == kRing ? 0 : ring + 1) {
                wait(&bar[B_G], cc & 1, ok);
                tc_fence_after();
                if (quad == 0) {
                    // gamma: a scan in pairs of floats, so that a decay that forgets everything leaves the
                    // differences after it exact.  e^-200 is zero, whatever lies below it
                    const float g0 = pg[0] < -200.f ? -200.f : pg[0], g1 = pg[1] < -200.f ? -200.f : pg[1];
                    float h = g0, l = 0.f;
                    dd_add(h, l, g1, 0.f);
#pragma unroll
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
                    float *rg = reinterpret_cast<float *>(sm + OFF_RING) + ring * 2 * kC;
                    const float hh[2] = {h0, h}, lw[2] = {l0, l};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = 2 * lane + e;
                        const float eg = expf(hh[e] + lw[e]);
                        ghi[t] = hh[e];
                        glo[t] = lw[e];
                        sbeta[t] = pb[e];
                        sbg[t] = pb[e] * eg;
                        rg[t] = p.scale * eg;
                        rg[kC + t] = expf((hl - hh[e]) + (ll - lw[e]));
                    }
                    if (lane == 0) el[cc & (kDecays - 1)] = expf(hl + ll);
                    if (c + 1 < x.chunks) fetch(c + 1);
                }
                named_sync(1, 128);
                const float gh = ghi[i], gl = glo[i], f = row < 64 ? sbeta[i] : p.scale;
                const int cols = (quad & 1) ? 64 : 32;  // rows 0..31 have nothing right of column 31
                uint32_t y[32];
#pragma unroll
                for (int j0 = 0; j0 < 64; j0 += 16) {
                    if (j0 < cols) {
                        uint32_t r[16];
                        tmem_ld16_nowait(tmem + lanes + TM_G + j0, r);
                        tmem_wait_ld_into(r);
                        float m[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int jj = j0 + j;
                            const float d = f * __expf((gh - ghi[jj]) + (gl - glo[jj]));
                            m[j] = jj < i + (row >> 6) ? d * __uint_as_float(r[j]) : 0.f;
                        }
                        if (row < 64) {
#pragma unroll
                            for (int j = 0; j < 16; j += 4) st4(A, i, j0 + j, make_float4(m[j], m[j + 1], m[j + 2], m[j + 3]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; j += 2) y[(j0 + j) >> 1] = pack_bf16(m[j], m[j + 1]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_GFREE]);
                if (row >= 64) {
                    if (cc >= 2) wait(&bar[B_O], (cc - 2) & 1, ok);
                    uint8_t *yt = sm + OFF_Y + (cc & 1) * kTile;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (q * 8 < cols)
                            *reinterpret_cast<uint4 *>(yt + sw(i, q)) = make_uint4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
                }
                named_sync(1, 128);
                // T, diagonal blocks of 16: warp w block w, lane r < 16 row r.  From T (I + A) = I,
                // t_j = -A_rj - sum_{j < k < r} t_k A_kj, for falling j
                {
                    const int b0 = quad * 16, r = lane & 15;
                    float t[16];
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 a = ld4(A, b0 + r, b0 + j);
                        t[j] = -a.x; t[j + 1] = -a.y; t[j + 2] = -a.z; t[j + 3] = -a.w;
                    }
#pragma unroll
                    for (int k = 14; k >= 1; --k) {
                        const float tk = k < r ? t[k] : 0.f;
#pragma unroll
                        for (int j = 0; j < k; j += 4) {
                            const float4 a = ld4(A, b0 + k, b0 + j);
                            t[j] = fmaf(-tk, a.x, t[j]);
                            if (j + 1 < k) t[j + 1] = fmaf(-tk, a.y, t[j + 1]);
                            if (j + 2 < k) t[j + 2] = fmaf(-tk, a.z, t[j + 2]);
                            if (j + 3 < k) t[j + 3] = fmaf(-tk, a.w, t[j + 3]);
                        }
                    }
                    __syncwarp();
                    if (lane < 16) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) t[j] = j < r ? t[j] : j == r ? 1.f : 0.f;
#pragma unroll
                        for (int j = 0; j < 16; j += 4) st4(A, b0 + r, b0 + j, make_float4(t[j], t[j + 1], t[j + 2], t[j + 3]));
                    }
                }
                named_sync(1, 128);
                // blocks of 32: T21 = -T22 (A21 T11); the products A21 T11 lie in the free upper right quarter
                {
                    const int pr = t128 >> 6, r = (t128 & 63) >> 2, c4 = (t128 & 3) * 4, b0 = pr * 32;
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 a = ld4(A, b0 + 16 + r, b0 + k);
                        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 t = ld4(A, b0 + k + e, b0 + c4);
                            s.x = fmaf(av[e], t.x, s.x); s.y = fmaf(av[e], t.y, s.y);
                            s.z = fmaf(av[e], t.z, s.z); s.w = fmaf(av[e], t.w, s.w);
                        }
                    }
                    st4(A, pr * 16 + r, 32 + c4, s);
                    named_sync(1, 128);
                    s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 a = ld4(A, b0 + 16 + r, b0 + 16 + k);
                        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 t = ld4(A, pr * 16 + k + e, 32 + c4);
                            s.x = fmaf(-av[e], t.x, s.x); s.y = fmaf(-av[e], t.y, s.y);
                            s.z = fmaf(-av[e], t.z, s.z); s.w = fmaf(-av[e], t.w, s.w);
                        }
                    }
                    st4(A, b0 + 16 + r, b0 + c4, s);
                }
                named_sync(1, 128);
                // the block of 64, the same
                {
                    const int r = t128 >> 2, c8 = (t128 & 3) * 8;
                    float s[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = 0.f;
#pragma unroll 4
                    for (int k = 0; k < 32; k += 4) {
                        const float4 a = ld4(A, 32 + r, k);
                        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 t = ld4(A, k + e, c8), u = ld4(A, k + e, c8 + 4);
                            s[0] = fmaf(av[e], t.x, s[0]); s[1] = fmaf(av[e], t.y, s[1]);
                            s[2] = fmaf(av[e], t.z, s[2]); s[3] = fmaf(av[e], t.w, s[3]);
                            s[4] = fmaf(av[e], u.x, s[4]); s[5] = fmaf(av[e], u.y, s[5]);
                            s[6] = fmaf(av[e], u.z, s[6]); s[7] = fmaf(av[e], u.w, s[7]);
                        }
                    }
                    st4(A, r, 32 + c8, make_float4(s[0], s[1], s[2], s[3]));
                    st4(A, r, 36 + c8, make_float4(s[4], s[5], s[6], s[7]));
                    named_sync(1, 128);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = 0.f;
#pragma unroll 4
                    for (int k = 0; k < 32; k += 4) {
                        const float4 a = ld4(A, 32 + r, 32 + k);
                        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 t = ld4(A, k + e, 32 + c8), u = ld4(A, k + e, 36 + c8);
                            s[0] = fmaf(-av[e], t.x, s[0]); s[1] = fmaf(-av[e], t.y, s[1]);
                            s[2] = fmaf(-av[e], t.z, s[2]); s[3] = fmaf(-av[e], t.w, s[3]);
                            s[4] = fmaf(-av[e], u.x, s[4]); s[5] = fmaf(-av[e], u.y, s[5]);
                            s[6] = fmaf(-av[e], u.z, s[6]); s[7] = fmaf(-av[e], u.w, s[7]);
                        }
                    }
                    st4(A, 32 + r, c8, make_float4(s[0], s[1], s[2], s[3]));
                    st4(A, 32 + r, c8 + 4, make_float4(s[4], s[5], s[6], s[7]));
                }
                named_sync(1, 128);
                // T' and -T'' as hi + lo tiles: thread (row r, half of the columns)
                if (cc > 0) wait(&bar[B_TFREE], (cc - 1) & 1, ok);
                {
                    const int r = t128 & 63, hf = t128 >> 6;
                    const bool zero = hf == 1 && r < 32;
                    uint8_t *tt = sm + OFF_T;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int j = hf * 32 + q * 8;
                        uint32_t h1[4] = {}, l1[4] = {}, h2[4] = {}, l2[4] = {};
                        if (!zero) {
#pragma unroll
                            for (int e = 0; e < 8; e += 4) {
                                const float4 t = ld4(A, r, j + e);
                                const float4 b = *reinterpret_cast<const float4 *>(sbeta + j + e);
                                const float4 bg = *reinterpret_cast<const float4 *>(sbg + j + e);
                                split2(t.x * b.x, t.y * b.y, h1[e / 2], l1[e / 2]);
                                split2(t.z * b.z, t.w * b.w, h1[e / 2 + 1], l1[e / 2 + 1]);
                                split2(-t.x * bg.x, -t.y * bg.y, h2[e / 2], l2[e / 2]);
                                split2(-t.z * bg.z, -t.w * bg.w, h2[e / 2 + 1], l2[e / 2 + 1]);
                            }
                        }
                        const uint32_t off = sw(r, hf * 4 + q);
                        *reinterpret_cast<uint4 *>(tt + off) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
                        *reinterpret_cast<uint4 *>(tt + kTile + off) = make_uint4(l1[0], l1[1], l1[2], l1[3]);
                        *reinterpret_cast<uint4 *>(tt + 2 * kTile + off) = make_uint4(h2[0], h2[1], h2[2], h2[3]);
                        *reinterpret_cast<uint4 *>(tt + 3 * kTile + off) = make_uint4(l2[0], l2[1], l2[2], l2[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_T]);
                named_sync(1, 128);  // the gates and A are read: the next chunk may write them
            }
        }
    } else if (warp < 12) {
        // -------------------------------------------------------------------- W to shared memory, outputs
        const int row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        auto outputs = [&](int cc, int ring, int tok, int nv, int h) {
            const float *rg = reinterpret_cast<const float *>(sm + OFF_RING) + ring * 2 * kC;
            float acc[64];
            wait(&bar[B_SQ], cc & 1, ok);
            tc_fence_after();
#pragma unroll
            for (int j0 = 0; j0 < 64; j0 += 16) {
                uint32_t r[16];
                tmem_ld16_nowait(tmem + lanes + TM_O + j0, r);
                tmem_wait_ld_into(r);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 e = *reinterpret_cast<const float4 *>(rg + j0 + j);
                    acc[j0 + j] = e.x * __uint_as_float(r[j]);
                    acc[j0 + j + 1] = e.y * __uint_as_float(r[j + 1]);
                    acc[j0 + j + 2] = e.z * __uint_as_float(r[j + 2]);
                    acc[j0 + j + 3] = e.w * __uint_as_float(r[j + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B_SQRD]);
            wait(&bar[B_O], cc & 1, ok);
            tc_fence_after();
            __nv_bfloat16 *dst = p.o + ((int64_t)tok * p.hv_n + h) * kD + row;
            const int64_t step = (int64_t)p.hv_n * kD;
#pragma unroll
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
                for (int j = 0; j < 16; ++j) {
                    if (j0 + j < nv) *dst = __float2bfloat16_rn(acc[j0 + j] + __uint_as_float(r[j]));
                    dst += step;
                }
            }
        };
        int cc = 0, ring = 0;
        int p_tok = 0, p_nv = 0, p_h = 0, p_ring = 0;  // the chunk whose outputs are still to come
        for (int idx = blockIdx.x; idx < p.items; idx += gridDim.x) {
            const Item x = item_of(p, idx);
            for (int c = 0; c < x.chunks; ++c, ++cc, ring = ring + 1 == kRing ? 0 : ring + 1) {
                wait(&bar[B_W], cc & 1, ok);
                if (cc > 0) wait(&bar[B_U], (cc - 1) & 1, ok);  // S W^T of the chunk before has read W
                tc_fence_after();
                uint8_t *wt = sm + OFF_W;
#pragma unroll
                for (int j0 = 0; j0 < 64; j0 += 16) {
                    uint32_t r[16];
                    tmem_ld16_nowait(tmem + lanes + TM_W + j0, r);
                    tmem_wait_ld_into(r);
                    uint32_t hi[8], lw[8];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) split2(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), hi[j / 2], lw[j / 2]);
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
                if (cc > 0) outputs(cc - 1, p_ring, p_tok, p_nv, p_h);
                p_tok = x.lo + c * kC;
                p_nv = x.n - c * kC;
                p_h = x.h;
                p_ring = ring;
            }
        }
        if (cc > 0) outputs(cc - 1, p_ring, p_tok, p_nv, p_h);
    } else {
        // -------------------------------------------------------------------- the state
        reg_alloc<128>();
        const int row = quad * 32 + lane, half = (warp - 12) >> 2;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const float *el = reinterpret_cast<const float *>(sm + OFF_EL);
        int cc = 0, ring = 0;
        for (int idx = blockIdx.x; idx < p.items; idx += gridDim.x) {
            const Item x = item_of(p, idx);
            if (x.err) continue;
            const int64_t mine = x.state + row * kD + half * 64;
            float s[64];
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
                const float4 v = x.zero ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4 *>(p.S0 + mine + j);
                s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
            }
            // s = e^gamma_63 s + dS of chunk number n
            auto advance = [&](int n) {
                wait(&bar[B_UPD], n & 1, ok);
                tc_fence_after();
                const float a = el[n & (kDecays - 1)];
#pragma unroll
                for (int j0 = 0; j0 < 64; j0 += 16) {
                    uint32_t r[16];
                    tmem_ld16_nowait(tmem + lanes + TM_DS + half * 64 + j0, r);
                    tmem_wait_ld_into(r);
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j0 + j] = fmaf(a, s[j0 + j], __uint_as_float(r[j]));
                }
            };
            for (int c = 0; c < x.chunks; ++c, ++cc, ring = ring + 1 == kRing ? 0 : ring + 1) {
                if (c > 0) advance(cc - 1);
                if (cc > 0) wait(&bar[B_O], (cc - 1) & 1, ok);  // U of the chunk before lies over S hi
                tc_fence_after();
#pragma unroll
                for (int j0 = 0; j0 < 64; j0 += 16) {
                    uint32_t hi[8], lw[8];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) split2(s[j0 + j], s[j0 + j + 1], hi[j / 2], lw[j / 2]);
                    tmem_st8(tmem + lanes + TM_SHI + half * 32 + j0 / 2, hi);
                    tmem_st8(tmem + lanes + TM_SLO + half * 32 + j0 / 2, lw);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_S]);

                const float *fd = reinterpret_cast<const float *>(sm + OFF_RING) + ring * 2 * kC + kC + half * 32;
                uint32_t ub[2][8];
                wait(&bar[B_U], cc & 1, ok);
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t r[16], hi[8], lw[8];
                    tmem_ld16_nowait(tmem + lanes + TM_U + half * 32 + q * 16, r);
                    tmem_wait_ld_into(r);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(fd + q * 16 + j);
                        const float a = __uint_as_float(r[j]), b = __uint_as_float(r[j + 1]), d = __uint_as_float(r[j + 2]),
                                    e = __uint_as_float(r[j + 3]);
                        ub[q][j / 2] = pack_bf16(a, b);
                        ub[q][j / 2 + 1] = pack_bf16(d, e);
                        split2(a * f.x, b * f.y, hi[j / 2], lw[j / 2]);
                        split2(d * f.z, e * f.w, hi[j / 2 + 1], lw[j / 2 + 1]);
                    }
                    tmem_st8(tmem + lanes + TM_UHI + half * 16 + q * 8, hi);
                    tmem_st8(tmem + lanes + TM_ULO + half * 16 + q * 8, lw);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_UST]);
                wait(&bar[B_SQ], cc & 1, ok);
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 2; ++q) tmem_st8(tmem + lanes + TM_UBF + half * 16 + q * 8, ub[q]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_UBF]);
            }
            if (x.chunks > 0) advance(cc - 1);
#pragma unroll
            for (int j = 0; j < 64; j += 4)
                *reinterpret_cast<float4 *>(p.S_new + mine + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        }
    }
    if (!ok) flag(p.status, GDN_DEV_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, 512);
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

int64_t token_stride(int64_t given, int heads) { return given ? given : (int64_t)heads * kD; }

}  // namespace

bool prefill_tc_supported(const gdn_prefill_args &a) {
    const int64_t qs = token_stride(a.q_stride, a.n_k_heads), ks = token_stride(a.k_stride, a.n_k_heads),
                  vs = token_stride(a.v_stride, a.n_v_heads);
    return a.qkv_dtype == GDN_BF16 && a.out_dtype == GDN_BF16 && a.d_k == kD && a.d_v == kD && a.total_tokens > 0 &&
           tiles::aligned16(a.q) && tiles::aligned16(a.k) && tiles::aligned16(a.v) && tiles::aligned16(a.S0) &&
           tiles::aligned16(a.S_new) && qs % 8 == 0 && ks % 8 == 0 && vs % 8 == 0 && std::max(qs, std::max(ks, vs)) < (1ll << 38) &&
           (int64_t)a.batch * a.n_v_heads <= 0x7fffffff && tensor_map_encoder() != nullptr;
}

cudaError_t launch_prefill_tc(const gdn_prefill_args &a, cudaStream_t stream) {
    CUtensorMap tmQ, tmK, tmV;
    if (!encode(&tmQ, a.q, a.n_k_heads, a.total_tokens, token_stride(a.q_stride, a.n_k_heads)) ||
        !encode(&tmK, a.k, a.n_k_heads, a.total_tokens, token_stride(a.k_stride, a.n_k_heads)) ||
        !encode(&tmV, a.v, a.n_v_heads, a.total_tokens, token_stride(a.v_stride, a.n_v_heads)))
        return cudaErrorInvalidValue;
    Params p = {};
    p.hk_n = a.n_k_heads; p.hv_n = a.n_v_heads; p.total = a.total_tokens; p.max_tokens = a.max_tokens;
    p.n_states = a.n_states; p.items = a.batch * a.n_v_heads; p.probe = wait_probe_polls();
    p.scale = a.scale;
    p.offsets = a.token_offsets; p.slots = a.slots; p.fresh = a.fresh;
    p.g = a.g; p.beta = a.beta; p.S0 = a.S0;
    p.o = static_cast<__nv_bfloat16 *>(a.o); p.S_new = a.S_new; p.status = a.dev_status;
    static int have[16];
    cudaError_t e = ensure_smem(prefill_tc_kernel, kSmem, have);
    if (e != cudaSuccess) return e;
    prefill_tc_kernel<<<(unsigned)std::min(p.items, sm_count()), kThreads, kSmem, stream>>>(tmQ, tmK, tmV, p);
    return cudaGetLastError();
}

}  // namespace gdn
