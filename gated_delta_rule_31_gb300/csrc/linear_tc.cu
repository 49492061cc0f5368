// linear_tc.cu - linear attention with a constant decay per head on the tensor cores, for bf16
// q, k, v: the segment summary and the mix passes of o and dv (linear.h).
//
// A CTA walks the 128-token chunks of one segment of one (b, value head), forwards for o
// (a, b, c = q, k, v) or backwards for dv (k, q, do), with the state S [Dv x Dk] (or its adjoint)
// in fp32 registers. Rows r and columns j of a chunk's products are its tokens in memory order,
// m of them valid; with l the head's decay, per chunk
//
//     P = a b^T                       128 x 128 x Dk
//     Y = P' c, P'_rj = f l^|r-j| P_rj for j <= r (reverse: j >= r)       128 x Dv x 128
//     X = a S^T                       128 x Dv x Dk
//     out_r = f' l^(r+1) X_r + Y_r    (reverse: l^(m-1-r))
//     S <- l^m S + c'^T b, c'_j = f'' l^(m-1-j) c_j (reverse: l^(j+1))    Dv x Dk x 128
//
// All four run as tcgen05 products with 128 rows. Rounding to bf16: P' (an operand kept in TMEM), the copy
// of S that X reads, and the result, one rounding each: the products take bf16 operands, and a second
// term of either would need as many products again and, for S, 32 KB of shared memory that the tiles
// have. (Error of o, relative to its norm: 0.0023; the result's rounding alone 0.0017.) c' would be a fourth, so
// it enters as the sum of bf16 terms: two (2^-17 off, below the other roundings) where the state only feeds X,
// three (the 24 bits of an fp32 product) where it is returned in fp32. Each chunk's sum starts from zero in TMEM
// and is added to the fp32 registers there, so the tensor core's own accumulation never runs over more than
// one chunk. X is scaled by its rows' decays in TMEM and Y accumulates onto it.
//
// c'^T is an operand in TMEM: transposing matrix loads give each thread two tokens of a channel,
// which is the operand's own layout, so the terms go from registers to TMEM with no pass
// through shared memory.
//
// Warps: 0-7 turn P into P' and finish the output (a thread is half a token row), 8-11 hold the
// state (a thread is a state row), 12-19 form c' in pieces of PIECE tokens (in the summary 0-7 do
// too), 20 and 23 copy tiles in, 21 issues the products, 22 stores the output tiles. The state rows need
// the registers: warps 12-23 give some up (setmaxnreg). The products of a chunk are issued as X, the next
// chunk's sum of the state, Y, the next chunk's P: each has the others' time to wait for the warps that
// feed it. Input tiles (128 tokens, two 64-channel panels, 32 KB) have three slots for c, which is wanted
// a chunk ahead and whose slot then takes the output tile, two for b and one for a (three for b in the
// summary). Channels past a head size of 32 read as zero (out of the tensor map's range), sizes of 32 and
// 64 use one panel. With 512 TMEM columns and 224 KB of shared memory one CTA runs per SM.
//
// T = 32768, Hk 16, Hv 32, D 128, four segments a head: the output pass 160 us (187 with the states kept),
// bound by the copies in and out (805 MB, 74% of a plain copy's rate, from 128 CTAs with about one
// chunk's tiles in flight each); the summary 101 us, bound by the waits between copy, decay, product and
// sum of a chunk (1.45 us; 85 us in all with two terms). Pieces of 32 tokens in a ring of five take 111 us
// for the summary, of 128 with one sum 118; the output tile in b's slot took 198 us for the output pass
// where c's took 172.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "kernels.h"
#include "linear.h"
#include "linear_dev.cuh"
#include "linear_host.h"

namespace gdr {

using namespace linear;

namespace {

constexpr int SLOTS = 6, SLOTS_C = 3;  // input tiles, those of c
constexpr uint32_t SLOT = TILE;
constexpr uint32_t AT_S = SLOTS * SLOT;     // bf16 state [128 x 128]
constexpr uint32_t AT_W = AT_S + 32768;     // weights of c' for 128 exponents, 8 bytes each
constexpr uint32_t BYTES = AT_W + 1024;
static_assert(BYTES + 1024 <= 232448, "shared memory");
constexpr int THREADS = 768;
// Registers a thread: 768 threads start with 80; 8 warps keep them, 4 go up, 8 and 4 go down.
constexpr int REGS = 80, REGS_STATE = 176, REGS_DECAY = 48, REGS_REST = 48;
static_assert(2 * REGS + REGS_STATE + 2 * REGS_DECAY + REGS_REST <= 6 * REGS, "registers of the launch");

struct TcArgs {
    LinearShape s;
    int reverse, panels_k, panels_v, first_seg;
    float fp, fx, fu;          // f, f', f''
    const float* start;        // state entering each segment [B, Hv, start_segs, Dv, Dk], or null (zero)
    int start_segs;
    float* z;                  // summary: what the segment adds to the state [B, Hv, nseg, Dv, Dk]
    float* last;               // mix: the state after all segments, or null
    void* out;                 // mix: [B, T, Hv, Dv]
    uint8_t* images;           // mix: the bf16 state that each chunk's X reads, or null (linear.h)
    int* status;
    int clear_status;          // the first kernel of a call clears the status word
};

// 16 lanes x 16 columns: r[2 i], r[2 i + 1] hold column 4 i + t % 4 of lanes t / 4 and t / 4 + 8.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
// The upper halves of two floats: bf16 values, rounded towards zero.
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
// Four transposed 8 x 8 tiles of 16-bit values, rows at the addresses of lanes 8 i .. 8 i + 7: thread t
// gets values (2 (t % 4), 2 (t % 4) + 1) of column t / 4 of each.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// TERMS: bf16 terms of c' (2 or 3). MIX: the output pass, else the summary.
template <bool MIX, int TERMS>
__global__ void __launch_bounds__(THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                     const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap mo, TcArgs a) {
    extern __shared__ __align__(1024) uint8_t sm[];  // swizzled tiles: no room for rounding up
    const uint32_t sb = smem_u32(sm);
    __shared__ uint64_t full[SLOTS], empty[SLOTS], bfull[4], bfree[4];
    __shared__ uint64_t pfull, xfull, pready, yfull, xready, staged, sfull[2], sfree[2], drain;
    __shared__ float tri[160];
    __shared__ uint32_t tmem_sh;
    __shared__ int failed, used[SLOTS];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const LinearShape& s = a.s;
    const int seg = a.first_seg + blockIdx.x;
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / (s.Hv / s.Hk);
    const size_t bh = (size_t)b * s.Hv + hv;
    if (sb & 1023u) {  // never on this layout; swizzled tiles would be read wrongly
        if (tid == 0) a.status[0] = -1;
        return;
    }
    // TMEM columns. Output pass: P (P' packed in the first half of each 64), X and then the output, the
    // chunk's sum of the state, a ring of pieces of c'. Summary: two sums and the ring.
    constexpr int PIECE = MIX && TERMS == 3 ? 32 : 64; // tokens of a piece
    constexpr int STEPS = PIECE / 16;                  // products of a piece and term
    constexpr uint32_t STEP = 8 * TERMS;               // columns of a step: its terms, eight each
    constexpr uint32_t COL_P = 0, COL_X = 128, COL_S = MIX ? 256 : 0, COL_C = MIX ? 384 : 256;
    constexpr int SUMS = MIX ? 1 : 2, RING = (512 - COL_C) / (STEPS * STEP);
    static_assert(RING == 2 && (TERMS == 2 || TERMS == 3), "pieces");
    constexpr int SLOTS_B = MIX ? 2 : 3;
    auto slot_c = [](int i) { return i % SLOTS_C; };
    auto slot_b = [](int i) { return SLOTS_C + i % SLOTS_B; };
    constexpr int slot_a = SLOTS - 1;
    constexpr int DECAY_WARPS = MIX ? 8 : 16;

    const int n = s.lengths ? min(max(s.lengths[b], 0), s.T) : s.T;
    const int begin = seg * s.seg_tokens, end = min(begin + s.seg_tokens, s.T);
    const int first = min(begin, n), last = min(end, n), nc = (last - first + C - 1) / C;
    // The summary, which may take a segment's chunks in any order, ends with those that the output pass begins
    // with: part of them it then finds in L2.
    auto chunk_of = [&](int i) { return (a.reverse != 0) == MIX ? nc - 1 - i : i; };
    auto tokens_of = [&](int i) { return min(C, last - first - chunk_of(i) * C); };

    if (tid == 0) {
        if (a.clear_status && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            for (int i = 0; i < 4; i++) a.status[i] = 0;  // a wait expires a second later at the earliest
        failed = 0;
        for (int i = 0; i < SLOTS; i++) {
            used[i] = 0;
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < RING; i++) {
            mbar_init(&bfull[i], DECAY_WARPS);
            mbar_init(&bfree[i], 1);
        }
        for (int i = 0; i < SUMS; i++) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sfree[i], 4);
        }
        mbar_init(&pfull, 1);
        mbar_init(&xfull, 1);
        mbar_init(&pready, 8);
        mbar_init(&staged, 8);
        mbar_init(&yfull, 1);
        mbar_init(&xready, 12);  // the copy of the state is written (4) and the last output read (8)
        mbar_init(&drain, 1);
        fence_barrier_init();
    }
    const float g = s.g[hv];
    // tri[31 + r - j] = f l^(r-j) of a pair in order, else 0; in reverse tri[127 + r - j] = f l^(j-r)
    const int tri_zero = a.reverse ? 127 : 31;
    if (tid < 160) {
        const int d = a.reverse ? tri_zero - tid : tid - tri_zero;
        tri[tid] = d >= 0 ? a.fp * power(g, d) : 0.f;
    }
    // f'' l^e for two tokens in a row, the first of exponent e (the next e - 1, in reverse e + 1): for three
    // terms in fp32, for two as bf16 parts, w1 and w2
    uint32_t* weights = reinterpret_cast<uint32_t*>(sm + AT_W);
    if (tid < 128) {
        const float x0 = a.fu * power(g, tid), x1 = a.fu * power(g, a.reverse ? tid + 1 : max(tid - 1, 0));
        const uint32_t w = pack_bf16(x0, x1);
        weights[2 * tid] = TERMS == 3 ? __float_as_uint(x0) : w;
        weights[2 * tid + 1] = TERMS == 3 ? __float_as_uint(x1) : pack_bf16(x0 - bf16lo(w), x1 - bf16hi(w));
    }
    if (warp == 20) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    next_kernel_may_start();
    const uint32_t tm = tmem_sh;

    // Pieces of c' into TMEM, by DECAY_WARPS warps of which this is number w (warp & 3 is its TMEM quarter).
    auto decay_pieces = [&](const int w) {
        const int quarter = w & 3, part = w >> 2;
        const uint32_t lanes = tm + ((uint32_t)(32 * quarter) << 16);
        constexpr int OWN = STEPS * 4 / DECAY_WARPS;  // steps of a piece for each warp
        // where this lane's matrix row lies in a step's 16 tokens of the tile of c
        const uint32_t at_row = sw128_chunk((lane >> 4) * 8 + (lane & 7), 4 * quarter + (lane >> 3 & 1), C);
        int piece = 0;
        for (int i = 0; i < nc; i++) {
            const int m = tokens_of(i), nj = (m + 15) / 16;
            const uint32_t ct = sb + slot_c(i) * SLOT, bt = sb + slot_b(i) * SLOT;
            bool ok = wait_phase(&full[slot_c(i)], i / SLOTS_C & 1, &failed, 60);
            if (m < C && s.lengths) {
                ok = ok && wait_phase(&full[slot_b(i)], i / SLOTS_B & 1, &failed, 61);
                // rows past the last token: zero in b, and in c where they enter the last 16-token step,
                // whatever they hold
                const int ch = lane & 15;
#pragma unroll 1
                for (int z = m + 2 * w + (lane >> 4); ok && z < C; z += 2 * DECAY_WARPS) {
                    if (z < 16 * nj && ch < 8 * a.panels_v) st_shared_v4(ct + sw128_chunk(z, ch, C), 0, 0, 0, 0);
                    if (ch < 8 * a.panels_k) st_shared_v4(bt + sw128_chunk(z, ch, C), 0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
#pragma unroll 1
            for (int j = 0; j < nj && ok; j += STEPS, piece++) {
                const int r = piece % RING;
                if (piece >= RING) ok = wait_phase(&bfree[r], (piece / RING + 1) & 1, &failed, 62);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int e = 0; e < OWN; e++) {
                    const int in = part * OWN + e, t = 16 * (j + in);  // step of the piece, its first token
                    if (t >= m || quarter >= 2 * a.panels_v) continue;
                    uint32_t v[2][4];
                    ldmatrix_x4_trans(ct + t * 128 + at_row, v[0]);
                    ldmatrix_x4_trans(ct + t * 128 + (at_row ^ 32u), v[1]);
                    const int u = t + 2 * (lane & 3);  // first token of v[.][0], v[.][1]; that of the others is u + 8
                    if (t + 16 > m) {                  // nothing past the last token, whatever it holds
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const int x = u + 8 * (k >> 1);
                            const uint32_t keep = x + 1 < m ? 0xffffffffu : x < m ? 0xffffu : 0u;
                            v[0][k] &= keep;
                            v[1][k] &= keep;
                        }
                    }
                    const uint2* table = reinterpret_cast<const uint2*>(weights);
                    const uint2 w[2] = {table[a.reverse ? u + 1 : max(m - 1 - u, 0)], table[a.reverse ? u + 9 : max(m - 9 - u, 0)]};
#pragma unroll
                    for (int g2 = 0; g2 < 2; g2++) {
                        uint32_t y[4 * TERMS];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint32_t x = v[g2][k];
                            const uint2 p = w[k >> 1];
                            if (TERMS == 2) {
                                y[k] = bf16x2_mul(x, p.x);
                                y[4 + k] = bf16x2_fma(x, p.y, bf16x2_fma(x, p.x, bf16x2_neg(y[k])));
                            } else {  // 24 bits cut into three times eight
                                float f0 = bf16lo(x) * __uint_as_float(p.x), f1 = bf16hi(x) * __uint_as_float(p.y);
#pragma unroll
                                for (int h = 0; h < 3; h++) {
                                    y[4 * h + k] = high_halves(f0, f1);
                                    f0 -= bf16hi(__float_as_uint(f0));
                                    f1 -= bf16hi(__float_as_uint(f1));
                                }
                            }
                        }
                        const uint32_t to = lanes + ((uint32_t)(16 * g2) << 16) + COL_C + (r * STEPS + in) * STEP;
                        tmem_st_16x128b_x4(to, y);
                        if (TERMS == 3) tmem_st_16x128b_x2(to + 16, y + 4 * (TERMS - 1));
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bfull[r]);
            }
            if (!ok) break;
        }
    };

    if (warp >= 20) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
        if (warp == 20 || warp == 23) {
            // Tiles are asked for as their slots come free: c by one warp, since it is wanted first and kept
            // longest, b and a by another (its steps: b of chunk 0, b 1, a 0, b 2, a 1, ..). In the output
            // pass, whose one slot for a is free for a short time only, a step also brings its tile two chunks
            // on into L2 (further ahead costs more than it hides: 227 us at six chunks, T = 32768).
            const bool for_c = warp == 20;
            const int steps = for_c ? nc : 2 * nc;
#pragma unroll 1
            for (int t = 0; t < steps; t++) {
                const bool is_a = MIX && !for_c && t > 0 && (t % 2 == 0 || t == 2 * nc - 1);
                if (!MIX && !for_c && t >= nc) break;
                const int i = for_c || !MIX ? t : is_a ? (t - 1) / 2 : (t + 1) / 2;
                const CUtensorMap* map = for_c ? &mc : is_a ? &ma : &mb;
                const int panels = for_c ? a.panels_v : a.panels_k, head = for_c ? hv : hk;
                const int k = for_c ? slot_c(i) : is_a ? slot_a : slot_b(i);
                const int use = for_c ? i / SLOTS_C : is_a ? i : i / SLOTS_B;  // tiles that the slot had before
                if (use > 0 && !wait_phase(&empty[k], (use + 1) & 1, &failed, 40)) break;
                if (lane == 0) {
                    const int t0 = first + chunk_of(i) * C, far = first + chunk_of(min(i + 2, nc - 1)) * C;
                    mbar_expect_tx(&full[k], panels * PANEL);
                    used[k] = use + 1;
#pragma unroll 1
                    for (int p = 0; p < panels; p++) {
                        tma_load_4d(sm + k * SLOT + p * PANEL, map, 64 * p, head, t0, b, &full[k]);
                        if (MIX) tma_prefetch_4d(map, 64 * p, head, far, b);
                    }
                }
                __syncwarp();
            }
        } else if (warp == 21) {
            const int dk = 64 * a.panels_k, dv = 64 * a.panels_v;
            const uint32_t id_p = idesc_bf16(128, 128, 0, 0), id_x = idesc_bf16(128, dv, 0, 0);
            const uint32_t id_y = idesc_bf16(128, dv, 0, 1), id_s = idesc_bf16(128, dk, 0, 1);
            int piece = 0;
            auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
                return wait_phase(bar, parity, &failed, site);
            };
            auto issue_p = [&](int i) {  // over P', which the Y product before has read
                if (!wait(&full[slot_a], i & 1, 42)) return false;  // b has been there for the sum
                tc_fence_after();
                const uint32_t ad = lo_kmajor(sb + slot_a * SLOT), bd = lo_kmajor(sb + slot_b(i) * SLOT);
#pragma unroll 1
                for (int p = 0; p < a.panels_k; p++)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        mma_ss(tm + COL_P, ad + p * (PANEL >> 4) + 2 * k, bd + p * (PANEL >> 4) + 2 * k, id_p, k > 0 ? 1u : p);
                commit(&pfull);
                commit(&empty[slot_b(i)]);  // the sum of the state read it before
                return true;
            };
            auto issue_s = [&](int i) {
                const int nj = (tokens_of(i) + 15) / 16;  // 16-token steps that hold tokens
                if (!wait(&full[slot_b(i)], i / SLOTS_B & 1, 43)) return false;
                if (i >= SUMS && !wait(&sfree[i % SUMS], (i / SUMS + 1) & 1, 44)) return false;
                const uint32_t sum = tm + COL_S + 128 * (i % SUMS);
                for (int j = 0; j < nj; j += STEPS, piece++) {
                    const int r = piece % RING;
                    if (!wait(&bfull[r], piece / RING & 1, 45)) return false;
                    tc_fence_after();
                    const uint32_t from = tm + COL_C + r * STEPS * STEP, bd = lo_mnmajor(sb + slot_b(i) * SLOT) + step_mnmajor(j);
#pragma unroll
                    for (int e = 0; e < STEPS; e++)
#pragma unroll
                        for (int t = TERMS - 1; t >= 0; t--)  // the smallest term first
                            if (j + e < nj)
                                mma_ts(sum, from + e * STEP + 8 * t, bd + step_mnmajor(e), id_s,
                                       e > 0 || t < TERMS - 1 ? 1u : j > 0);
                    commit(&bfree[r]);
                }
                commit(&sfull[i % SUMS]);
                if (!MIX) {
                    commit(&empty[slot_b(i)]);
                    commit(&empty[slot_c(i)]);
                }
                return true;
            };
#pragma unroll 1
            for (int i = -1; i < nc; i++) {
                const bool now = MIX && i >= 0;
                if (now) {
                    if (!wait(&xready, i & 1, 46)) break;
                    tc_fence_after();
                    const uint32_t ad = lo_kmajor(sb + slot_a * SLOT), sd = lo_kmajor(sb + AT_S);
#pragma unroll 1
                    for (int p = 0; p < a.panels_k; p++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            mma_ss(tm + COL_X, ad + p * (PANEL >> 4) + 2 * k, sd + p * (PANEL >> 4) + 2 * k, id_x, k > 0 ? 1u : p);
                    commit(&xfull);
                    commit(&empty[slot_a]);  // P read it before
                }
                if (i + 1 < nc && !issue_s(i + 1)) break;
                if (now) {
                    const int nj = (tokens_of(i) + 15) / 16;
                    if (!wait(&pready, i & 1, 48)) break;
                    tc_fence_after();
                    const uint32_t cd = lo_mnmajor(sb + slot_c(i) * SLOT);
#pragma unroll 1
                    for (int h = 0; 4 * h < nj; h++)  // P' of tokens 64 .. starts at column 64
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            if (4 * h + j < nj)
                                mma_ts(tm + COL_X, tm + COL_P + 64 * h + 8 * j, cd + h * step_mnmajor(4) + step_mnmajor(j), id_y, 1);
                    commit(&yfull);
                }
                if (MIX && i + 1 < nc && !issue_p(i + 1)) break;
            }
            commit(&drain);  // every product issued so far has completed before TMEM is released
            int never = 0;
            wait_phase(&drain, 0, &never, 1);
        } else if (MIX && warp == 22) {
            for (int i = 0; i < nc; i++) {
                if (!wait_phase(&staged, i & 1, &failed, 48)) break;
                if (lane == 0) {
                    for (int p = 0; p < a.panels_v; p++)
                        tma_store_4d(&mo, sm + slot_c(i) * SLOT + p * PANEL, 64 * p, hv, first + chunk_of(i) * C, b);
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(&empty[slot_c(i)]);
                }
                __syncwarp();
            }
            if (lane == 0) bulk_wait_all();
        }
    } else if (warp >= 12 || (!MIX && warp < 8)) {
        if (warp >= 12) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_DECAY));
        decay_pieces(warp >= 12 ? warp - 12 : 8 + warp);
    } else if (warp < 8) {
        if (MIX) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
            for (int t = max(begin, first + nc * C) + warp; t < end; t += 8)  // past the last chunk: zero
                for (int d = 8 * lane; d < s.Dv; d += 256)
                    *reinterpret_cast<uint4*>(out + (((size_t)b * s.T + t) * s.Hv + hv) * s.Dv + d) = make_uint4(0, 0, 0, 0);
            const int quarter = warp & 3, half = warp >> 2;
            const int r = 32 * quarter + lane;  // token row; columns 64 half ..
            const uint32_t row = tm + ((uint32_t)(32 * quarter) << 16);
            if (lane == 0) mbar_arrive(&xready);
            for (int i = 0; i < nc; i++) {
                const int m = tokens_of(i);
                bool ok = wait_phase(&pfull, i & 1, &failed, 50);
                tc_fence_after();
                if (ok) {
#pragma unroll 1
                    for (int h = 0; h < 2; h++) {
                        const int cb = 2 * half + h;  // columns 32 cb ..
                        uint32_t w[16];
                        if (a.reverse ? cb < quarter : cb > quarter) {  // no pair of tokens in order
#pragma unroll
                            for (int e = 0; e < 16; e++) w[e] = 0;
                        } else {
                            float p[32];
                            tmem_ld32(row + COL_P + 32 * cb, p);
                            tmem_wait_ld();
                            const float* in = tri + tri_zero + r - 32 * cb;
#pragma unroll
                            for (int e = 0; e < 32; e++) p[e] *= in[-e];
#pragma unroll
                            for (int e = 0; e < 16; e++) w[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
                        }
                        // onto columns of P that this warp alone reads, and has read
                        tmem_st16(row + COL_P + 64 * half + 16 * h, w);
                    }
                }
                ok = ok && wait_phase(&xfull, i & 1, &failed, 52);
                tc_fence_after();
                if (ok) {
                    if (half < a.panels_v) {
                        const float f = a.fx * power(g, a.reverse ? max(m - 1 - r, 0) : r + 1);
#pragma unroll 1
                        for (int h = 0; h < 2; h++) {
                            float x[32];
                            tmem_ld32(row + COL_X + 64 * half + 32 * h, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; e += 2) scale2(x + e, f);
                            tmem_st32(row + COL_X + 64 * half + 32 * h, x);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pready);
                }
                ok = ok && wait_phase(&yfull, i & 1, &failed, 51);
                tc_fence_after();
                if (ok) {
                    if (half < a.panels_v) {
                        const uint32_t stage = sb + slot_c(i) * SLOT;
#pragma unroll 1
                        for (int h = 0; h < 2; h++) {
                            float x[32];
                            tmem_ld32(row + COL_X + 64 * half + 32 * h, x);
                            tmem_wait_ld();
                            if (r >= m)
#pragma unroll
                                for (int e = 0; e < 32; e++) x[e] = 0.f;
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                st_chunk(stage + sw128_chunk(r, 8 * half + 4 * h + e, C), x + 8 * e, 1.f);
                        }
                    }
                    tc_fence_before();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&xready);
                        mbar_arrive(&staged);
                    }
                }
                if (!ok) break;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_STATE));
        const int row = tid - 256;  // state row
        const uint32_t lanes = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const size_t state = (size_t)s.Dv * s.Dk;
        float S[128];
        wait_kernel_before();  // the states that enter the segments; the inputs come from before the call
        {
            const float* p = a.start ? a.start + (bh * a.start_segs + (a.start_segs > 1 ? seg : 0)) * state : nullptr;
#pragma unroll
            for (int e = 0; e < 128; e += 4) {
                const bool in = MIX && p && row < s.Dv && e < s.Dk;
                const float4 x = in ? *reinterpret_cast<const float4*>(p + (size_t)row * s.Dk + e)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
            }
        }
        auto write_state = [&]() {  // the bf16 copy that X reads
#pragma unroll
            for (int e = 0; e < 16; e++)
                if (e < 8 * a.panels_k) st_chunk(sb + AT_S + sw128_chunk(row, e, C), S + 8 * e, 1.f);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&xready);
        };
        // The copy of chunk i, and its image. The four warps decide together whether to go on.
        auto share_state = [&](int i, bool ok) {
            if (a.images && row == 0) bulk_wait_read_all();  // the last image has been read
            if (bar_sync_or(2, 128, !ok)) return false;
            write_state();
            if (a.images) {
                bar_sync_or(2, 128, false);
                if (row == 0) {
                    const size_t chunk = (bh * ((s.T + C - 1) / C) + first / C + chunk_of(i)) * TILE;
                    bulk_store(a.images + chunk, sm + AT_S, a.panels_k * PANEL);
                    bulk_commit();
                }
            }
            return true;
        };
        bool go = !MIX || nc == 0 || share_state(0, true);
        for (int i = 0; i < nc && go; i++) {
            bool ok = wait_phase(&sfull[i % SUMS], i / SUMS & 1, &failed, 63);
            if (ok) {
                tc_fence_after();
                // output pass: S <- l^m S + sum; summary: S <- S + l^(tokens of the segment after the chunk) sum
                const int t0 = chunk_of(i) * C, tokens = last - first;
                const float over = power(g, MIX ? tokens_of(i) : a.reverse ? t0 : max(tokens - t0 - C, 0));
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    if (h >= 2 * a.panels_k) continue;
                    float d[32];
                    tmem_ld32(lanes + COL_S + 128 * (i % SUMS) + 32 * h, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) axpy2<MIX>(S + 32 * h + e, over, d + e);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfree[i % SUMS]);
            }
            if (MIX && i + 1 < nc) {
                ok = ok && wait_phase(&xfull, i & 1, &failed, 64);  // X has read the last copy
                ok = share_state(i + 1, ok);
            }
            go = ok;
        }
        if (MIX && a.images && row == 0) bulk_wait_all();
        float* to = nullptr;
        if (!MIX) to = a.z + (bh * s.nseg + seg) * state;
        else if (a.last && seg == (a.reverse ? 0 : s.nseg - 1)) to = a.last + bh * state;
        if (to && row < s.Dv)
#pragma unroll
            for (int e = 0; e < 128; e += 4)
                if (e < s.Dk)
                    *reinterpret_cast<float4*>(to + (size_t)row * s.Dk + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
    tc_fence_before();
    __syncthreads();
    if (failed && tid == 0) {
        if (atomicCAS(a.status, 0, DEV_TIMEOUT) == 0) {
            a.status[1] = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
            a.status[2] = failed;
        }
        int never = 0;
        for (int k = 0; k < SLOTS; k++)  // copies still in flight must land first
            if (used[k]) mbar_wait(&full[k], (used[k] - 1) & 1, &never, nullptr, 0);
    }
    __syncthreads();
    if (warp == 20) tmem_dealloc(tm, 512);
}

// Before the tensor maps: the first runtime call of a host thread (autograd's, say) makes the device's
// context current there, which encoding a map needs.
template <bool MIX, int TERMS>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(linear_tc_kernel<MIX, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
}

template <bool MIX, int TERMS>
cudaError_t launch(const CUtensorMap* maps, const TcArgs& a, int segs, const char* name, bool overlap, cudaStream_t st) {
    trace_begin(name, st);
    const cudaError_t e = launch_after(linear_tc_kernel<MIX, TERMS>, dim3(segs, a.s.Hv, a.s.B), THREADS, BYTES, st, overlap,
                                       maps[0], maps[1], maps[2], maps[3], a);
    trace_end(st);
    return e;
}

}  // namespace

cudaError_t launch_linear_tc_summary(const LinearSummaryArgs& x, bool all, int* status, bool clear, cudaStream_t st) {
    if (cudaError_t e = allow_smem<false, 3>()) return e;
    CUtensorMap maps[4];
    memset(maps, 0, sizeof(maps));
    if (!tile_map(&maps[1], x.cols, x.s, x.s.Hk, x.s.Dk) || !tile_map(&maps[2], x.rows, x.s, x.s.Hv, x.s.Dv))
        return cudaErrorInvalidValue;
    TcArgs a = {};
    a.s = x.s;
    a.reverse = x.reverse;
    a.panels_k = panels(x.s.Dk);
    a.panels_v = panels(x.s.Dv);
    a.fu = x.factor;
    a.z = x.z;
    a.status = status;
    a.clear_status = clear;
    a.first_seg = all || !x.reverse ? 0 : 1;
    return launch<false, 3>(maps, a, all ? x.s.nseg : x.s.nseg - 1, "linear_summary", false, st);
}

cudaError_t launch_linear_tc_mix(const LinearMixArgs& x, const float* start, int start_segs, float* last, int* status,
                                 bool clear, bool overlap, cudaStream_t st) {
    const bool rev = x.pass == LINEAR_DV;
    // One segment carries the state that leaves the call, with three terms (also where the caller does not
    // want it, so that the kept states are the same); with several it comes from the summary, with three too.
    const bool one = x.s.nseg == 1;
    if (cudaError_t e = one ? allow_smem<true, 3>() : allow_smem<true, 2>()) return e;
    CUtensorMap maps[4];
    if (!tile_map(&maps[0], rev ? x.k : x.q, x.s, x.s.Hk, x.s.Dk) || !tile_map(&maps[1], rev ? x.q : x.k, x.s, x.s.Hk, x.s.Dk) ||
        !tile_map(&maps[2], rev ? x.do_ : x.v, x.s, x.s.Hv, x.s.Dv) || !tile_map(&maps[3], x.out, x.s, x.s.Hv, x.s.Dv))
        return cudaErrorInvalidValue;
    TcArgs a = {};
    a.s = x.s;
    a.reverse = rev;
    a.panels_k = panels(x.s.Dk);
    a.panels_v = panels(x.s.Dv);
    a.fp = x.scale;
    a.fx = rev ? 1.f : x.scale;
    a.fu = rev ? x.scale : 1.f;
    a.start = start;
    a.start_segs = start_segs;
    a.last = last;
    a.out = x.out;
    a.images = static_cast<uint8_t*>(x.images);
    a.status = status;
    a.clear_status = clear;
    const char* name = rev ? "linear_dv" : "linear_o";
    return one ? launch<true, 3>(maps, a, x.s.nseg, name, overlap, st) : launch<true, 2>(maps, a, x.s.nseg, name, overlap, st);
}

// Segments of whole chunks, one CTA each, on 152 SMs. In units of one chunk of the output pass (2.4 us): a
// wave of it takes a segment's chunks and about four for its start and end; with several segments there is
// the summary too, at about 0.6 a chunk, and the combine step, which reads every segment's state. At
// T = 32768 and 32 heads 4 segments take 101 + 8 + 160 us, 9 take 104 + 10 + 162, 19 take 114 + 16 + 180.
int linear_tc_segments(int B, int T, int Hv) {
    const long long chunks = (T + C - 1) / C, heads = (long long)B * Hv;
    if (chunks <= 1 || heads <= 0) return 1;
    int best = 1;
    double least = 1e300;
    for (long long n = 1; n <= chunks && (n == 1 || heads * n <= 8 * 152); n++) {
        const long long len = (chunks + n - 1) / n, real = (chunks + len - 1) / len;
        const double mix = (double)((heads * real + 151) / 152) * (len + 4);
        const double sum = real > 1 ? (double)((heads * (real - 1) + 151) / 152) * (0.6 * len + 5) + 3 + 0.2 * real : 0.0;
        if (mix + sum < least) {
            least = mix + sum;
            best = (int)real;
        }
    }
    return best;
}

}  // namespace gdr
