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
//     S <- l^m S + c^T B, B_j = f'' l^(m-1-j) b_j (reverse: l^(j+1))      Dv x Dk x 128
//
// All four run as tcgen05 products with 128 rows. Rounding to bf16: P' (an operand kept in TMEM), the copy
// of S that X reads, and the result, one rounding each. B would be a fourth, and the state is
// returned in fp32, so it enters as the sum of three bf16 terms (B to 2^-26): three products in
// place of one, which the tensor pipe has room for beside the memory traffic. Each chunk's sum
// starts from zero in TMEM and is added to the fp32 registers there, so the tensor core's own
// accumulation never runs over more than one chunk.
//
// Warps: 0-3 turn P into P' and finish the output (a thread is a token row), 4-11 hold the state
// (a thread is half a state row) and form B in 16-token pieces, 12 copies tiles in, 13 issues the
// products. Input tiles (128 tokens, two 64-channel panels, 32 KB) go through a ring of five
// slots in the order b, a, c; the a slot takes the output tile once its products are done.
// Channels past a head size of 32 read as zero (out of the tensor map's range), sizes of 32 and 64
// use one panel. With 512 TMEM columns and 217 KB of shared memory one CTA runs per SM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "chunk_dev.cuh"
#include "common.cuh"
#include "kernels.h"
#include "linear.h"
#include "tma_host.h"

namespace gdr {

namespace {

constexpr int C = 128;     // tokens of a chunk
constexpr int SLOTS = 5;   // input tiles
constexpr uint32_t SLOT = 32768, PANEL = 16384;
constexpr uint32_t AT_S = SLOTS * SLOT;      // bf16 state [128 x 128]
constexpr uint32_t AT_B = AT_S + 32768;      // two pieces of B: three terms of [16 x 128]
constexpr uint32_t TERM = 4096, PIECE = 3 * TERM;
constexpr uint32_t AT_PW = AT_B + 2 * PIECE; // l^0 .. l^128, then l^31 .. l^0 (16-byte aligned)
constexpr uint32_t BYTES = AT_PW + 1024;
static_assert(BYTES + 1024 + 512 <= 232448, "shared memory");
constexpr int THREADS = 448;
constexpr uint32_t COL_P = 0, COL_X = 128, COL_Y = 256, COL_S = 384;

struct TcArgs {
    LinearShape s;
    int reverse, panels_k, panels_v;
    float fp, fx, fu;          // f, f', f''
    const float* start;        // state entering each segment [B, Hv, start_segs, Dv, Dk], or null (zero)
    int start_segs;
    float* z;                  // summary: what the segment adds to the state [B, Hv, nseg, Dv, Dk]
    float* last;               // mix: the state after all segments, or null
    void* out;                 // mix: [B, T, Hv, Dv]
    int* status;
    int clear_status;          // the first kernel of a call clears the status word
};

__device__ __forceinline__ float power(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }

__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// x, as the sum of three bf16 terms: two values packed in each word.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack_bf16(x0, x1);
    const float y0 = x0 - bf16lo(hi), y1 = x1 - bf16hi(hi);
    mid = pack_bf16(y0, y1);
    lo = pack_bf16(y0 - bf16lo(mid), y1 - bf16hi(mid));
}

template <bool MIX>
__global__ void __launch_bounds__(THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                     const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap mo, TcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = align1024(smem_raw);
    const uint32_t sb = smem_u32(sm);
    __shared__ uint64_t full[SLOTS], empty[SLOTS], bfull[2], bfree[2];
    __shared__ uint64_t pfull, pready, xdone, yfull, yfree, sfull, sfree, sready, drain;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const LinearShape& s = a.s;
    const int seg = MIX || !a.reverse ? blockIdx.x : blockIdx.x + 1;  // the summary leaves out the last segment
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / (s.Hv / s.Hk);
    const size_t bh = (size_t)b * s.Hv + hv;
    constexpr int TILES = MIX ? 3 : 2;  // b, a, c or b, c
    constexpr uint32_t COLS = MIX ? 512 : 128, CS = MIX ? COL_S : 0;

    const int n = s.lengths ? min(max(s.lengths[b], 0), s.T) : s.T;
    const int begin = seg * s.seg_tokens, end = min(begin + s.seg_tokens, s.T);
    const int first = min(begin, n), last = min(end, n), nc = (last - first + C - 1) / C;
    auto chunk_of = [&](int i) { return a.reverse ? nc - 1 - i : i; };
    auto tokens_of = [&](int i) { return min(C, last - first - chunk_of(i) * C); };

    if (tid == 0) {
        if (a.clear_status && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            for (int i = 0; i < 4; i++) a.status[i] = 0;  // a wait expires a second later at the earliest
        abort_sh = 0;
        for (int i = 0; i < SLOTS; i++) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&bfull[i], 8);
            mbar_init(&bfree[i], 1);
        }
        mbar_init(&pfull, 1);
        mbar_init(&pready, 4);
        mbar_init(&xdone, 1);
        mbar_init(&yfull, 1);
        mbar_init(&yfree, 4);
        mbar_init(&sfull, 1);
        mbar_init(&sfree, 8);
        mbar_init(&sready, 8);
        mbar_init(&drain, 1);
        fence_barrier_init();
    }
    float* pw = reinterpret_cast<float*>(sm + AT_PW);  // pw[i] = l^i
    float* pd = pw + 132;                              // pd[i] = l^(31-i)
    if (tid <= C) pw[tid] = power(s.g[hv], tid);
    if (tid < 32) pd[tid] = power(s.g[hv], 31 - tid);
    if (warp == 12) {
        tmem_alloc(&tmem_sh, COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_sh;
    int loaded = 0;  // tiles asked for (warp 12)

    if (warp == 12) {
        if (lane == 0) {
            bool ok = true;
            for (int i = 0; i < nc && ok; i++) {
                const int t0 = first + chunk_of(i) * C;
#pragma unroll
                for (int t = 0; t < TILES; t++) {
                    const int k = loaded % SLOTS;
                    if (loaded >= SLOTS && !mbar_wait(&empty[k], (loaded / SLOTS + 1) & 1, &abort_sh, a.status, 40)) {
                        ok = false;
                        break;
                    }
                    const bool is_c = t == TILES - 1;
                    const int panels = is_c ? a.panels_v : a.panels_k;
                    const CUtensorMap* map = is_c ? &mc : t == 0 ? &mb : &ma;
                    mbar_expect_tx(&full[k], panels * PANEL);
                    for (int p = 0; p < panels; p++)
                        tma_load_4d(sm + k * SLOT + p * PANEL, map, 64 * p, is_c ? hv : hk, t0, b, &full[k]);
                    loaded++;
                }
            }
        }
    } else if (warp == 13) {
        if (lane == 0) {
            const int dk = 64 * a.panels_k, dv = 64 * a.panels_v;
            const uint32_t id_p = idesc_bf16(128, 128, 0, 0), id_x = idesc_bf16(128, dv, 0, 0);
            const uint32_t id_y = idesc_bf16(128, dv, 0, 1), id_s = idesc_bf16(128, dk, 1, 1);
            int piece = 0;
            for (int i = 0; i < nc; i++) {
                const int tb = i * TILES, ta = tb + 1, tc = tb + TILES - 1;
                const uint32_t bt = sb + tb % SLOTS * SLOT, at = sb + ta % SLOTS * SLOT, ct = sb + tc % SLOTS * SLOT;
                const int nj = (tokens_of(i) + 15) / 16;  // 16-token steps that hold tokens
                if (!mbar_wait(&full[tb % SLOTS], tb / SLOTS & 1, &abort_sh, a.status, 41)) break;
                if (MIX) {
                    if (!mbar_wait(&full[ta % SLOTS], ta / SLOTS & 1, &abort_sh, a.status, 42)) break;
                    tc_fence_after();
                    // P takes the columns of the previous P', which the Y product before it has read
                    for (int k0 = 0; k0 < dk; k0 += 16)
                        mma_bf16(tm + COL_P, desc_kmajor(at, C, 0, k0), desc_kmajor(bt, C, 0, k0), id_p, k0 > 0);
                    mma_commit(&pfull);
                }
                if (!mbar_wait(&full[tc % SLOTS], tc / SLOTS & 1, &abort_sh, a.status, 43)) break;
                if (i > 0 && !mbar_wait(&sfree, (i - 1) & 1, &abort_sh, a.status, 44)) break;
                bool ok = true;
                for (int j = 0; j < nj; j++, piece++) {
                    const int r = piece & 1;
                    if (!(ok = mbar_wait(&bfull[r], piece / 2 & 1, &abort_sh, a.status, 45))) break;
                    tc_fence_after();
                    const uint32_t p = sb + AT_B + r * PIECE;
                    for (int t = 2; t >= 0; t--)  // the smallest term first
                        mma_bf16(tm + CS, desc_mnmajor(ct, C, 0, 16 * j), desc_mnmajor(p + t * TERM, 16, 0, 0), id_s,
                                 j > 0 || t < 2);
                    mma_commit(&bfree[r]);
                }
                if (!ok) break;
                mma_commit(&sfull);
                mma_commit(&empty[tb % SLOTS]);  // every piece has been formed from b
                if (MIX) {
                    if (!mbar_wait(&sready, i & 1, &abort_sh, a.status, 46)) break;
                    if (i > 0 && !mbar_wait(&yfree, (i - 1) & 1, &abort_sh, a.status, 47)) break;
                    tc_fence_after();
                    for (int k0 = 0; k0 < dk; k0 += 16)
                        mma_bf16(tm + COL_X, desc_kmajor(at, C, 0, k0), desc_kmajor(sb + AT_S, C, 0, k0), id_x, k0 > 0);
                    mma_commit(&xdone);
                    if (!mbar_wait(&pready, i & 1, &abort_sh, a.status, 48)) break;
                    tc_fence_after();
                    for (int j = 0; j < nj; j++)
                        mma_bf16_ts(tm + COL_Y, tm + COL_P + 8 * j, desc_mnmajor(ct, C, 0, 16 * j), id_y, j > 0);
                    mma_commit(&yfull);
                }
                mma_commit(&empty[tc % SLOTS]);
            }
            mma_commit(&drain);  // every product issued so far has completed before TMEM is released
            volatile int never = 0;
            mbar_wait(&drain, 0, &never, nullptr, 0);
        }
    } else if (warp < 4) {
        if (MIX) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
            for (int t = max(begin, first + nc * C) + warp; t < end; t += 4)  // past the last chunk: zero
                for (int d = 8 * lane; d < s.Dv; d += 256)
                    *reinterpret_cast<uint4*>(out + (((size_t)b * s.T + t) * s.Hv + hv) * s.Dv + d) = make_uint4(0, 0, 0, 0);
            const int r = tid;
            const uint32_t row = tm + ((uint32_t)(32 * warp) << 16);
            bool bad = false;
            for (int i = 0; i < nc && !bad; i++) {
                const int m = tokens_of(i), ta = i * TILES + 1;
                bool ok = __all_sync(0xffffffffu, mbar_wait(&pfull, i & 1, &abort_sh, a.status, 50));
                tc_fence_after();
                if (ok) {
#pragma unroll 1
                    for (int cb = 0; cb < 4; cb++) {
                        uint32_t w[16];
                        if (a.reverse ? cb < warp : cb > warp) {  // no pair of tokens in order
#pragma unroll
                            for (int e = 0; e < 16; e++) w[e] = 0;
                        } else {
                            float p[32];
                            tmem_ld32(row + COL_P + 32 * cb, p);
                            tmem_wait_ld();
                            if (cb == warp) {
#pragma unroll
                                for (int e = 0; e < 32; e++) {
                                    const int d = a.reverse ? e - lane : lane - e;
                                    p[e] = d >= 0 && 32 * cb + e < m ? a.fp * pw[max(d, 0)] * p[e] : 0.f;
                                }
                            } else {  // l^|r-j| as l to the tokens up to this block of columns, times l to those in it
                                const float f = a.fp * (a.reverse ? pw[32 * cb - r] : pw[r - 32 * cb - 31]);
                                const float* in = a.reverse ? pw : pd;
#pragma unroll
                                for (int e = 0; e < 32; e += 4) {
                                    const float4 x = *reinterpret_cast<const float4*>(in + e);
                                    p[e] *= f * x.x;
                                    p[e + 1] *= f * x.y;
                                    p[e + 2] *= f * x.z;
                                    p[e + 3] *= f * x.w;
                                }
                                if (32 * cb + 32 > m)
#pragma unroll
                                    for (int e = 0; e < 32; e++) p[e] = 32 * cb + e < m ? p[e] : 0.f;
                            }
#pragma unroll
                            for (int e = 0; e < 16; e++) w[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
                        }
                        // the packed block lands on columns of P that this warp has already read
                        tmem_st16(row + COL_P + 16 * cb, w);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pready);
                }
                ok = ok && __all_sync(0xffffffffu, mbar_wait(&yfull, i & 1, &abort_sh, a.status, 51));
                tc_fence_after();
                const uint32_t stage = sb + ta % SLOTS * SLOT;
                if (ok) {
                    const float f = a.fx * pw[a.reverse ? max(m - 1 - r, 0) : r + 1];
#pragma unroll 1
                    for (int cb = 0; cb < 2 * a.panels_v; cb++) {
                        float x[32], y[32];
                        tmem_ld32(row + COL_X + 32 * cb, x);
                        tmem_ld32(row + COL_Y + 32 * cb, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e++) x[e] = r < m ? f * x[e] + y[e] : 0.f;
#pragma unroll
                        for (int e = 0; e < 4; e++) st_chunk(stage + sw128_chunk(r, 4 * cb + e, C), x + 8 * e, 1.f);
                    }
                    tc_fence_before();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&yfree);
                }
                bad = bar_sync_or(1, 128, !ok || abort_sh);
                if (!bad && tid == 0) {
                    for (int p = 0; p < a.panels_v; p++)
                        tma_store_4d(&mo, sm + ta % SLOTS * SLOT + p * PANEL, 64 * p, hv, first + chunk_of(i) * C, b);
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(&empty[ta % SLOTS]);
                }
            }
            if (tid == 0) bulk_wait_all();
        }
    } else {
        const int et = tid - 128, half = (warp - 4) >> 2;
        const int row = 32 * (warp & 3) + lane;  // state row; columns 64 half ..
        const bool mine = half < a.panels_k;
        const uint32_t acc = tm + ((uint32_t)(32 * (warp & 3)) << 16) + CS + 64 * half;
        const size_t state = (size_t)s.Dv * s.Dk;
        float S[64];
        {
            const float* p = a.start ? a.start + (bh * a.start_segs + (a.start_segs > 1 ? seg : 0)) * state : nullptr;
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                const bool in = MIX && p && row < s.Dv && 64 * half + e < s.Dk;
                const float4 x = in ? *reinterpret_cast<const float4*>(p + (size_t)row * s.Dk + 64 * half + e)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
            }
        }
        auto write_state = [&]() {  // the bf16 copy that X reads
            if (mine)
#pragma unroll
                for (int e = 0; e < 8; e++) st_chunk(sb + AT_S + sw128_chunk(row, 8 * half + e, C), S + 8 * e, 1.f);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sready);
        };
        if (MIX) write_state();
        int piece = 0;
        const int u = et >> 4, ch = et & 15;  // this thread's token row and 16-byte chunk of a piece
        for (int i = 0; i < nc; i++) {
            const int m = tokens_of(i), tb = i * TILES, tc = tb + TILES - 1, nj = (m + 15) / 16;
            bool ok = __all_sync(0xffffffffu, mbar_wait(&full[tb % SLOTS], tb / SLOTS & 1, &abort_sh, a.status, 60));
            if (ok && (m & 15) && s.lengths) {
                // rows of c past the last token enter the last 16-token step: zero, whatever they hold
                ok = __all_sync(0xffffffffu, mbar_wait(&full[tc % SLOTS], tc / SLOTS & 1, &abort_sh, a.status, 61));
                const int z = m + u;
                if (ok && z < 16 * nj && ch < 8 * a.panels_v)
                    st_shared_v4(sb + tc % SLOTS * SLOT + sw128_chunk(z, ch, C), 0, 0, 0, 0);
            }
            for (int j = 0; j < nj && ok; j++, piece++) {
                const int r = piece & 1;
                if (piece >= 2)
                    ok = __all_sync(0xffffffffu, mbar_wait(&bfree[r], (piece / 2 + 1) & 1, &abort_sh, a.status, 62));
                if (!ok) break;
                if (ch < 8 * a.panels_k) {
                    const int t = 16 * j + u;
                    const uint4 v = ld_shared_v4(sb + tb % SLOTS * SLOT + sw128_chunk(t, ch, C));
                    const float w = t < m ? a.fu * pw[a.reverse ? t + 1 : m - 1 - t] : 0.f;
                    float x[8];
                    unpack8(v, x);
                    uint32_t h[4], d[4], l[4];
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        split3(t < m ? w * x[2 * e] : 0.f, t < m ? w * x[2 * e + 1] : 0.f, h[e], d[e], l[e]);
                    const uint32_t to = sb + AT_B + r * PIECE + sw128_chunk(u, ch, 16);
                    st_shared_v4(to, h[0], h[1], h[2], h[3]);
                    st_shared_v4(to + TERM, d[0], d[1], d[2], d[3]);
                    st_shared_v4(to + 2 * TERM, l[0], l[1], l[2], l[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bfull[r]);
            }
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&sfull, i & 1, &abort_sh, a.status, 63));
            if (!ok) break;
            tc_fence_after();
            const float over = pw[m];
            if (mine) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float d[32];
                    tmem_ld32(acc + 32 * h, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e++) S[32 * h + e] = over * S[32 * h + e] + d[e];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfree);
            if (MIX && i + 1 < nc) {
                if (!__all_sync(0xffffffffu, mbar_wait(&xdone, i & 1, &abort_sh, a.status, 64))) break;
                write_state();
            }
        }
        float* to = nullptr;
        if (!MIX) to = a.z + (bh * s.nseg + seg) * state;
        else if (a.last && seg == (a.reverse ? 0 : s.nseg - 1)) to = a.last + bh * state;
        if (to && mine && row < s.Dv)
#pragma unroll
            for (int e = 0; e < 64; e += 4)
                if (64 * half + e < s.Dk)
                    *reinterpret_cast<float4*>(to + (size_t)row * s.Dk + 64 * half + e) =
                        make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
    tc_fence_before();
    __syncthreads();
    if (abort_sh && warp == 12 && lane == 0) {  // copies still in flight must land first
        volatile int never = 0;
        for (int i = loaded > SLOTS ? loaded - SLOTS : 0; i < loaded; i++)
            mbar_wait(&full[i % SLOTS], i / SLOTS & 1, &never, nullptr, 0);
    }
    __syncthreads();
    if (warp == 12) tmem_dealloc(tm, COLS);
}

// Tiles of one 64-channel panel and 128 tokens of a [B, T, H, D] tensor.
bool tile_map(CUtensorMap* m, const void* p, const LinearShape& s, int H, int D) {
    return make_map_4d_bf16(m, p, D, H, s.T, s.B, 64, C, CU_TENSOR_MAP_SWIZZLE_128B);
}

int panels(int d) { return d > 64 ? 2 : 1; }

// Before the tensor maps: the first runtime call of a host thread (autograd's, say) makes the device's
// context current there, which encoding a map needs.
template <bool MIX>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(linear_tc_kernel<MIX>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES + 1024);
}

template <bool MIX>
cudaError_t launch(const CUtensorMap* maps, const TcArgs& a, int segs, const char* name, cudaStream_t st) {
    trace_begin(name, st);
    linear_tc_kernel<MIX><<<dim3(segs, a.s.Hv, a.s.B), THREADS, BYTES + 1024, st>>>(maps[0], maps[1], maps[2], maps[3], a);
    trace_end(st);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_tc_summary(const LinearSummaryArgs& x, int* status, bool clear, cudaStream_t st) {
    if (cudaError_t e = allow_smem<false>()) return e;
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
    return launch<false>(maps, a, x.s.nseg - 1, "linear_summary", st);
}

cudaError_t launch_linear_tc_mix(const LinearMixArgs& x, const float* start, int start_segs, float* last, int* status,
                                 bool clear, cudaStream_t st) {
    const bool rev = x.pass == LINEAR_DV;
    if (cudaError_t e = allow_smem<true>()) return e;
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
    a.status = status;
    a.clear_status = clear;
    return launch<true>(maps, a, x.s.nseg, rev ? "linear_dv" : "linear_o", st);
}

// Segments of whole chunks, one CTA each, on 152 SMs. In units of one chunk of the mix pass: a wave
// of it takes a segment's chunks and about three for its start, with several segments there is
// the summary too, at about 0.6 a chunk, and the combine step reads every segment's state.
int linear_tc_segments(int B, int T, int Hv) {
    const long long chunks = (T + C - 1) / C, heads = (long long)B * Hv;
    if (chunks <= 1 || heads <= 0) return 1;
    int best = 1;
    double least = 1e300;
    for (long long n = 1; n <= chunks && (n == 1 || heads * n <= 8 * 152); n++) {
        const long long len = (chunks + n - 1) / n, real = (chunks + len - 1) / len;
        const double mix = (double)((heads * real + 151) / 152) * (len + 3);
        const double sum = real > 1 ? (double)((heads * (real - 1) + 151) / 152) * (0.6 * len + 3) + 3 + 0.2 * real : 0.0;
        if (mix + sum < least) {
            least = mix + sum;
            best = (int)real;
        }
    }
    return best;
}

}  // namespace gdr
