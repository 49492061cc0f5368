// linear_grad.cu - dq and dk of linear attention with a constant decay per head, for bf16, from the states
// that the o and dv passes kept for each 128-token chunk (linear.h).
//
// With S the state before a chunk and D the adjoint of the state after it, per (b, key head,
// chunk) and value head h that shares the key head, tokens r, j of the chunk, m of them valid,
//
//     P = do v^T,   P'_rj = scale l^(r-j) P_rj for j <= r, else 0
//     dq_r = sum_h scale l^(r+1) (do S)_r + (P' k)_r
//     dk_j = sum_h l^(m-1-j) (v D)_j + (P'^T q)_j
//
// with do, v as [tokens, Dv] and S, D as [Dv, Dk]. A CTA owns one (b, key head, chunk), so
// the sum over value heads needs no atomics and its order is fixed: the P' products accumulate
// over the heads in TMEM, the state products, which every row scales by its own decay, in fp32
// registers. Rounding to bf16: P', the kept states and the results.
//
// HBM bounds it: per value head do, v and the two states (128 KB), per key head q, k, dq, dk. The
// tiles of the next head are copied in as each product releases its operand, and the products of
// P' are issued a head late, between the next head's, so that the tensor pipe works while P' is formed.
// Warps 0-15 form P' (a thread is a quarter of a row); then 0-7 hold dq and 8-15 dk (half a row each);
// 16 copies, 17 issues.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "linear.h"
#include "linear_dev.cuh"
#include "linear_host.h"

namespace gdr {

using namespace linear;

namespace {

constexpr int THREADS = 640, ROWS = 512;  // threads; those that hold rows
constexpr int REGS_ROWS = 104, REGS_REST = 64;
static_assert(4 * REGS_ROWS + REGS_REST <= 5 * 96, "registers of the launch");
// Tiles: q, k and P' for the whole CTA; do, v, S, D of one value head.
constexpr uint32_t AT_Q = 0, AT_K = TILE, AT_P = 2 * TILE, AT_HEAD = 3 * TILE;
constexpr uint32_t BYTES = 7 * TILE;
static_assert(BYTES + 1536 <= 232448, "shared memory");
enum { DO = 0, V = 1, S0 = 2, D1 = 3 };  // tiles of a head
constexpr uint32_t COL_P = 0, COL_X = 128, COL_DQ = 256, COL_DK = 384;

struct GradArgs {
    LinearShape s;
    float scale;
    const uint8_t *states, *adjoints;
    int panels_k, panels_v;
    int* status;
};

__global__ void __launch_bounds__(THREADS, 1)
    linear_grad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                       const __grid_constant__ CUtensorMap mdq, const __grid_constant__ CUtensorMap mdk, GradArgs a) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    __shared__ uint64_t qk, full[4], empty[4], pfull, pready, pfree, xfull, xread, yfull, yread, done, drain;
    __shared__ float tables[2][96];
    __shared__ uint32_t tmem_sh;
    __shared__ int failed, used[4];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const LinearShape& s = a.s;
    const int chunk = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, G = s.Hv / s.Hk;
    const int n = s.lengths ? min(max(s.lengths[b], 0), s.T) : s.T;
    const int t0 = chunk * C, m = min(max(n - t0, 0), C), nj = (m + 15) / 16;
    if (sb & 1023u) {  // never on this layout; swizzled tiles would be read wrongly
        if (tid == 0) a.status[0] = -1;
        return;
    }
    if (tid == 0) {
        failed = 0;
        for (int i = 0; i < 4; i++) {
            used[i] = 0;
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&qk, 1);
        mbar_init(&pfull, 1);
        mbar_init(&pready, 16);
        mbar_init(&pfree, 1);
        mbar_init(&xfull, 1);
        mbar_init(&xread, 8);
        mbar_init(&yfull, 1);
        mbar_init(&yread, 8);
        mbar_init(&done, 1);
        mbar_init(&drain, 1);
        fence_barrier_init();
    }
    if (warp == 16) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_sh;

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
        if (warp == 16 && m > 0) {
            if (lane == 0) {
                mbar_expect_tx(&qk, 2 * a.panels_k * PANEL);
                for (int p = 0; p < a.panels_k; p++) {
                    tma_load_4d(sm + AT_Q + p * PANEL, &mq, 64 * p, hk, t0, b, &qk);
                    tma_load_4d(sm + AT_K + p * PANEL, &mk, 64 * p, hk, t0, b, &qk);
                }
            }
            const int NC = (s.T + C - 1) / C;
            for (int h = 0; h < G; h++) {
                const int hv = hk * G + h;
                const size_t image = (((size_t)b * s.Hv + hv) * NC + chunk) * TILE;
                bool ok = true;
                for (int t = 0; t < 4; t++) {  // do, v, S, D
                    ok = ok && (h == 0 || wait_phase(&empty[t], (h + 1) & 1, &failed, 70));
                    if (ok && lane == 0) {
                        uint8_t* to = sm + AT_HEAD + t * TILE;
                        mbar_expect_tx(&full[t], (t < 2 ? a.panels_v : a.panels_k) * PANEL);
                        if (t < 2)
                            for (int p = 0; p < a.panels_v; p++)
                                tma_load_4d(to + p * PANEL, t == DO ? &mdo : &mv, 64 * p, hv, t0, b, &full[t]);
                        else
                            bulk_load(to, (t == S0 ? a.states : a.adjoints) + image, a.panels_k * PANEL, &full[t]);
                        used[t] = h + 1;
                    }
                }
                if (!ok) break;
            }
        } else if (warp == 17 && m > 0) {
            const int dk = 64 * a.panels_k;
            const uint32_t id_p = idesc_bf16(128, 128, 0, 0), id_x = idesc_bf16(128, dk, 0, 1);
            const uint32_t id_t = idesc_bf16(128, dk, 1, 1);
            auto wait = [&](uint64_t* bar, int parity, int site) { return wait_phase(bar, parity & 1, &failed, site); };
            auto tile = [&](int t) { return sb + AT_HEAD + t * TILE; };
            // rows of `x` times the kept state in tile t
            auto state_product = [&](int x, int t) {
                const uint32_t ad = lo_kmajor(tile(x)), bd = lo_mnmajor(tile(t));
#pragma unroll 1
                for (int p = 0; p < a.panels_v; p++)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        mma_ss(tm + COL_X, ad + p * (PANEL >> 4) + 2 * k, bd + p * step_mnmajor(4) + step_mnmajor(k), id_x,
                               k > 0 ? 1u : p);
            };
            bool ok = wait(&qk, 0, 71);
            for (int h = 0; h <= G && ok; h++) {
                if (h < G) {
                    if (!wait(&full[DO], h, 72) || !wait(&full[V], h, 73)) break;
                    if (h > 0 && !wait(&pready, h - 1, 74)) break;  // P has been read
                    tc_fence_after();
                    const uint32_t ad = lo_kmajor(tile(DO)), bd = lo_kmajor(tile(V));
#pragma unroll 1
                    for (int p = 0; p < a.panels_v; p++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            mma_ss(tm + COL_P, ad + p * (PANEL >> 4) + 2 * k, bd + p * (PANEL >> 4) + 2 * k, id_p, k > 0 ? 1u : p);
                    commit(&pfull);
                    if (!wait(&full[S0], h, 75)) break;
                    if (h > 0 && !wait(&yread, h - 1, 76)) break;
                    tc_fence_after();
                    state_product(DO, S0);
                    commit(&xfull);
                    commit(&empty[DO]);
                    commit(&empty[S0]);
                }
                if (h > 0) {
                    if (!wait(&pready, h - 1, 77)) break;
                    tc_fence_after();
                    const uint32_t pk = lo_kmajor(sb + AT_P), pm = lo_mnmajor(sb + AT_P);
                    const uint32_t kd = lo_mnmajor(sb + AT_K), qd = lo_mnmajor(sb + AT_Q);
#pragma unroll 1
                    for (int j = 0; j < nj; j++) {
                        mma_ss(tm + COL_DQ, pk + (j >> 2) * (PANEL >> 4) + 2 * (j & 3), kd + step_mnmajor(j), id_x, h > 1 || j > 0);
                        mma_ss(tm + COL_DK, pm + step_mnmajor(j), qd + step_mnmajor(j), id_t, h > 1 || j > 0);
                    }
                    commit(h == G ? &done : &pfree);
                }
                if (h < G) {
                    if (!wait(&full[D1], h, 78) || !wait(&xread, h, 79)) break;
                    tc_fence_after();
                    state_product(V, D1);
                    commit(&yfull);
                    commit(&empty[V]);
                    commit(&empty[D1]);
                }
            }
            commit(&drain);  // every product issued so far has completed before TMEM is released
            int never = 0;
            wait_phase(&drain, 0, &never, 1);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_ROWS));
        const int quarter = warp & 3, r = 32 * quarter + lane;  // row of P and of dq or dk
        const int cb = warp >> 2;                               // columns 32 cb .. of P
        const bool is_k = warp >= 8;                            // holds dk, else dq
        const int half = cb & 1;                                // columns 64 half .. of it
        const uint32_t row = tm + ((uint32_t)(32 * quarter) << 16);
        // l^(31-i) for i < 32; at 64 + r - j for rows and columns of a diagonal block: scale l^(r-j) for j <= r, else 0
        auto make_table = [&](int h) {
            const float g = s.g[hk * G + h];
            float* t = tables[h & 1];
            if (tid < 32) t[tid] = power(g, 31 - tid);
            else if (tid < 96) t[tid] = tid >= 64 ? a.scale * power(g, tid - 64) : 0.f;
        };
        float acc[64];
#pragma unroll
        for (int e = 0; e < 64; e++) acc[e] = 0.f;
        bool bad = m == 0;
        if (!bad) {
            make_table(0);
            // rows past the last token that enter the last 16-token step of a sum over tokens: zero
            bool ok = wait_phase(&qk, 0, &failed, 80);
            const int z = m + (tid >> 5), ch = tid & 15;
            if (ok && (m & 15) && z < 16 * nj && ch < 8 * a.panels_k)
                st_shared_v4(sb + (tid & 16 ? AT_Q : AT_K) + sw128_chunk(z, ch, C), 0, 0, 0, 0);
            bad = bar_sync_or(1, ROWS, !ok);
        }
#pragma unroll 1
        for (int h = 0; h < G && !bad; h++) {
            const float g = s.g[hk * G + h];
            const float* table = tables[h & 1];
            bool ok = wait_phase(&pfull, h & 1, &failed, 81);
            tc_fence_after();
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; e++) w[e] = 0;
            if (ok && cb <= quarter) {
                float p[32];
                tmem_ld32(row + COL_P + 32 * cb, p);
                tmem_wait_ld();
                if (32 * cb + 32 > m || r >= m)  // past the last token, whatever was there
#pragma unroll
                    for (int e = 0; e < 32; e++) p[e] = 32 * cb + e < m && r < m ? p[e] : 0.f;
                if (cb == quarter) {
                    const float* in = table + 64 + lane;
#pragma unroll
                    for (int e = 0; e < 32; e++) p[e] *= in[-e];
                } else {  // l^(r-j) as l to the tokens up to this block of columns, times l to those in it
                    const float f = a.scale * power(g, r - 32 * cb - 31);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(table + e);
                        scale2(p + e, x.x, x.y);
                        scale2(p + e + 2, x.z, x.w);
                        scale2(p + e, f);
                        scale2(p + e + 2, f);
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; e++) w[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
            }
            tc_fence_before();
            if (h > 0) ok = ok && wait_phase(&pfree, (h - 1) & 1, &failed, 82);  // the last P' has been read
#pragma unroll
            for (int e = 0; e < 4; e++)
                st_shared_v4(sb + AT_P + sw128_chunk(r, 4 * cb + e, C), w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pready);
            ok = ok && wait_phase(is_k ? &yfull : &xfull, h & 1, &failed, 83);
            tc_fence_after();
            if (ok && half < a.panels_k) {
                const float f = is_k ? power(g, max(m - 1 - r, 0)) : a.scale * power(g, r + 1);
#pragma unroll
                for (int e = 0; e < 64; e += 16) {
                    float x[16];
                    tmem_ld16(row + COL_X + 64 * half + e, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i++) acc[e + i] += f * x[i];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(is_k ? &yread : &xread);
            if (h + 1 < G) make_table(h + 1);
            bad = bar_sync_or(1, ROWS, !ok || failed);
        }
        if (m == 0 || !bad) {
            bool ok = m == 0 || wait_phase(&done, 0, &failed, 84);
            tc_fence_after();
            const uint32_t stage = sb + AT_HEAD + (is_k ? TILE : 0);  // the head's tiles have been read
            if (ok && half < a.panels_k) {
#pragma unroll
                for (int e = 0; e < 64; e += 16) {
                    float x[16];
                    if (m > 0) {
                        tmem_ld16(row + (is_k ? COL_DK : COL_DQ) + 64 * half + e, x);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < 16; i++) x[i] = r < m ? x[i] + acc[e + i] : 0.f;
                    st_chunk(stage + sw128_chunk(r, 8 * half + e / 8, C), x, 1.f);
                    st_chunk(stage + sw128_chunk(r, 8 * half + e / 8 + 1, C), x + 8, 1.f);
                }
            }
            fence_proxy_async_smem();
            bad = bar_sync_or(1, ROWS, !ok);
            if (!bad && tid == 0) {
                for (int p = 0; p < a.panels_k; p++) {
                    tma_store_4d(&mdq, sm + AT_HEAD + p * PANEL, 64 * p, hk, t0, b);
                    tma_store_4d(&mdk, sm + AT_HEAD + TILE + p * PANEL, 64 * p, hk, t0, b);
                }
                bulk_commit();
                bulk_wait_all();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (failed && tid == 0) {
        if (atomicCAS(a.status, 0, DEV_TIMEOUT) == 0) {
            a.status[1] = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
            a.status[2] = failed;
        }
        int never = 0;  // copies still in flight must land first
        mbar_wait(&qk, 0, &never, nullptr, 0);
        for (int t = 0; t < 4; t++)
            if (used[t]) mbar_wait(&full[t], (used[t] - 1) & 1, &never, nullptr, 0);
    }
    __syncthreads();
    if (warp == 16) tmem_dealloc(tm, 512);
}

}  // namespace

cudaError_t launch_linear_tc_grad(const LinearGradArgs& x, cudaStream_t st) {
    // before the tensor maps: see linear_tc.cu
    if (cudaError_t e = cudaFuncSetAttribute(linear_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES)) return e;
    CUtensorMap mq, mk, mv, mdo, mdq, mdk;
    const LinearShape& s = x.s;
    if (!tile_map(&mq, x.q, s, s.Hk, s.Dk) || !tile_map(&mk, x.k, s, s.Hk, s.Dk) || !tile_map(&mv, x.v, s, s.Hv, s.Dv) ||
        !tile_map(&mdo, x.do_, s, s.Hv, s.Dv) || !tile_map(&mdq, x.dq, s, s.Hk, s.Dk) || !tile_map(&mdk, x.dk, s, s.Hk, s.Dk))
        return cudaErrorInvalidValue;
    GradArgs a;
    a.s = s;
    a.scale = x.scale;
    a.states = static_cast<const uint8_t*>(x.states);
    a.adjoints = static_cast<const uint8_t*>(x.adjoints);
    a.panels_k = panels(s.Dk);
    a.panels_v = panels(s.Dv);
    a.status = x.status;
    trace_begin("linear_grad", st);
    linear_grad_kernel<<<dim3((s.T + C - 1) / C, s.Hk, s.B), THREADS, BYTES, st>>>(mq, mk, mv, mdo, mdq, mdk, a);
    trace_end(st);
    return cudaGetLastError();
}

}  // namespace gdr
