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
// registers. Rounding to bf16: P', the kept states (operands of the products; the states themselves are
// carried in fp32 by the passes that keep these copies) and the results, one rounding each.
//
// HBM bounds it: per value head do, v and the two states (128 KB), per key head q, k, dq, dk. One CTA per
// SM takes the (b, chunk, key head) units in turn, key heads fastest, so that the CTAs at work read
// neighbouring rows, and its value heads run as one stream across them: the tiles of the next head are
// copied in as each product releases its operand, the products of P' are issued a head late, between
// the next head's, so that the tensor pipe works while P' is formed, and the results leave through the
// slots of q and k while the next unit's first head is under way. (One CTA per unit, each with its
// own start and end: 354 us at T = 32768, Hk 16, Hv 32, D 128; so 274, 1.57 GB at 85% of a plain
// copy's rate.)
// Warps 0-15 form P' (a thread is a quarter of a row); then 0-7 hold dq and 8-15 dk (half a row each);
// 16 copies, 17 issues, 18 stores.
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
    void *dq, *dk;
    int panels_k, panels_v;
    int* status;
};

__global__ void __launch_bounds__(THREADS, 1)
    linear_grad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                       const __grid_constant__ CUtensorMap mdq, const __grid_constant__ CUtensorMap mdk, GradArgs a) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    // counted by head of the stream: full .. yread; by unit: qk .. accfree
    __shared__ uint64_t full[4], empty[4], pfull, pready, pfree, xfull, xread, yfull, yread;
    __shared__ uint64_t qk, done, staged, qkfree, accfree, drain;
    __shared__ float tables[2][160];
    __shared__ uint32_t tmem_sh;
    __shared__ int failed, used[5];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const LinearShape& s = a.s;
    const int G = s.Hv / s.Hk, NC = (s.T + C - 1) / C;
    const long long units = (long long)s.B * NC * s.Hk;
    struct Unit {
        int b, chunk, hk, m;  // m: its tokens
    };
    auto unit_at = [&](long long u) {
        Unit x;
        x.hk = (int)(u % s.Hk);
        x.chunk = (int)(u / s.Hk % NC);
        x.b = (int)(u / s.Hk / NC);
        const int n = s.lengths ? min(max(s.lengths[x.b], 0), s.T) : s.T;
        x.m = min(max(n - x.chunk * C, 0), C);
        return x;
    };
    // tables[.][31 + r - j] = scale l^(r-j) for j <= r, else 0, of value head hv
    auto make_table = [&](int which, int hv, int i) {
        if (i < 160) tables[which][i] = i >= 31 ? a.scale * power(s.g[hv], i - 31) : 0.f;
    };
    if (sb & 1023u) {  // never on this layout; swizzled tiles would be read wrongly
        if (tid == 0) a.status[0] = -1;
        return;
    }
    if (tid == 0) {
        failed = 0;
        for (int i = 0; i < 4; i++) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 5; i++) used[i] = 0;
        mbar_init(&pfull, 1);
        mbar_init(&pready, 16);
        mbar_init(&pfree, 1);
        mbar_init(&xfull, 1);
        mbar_init(&xread, 8);
        mbar_init(&yfull, 1);
        mbar_init(&yread, 8);
        mbar_init(&qk, 1);
        mbar_init(&done, 1);
        mbar_init(&staged, 16);
        mbar_init(&qkfree, 1);
        mbar_init(&accfree, 16);
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
    auto wait = [&](uint64_t* bar, int phase, int site) { return wait_phase(bar, phase & 1, &failed, site); };

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
        if (warp == 16) {
            wait_kernel_before();  // the adjoints
            int t = 0, k = 0;  // heads and units so far
            bool ok = true;
#pragma unroll 1
            for (long long u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit x = unit_at(u);
                if (x.m == 0) continue;
                const int t0 = x.chunk * C;
#pragma unroll 1
                for (int h = 0; h < G && ok; h++, t++) {
                    const int hv = x.hk * G + h;
                    const size_t image = (((size_t)x.b * s.Hv + hv) * NC + x.chunk) * TILE;
#pragma unroll 1
                    for (int i = 0; i < 4 && ok; i++) {  // do, v, S, D
                        ok = t == 0 || wait(&empty[i], t - 1, 70);
                        if (ok && lane == 0) {
                            uint8_t* to = sm + AT_HEAD + i * TILE;
                            mbar_expect_tx(&full[i], (i < 2 ? a.panels_v : a.panels_k) * PANEL);
                            used[i] = t + 1;
                            if (i < 2) {
#pragma unroll 1
                                for (int p = 0; p < a.panels_v; p++)
                                    tma_load_4d(to + p * PANEL, i == DO ? &mdo : &mv, 64 * p, hv, t0, x.b, &full[i]);
                            } else {
                                bulk_load(to, (i == S0 ? a.states : a.adjoints) + image, a.panels_k * PANEL, &full[i]);
                            }
                        }
                        __syncwarp();
                    }
                    if (h > 0 || !ok) continue;
                    ok = k == 0 || wait(&qkfree, k - 1, 71);
                    if (ok && lane == 0) {
                        mbar_expect_tx(&qk, 2 * a.panels_k * PANEL);
                        used[4] = k + 1;
#pragma unroll 1
                        for (int p = 0; p < a.panels_k; p++) {
                            tma_load_4d(sm + AT_Q + p * PANEL, &mq, 64 * p, x.hk, t0, x.b, &qk);
                            tma_load_4d(sm + AT_K + p * PANEL, &mk, 64 * p, x.hk, t0, x.b, &qk);
                        }
                    }
                    __syncwarp();
                    k++;
                }
            }
        } else if (warp == 17) {
            const int dk = 64 * a.panels_k;
            const uint32_t id_p = idesc_bf16(128, 128, 0, 0), id_x = idesc_bf16(128, dk, 0, 1);
            const uint32_t id_t = idesc_bf16(128, dk, 1, 1);
            auto tile = [&](int i) { return sb + AT_HEAD + i * TILE; };
            int t = 0, k = 0;
            // the products of P' of head t, the h-th of its unit
            auto issue_p = [&](int t, int h, int nj) {
                if (h == 0 && (!wait(&qk, k, 72) || (k > 0 && !wait(&accfree, k - 1, 73)))) return false;
                if (!wait(&pready, t, 77)) return false;
                tc_fence_after();
                const uint32_t pk = lo_kmajor(sb + AT_P), pm = lo_mnmajor(sb + AT_P);
                const uint32_t kd = lo_mnmajor(sb + AT_K), qd = lo_mnmajor(sb + AT_Q);
#pragma unroll 1
                for (int j = 0; j < nj; j++) {
                    mma_ss(tm + COL_DQ, pk + (j >> 2) * (PANEL >> 4) + 2 * (j & 3), kd + step_mnmajor(j), id_x, h > 0 || j > 0);
                    mma_ss(tm + COL_DK, pm + step_mnmajor(j), qd + step_mnmajor(j), id_t, h > 0 || j > 0);
                }
                commit(&pfree);
                return true;
            };
            bool ok = true;
#pragma unroll 1
            for (long long u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit x = unit_at(u);
                const int nj = (x.m + 15) / 16;
                if (x.m == 0) continue;
#pragma unroll 1
                for (int h = 0; h < G && ok; h++, t++) {
                    ok = wait(&full[DO], t, 74) && wait(&full[V], t, 75) && (t == 0 || wait(&pready, t - 1, 76));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t od = lo_kmajor(tile(DO)), vd = lo_kmajor(tile(V));
#pragma unroll 1
                    for (int p = 0; p < a.panels_v; p++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            mma_ss(tm + COL_P, od + p * (PANEL >> 4) + 2 * e, vd + p * (PANEL >> 4) + 2 * e, id_p, e > 0 ? 1u : p);
                    commit(&pfull);
#pragma unroll 1
                    for (int y = 0; y < 2 && ok; y++) {  // do S, then v D, in the same columns
                        if (y == 1 && h > 0) ok = issue_p(t - 1, h - 1, nj);
                        ok = ok && wait(&full[S0 + y], t, 78) && (y == 0 ? t == 0 || wait(&yread, t - 1, 79) : wait(&xread, t, 80));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t ad = lo_kmajor(tile(DO + y)), bd = lo_mnmajor(tile(S0 + y));
#pragma unroll 1
                        for (int p = 0; p < a.panels_v; p++)
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                mma_ss(tm + COL_X, ad + p * (PANEL >> 4) + 2 * e, bd + p * step_mnmajor(4) + step_mnmajor(e), id_x,
                                       e > 0 ? 1u : p);
                        commit(y == 0 ? &xfull : &yfull);
                        commit(&empty[DO + y]);
                        commit(&empty[S0 + y]);
                    }
                }
                ok = ok && issue_p(t - 1, G - 1, nj);
                if (ok) commit(&done);
                k++;
            }
            commit(&drain);  // every product issued so far has completed before TMEM is released
            int never = 0;
            wait_phase(&drain, 0, &never, 1);
        } else if (warp == 18) {
            int k = 0;
#pragma unroll 1
            for (long long u = blockIdx.x; u < units; u += gridDim.x) {
                const Unit x = unit_at(u);
                if (x.m == 0) continue;
                if (!wait(&staged, k++, 81)) break;
                if (lane == 0) {
#pragma unroll 1
                    for (int p = 0; p < a.panels_k; p++) {
                        tma_store_4d(&mdq, sm + AT_Q + p * PANEL, 64 * p, x.hk, x.chunk * C, x.b);
                        tma_store_4d(&mdk, sm + AT_K + p * PANEL, 64 * p, x.hk, x.chunk * C, x.b);
                    }
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(&qkfree);
                }
                __syncwarp();
            }
            if (lane == 0) bulk_wait_all();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_ROWS));
        const int quarter = warp & 3, r = 32 * quarter + lane;  // row of P and of dq or dk
        const int cb = warp >> 2;                               // columns 32 cb .. of P
        const bool is_k = warp >= 8;                            // holds dk, else dq
        const int half = cb & 1;                                // columns 64 half .. of it
        const bool mine = half < a.panels_k;
        const uint32_t row = tm + ((uint32_t)(32 * quarter) << 16);
        int t = 0, k = 0;
        bool ok = true;
#pragma unroll 1
        for (long long u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const Unit x = unit_at(u);
            const int m = x.m, nj = (m + 15) / 16;
            if (m == 0) {  // past the length: zero
                const int per = s.Dk / 8;  // 16-byte chunks of a row
                for (int i = tid; i < 2 * min(C, s.T - x.chunk * C) * per; i += ROWS) {
                    const int at = i >> 1;
                    uint8_t* to = static_cast<uint8_t*>(i & 1 ? a.dk : a.dq);
                    const size_t token = (size_t)x.b * s.T + x.chunk * C + at / per;
                    *reinterpret_cast<uint4*>(to + ((token * s.Hk + x.hk) * s.Dk + at % per * 8) * 2) = make_uint4(0, 0, 0, 0);
                }
                continue;
            }
            if (s.lengths && (m & 15)) {
                // rows past the last token that enter the last 16-token step of a sum over tokens: zero
                ok = wait(&qk, k, 82);
                const int z = m + (tid >> 5), ch = tid & 15;
                if (ok && z < 16 * nj && ch < 8 * a.panels_k)
                    st_shared_v4(sb + (tid & 16 ? AT_Q : AT_K) + sw128_chunk(z, ch, C), 0, 0, 0, 0);
            }
            float acc[64];
#pragma unroll
            for (int e = 0; e < 64; e++) acc[e] = 0.f;
#pragma unroll 1
            for (int h = 0; h < G && ok; h++, t++) {
                const int hv = x.hk * G + h;
                const float g = s.g[hv];
                // This head's table, by each warp for itself alone: the same values in the same places.
                // (Heads two apart share a buffer; the products of P' lie between them.)
#pragma unroll 1
                for (int i = lane; i < 160; i += 32) make_table(t & 1, hv, i);
                __syncwarp();
                ok = wait(&pfull, t, 83);
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
                    const float* in = tables[t & 1] + 31 + r - 32 * cb;
#pragma unroll
                    for (int e = 0; e < 32; e++) p[e] *= in[-e];
#pragma unroll
                    for (int e = 0; e < 16; e++) w[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
                }
                tc_fence_before();
                if (t > 0) ok = ok && wait(&pfree, t - 1, 84);  // the last P' has been read
                if (!ok) break;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    st_shared_v4(sb + AT_P + sw128_chunk(r, 4 * cb + e, C), w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pready);
                if (!(ok = wait(is_k ? &yfull : &xfull, t, 85))) break;
                tc_fence_after();
                if (mine) {
                    const float f = is_k ? power(g, max(m - 1 - r, 0)) : a.scale * power(g, r + 1);
#pragma unroll
                    for (int e = 0; e < 64; e += 16) {
                        float v[16];
                        tmem_ld16(row + COL_X + 64 * half + e, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i++) acc[e + i] += f * v[i];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(is_k ? &yread : &xread);
            }
            ok = ok && wait(&done, k++, 86);
            if (!ok) break;
            tc_fence_after();
            if (mine) {  // q and k have been read
                const uint32_t stage = sb + (is_k ? AT_K : AT_Q);
#pragma unroll
                for (int e = 0; e < 64; e += 16) {
                    float v[16];
                    tmem_ld16(row + (is_k ? COL_DK : COL_DQ) + 64 * half + e, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i++) v[i] = r < m ? v[i] + acc[e + i] : 0.f;
                    st_chunk(stage + sw128_chunk(r, 8 * half + e / 8, C), v, 1.f);
                    st_chunk(stage + sw128_chunk(r, 8 * half + e / 8 + 1, C), v + 8, 1.f);
                }
            }
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&accfree);
                mbar_arrive(&staged);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (failed && tid == 0) {
        if (atomicCAS(a.status, 0, DEV_TIMEOUT) == 0) {
            a.status[1] = blockIdx.x;
            a.status[2] = failed;
        }
        int never = 0;  // copies still in flight must land first
        for (int i = 0; i < 5; i++)
            if (used[i]) mbar_wait(i < 4 ? &full[i] : &qk, (used[i] - 1) & 1, &never, nullptr, 0);
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
    a.dq = x.dq;
    a.dk = x.dk;
    a.panels_k = panels(s.Dk);
    a.panels_v = panels(s.Dv);
    a.status = x.status;
    trace_begin("linear_grad", st);
    const long long units = (long long)s.B * ((s.T + C - 1) / C) * s.Hk;
    const cudaError_t e = launch_after(linear_grad_kernel, dim3((unsigned)(units < 152 ? units : 152)), THREADS, BYTES, st,
                                       true, mq, mk, mv, mdo, mdq, mdk, a);
    trace_end(st);
    return e;
}

}  // namespace gdr
