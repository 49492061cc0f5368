// window_grad.cu - VJP of window attention on the tensor cores, for bf16 (gdr_window_bwd), from lse and
// delta = sum do o: with c = scale log2 e, per pair of 128-token tiles of queries and keys
//
//     P = 2^(c Q K^T - log2 e lse),  dS = P (dO V^T - delta),  dQ += scale dS K,  dV += P^T dO,  dK += scale dS^T Q.
//
// Two kernels walk the pairs, dq by query tiles and dkv by key tiles, 3 and 4 products a pair: one walk would need 5
// but add one of its results into memory in an order that changes, or hand it on in fp32 through memory. Here each result
// is summed in TMEM, over the heads that share a key head too, and written once.
//
// dkv forms S^T and dP^T (rows: keys), so that P^T and dS^T, over them in TMEM as bf16, are the operands of the sums as
// they are. In order per pair: dV, the next pair's S^T, dK, the next dP^T: each half has the other's time to wait for the
// rows' arithmetic. dq keeps two S, and puts dS over the one that is done with: dP of the next pair, dQ, S of the pair after it.
// dq comes first and forms delta too, from the copy of do that it has.
// Eight warps do the arithmetic, a thread for a row and half of the columns; 8 copies tiles in, 9 issues products, and in dkv 10 fetches
// lse and delta, which lie along the columns there. Units are taken in turn by CTAs that stay, longest first, as one stream.
//
// Where a key tile's queries are many (first tokens that all see) or the units few, a key tile is cut: its pieces leave fp32 sums,
// which a third kernel adds in order.
// Rounding to bf16: P and dS as operands, and the results.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "kernels.h"
#include "linear.h"
#include "window_dev.cuh"
#include "window_host.h"

namespace gdr {

using namespace window;

namespace {

constexpr int THREADS = 384, SLOTS = 5, SMS = 152;
constexpr uint32_t AT_RING = 2 * TILE, BYTES = AT_RING + SLOTS * TILE;  // two operands that stay, then the ring
static_assert(BYTES + 3072 <= 232448, "shared memory");
constexpr int REGS_ROWS = 208, REGS_REST = 80;  // of 168 at the launch
static_assert(2 * REGS_ROWS + REGS_REST <= 3 * 168, "registers of the launch");

struct GradArgs {
    WindowShape s;
    int tiles;            // of the sequence
    int cut, pieces_cut;  // key tiles from the start, pieces of each
    int pieces;           // pieces of the others
    long long units;
    const float* lse;
    const void *o, *rest;
    float* delta;
    void *dq, *dk, *dv;
    float* parts;  // of a cut key tile's pieces: dv, dk [2, 128, D] each
    int* status;
};

__device__ __forceinline__ long long unit_of(long long round) {  // every other round in reverse
    return round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// dq: 128 queries of a head, and the key tiles that they see.
struct QueryUnit {
    int b, h, hk, n, t0;
    KeyTiles tiles;
    __device__ __forceinline__ void set(const GradArgs& a, long long u) {
        const WindowShape& s = a.s;
        const long long per = (long long)s.Hq * s.B;
        const int rest = (int)(u % per);
        t0 = (a.tiles - 1 - (int)(u / per)) * C;
        h = rest % s.Hq;
        b = rest / s.Hq;
        hk = h / (s.Hq / s.Hk);
        n = s.tokens(b);
        tiles = KeyTiles(C, s.window, s.sinks, t0, min(t0 + C, n));
    }
    __device__ __forceinline__ int count() const { return tiles.count(); }
};

// dkv: 128 keys of a head, a piece of the (query head, query tile) pairs that see them.
struct KeyUnit {
    int b, hk, n, j0, per, begin, end;  // pairs begin .. end - 1, `per` query tiles a head
    long long part;                     // index of its piece of `parts`, or -1
    __device__ __forceinline__ void set(const GradArgs& a, long long u) {
        const WindowShape& s = a.s;
        const long long heads = (long long)s.Hk * s.B, cut = heads * a.cut * a.pieces_cut;
        const bool in_cut = u < cut;
        const int pieces = in_cut ? a.pieces_cut : a.pieces;
        const long long v = in_cut ? u : u - cut;
        const int head = (int)(v % heads), piece = (int)(v / heads % pieces), tile = (int)(v / heads / pieces) + (in_cut ? 0 : a.cut);
        hk = head % s.Hk;
        b = head / s.Hk;
        n = s.tokens(b);
        j0 = tile * C;
        per = j0 < n ? (queries_end(C, s.window, s.sinks, j0, n) - j0 + C - 1) / C : 0;
        const long long all = (long long)per * (s.Hq / s.Hk);
        begin = (int)(all * piece / pieces);
        end = (int)(all * (piece + 1) / pieces);
        part = pieces == 1 ? -1 : in_cut || a.pieces_cut == 1 ? v : u;
    }
    __device__ __forceinline__ int count() const { return end - begin; }
    __device__ __forceinline__ int head(const WindowShape& s, int i) const { return hk * (s.Hq / s.Hk) + (begin + i) / per; }
    __device__ __forceinline__ int query(int i) const { return j0 + (begin + i) % per * C; }
};

// A pair of tiles as the product warp needs it.
struct Pair {
    bool some, first, last;
    int m;  // rows of the streamed tiles that hold tokens
};

// The stream of pairs of a CTA's units.
template <typename U>
struct Stream {
    U x;
    long long round = -1;
    int i = 0, count = 0;
    __device__ __forceinline__ Pair next(const GradArgs& a) {
        i++;
        while (i >= count) {
            round++;
            if (round * gridDim.x >= a.units) return Pair{false, false, false, 0};
            const long long u = unit_of(round);
            if (u >= a.units) continue;
            x.set(a, u);
            i = 0;
            count = x.count();
        }
        return Pair{true, i == 0, i + 1 == count, x.n - row0()};
    }
    __device__ __forceinline__ int row0() const;
};
template <>
__device__ __forceinline__ int Stream<QueryUnit>::row0() const { return x.tiles.at(i) * C; }
template <>
__device__ __forceinline__ int Stream<KeyUnit>::row0() const { return x.query(i); }

__device__ __forceinline__ void product_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t id, int ksteps) {  // a b^T over channels
    const uint32_t ad = lo_kmajor(a), bd = lo_kmajor(b);
#pragma unroll
    for (int k = 0; k < 8; k++)
        if (k < ksteps)
            mma_ss(d, ad + (k >> 2) * (PANEL >> 4) + 2 * (k & 3), bd + (k >> 2) * (PANEL >> 4) + 2 * (k & 3), id, k > 0);
}
// += p b over the rows of b, p in TMEM: the columns of each half of 64 start at column 64 of it
__device__ __forceinline__ void product_sum(uint32_t d, uint32_t p, uint32_t b, uint32_t id, int m, bool begin) {
    const uint32_t bd = lo_mnmajor(b);
    const int steps = m < C ? (m + 15) / 16 : 8;
#pragma unroll
    for (int k = 0; k < 8; k++)
        if (k < steps) mma_ts(d, p + 64 * (k >> 2) + 8 * (k & 3), bd + step_mnmajor(k), id, k > 0 || !begin);
}

struct Bars {
    uint64_t keep[2], kept[2];  // operands that stay for a unit: there; free
    uint64_t full[SLOTS], empty[SLOTS];
    uint64_t sfull[2], dpfull, pready, dsready, sumfull, sumfree, drain;
    uint64_t lfull[2], lfree[2];
};

// 64 columns of p - or of their seen part - as bf16 to TMEM
__device__ __forceinline__ void put_half(uint32_t at, const float (&x)[64]) {
#pragma unroll
    for (int e = 0; e < 2; e++) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; k++) w[k] = pack_bf16(x[32 * e + 2 * k], x[32 * e + 2 * k + 1]);
        tmem_st16(at + 16 * e, w);
    }
}

template <bool KEYS>
__global__ void __launch_bounds__(THREADS, 1)
    window_grad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mg, GradArgs a) {
    using U = typename std::conditional<KEYS, KeyUnit, QueryUnit>::type;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    __shared__ Bars bar;
    __shared__ __align__(16) float2 stats[KEYS ? 2 : 1][KEYS ? C : 1];  // (- log2 e lse, - delta) of the queries
    __shared__ float half_sums[KEYS ? 1 : 2][2][KEYS ? 1 : C];  // of do o over the channels
    __shared__ uint32_t tmem_sh;
    __shared__ int failed, used[SLOTS], used_keep[2];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const WindowShape& s = a.s;
    if (sb & 1023u) {  // never on this layout; swizzled tiles would be read wrongly
        if (tid == 0) a.status[0] = -1;
        return;
    }
    if (tid == 0) {
        if (!KEYS && blockIdx.x == 0)
            for (int i = 0; i < 4; i++) a.status[i] = 0;  // a wait expires a second later at the earliest
        failed = 0;
        for (int i = 0; i < SLOTS; i++) {
            used[i] = 0;
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            used_keep[i] = 0;
            mbar_init(&bar.keep[i], 1);
            mbar_init(&bar.kept[i], !KEYS && i == 1 ? 9 : 1);  // dq: do is read by the rows' warps too
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.lfull[i], 32);
            mbar_init(&bar.lfree[i], 8);
        }
        mbar_init(&bar.dpfull, 1);
        mbar_init(&bar.pready, 8);
        mbar_init(&bar.dsready, 8);
        mbar_init(&bar.sumfull, 1);
        mbar_init(&bar.sumfree, 8);
        mbar_init(&bar.drain, 1);
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_sh;
    const int panels = s.D > 64 ? 2 : 1;
    // TMEM columns. dkv: S^T (P^T), dP^T (dS^T), dV, dK. dq: two S (dS), dP, dQ.
    constexpr uint32_t COL_S = 0, COL_DP = KEYS ? 128 : 256, COL_V = 256, COL_SUM = 384;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
        if (warp == 8) {
            // dkv keeps K and V and streams q, do; dq keeps q, do and streams K, V.
            int pos = 0, units = 0;
            bool ok = true;
            auto put = [&](uint32_t at, const CUtensorMap* map, int head, int t, int b, uint64_t* full, int* count) {
                if (ok && lane == 0) {
                    mbar_expect_tx(full, panels * PANEL);
                    (*count)++;
                    for (int p = 0; p < panels; p++) tma_load_4d(sm + at + p * PANEL, map, 64 * p, head, t, b, full);
                }
                __syncwarp();
            };
            auto stream = [&](const CUtensorMap* map, int head, int t, int b) {
                const int k = pos % SLOTS, use = pos / SLOTS;
                if (use > 0) ok = ok && wait_phase(&bar.empty[k], (use + 1) & 1, &failed, 90);
                put(AT_RING + k * TILE, map, head, t, b, &bar.full[k], &used[k]);
                pos++;
            };
#pragma unroll 1
            for (long long round = 0; ok; round++) {
                const long long u = unit_of(round);
                if (u >= a.units) {
                    if (round * gridDim.x >= a.units) break;
                    continue;
                }
                U x;
                x.set(a, u);
                const int count = x.count();
#pragma unroll 1
                for (int i = 0; i < count && ok; i++) {
                    int head, t;
                    if constexpr (KEYS) {
                        head = x.head(s, i);
                        t = x.query(i);
                    } else {
                        head = x.hk;
                        t = x.tiles.at(i) * C;
                    }
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        if (i == 0) {
                            if (units > 0) ok = ok && wait_phase(&bar.kept[w], (units + 1) & 1, &failed, 91);
                            if constexpr (KEYS) put(w * TILE, w ? &mv : &mk, x.hk, x.j0, x.b, &bar.keep[w], &used_keep[w]);
                            else put(w * TILE, w ? &mg : &mq, x.h, x.t0, x.b, &bar.keep[w], &used_keep[w]);
                        }
                        stream(KEYS ? (w ? &mg : &mq) : (w ? &mv : &mk), head, t, x.b);
                    }
                }
                if (count > 0) units++;
            }
        } else if (warp == 9) {
            const uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, s.D, 0, 1);
            const int ksteps = s.D / 16;
            Stream<U> stream;
            int started[2] = {0, 0}, summed = 0;  // units begun by S, by dP, by the sums
            bool ok = true;
            const bool ragged = s.lengths != nullptr;
            auto slot = [&](int pos, int w) { return sb + AT_RING + (2 * pos + w) % SLOTS * TILE; };
            auto there = [&](int pos, int w, int m) {  // the streamed tile, finite past its tokens
                ok = ok && wait_phase(&bar.full[(2 * pos + w) % SLOTS], (2 * pos + w) / SLOTS & 1, &failed, 92);
                if (ok && ragged && m < C) zero_rows(slot(pos, w), m, panels, lane);
            };
            auto done = [&](int pos, int w) { commit(&bar.empty[(2 * pos + w) % SLOTS]); };
            // w 0: S, w 1: dP, of pair p, the pos-th
            auto issue = [&](int w, const Pair& p, int pos, uint32_t to, uint64_t* full) {
                if (!ok || !p.some) return;
                if (p.first) ok = wait_phase(&bar.keep[w], started[w]++ & 1, &failed, 93);
                there(pos, w, p.m);
                if (!ok) return;
                tc_fence_after();
                // the rows are those of the operand that stays
                product_rows(tm + to, sb + w * TILE, slot(pos, w), id_s, ksteps);
                commit(full);
                if (p.last) commit(&bar.kept[w]);
            };
            auto sums_begin = [&](const Pair& p) {
                if (p.first && summed++ > 0) ok = ok && wait_phase(&bar.sumfree, summed & 1, &failed, 94);
            };
            Pair cur = stream.next(a);
            if constexpr (KEYS) {
                issue(0, cur, 0, COL_S, &bar.sfull[0]);
                issue(1, cur, 0, COL_DP, &bar.dpfull);
#pragma unroll 1
                for (int pos = 0; cur.some && ok; pos++) {
                    const Pair nxt = stream.next(a);
                    sums_begin(cur);
                    ok = ok && wait_phase(&bar.pready, pos & 1, &failed, 95);
                    if (!ok) break;
                    tc_fence_after();
                    product_sum(tm + COL_V, tm + COL_S, slot(pos, 1), id_o, cur.m, cur.first);
                    done(pos, 1);
                    issue(0, nxt, pos + 1, COL_S, &bar.sfull[0]);
                    ok = ok && wait_phase(&bar.dsready, pos & 1, &failed, 96);
                    if (!ok) break;
                    tc_fence_after();
                    product_sum(tm + COL_SUM, tm + COL_DP, slot(pos, 0), id_o, cur.m, cur.first);
                    done(pos, 0);
                    if (cur.last) commit(&bar.sumfull);
                    issue(1, nxt, pos + 1, COL_DP, &bar.dpfull);
                    cur = nxt;
                }
            } else {
                Pair nxt = cur.some ? stream.next(a) : cur;
                issue(0, cur, 0, COL_S, &bar.sfull[0]);
                issue(1, cur, 0, COL_DP, &bar.dpfull);
                if (cur.some) done(0, 1);
                issue(0, nxt, 1, COL_S + 128, &bar.sfull[1]);
#pragma unroll 1
                for (int pos = 0; cur.some && ok; pos++) {
                    const Pair far = nxt.some ? stream.next(a) : nxt;
                    const uint32_t at = COL_S + 128 * (pos & 1);
                    ok = wait_phase(&bar.dsready, pos & 1, &failed, 96);
                    issue(1, nxt, pos + 1, COL_DP, &bar.dpfull);
                    if (ok && nxt.some) done(pos + 1, 1);
                    sums_begin(cur);
                    if (!ok) break;
                    tc_fence_after();
                    product_sum(tm + COL_SUM, tm + at, slot(pos, 0), id_o, cur.m, cur.first);
                    done(pos, 0);
                    if (cur.last) commit(&bar.sumfull);
                    issue(0, far, pos + 2, at, &bar.sfull[pos & 1]);
                    cur = nxt;
                    nxt = far;
                }
            }
            commit(&bar.drain);  // every product issued so far has completed before TMEM is released
            int never = 0;
            wait_phase(&bar.drain, 0, &never, 1);
        } else if (KEYS && warp == 10) {
            if constexpr (KEYS) {
                Stream<KeyUnit> stream;
                for (int pos = 0;; pos++) {
                    const Pair p = stream.next(a);
                    if (!p.some) break;
                    const int t0 = stream.row0();
                    const size_t row = ((size_t)stream.x.b * s.Hq + stream.x.head(s, stream.i)) * s.T + t0;
                    float2 x[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int r = lane + 32 * e;
                        // queries past the end weigh nothing: 2^-inf
                        x[e] = r < p.m ? make_float2(-LOG2E * a.lse[row + r], -a.delta[row + r]) : make_float2(-INFINITY, 0.f);
                    }
                    if (pos >= 2 && !wait_phase(&bar.lfree[pos & 1], (pos / 2 + 1) & 1, &failed, 97)) break;
#pragma unroll
                    for (int e = 0; e < 4; e++) stats[pos & 1][lane + 32 * e] = x[e];
                    mbar_arrive(&bar.lfull[pos & 1]);
                    __syncwarp();
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_ROWS));
        const int half = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lanes = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const float c = s.scale * LOG2E;
        const uint64_t c2 = pair(c, c);
        int np = 0, units = 0;
        bool ok = true;
#pragma unroll 1
        for (long long round = 0; ok; round++) {
            const long long u = unit_of(round);
            if (u >= a.units) {
                if (round * gridDim.x >= a.units) break;
                continue;
            }
            U x;
            x.set(a, u);
            const int count = x.count(), n = x.n;
            uint64_t b2 = 0, d2 = 0;  // dq: - log2 e lse and - delta of the thread's row, twice
            if constexpr (!KEYS) {
                const int t = x.t0 + row;
                const size_t at = ((size_t)x.b * s.Hq + x.h) * s.T + t;
                const float l = t < n ? -LOG2E * a.lse[at] : 0.f;
                b2 = pair(l, l);
                if (count > 0) {
                    // a thread's half of the row's do o: channels 64 half .. (32 half .. of at most 64)
                    const int width = s.D > 64 ? 64 : s.D / 2, from = width * half;
                    const size_t to = (((size_t)x.b * s.T + t) * s.Hq + x.h) * s.D + from;
                    const __nv_bfloat16 *o = static_cast<const __nv_bfloat16*>(a.o) + to, *rest = static_cast<const __nv_bfloat16*>(a.rest) + to;
                    float sum = 0.f;
                    ok = wait_phase(&bar.keep[1], units & 1, &failed, 101);
                    if (ok && t < n)
#pragma unroll 4
                        for (int e = 0; e < width; e += 8) {
                            float y[8], z[8] = {}, g[8];
                            unpack8(*reinterpret_cast<const uint4*>(o + e), y);
                            if (a.rest) unpack8(*reinterpret_cast<const uint4*>(rest + e), z);
                            unpack8(ld_shared_v4(sb + TILE + sw128_chunk(row, (from + e) / 8, C)), g);
#pragma unroll
                            for (int k = 0; k < 8; k++) sum = fmaf(g[k], y[k] + z[k], sum);
                        }
                    half_sums[units & 1][half][row] = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.kept[1]);
                    if (bar_sync_or(1, 256, !ok)) {  // all go on, or none
                        ok = false;
                        break;
                    }
                    const float d = -(half_sums[units & 1][0][row] + half_sums[units & 1][1][row]);
                    d2 = pair(d, d);
                    if (half == 0 && t < n) a.delta[at] = -d;
                }
            }
#pragma unroll 1
            for (int i = 0; i < count; i++, np++) {
                const int buffer = KEYS ? 0 : np & 1;
                const uint32_t at_s = lanes + COL_S + 128 * buffer + 64 * half, at_dp = lanes + COL_DP + 64 * half;
                if (KEYS) ok = wait_phase(&bar.lfull[np & 1], np / 2 & 1, &failed, 97);
                ok = ok && wait_phase(&bar.sfull[buffer], (KEYS ? np : np / 2) & 1, &failed, 98);
                if (!ok) break;
                tc_fence_after();
                float p[64];
                tmem_ld32(at_s, p);
                tmem_ld32(at_s + 32, p + 32);
                int t0, j0;
                if constexpr (KEYS) {
                    t0 = x.query(i);
                    j0 = x.j0;
                } else {
                    t0 = x.t0;
                    j0 = x.tiles.at(i) * C;
                }
                const bool all = all_seen(s, t0, j0, n);
                const float4* st = reinterpret_cast<const float4*>(stats[KEYS ? np & 1 : 0]) + (KEYS ? 32 * half : 0);  // two queries each
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k++) {
                    uint64_t lse = b2;
                    if (KEYS) {
                        const float4 f = st[k];
                        lse = pair(f.x, f.z);
                    }
                    unpair(fma2(pair(p[2 * k], p[2 * k + 1]), c2, lse), p[2 * k], p[2 * k + 1]);
                }
#pragma unroll
                for (int k = 0; k < 64; k++) p[k] = exp2_fast(p[k]);
                if (!all) {
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int col = 64 * half + 32 * e;
                        const uint32_t w = KEYS ? seen_by(s, t0 + col, j0 + row, n) : keys_seen(s, t0 + row, j0 + col, n);
#pragma unroll
                        for (int k = 0; k < 32; k++)
                            if (!(w >> k & 1)) p[32 * e + k] = 0.f;
                    }
                }
                if (KEYS) {
                    put_half(at_s, p);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.pready);
                }
                ok = wait_phase(&bar.dpfull, np & 1, &failed, 99);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float d[32];
                    tmem_ld32(at_dp + 32 * e, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k++) {
                        uint64_t delta = d2;
                        if (KEYS) {
                            const float4 f = st[16 * e + k];
                            delta = pair(f.y, f.w);
                        }
                        float* q = p + 32 * e + 2 * k;
                        unpair(mul2(pair(q[0], q[1]), add2(pair(d[2 * k], d[2 * k + 1]), delta)), q[0], q[1]);
                    }
                }
                put_half(KEYS ? at_dp : at_s, p);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.dsready);
                    if (KEYS) mbar_arrive(&bar.lfree[np & 1]);
                }
            }
            if (!ok) break;
            if (count > 0) {
                ok = wait_phase(&bar.sumfull, units & 1, &failed, 100);
                if (!ok) break;
                tc_fence_after();
                units++;
            }
            // dkv: the first four warps write dv, the others dk; dq: every other 32 channels each
            const float f = KEYS && half == 0 ? 1.f : s.scale;
            if constexpr (KEYS) {
                const int j = x.j0 + row;
                const bool there = j < n;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(half ? a.dk : a.dv) + (((size_t)x.b * s.T + j) * s.Hk + x.hk) * s.D;
                float* part = a.parts + (((size_t)x.part * 2 + half) * C + row) * s.D;
#pragma unroll 1
                for (int e = 0; e < s.D; e += 32) {
                    float o[32];
                    if (count > 0) {
                        tmem_ld32(lanes + (half ? COL_SUM : COL_V) + e, o);
                        tmem_wait_ld();
                    }
                    if (count == 0 || !there)
#pragma unroll
                        for (int k = 0; k < 32; k++) o[k] = 0.f;
                    if (x.part >= 0) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) *reinterpret_cast<float4*>(part + e + k) = make_float4(f * o[k], f * o[k + 1], f * o[k + 2], f * o[k + 3]);
                    } else if (j < s.T) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) *reinterpret_cast<uint4*>(out + e + k) = pack8(o + k, f);
                    }
                }
            } else {
                const int q = x.t0 + row;
                const bool there = q < n;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dq) + (((size_t)x.b * s.T + q) * s.Hq + x.h) * s.D;
#pragma unroll 1
                for (int e = 32 * half; e < s.D; e += 64) {
                    float o[32];
                    if (count > 0) {
                        tmem_ld32(lanes + COL_SUM + e, o);
                        tmem_wait_ld();
                    }
                    if (q < s.T)
#pragma unroll
                        for (int k = 0; k < 32; k += 8) *reinterpret_cast<uint4*>(out + e + k) = there ? pack8(o + k, f) : make_uint4(0, 0, 0, 0);
                }
            }
            if (count > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.sumfree);
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
        int never = 0;
        for (int k = 0; k < SLOTS; k++)  // copies still in flight must land first
            if (used[k]) mbar_wait(&bar.full[k], (used[k] - 1) & 1, &never, nullptr, 0);
        for (int k = 0; k < 2; k++)
            if (used_keep[k]) mbar_wait(&bar.keep[k], (used_keep[k] - 1) & 1, &never, nullptr, 0);
    }
    __syncthreads();
    if (warp == 8) tmem_dealloc(tm, 512);
}

// The sums of the pieces of a cut key tile, in order: a CTA for 8 of its 128 rows.
__global__ void __launch_bounds__(256) window_join_kernel(GradArgs a, int first, int pieces, long long part0) {
    const WindowShape& s = a.s;
    const int heads = s.Hk * s.B, head = blockIdx.y, tile = first + blockIdx.z, hk = head % s.Hk, b = head / s.Hk;
    const int row = blockIdx.x * 8 + threadIdx.x / 32, which = threadIdx.x / 16 % 2, lane = threadIdx.x % 16, j = tile * C + row;
    if (j >= s.T) return;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(which ? a.dk : a.dv) + (((size_t)b * s.T + j) * s.Hk + hk) * s.D;
    for (int d = 4 * lane; d < s.D; d += 64) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < pieces; p++) {
            const size_t part = part0 + ((size_t)blockIdx.z * pieces + p) * heads + head;
            const float4 y = *reinterpret_cast<const float4*>(a.parts + ((part * 2 + which) * C + row) * s.D + d);
            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        *reinterpret_cast<uint2*>(out + d) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
    }
}

// How key tiles are cut.
struct Cut {
    int tiles, cut, pieces_cut, pieces;
    long long parts;  // pieces that leave sums, without and with those of the first tiles
    explicit Cut(const WindowShape& s) {
        const long long group = s.Hq / s.Hk, heads = (long long)s.B * s.Hk;
        tiles = (s.T + C - 1) / C;
        // a tile that holds first tokens is seen by all later queries, others by those within the window
        cut = s.window < s.T ? (s.sinks + C - 1) / C : 0;
        const long long reach = (C - 1 + (long long)s.window + C - 1) / C + 1, near_ = reach < tiles ? reach : tiles;
        const long long rest = tiles - cut, tail = rest < near_ ? rest : near_;  // of the others the last ones are seen by fewer
        const long long pairs = (long long)cut * tiles - (long long)cut * (cut - 1) / 2 + tail * (tail + 1) / 2 + (rest - tail) * near_;
        // no piece longer than a third of a CTA's share, or shorter than 8 pairs, below which writing and adding its sums costs more
        long long most = heads * group * pairs / (3 * SMS);
        if (most < 8) most = 8;
        pieces_cut = (int)((group * tiles + most - 1) / most);
        pieces = (int)((group * near_ + most - 1) / most);
        if (cut == 0) pieces_cut = 1;
        parts = (pieces_cut > 1 ? heads * cut * pieces_cut : 0) + (pieces > 1 ? heads * (tiles - cut) * pieces : 0);
    }
};

template <bool KEYS>
cudaError_t launch(const CUtensorMap* maps, const GradArgs& a, const char* name, cudaStream_t st) {
    trace_begin(name, st);
    window_grad_kernel<KEYS><<<(unsigned)(a.units < SMS ? a.units : SMS), THREADS, BYTES, st>>>(maps[0], maps[1], maps[2], maps[3], a);
    trace_end(st);
    return cudaGetLastError();
}

}  // namespace

size_t window_parts_bytes(const WindowShape& s) {
    return s.bf16 && s.B > 0 && s.T > 0 ? (size_t)Cut(s).parts * 2 * C * s.D * sizeof(float) : 0;
}

cudaError_t launch_window_bwd_tc(const WindowArgs& x, cudaStream_t st) {
    // before the tensor maps: the first runtime call of a host thread makes the device's context current there
    if (cudaError_t e = cudaFuncSetAttribute(window_grad_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES)) return e;
    if (cudaError_t e = cudaFuncSetAttribute(window_grad_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES)) return e;
    CUtensorMap maps[4];
    if (!rows_map(&maps[0], x.q, x.s, x.s.Hq) || !rows_map(&maps[1], x.k, x.s, x.s.Hk) || !rows_map(&maps[2], x.v, x.s, x.s.Hk) ||
        !rows_map(&maps[3], x.do_, x.s, x.s.Hq))
        return cudaErrorInvalidValue;
    const Cut cut(x.s);
    GradArgs a = {};
    a.s = x.s;
    a.tiles = cut.tiles;
    a.cut = cut.cut;
    a.pieces_cut = cut.pieces_cut;
    a.pieces = cut.pieces;
    a.lse = x.lse;
    a.o = x.o;
    a.rest = x.rest;
    a.delta = x.delta;
    a.dq = x.dq;
    a.dk = x.dk;
    a.dv = x.dv;
    a.parts = x.parts;
    a.status = x.status;
    a.units = (long long)x.s.B * x.s.Hq * cut.tiles;
    if (cudaError_t e = launch<false>(maps, a, "window_dq_tc", st)) return e;
    const long long heads = (long long)x.s.B * x.s.Hk, first = heads * cut.cut * cut.pieces_cut;
    a.units = first + heads * (cut.tiles - cut.cut) * cut.pieces;
    if (cudaError_t e = launch<true>(maps, a, "window_dkv_tc", st)) return e;
    const struct { int first, tiles, pieces; long long part0; } joins[2] = {
        {0, cut.cut, cut.pieces_cut, 0}, {cut.cut, cut.tiles - cut.cut, cut.pieces, cut.pieces_cut > 1 ? first : 0}};
    for (const auto& j : joins) {
        if (j.pieces == 1 || j.tiles == 0) continue;
        trace_begin("window_join", st);
        window_join_kernel<<<dim3(C / 8, (unsigned)heads, j.tiles), 256, 0, st>>>(a, j.first, j.pieces, j.part0);
        trace_end(st);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    return cudaSuccess;
}

}  // namespace gdr
