// window_grad.cu - VJP of window attention on the tensor cores, for bf16 (gdr_window_bwd), from lse and o: with delta = sum do o,
// c = scale log2 e, per pair of 128-token tiles of queries and keys
//
//     P = 2^(c Q K^T - log2 e lse),  dS = P (dO V^T - delta),  dQ += scale dS K,  dV += P^T dO,  dK += scale dS^T Q.
//
// Two kernels walk the pairs, dq by query tiles and dkv by key tiles, 3 and 4 products a pair: one walk would need 5
// but add one of its results into memory in an order that changes, or hand it on in fp32 through memory. Here each result
// is summed in TMEM, over the heads that share a key head too, and written once.
//
// Eight warps do the arithmetic, a thread for a row and half of a pair's columns.
//
// dkv forms S^T and dP^T (rows: keys), so that P^T and dS^T, over them in TMEM as bf16, are the operands of the sums as
// they are. In order per pair: dV, the next pair's S^T; dK, the next dP^T: each half has the other's time to wait for the
// rows' arithmetic. 2080 cycles of products a pair. (By halves of 64 columns with barriers of their own, as in dq, a product of two
// operands in shared memory takes 49 cycles a 16-channel step, not 33, bound by reading K or V again.)
// dq has Q and dO in TMEM, where there is no such bound, and goes by halves: in order, for each, the next S, dQ, the next dP, so one
// group of four warps has the other's time. 1560 cycles a pair. It comes first and forms delta for both, from tiles of o and what
// its rounding left that come through the ring ahead of a unit's keys.
//
// Warp 8 copies tiles in, 9 issues products, and in dkv 10 brings lse and delta, which lie along the columns there. Units are taken
// in turn by CTAs that stay, longest first, as one stream.
//
// 32768 tokens, 32 heads on 8 of 128, a window of 1024 and 4 first tokens: dq 820 us, dkv 850, their sums of pieces 14. A pair more takes
// 1.03 us in dq and 1.28 in dkv, 1.9 and 2.0 PFLOP/s; the rest is a unit's beginning and end (dq: 7000 of 26000 cycles). dq reads
// 64 KB from L2 for each pair, 8 TB/s over all SMs: without these copies it would take 750 us. Measured and not kept: two warps to
// issue products (dq 1.31 us a pair, dkv 1.47); four more warps in dq for delta and for what is written (810 us, but 362 for 335 at a
// window of 128).
//
// Where a key tile's queries are many (first tokens that all see) or the units few, a key tile is cut: its pieces leave fp32 sums,
// which a third kernel adds in order.
// Rounding to bf16: P and dS as operands (kTwoTerms), and the results.
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

constexpr int THREADS = 384, SMS = 152;
// Shared memory: two operands that stay, then the ring: five slots in dq (four: 5% slower), four in dkv, and there 4 KB for each
// warp that writes rows (dq: where Q was).
constexpr int slots(bool keys) { return keys ? 4 : 5; }
constexpr uint32_t AT_RING = 2 * TILE, BYTES = AT_RING + 5 * TILE;
static_assert(BYTES + 3072 <= 232448, "shared memory");
constexpr int REGS_ROWS = 208, REGS_REST = 80;  // of 168 at the launch
static_assert(2 * REGS_ROWS + REGS_REST <= 3 * 168, "registers of the launch");

struct GradArgs {
    WindowShape s;
    int tiles;            // of the sequence
    int cut, pieces_cut;  // key tiles from the start, pieces of each
    int pieces;           // pieces of the others
    int units;
    int heavy, light;  // dkv with first tiles that are cut: pairs of a piece and of another tile; heavy 0: not
    const float* lse;
    int rest;  // dq: what the rounding of o left is there
    float* delta;
    void *dq, *dk, *dv;
    float* parts;  // of a cut key tile's pieces: dv, dk [2, 128, D] each
    int* status;
};

// The units of a CTA, in turn: one of each round of them, every other round in reverse, so that long and short ones even out. Where
// there are long ones first and then equal ones, the CTAs that get one long one more than others join the rounds of the equal ones
// as many rounds later as that is worth. (CTAs that take neighbouring units instead share no tiles in L2: 1170 us for 865.)
template <bool KEYS>
struct Share {
    int mine, pieces, more, late;  // this CTA's long ones; of all; CTAs with one more; rounds that they are late
    __device__ __forceinline__ explicit Share(const GradArgs& a) : mine(0), pieces(0), more(0), late(0) {
        if (KEYS && a.heavy) {
            const int n = gridDim.x, c = blockIdx.x;
            pieces = a.s.Hk * a.s.B * a.cut * a.pieces_cut;
            more = pieces % n;
            mine = pieces / n + (c < more);
            late = more ? (a.heavy + a.light / 2) / a.light : 0;
        }
    }
    // The unit of a round: -1 for none in this round; false after the last.
    __device__ __forceinline__ bool unit(const GradArgs& a, int round, int& u) const {
        const int n = gridDim.x, c = blockIdx.x;
        if (KEYS && a.heavy) {
            if (round < mine) {
                u = round * n + c;
                return true;
            }
            const int r = round - mine + (c < more ? late : 0);
            u = pieces + (r < late ? r * (n - more) + c - more : late * (n - more) + (r - late) * n + c);
            return u < a.units;
        }
        u = round * n + (round & 1 ? n - 1 - c : c);
        if (u < a.units) return true;
        u = -1;
        return round * n < a.units;
    }
};

// dq: 128 queries of a head, and the key tiles that they see.
struct QueryUnit {
    int b, h, hk, n, t0;
    KeyTiles tiles;
    __device__ __forceinline__ void set(const GradArgs& a, int u) {
        const WindowShape& s = a.s;
        const int per = s.Hq * s.B, from_top = u / per, rest = u - from_top * per;
        t0 = (a.tiles - 1 - from_top) * C;
        b = rest / s.Hq;
        h = rest - b * s.Hq;
        hk = h / (s.Hq / s.Hk);
        n = s.tokens(b);
        tiles = KeyTiles(C, s.window, s.sinks, t0, min(t0 + C, n));
    }
    __device__ __forceinline__ int count() const { return tiles.count(); }
};

// dkv: 128 keys of a head, a piece of the (query head, query tile) pairs that see them.
struct KeyUnit {
    int b, hk, n, j0, per, begin, end;  // pairs begin .. end - 1, `per` query tiles a head
    int part;                           // index of its piece of `parts`, or -1
    __device__ __forceinline__ void set(const GradArgs& a, int u) {
        const WindowShape& s = a.s;
        const int heads = s.Hk * s.B, cut = heads * a.cut * a.pieces_cut;
        const bool in_cut = u < cut;
        const int pieces = in_cut ? a.pieces_cut : a.pieces;
        const int v = in_cut ? u : u - cut, of_heads = v / heads, head = v - of_heads * heads;
        const int of_tile = of_heads / pieces, piece = of_heads - of_tile * pieces, tile = of_tile + (in_cut ? 0 : a.cut);
        b = head / s.Hk;
        hk = head - b * s.Hk;
        n = s.tokens(b);
        j0 = tile * C;
        per = j0 < n ? (queries_end(C, s.window, s.sinks, j0, n) - j0 + C - 1) / C : 0;
        const int all = per * (s.Hq / s.Hk);
        begin = pieces == 1 ? 0 : (int)((long long)all * piece / pieces);
        end = pieces == 1 ? all : (int)((long long)all * (piece + 1) / pieces);
        part = pieces == 1 ? -1 : in_cut || a.pieces_cut == 1 ? v : u;
    }
    __device__ __forceinline__ int count() const { return end - begin; }
};
// The pairs of a KeyUnit in order: query head (of those that share the key head) and tile.
struct Queries {
    int g, tile;
    __device__ __forceinline__ void begin(const KeyUnit& x) {
        g = x.per > 0 ? x.begin / x.per : 0;
        tile = x.begin - g * x.per;
    }
    __device__ __forceinline__ void next(const KeyUnit& x) {
        if (++tile == x.per) {
            tile = 0;
            g++;
        }
    }
    __device__ __forceinline__ int head(const WindowShape& s, const KeyUnit& x) const { return x.hk * (s.Hq / s.Hk) + g; }
    __device__ __forceinline__ int query(const KeyUnit& x) const { return x.j0 + tile * C; }
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
    Queries at;
    Share<std::is_same<U, KeyUnit>::value> share;
    int round = -1, i = 0, count = 0;
    __device__ __forceinline__ explicit Stream(const GradArgs& a) : share(a) {}
    __device__ __forceinline__ Pair next(const GradArgs& a) {
        if (++i < count) {
            if constexpr (std::is_same<U, KeyUnit>::value) at.next(x);
        }
        while (i >= count) {
            int u;
            if (!share.unit(a, ++round, u)) return Pair{false, false, false, 0};
            if (u < 0) continue;
            x.set(a, u);
            i = 0;
            count = x.count();
            if constexpr (std::is_same<U, KeyUnit>::value) at.begin(x);
        }
        return Pair{true, i == 0, i + 1 == count, x.n - row0()};
    }
    __device__ __forceinline__ int row0() const {  // of the streamed tiles
        if constexpr (std::is_same<U, KeyUnit>::value) return at.query(x);
        else return x.tiles.at(i) * C;
    }
};

template <int SLOTS>
struct Bars {
    uint64_t keep[2], kept[2];  // operands that stay for a unit: there; free
    uint64_t full[SLOTS], empty[SLOTS];
    uint64_t sfull[2], dpfull[2], pready, dsready[2], sumfull, sumfree, drain;  // dq: of each half
    uint64_t aready;              // dq: the operands that stay are in TMEM
    uint64_t lfull[2], lfree[2];  // dkv: statistics
};

// 64 columns as bf16 to TMEM, the second terms 32 columns on (both: of a second half, which is empty with two terms, none are read)
template <int TERMS>
__device__ __forceinline__ void put_half(uint32_t at, const float (&x)[64]) {
#pragma unroll
    for (int e = 0; e < 2; e++) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; k++) w[k] = pack_bf16(x[32 * e + 2 * k], x[32 * e + 2 * k + 1]);
        tmem_st16(at + 16 * e, w);
        if (TERMS == 2) {
#pragma unroll
            for (int k = 0; k < 16; k++) w[k] = second_term(w[k], x[32 * e + 2 * k], x[32 * e + 2 * k + 1]);
            tmem_st16(at + 32 + 16 * e, w);
        }
    }
}

template <bool KEYS, int D, int TERMS>
__global__ void __launch_bounds__(THREADS, 1)
    window_grad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap mr,
                       GradArgs a) {
    using U = typename std::conditional<KEYS, KeyUnit, QueryUnit>::type;
    constexpr int SLOTS = slots(KEYS);
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    __shared__ Bars<SLOTS> bar;
    // dkv: - log2 e lse and - delta of a pair's queries; dq: the halves of delta
    __shared__ __align__(16) float lse_sh[2][C], delta_sh[2][C];
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
            mbar_init(&bar.kept[i], KEYS ? 1 : 8);  // dq: the rows' warps read dO, and write over Q
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.dpfull[i], 1);
            mbar_init(&bar.dsready[i], KEYS ? 8 : 4);
            mbar_init(&bar.lfull[i], 1);
            mbar_init(&bar.lfree[i], 8);
        }
        mbar_init(&bar.pready, 8);
        mbar_init(&bar.sumfull, 1);
        mbar_init(&bar.sumfree, 8);
        mbar_init(&bar.aready, 8);
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
    constexpr int panels = D > 64 ? 2 : 1;
    // TMEM columns, S and dP in halves of 64. dkv: S^T (P^T), dP^T (dS^T), dV, dK. dq: Q, dO, S, dP (dS), dQ.
    constexpr uint32_t COL_Q = 0, COL_G = 64, COL_S = KEYS ? 0 : 128, COL_DP = KEYS ? 128 : 256, COL_V = 256, COL_SUM = 384;

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
                if (use > 0) ok = ok && wait_for(&bar.empty[k], (use + 1) & 1, &failed, 90);
                put(AT_RING + k * TILE, map, head, t, b, &bar.full[k], &used[k]);
                pos++;
            };
            const Share<KEYS> share(a);
#pragma unroll 1
            for (int round = 0, u; ok && share.unit(a, round, u); round++) {
                if (u < 0) continue;
                U x;
                x.set(a, u);
                const int count = x.count();
                Queries at;
                if constexpr (KEYS) at.begin(x);
#pragma unroll 1
                for (int i = 0; i < count && ok; i++) {
                    int head, t;
                    if constexpr (KEYS) {
                        head = at.head(s, x);
                        t = at.query(x);
                        at.next(x);
                    } else {
                        head = x.hk;
                        t = x.tiles.at(i) * C;
                    }
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        if (i == 0) {
                            if (units > 0) ok = ok && wait_for(&bar.kept[w], (units + 1) & 1, &failed, 91);
                            if constexpr (KEYS) {
                                put(w * TILE, w ? &mv : &mk, x.hk, x.j0, x.b, &bar.keep[w], &used_keep[w]);
                            } else {
                                put(w * TILE, w ? &mg : &mq, x.h, x.t0, x.b, &bar.keep[w], &used_keep[w]);
                                if (w == 0) {
                                    stream(&mo, x.h, x.t0, x.b);
                                    if (a.rest) stream(&mr, x.h, x.t0, x.b);
                                }
                            }
                        }
                        stream(KEYS ? (w ? &mg : &mq) : (w ? &mv : &mk), head, t, x.b);
                    }
                }
                if (count > 0) units++;
            }
        } else if (warp == 9) {
            constexpr uint32_t id_s = idesc_bf16(128, KEYS ? 128 : 64, 0, 0), id_o = idesc_bf16(128, D, 0, 1);
            const int extra = KEYS ? 0 : a.rest ? 2 : 1;  // tiles of the ring ahead of a unit's pairs
            Stream<U> stream(a);
            int started = 0, summed = 0;  // units begun by S and dP, by the sums
            int pos = 0;                  // pairs so far
            int ring = 0;                 // place in the ring of the current pair's first tile
            bool ok = true;
            const bool ragged = s.lengths != nullptr;
            auto slot = [&](int at) { return sb + AT_RING + at % SLOTS * TILE; };
            auto there = [&](int at, int m) {  // the streamed tile, finite past its tokens
                ok = ok && wait_for(&bar.full[at % SLOTS], at / SLOTS & 1, &failed, 92);
                if (ok && ragged && m < C) zero_rows(slot(at), m, panels, lane);
            };
            auto done = [&](int at) { commit(&bar.empty[at % SLOTS]); };
            auto rows_ready = [&](uint64_t* b, int site) {
                ok = ok && wait_for(b, pos & 1, &failed, site);
                tc_fence_after();
                return ok;
            };
            auto sums_begin = [&](const Pair& p) {
                if (p.first && summed++ > 0) ok = ok && wait_for(&bar.sumfree, summed & 1, &failed, 94);
            };
            Pair cur = stream.next(a);
            if constexpr (KEYS) {
                // w 0: S^T, w 1: dP^T, of a pair whose tile is at `at`
                auto issue = [&](int w, const Pair& p, int at) {
                    if (!ok || !p.some) return;
                    if (p.first) {
                        ok = wait_for(&bar.keep[w], started & 1, &failed, 93);
                        started += w;
                    }
                    there(at, p.m);
                    if (!ok) return;
                    tc_fence_after();
                    product_ss<D>(tm + (w ? COL_DP : COL_S), lo_kmajor(sb + w * TILE), lo_kmajor(slot(at)), id_s);
                    commit(w ? &bar.dpfull[0] : &bar.sfull[0]);
                    if (p.last) commit(&bar.kept[w]);
                };
                auto sum = [&](int w, uint32_t from, int at) {  // both halves' columns, each from its column 64
                    const uint32_t d = tm + (w ? COL_SUM : COL_V), bd = lo_mnmajor(slot(at));
                    product_sum64(d, tm + from, bd, id_o, cur.m, cur.first);
                    if (TERMS == 2) product_sum64(d, tm + from + 32, bd, id_o, cur.m, false);
                    else product_sum64(d, tm + from + 64, bd + step_mnmajor(4), id_o, cur.m - 64, false);
                    done(at);
                };
                issue(0, cur, 0);
                issue(1, cur, 1);
#pragma unroll 1
                for (; cur.some && ok; pos++, ring += 2) {
                    const Pair nxt = stream.next(a);
                    sums_begin(cur);
                    if (!rows_ready(&bar.pready, 95)) break;
                    sum(0, COL_S, ring + 1);
                    issue(0, nxt, ring + 2);
                    if (!rows_ready(&bar.dsready[0], 96)) break;
                    sum(1, COL_DP, ring);
                    if (cur.last) commit(&bar.sumfull);
                    issue(1, nxt, ring + 3);
                    cur = nxt;
                }
            } else {
                auto issue = [&](int w, int half, int at) {  // w 0: S, w 1: dP
                    product_ts<D>(tm + (w ? COL_DP : COL_S) + 64 * half, tm + (w ? COL_G : COL_Q), lo_kmajor(slot(at)) + half * (64 * 128 >> 4), id_s);
                    commit(w ? &bar.dpfull[half] : &bar.sfull[half]);
                };
                auto begin_unit = [&]() {  // S and dP of a unit's first pair
                    if (!ok || !cur.some) return;
                    ring += extra;
                    ok = wait_for(&bar.aready, started++ & 1, &failed, 93);
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        there(ring + w, cur.m);
                        if (!ok) return;
                        tc_fence_after();
                        issue(w, 0, ring + w);
                        issue(w, 1, ring + w);
                    }
                    done(ring + 1);
                };
                begin_unit();
#pragma unroll 1
                for (; cur.some && ok; pos++) {
                    const Pair nxt = stream.next(a);
                    const bool on = nxt.some && !nxt.first;
                    sums_begin(cur);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        if (!rows_ready(&bar.dsready[h], 96)) break;
                        if (on) {
                            if (h == 0) there(ring + 2, nxt.m);
                            if (!ok) break;
                            tc_fence_after();
                            issue(0, h, ring + 2);
                        }
                        if (TERMS == 1 || h == 0)
                            product_sum64(tm + COL_SUM, tm + COL_DP + 64 * h, lo_mnmajor(slot(ring)) + h * step_mnmajor(4), id_o, cur.m - 64 * h, cur.first && h == 0);
                        if (TERMS == 2 && h == 0) product_sum64(tm + COL_SUM, tm + COL_DP + 32, lo_mnmajor(slot(ring)), id_o, cur.m, false);
                        if (h == 1) {
                            done(ring);
                            if (cur.last) commit(&bar.sumfull);
                        }
                        if (on) {
                            if (h == 0) there(ring + 3, nxt.m);
                            if (!ok) break;
                            tc_fence_after();
                            issue(1, h, ring + 3);
                        }
                    }
                    if (ok && on) done(ring + 3);
                    ring += 2;
                    cur = nxt;
                    if (!on) begin_unit();
                }
            }
            commit(&bar.drain);  // every product issued so far has completed before TMEM is released
            int never = 0;
            wait_for(&bar.drain, 0, &never, 1);
        } else if (KEYS && warp == 10) {
            if constexpr (KEYS) {
                Stream<KeyUnit> stream(a);
                for (int pos = 0;; pos++) {
                    const Pair p = stream.next(a);
                    if (!p.some) break;
                    const size_t row = ((size_t)stream.x.b * s.Hq + stream.at.head(s, stream.x)) * s.T + stream.row0();
                    float l[4], d[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {  // queries past the end weigh nothing: 2^-inf
                        const int r = lane + 32 * e;
                        l[e] = r < p.m ? -LOG2E * a.lse[row + r] : -INFINITY;
                        d[e] = r < p.m ? -a.delta[row + r] : 0.f;
                    }
                    if (pos >= 2 && !wait_for(&bar.lfree[pos & 1], (pos / 2 + 1) & 1, &failed, 97)) break;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        lse_sh[pos & 1][lane + 32 * e] = l[e];
                        delta_sh[pos & 1][lane + 32 * e] = d[e];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.lfull[pos & 1]);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_ROWS));
        const int half = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lanes = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t at_s = lanes + COL_S + 64 * half, at_dp = lanes + COL_DP + 64 * half;
        const float c = s.scale * LOG2E;
        const uint64_t c2 = pair(c, c);
        int np = 0, units = 0;
        bool ok = true;
        // dq: the rows that are still to be written, a unit later
        int late_t = 0, late_n = 0, late_b = 0, late_h = 0;
        // Channels of the rows that this half writes, by way of Q's place in shared memory, 4 KB for each warp.
        constexpr int WIDTH = D > 32 ? D / 2 : D;
        auto write_dq = [&](bool sums, int t, int n, int b, int h) {
            if (D == 32 && half) return;
            const uint32_t stage = sb + warp * 4096;
            if (sums) {
#pragma unroll
                for (int e = 0; e < WIDTH; e += 32) {
                    float o[32];
                    tmem_ld32(lanes + COL_SUM + WIDTH * half + e, o);
                    tmem_wait_ld();
                    const uint4 y[4] = {pack8(o, s.scale), pack8(o + 8, s.scale), pack8(o + 16, s.scale), pack8(o + 24, s.scale)};
                    stage_row(stage, e, y, lane);
                }
                __syncwarp();
            }
            const int first = t - lane;
            store_rows<WIDTH>(static_cast<__nv_bfloat16*>(a.dq) + (((size_t)b * s.T + first) * s.Hq + h) * D + WIDTH * half, (size_t)s.Hq * D,
                              stage, s.T - first, sums ? n - first : 0, lane);
        };
        auto write_late = [&]() {  // of unit number `units`, counted from 1
            ok = wait_for(&bar.sumfull, (units + 1) & 1, &failed, 100);
            if (!ok) return;
            tc_fence_after();
            write_dq(true, late_t, late_n, late_b, late_h);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sumfree);
        };
        const Share<KEYS> share(a);
#pragma unroll 1
        for (int round = 0, u; ok && share.unit(a, round, u); round++) {
            if (u < 0) continue;
            U x;
            x.set(a, u);
            const int count = x.count(), n = x.n;
            uint64_t b2 = 0, d2 = 0;  // dq: - log2 e lse and - delta of the thread's row, twice
            if constexpr (!KEYS) {
                if (count == 0) {
                    write_dq(false, x.t0 + row, n, x.b, x.h);
                    continue;
                }
                const int t = x.t0 + row;
                const size_t stat = ((size_t)x.b * s.Hq + x.h) * s.T + t;
                const float lse = t < n ? a.lse[stat] : 0.f;  // used, and waited for, only below
                // the row of Q (first half) or dO into TMEM: the unit before has done with it, on both sides
                ok = wait_for(&bar.keep[half], units & 1, &failed, 101);
                if (bar_sync_or(1, 256, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < D / 2; e += 16) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const uint4 y = ld_shared_v4(sb + half * TILE + sw128_chunk(row, e / 4 + k, C));
                        w[4 * k] = y.x; w[4 * k + 1] = y.y; w[4 * k + 2] = y.z; w[4 * k + 3] = y.w;
                    }
                    tmem_st16(lanes + (half ? COL_G : COL_Q) + e, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.aready);
                }
                // half of the row's sum of do o, o with what its rounding left
                constexpr int width = D / 16;
                const int extra = a.rest ? 2 : 1, o_at = 2 * np + extra * units;  // chunks of 8 channels; place in the ring
                ok = wait_for(&bar.keep[1], units & 1, &failed, 102);
                for (int k = 0; k < extra; k++) ok = ok && wait_for(&bar.full[(o_at + k) % SLOTS], (o_at + k) / SLOTS & 1, &failed, 103);
                float d = 0.f;
                if (ok && t < n) {
                    const uint32_t at_o = sb + AT_RING + o_at % SLOTS * TILE, at_r = sb + AT_RING + (o_at + 1) % SLOTS * TILE;
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < width; e++) {
                        const uint32_t chunk = sw128_chunk(row, half * width + e, C);
                        const uint4 y = ld_shared_v4(at_o + chunk), g = ld_shared_v4(sb + TILE + chunk);
                        const uint4 z = a.rest ? ld_shared_v4(at_r + chunk) : make_uint4(0, 0, 0, 0);
                        const uint32_t ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w}, gs[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint64_t w = pair(bf16lo(gs[k]), bf16hi(gs[k]));
                            sum[0] = fma2(w, pair(bf16lo(ys[k]), bf16hi(ys[k])), sum[0]);
                            sum[1] = fma2(w, pair(bf16lo(zs[k]), bf16hi(zs[k])), sum[1]);
                        }
                    }
                    float s0, s1;
                    unpair(add2(sum[0], sum[1]), s0, s1);
                    d = s0 + s1;
                }
                float(*halves)[C] = units & 1 ? lse_sh : delta_sh;
                halves[half][row] = d;
                if (bar_sync_or(1, 256, !ok)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive(&bar.kept[1]);
                if (tid == 0)
                    for (int k = 0; k < extra; k++) mbar_arrive(&bar.empty[(o_at + k) % SLOTS]);
                d = halves[0][row] + halves[1][row];
                if (half == 0 && t < n) a.delta[stat] = d;
                if (units > 0) write_late();
                if (!ok) break;
                fence_proxy_async_smem();  // the next copy of Q comes over what was written there
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.kept[0]);
                b2 = pair(-LOG2E * lse, -LOG2E * lse);
                d2 = pair(-d, -d);
                late_t = x.t0 + row;
                late_n = n;
                late_b = x.b;
                late_h = x.h;
            }
            Queries at;
            if constexpr (KEYS) at.begin(x);
#pragma unroll 1
            for (int i = 0; i < count; i++, np++) {
                if (KEYS) ok = wait_for(&bar.lfull[np & 1], np / 2 & 1, &failed, 97);
                ok = ok && wait_for(&bar.sfull[KEYS ? 0 : half], np & 1, &failed, 98);
                if (!ok) break;
                tc_fence_after();
                float p[64];
                tmem_ld32(at_s, p);
                tmem_ld32(at_s + 32, p + 32);
                int t0, j0;
                if constexpr (KEYS) {
                    t0 = at.query(x);
                    j0 = x.j0;
                    at.next(x);
                } else {
                    t0 = x.t0;
                    j0 = x.tiles.at(i) * C;
                }
                const bool all = all_seen(s, t0, j0, n);
                const float4* st = reinterpret_cast<const float4*>(lse_sh[np & 1]) + 16 * half;  // dkv: four columns each
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k++) {
                    uint64_t l0 = b2, l1 = b2;
                    if (KEYS) {
                        const float4 f = st[k];
                        l0 = pair(f.x, f.y);
                        l1 = pair(f.z, f.w);
                    }
                    unpair(fma2(pair(p[4 * k], p[4 * k + 1]), c2, l0), p[4 * k], p[4 * k + 1]);
                    unpair(fma2(pair(p[4 * k + 2], p[4 * k + 3]), c2, l1), p[4 * k + 2], p[4 * k + 3]);
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
                    put_half<TERMS>(at_s, p);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.pready);
                }
                ok = wait_for(&bar.dpfull[KEYS ? 0 : half], np & 1, &failed, 99);
                if (!ok) break;
                tc_fence_after();
                const float4* dt = reinterpret_cast<const float4*>(delta_sh[np & 1]) + 16 * half;
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float d[32];
                    tmem_ld32(at_dp + 32 * e, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        uint64_t d0 = d2, d1 = d2;
                        if (KEYS) {
                            const float4 f = dt[8 * e + k];
                            d0 = pair(f.x, f.y);
                            d1 = pair(f.z, f.w);
                        }
                        float* q = p + 32 * e + 4 * k;
                        unpair(mul2(pair(q[0], q[1]), add2(pair(d[4 * k], d[4 * k + 1]), d0)), q[0], q[1]);
                        unpair(mul2(pair(q[2], q[3]), add2(pair(d[4 * k + 2], d[4 * k + 3]), d1)), q[2], q[3]);
                    }
                }
                put_half<TERMS>(at_dp, p);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.dsready[KEYS ? 0 : half]);
                    if (KEYS) mbar_arrive(&bar.lfree[np & 1]);
                }
            }
            if (!ok) break;
            if (count > 0) units++;
            if constexpr (KEYS) {  // the first four warps write dv, the others dk
                if (count > 0) {
                    ok = wait_for(&bar.sumfull, (units + 1) & 1, &failed, 100);
                    if (!ok) break;
                    tc_fence_after();
                }
                const int first = x.j0 + row - lane;
                const float f = half ? s.scale : 1.f;
                const size_t stride = (size_t)s.Hk * D;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(half ? a.dk : a.dv) + (((size_t)x.b * s.T + first) * s.Hk + x.hk) * D;
                float* part = a.parts + (((size_t)x.part * 2 + half) * C + row) * D;
                const uint32_t stage = sb + AT_RING + SLOTS * TILE + warp * 4096;
                constexpr int WIDTH = D > 64 ? 64 : D;  // channels staged at once
#pragma unroll 1
                for (int e = 0; e < D; e += WIDTH) {
#pragma unroll
                    for (int k = 0; k < WIDTH; k += 32) {
                        float o[32];
                        if (count > 0) {
                            tmem_ld32(lanes + (half ? COL_SUM : COL_V) + e + k, o);
                            tmem_wait_ld();
                        }
                        if (x.part >= 0) {
                            const bool there = count > 0 && first + lane < n;
#pragma unroll
                            for (int d = 0; d < 32; d += 4)
                                *reinterpret_cast<float4*>(part + e + k + d) =
                                    there ? make_float4(f * o[d], f * o[d + 1], f * o[d + 2], f * o[d + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                        } else {
                            const uint4 y[4] = {pack8(o, f), pack8(o + 8, f), pack8(o + 16, f), pack8(o + 24, f)};
                            stage_row(stage, k, y, lane);
                        }
                    }
                    __syncwarp();
                    if (x.part < 0) store_rows<WIDTH>(out + e, stride, stage, s.T - first, count > 0 ? n - first : 0, lane);
                    __syncwarp();
                }
                if (count > 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.sumfree);
                }
            }
        }
        if (!KEYS && ok && units > 0) write_late();
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

// Before the tensor maps: the first runtime call of a host thread makes the device's context current there.
template <int D, int TERMS>
cudaError_t allow_smem() {
    if (cudaError_t e = cudaFuncSetAttribute(window_grad_kernel<false, D, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES)) return e;
    return cudaFuncSetAttribute(window_grad_kernel<true, D, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
}

template <bool KEYS, int D, int TERMS>
cudaError_t launch(const CUtensorMap* maps, const GradArgs& a, const char* name, cudaStream_t st) {
    trace_begin(name, st);
    window_grad_kernel<KEYS, D, TERMS><<<(unsigned)(a.units < SMS ? a.units : SMS), THREADS, BYTES, st>>>(maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], a);
    trace_end(st);
    return cudaGetLastError();
}

template <int D, int TERMS>
cudaError_t launch_bwd(const WindowArgs& x, cudaStream_t st) {
    if (cudaError_t e = allow_smem<D, TERMS>()) return e;
    CUtensorMap maps[6];
    if (!rows_map(&maps[4], x.o, x.s, x.s.Hq) || !rows_map(&maps[5], x.rest ? x.rest : x.o, x.s, x.s.Hq)) return cudaErrorInvalidValue;
    if (!rows_map(&maps[0], x.q, x.s, x.s.Hq) || !rows_map(&maps[1], x.k, x.s, x.s.Hk) || !rows_map(&maps[2], x.v, x.s, x.s.Hk) ||
        !rows_map(&maps[3], x.do_, x.s, x.s.Hq))
        return cudaErrorInvalidValue;
    const Cut cut(x.s, C, SMS, 8);
    GradArgs a = {};
    a.s = x.s;
    a.tiles = cut.tiles;
    a.cut = cut.cut;
    a.pieces_cut = cut.pieces_cut;
    a.pieces = cut.pieces;
    a.lse = x.lse;
    a.rest = x.rest != nullptr;
    a.delta = x.delta;
    a.dq = x.dq;
    a.dk = x.dk;
    a.dv = x.dv;
    a.parts = x.parts;
    a.status = x.status;
    a.units = x.s.B * x.s.Hq * cut.tiles;
    if (cudaError_t e = launch<false, D, TERMS>(maps, a, "window_dq_tc", st)) return e;
    const int heads = x.s.B * x.s.Hk, first = heads * cut.cut * cut.pieces_cut;
    a.units = first + heads * (cut.tiles - cut.cut) * cut.pieces;
    a.heavy = cut.heavy;
    a.light = cut.light;
    if (cudaError_t e = launch<true, D, TERMS>(maps, a, "window_dkv_tc", st)) return e;
    const struct { int first, tiles, pieces, part0; } joins[2] = {
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

}  // namespace

size_t window_parts_bytes_tc(const WindowShape& s) {
    return s.B > 0 && s.T > 0 ? (size_t)Cut(s, C, SMS, 8).parts * 2 * C * s.D * sizeof(float) : 0;
}

cudaError_t launch_window_bwd_tc(const WindowArgs& x, cudaStream_t st) {
    if (x.s.T <= kTwoTerms) return x.s.D == 32 ? launch_bwd<32, 2>(x, st) : x.s.D == 64 ? launch_bwd<64, 2>(x, st) : launch_bwd<128, 2>(x, st);
    return x.s.D == 32 ? launch_bwd<32, 1>(x, st) : x.s.D == 64 ? launch_bwd<64, 1>(x, st) : launch_bwd<128, 1>(x, st);
}

}  // namespace gdr
