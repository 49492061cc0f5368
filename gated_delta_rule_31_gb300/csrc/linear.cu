// linear.cu - linear attention with a constant decay per head on the CUDA cores, for fp32: the segment
// summary and the mix pass (linear.h); and the combine step of both types.
//
// A chunk holds up to 32 tokens in processing order (u = 0 is the first token of the chunk, or
// its last one in reverse), so both directions run the same sums over j <= r:
//     P_rj = f l^(r-j) (a_r . b_j),   out_r = f' l^(r+1-s) a_r X + sum_{j<=r} P_rj c_j,
//     X <- l^m X + f'' sum_j l^(m-1-j+s) b_j c_j^T          (m tokens in the chunk; s = reverse)
// with f = scale, and (f', f'') = (scale, 1) forwards, (1, scale) in reverse: in reverse X is the
// adjoint of the state after the chunk, which reaches token 0 (the last one) undecayed. Every
// power of l has an exponent >= 0, so no decay overflows, and l^0 = 1 also where l = 0.
//
// fp32 FMA bounds it (a chunk of 32 tokens and 64 of 128 columns: 721 thousand FMAs, 0.15 ms in all at
// T = 4096 and 32 heads of 128), then shared-memory reads, so threads hold tiles of 4 x 4 and more whose
// operands are read as 16-byte vectors from different banks, lanes that share a tile's sum taking
// different parts of k; and the state stays in registers with a copy in shared memory for a X. Arithmetic
// is on fp32 pairs, along the direction in which they were loaded (for the state, the other direction
// takes 352 us instead of 301). Tiles are copied asynchronously, one chunk ahead. Chunks of 32 need fewer
// FMAs than chunks of 64 (half of P is masked) and leave room for two CTAs per SM. T = 4096, 32 heads of
// 128: summary 111 us, mix pass 301. (With synchronous loads and P and a X in strided tiles of 2 x 2 and
// 2 x 4: 209 and 604. With 64-token chunks, one CTA per SM: 1171 in all.) The VJP takes 1152 us, with two value heads a
// key head 1284: dq and dk then swap the heads' states through global memory after every chunk (371 instead of 303 each).
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "linear.h"
#include "linear_dev.cuh"

namespace gdr {

namespace {

constexpr int LC = 32;  // tokens of a chunk

using linear::power;

__device__ __forceinline__ int valid_tokens(const LinearShape& s, int b) {
    return s.lengths ? min(max(s.lengths[b], 0), s.T) : s.T;
}

// Clears the status word of a call, from one of the blocks of its first kernel. (No wait of the fp32 kernels
// is one that could expire, so nothing else is ever written there.)
__device__ __forceinline__ void clear_status(int* status) {
    if (status && threadIdx.x < 4 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) status[threadIdx.x] = 0;
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }

// N contiguous floats (N a multiple of 4, or 2).
template <int N>
__device__ __forceinline__ void load_n(const float* p, float* x) {
    if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        x[0] = v.x; x[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = load4(p + i);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float* x) {
    if constexpr (N == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) store4(p + i, make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
    }
}

// Threads' places in a 16 x 16 grid of state tiles: a warp takes 4 x 8 of them, so that each of its reads
// of a tile's row or column is one wavefront.
__device__ __forceinline__ int grid_row() { return (threadIdx.x >> 5 & 3) * 4 + (threadIdx.x >> 3 & 3); }
__device__ __forceinline__ int grid_col() { return (threadIdx.x >> 7) * 8 + (threadIdx.x & 7); }

// The N columns of thread tx of 16 in a row: runs of four, 64 apart, so that neighbours read without conflicts.
template <int N>
__device__ __forceinline__ void load_cols(const float* row, int tx, float* x) {
    if constexpr (N == 8) {
        load_n<4>(row + 4 * tx, x);
        load_n<4>(row + 64 + 4 * tx, x + 4);
    } else {
        load_n<N>(row + N * tx, x);
    }
}
template <int N>
__device__ __forceinline__ void store_cols(float* row, int tx, const float* x) {
    if constexpr (N == 8) {
        store_n<4>(row + 4 * tx, x);
        store_n<4>(row + 64 + 4 * tx, x + 4);
    } else {
        store_n<N>(row + N * tx, x);
    }
}

// Starts the copies of columns [c0, c0 + D) of a chunk's tokens of one head, in processing order, to rows
// of stride D + 4; rows m .. 31 become zero.
template <int D>
__device__ __forceinline__ void fetch_tile(float* dst, const float* src, size_t token0, size_t token_stride, int c0, int m,
                                           int reverse) {
    constexpr int V = D / 4;
#pragma unroll
    for (int i = threadIdx.x; i < LC * V; i += 256) {
        const int u = i / V, c = 4 * (i % V), row = u < m ? (reverse ? m - 1 - u : u) : 0;
        cp_async16(dst + u * (D + 4) + c, src + (token0 + row) * token_stride + c0 + c, u < m);
    }
}

__device__ __forceinline__ float at(const float4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// grid (nseg * Dv / RS, Hv, B): rows [RS * i, ...) of the state's sum over one segment; a thread holds
// RS / 16 x DK / 16 of it.
template <int DK, int RS>
__global__ void __launch_bounds__(256) linear_summary_kernel(LinearSummaryArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int XS = LC * (RS + 4), YS = LC * (DK + 4);
    float* pw = sm + 2 * (XS + YS);  // l^0 .. l^32, after two buffers of X [32][RS + 4] and Y [32][DK + 4]
    const LinearShape& s = a.s;
    const int nr = s.Dv / RS, seg = blockIdx.x / nr, r0 = (blockIdx.x % nr) * RS;
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / (s.Hv / s.Hk);
    constexpr int TR = RS / 16, TC = DK / 16;
    const int ty = grid_row(), tx = grid_col();
    if (threadIdx.x <= LC) pw[threadIdx.x] = power(s.g[hv], threadIdx.x);
    const int first = min(seg * s.seg_tokens, valid_tokens(s, b));
    const int last = min(first + s.seg_tokens, valid_tokens(s, b));
    const int nc = (last - first + LC - 1) / LC;
    const float* rows = static_cast<const float*>(a.rows) + ((size_t)b * s.T * s.Hv + hv) * s.Dv;
    const float* cols = static_cast<const float*>(a.cols) + ((size_t)b * s.T * s.Hk + hk) * s.Dk;
    auto fetch = [&](int i) {
        if (i >= nc) return;
        const int t0 = first + (a.reverse ? nc - 1 - i : i) * LC, m = min(LC, last - t0);
        float* X = sm + (i & 1) * (XS + YS);
        fetch_tile<RS>(X, rows, t0, (size_t)s.Hv * s.Dv, r0, m, a.reverse);
        fetch_tile<DK>(X + XS, cols, t0, (size_t)s.Hk * s.Dk, 0, m, a.reverse);
    };
    linear::next_kernel_may_start();
    clear_status(a.clear);
    float z[TR][TC] = {};
    fetch(0);
    for (int i = 0; i < nc; i++) {
        const int t0 = first + (a.reverse ? nc - 1 - i : i) * LC, m = min(LC, last - t0);
        cp_async_wait_all();
        __syncthreads();  // chunk i is there, and chunk i - 1's buffer is free
        fetch(i + 1);
        const float *X = sm + (i & 1) * (XS + YS), *Y = X + XS;
        const float over = pw[m];
#pragma unroll
        for (int r = 0; r < TR; r++)
#pragma unroll
            for (int c = 0; c < TC; c++) z[r][c] *= over;
#pragma unroll 4
        for (int u = 0; u < m; u++) {
            const float w = a.factor * pw[m - 1 - u + a.reverse];
            float x[TR], y[TC];
            load_n<TR>(X + u * (RS + 4) + ty * TR, x);
            load_cols<TC>(Y + u * (DK + 4), tx, y);
#pragma unroll
            for (int r = 0; r < TR; r++) {
                x[r] *= w;
#pragma unroll
                for (int c = 0; c < TC; c += 2) linear::axpy2<false>(&z[r][c], x[r], y + c);
            }
        }
    }
    float* out = a.z + ((((size_t)b * s.Hv + hv) * s.nseg + seg) * s.Dv + r0) * s.Dk;
#pragma unroll
    for (int r = 0; r < TR; r++) store_cols<TC>(out + (size_t)(ty * TR + r) * s.Dk, tx, z[r]);
}

// grid (ceil(Dv Dk / 1024), Hv, B): four state elements a thread, the segments in processing order.
__global__ void __launch_bounds__(256) linear_combine_kernel(LinearCombineArgs a) {
    const LinearShape& s = a.s;
    const int i = (blockIdx.x * 256 + threadIdx.x) * 4, D = s.Dv * s.Dk;
    linear::next_kernel_may_start();
    linear::wait_kernel_before();
    if (i >= D) return;
    const int n = valid_tokens(s, blockIdx.z);
    const size_t bh = (size_t)blockIdx.z * s.Hv + blockIdx.y;
    const float g = s.g[blockIdx.y];
    float4 x = a.init ? load4(a.init + bh * D + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < s.nseg; k0 += 8) {  // eight segments' loads in flight
        float4 z[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int k = k0 + e, seg = a.reverse ? s.nseg - 1 - k : k;
            if (k < s.nseg && (k + 1 < s.nseg || a.last)) z[e] = load4(a.z + (bh * s.nseg + seg) * D + i);
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int k = k0 + e, seg = a.reverse ? s.nseg - 1 - k : k;
            if (k >= s.nseg) break;
            store4(a.z + (bh * s.nseg + seg) * D + i, x);
            if (k + 1 == s.nseg && !a.last) break;
            const float over = power(g, max(0, min(s.seg_tokens, n - seg * s.seg_tokens)));
            x = make_float4(over * x.x + z[e].x, over * x.y + z[e].y, over * x.z + z[e].z, over * x.w + z[e].w);
        }
    }
    if (a.last) store4(a.last + bh * D + i, x);
}

// Rows of a thread's output tile, from its first: pairs, 8 apart, so that the four pairs of a warp and two
// runs of k lie in different banks.
__device__ __forceinline__ constexpr int row_of(int r) { return (r & 1) + 8 * (r >> 1); }

// y[r] += sum over four k of a[row_of(r)][k] x[k], rows at strides sa, sx; a points to column k, x to row k.
template <int R>
__device__ __forceinline__ void add_product(float (&y)[R][4], const float* a, int sa, const float* x, int sx, int row) {
    float4 av[R];
#pragma unroll
    for (int r = 0; r < R; r++) av[r] = load4(a + (row + row_of(r)) * sa);
#pragma unroll
    for (int e = 0; e < 4; e++) {
        float xv[4];
        load_n<4>(x + e * sx, xv);
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int c = 0; c < 4; c += 2) linear::axpy2<false>(&y[r][c], at(av[r], e), xv + c);
    }
}

// Adds lane pairs' sums of N rows: the lane with bit `mask` keeps the upper half of them, in y[0 .. N / 2).
template <int N, int R>
__device__ __forceinline__ void add_halves(float (&y)[R][4], int mask) {
    const bool up = threadIdx.x & mask;
#pragma unroll
    for (int r = 0; r < N / 2; r++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const float send = up ? y[r][c] : y[r + N / 2][c], keep = up ? y[r + N / 2][c] : y[r][c];
            y[r][c] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
        }
}

struct MixView {  // the roles of a pass (linear.h)
    const void *a, *b, *c;
    int ha, hc, ho;  // heads of a and b, of c, and of the output
    int reverse;
    float fp, fx, fu;  // factors of P, of a X and of the state's update
};

// grid (nseg * D2 / CS, output heads, B). D1: width of a and b; a CTA forms CS of the D2 output columns.
// ROWS1: the state's rows (Dv) run along D1 (dq, dk), else along D2 (o, dv). A thread holds D1 / 16 x
// CS / 16 of the state, a lane pair CS / 16 x 4 of the output, and four lanes 4 x 4 of P.
template <int D1, int CS, bool ROWS1>
__global__ void __launch_bounds__(256, 2) linear_mix_kernel(LinearMixArgs args, MixView w) {
    extern __shared__ __align__(16) float sm[];
    constexpr int BS = LC * (D1 + 4), CZ = LC * (CS + 4);
    float* A = sm;              // [32][D1 + 4]
    float* Bs = A + BS;         // two of [32][D1 + 4]
    float* Cs = Bs + 2 * BS;    // two of [32][CS + 4]
    float* X = Cs + 2 * CZ;     // [D1][CS + 4]
    float* P = X + D1 * (CS + 4);   // [32][36]
    float* pws = P + LC * (LC + 4); // two of l^0 .. l^32
    const LinearShape& s = args.s;
    const int D2 = ROWS1 ? s.Dk : s.Dv;
    const int ns = D2 / CS, seg = blockIdx.x / ns, c0 = (blockIdx.x % ns) * CS;
    const int ho = blockIdx.y, b = blockIdx.z, heads = s.Hv / w.ho;  // value heads summed into this output
    const int G = s.Hv / s.Hk;
    const int ty = grid_row(), tx = grid_col();
    constexpr int TC = CS / 16, TK = D1 / 16;
    const int n = valid_tokens(s, b);
    const int begin = seg * s.seg_tokens, end = min(begin + s.seg_tokens, s.T);
    const int first = min(begin, n), last = min(end, n), nc = (last - first + LC - 1) / LC;
    float* out = static_cast<float*>(args.out) + ((size_t)b * s.T * w.ho + ho) * D2 + c0;
    const size_t out_stride = (size_t)w.ho * D2;
    const size_t head_floats = (size_t)s.Dv * s.Dk;
    auto start_of = [&](int hv) { return args.starts + (((size_t)b * s.Hv + hv) * s.nseg + seg) * head_floats; };
    float x[TK][TC];  // rows ty TK .., columns tx TC .. of X
    // One segment: it starts from the state before the call, and ends with the one after it.
    auto state_before = [&](int i, int hv) {
        if (s.nseg > 1 || i > 0) return (const float*)start_of(hv);
        return args.init ? args.init + ((size_t)b * s.Hv + hv) * head_floats : nullptr;
    };
    auto state_from = [&](const float* p) {
        if (ROWS1) {
#pragma unroll
            for (int r = 0; r < TK; r++) {
                if (p) load_n<TC>(p + (size_t)(ty * TK + r) * s.Dk + c0 + tx * TC, x[r]);
#pragma unroll
                for (int c = 0; c < TC; c++) x[r][c] = p ? x[r][c] : 0.f;
            }
        } else {
#pragma unroll
            for (int c = 0; c < TC; c++) {
                float col[TK];
                if (p) load_n<TK>(p + (size_t)(c0 + tx * TC + c) * s.Dk + ty * TK, col);
#pragma unroll
                for (int r = 0; r < TK; r++) x[r][c] = p ? col[r] : 0.f;
            }
        }
    };
    auto state_to = [&](float* p) {
        if (ROWS1) {
#pragma unroll
            for (int r = 0; r < TK; r++) store_n<TC>(p + (size_t)(ty * TK + r) * s.Dk + c0 + tx * TC, x[r]);
        } else {
#pragma unroll
            for (int c = 0; c < TC; c++) {
                float col[TK];
#pragma unroll
                for (int r = 0; r < TK; r++) col[r] = x[r][c];
                store_n<TK>(p + (size_t)(c0 + tx * TC + c) * s.Dk + ty * TK, col);
            }
        }
    };
    auto share_state = [&] {
#pragma unroll
        for (int r = 0; r < TK; r++) store_n<TC>(X + (ty * TK + r) * (CS + 4) + tx * TC, x[r]);
    };
    // Step n: value head n % heads of chunk n / heads.
    const int steps = nc * heads;
    auto fetch = [&](int n, bool fetch_a) {
        if (n >= steps) return;
        const int i = n / heads, hv = ho * heads + n % heads, hk = hv / G;
        const int ia = w.ha == s.Hv ? hv : hk, ic = w.hc == s.Hv ? hv : hk;
        const int t0 = first + (w.reverse ? nc - 1 - i : i) * LC, m = min(LC, last - t0);
        const size_t at1 = ((size_t)b * s.T * w.ha + ia) * D1, at2 = ((size_t)b * s.T * w.hc + ic) * D2;
        if (fetch_a) {
            fetch_tile<D1>(A, static_cast<const float*>(w.a) + at1, t0, (size_t)w.ha * D1, 0, m, w.reverse);
        } else {
            fetch_tile<D1>(Bs + (n & 1) * BS, static_cast<const float*>(w.b) + at1, t0, (size_t)w.ha * D1, 0, m, w.reverse);
            fetch_tile<CS>(Cs + (n & 1) * CZ, static_cast<const float*>(w.c) + at2, t0, (size_t)w.hc * D2, c0, m, w.reverse);
            if (threadIdx.x <= LC) pws[(n & 1) * (LC + 1) + threadIdx.x] = power(s.g[hv], threadIdx.x);
        }
    };
    fetch(0, false);
    fetch(0, true);
    clear_status(args.clear);
    linear::wait_kernel_before();  // the states, and what the outputs' memory held
    for (int i = threadIdx.x; i < (end - max(begin, n)) * (CS / 4); i += 256)  // past the length: zero
        store4(out + (size_t)(max(begin, n) + i / (CS / 4)) * out_stride + 4 * (i % (CS / 4)),
               make_float4(0.f, 0.f, 0.f, 0.f));
    if (nc > 0 || heads == 1) state_from(state_before(0, ho * heads));
    share_state();
    // The output: a warp forms 4 RI x 16 of it.
    constexpr int RI = CS / 16, OW = CS / 16;  // rows of a thread's tile; warps side by side
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int orow = 4 * RI * (warp / OW) + 2 * (lane >> 3), oc = 16 * (warp % OW) + 4 * (lane >> 1 & 3);
    const int last_p = 4 * RI * (warp / OW + 1);  // P is zero from this column on in the warp's rows
    auto out_row = [&](int r) { return orow + row_of(r); };
    float acc[RI][4] = {};
    for (int i = 0; i < nc; i++) {
        const int t0 = first + (w.reverse ? nc - 1 - i : i) * LC, m = min(LC, last - t0);
        for (int h = 0; h < heads; h++) {
            const int step = i * heads + h;
            const float *Bm = Bs + (step & 1) * BS, *Cm = Cs + (step & 1) * CZ, *pw = pws + (step & 1) * (LC + 1);
            cp_async_wait_all();
            __syncthreads();  // the step's tiles and X are there, and the buffers of the step before are free
            fetch(step + 1, false);
            // P: a warp forms 8 x 16 of it, in tiles of 4 x 4 whose sums four lanes share, every fourth
            // run of four k each; what lies above the diagonal is not formed where no warp reads it.
            if (16 * (warp & 1) <= 8 * (warp >> 1)) {
                const int row = 8 * (warp >> 1) + 4 * (lane >> 4), col = 16 * (warp & 1) + 4 * (lane >> 2 & 3);
                float p[4][4] = {};
#pragma unroll 2
                for (int k = 4 * (lane & 3); k < D1; k += 16) {
                    float4 u[4], v[4];
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        u[r] = load4(A + (row + r) * (D1 + 4) + k);
                        v[r] = load4(Bm + (col + r) * (D1 + 4) + k);
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++)
#pragma unroll
                        for (int r = 0; r < 4; r++)
#pragma unroll
                            for (int j = 0; j < 4; j++) p[r][j] += at(u[r], e) * at(v[j], e);
                }
                add_halves<4>(p, 1);
                add_halves<2>(p, 2);
                const int u = row + 2 * (lane & 1) + (lane >> 1 & 1);
#pragma unroll
                for (int j = 0; j < 4; j++) p[0][j] = col + j <= u ? w.fp * pw[u - col - j] * p[0][j] : 0.f;
                store_n<4>(P + u * (LC + 4) + col, p[0]);
            }
            {  // a X: the sums of a tile of RI x 4 are shared by two lanes, every other run of four k each
                float y[RI][4] = {};
#pragma unroll 2
                for (int k = 4 * (lane & 1); k < D1; k += 8) add_product<RI>(y, A + k, D1 + 4, X + k * (CS + 4) + oc, CS + 4, orow);
#pragma unroll
                for (int r = 0; r < RI; r++) {
                    const float f = w.fx * pw[out_row(r) + 1 - w.reverse];
#pragma unroll
                    for (int c = 0; c < 4; c++) acc[r][c] += f * y[r][c];
                }
            }
            __syncthreads();  // P is written; A and X are free
            fetch(step + 1, true);
#pragma unroll 2
            for (int k = 4 * (lane & 1); k < last_p; k += 8)  // P c
                add_product<RI>(acc, P + k, LC + 4, Cm + k * (CS + 4) + oc, CS + 4, orow);
            {  // the state over this chunk
                const float over = pw[m];
#pragma unroll
                for (int r = 0; r < TK; r++)
#pragma unroll
                    for (int c = 0; c < TC; c++) x[r][c] *= over;
#pragma unroll 2
                for (int u = 0; u < m; u++) {
                    const float f = w.fu * pw[m - 1 - u + w.reverse];
                    float bv[TK], cv[TC];
                    load_n<TK>(Bm + u * (D1 + 4) + ty * TK, bv);
                    load_n<TC>(Cm + u * (CS + 4) + tx * TC, cv);
#pragma unroll
                    for (int c = 0; c < TC; c++) cv[c] *= f;
#pragma unroll
                    for (int r = 0; r < TK; r += ROWS1 ? 1 : 2)
#pragma unroll
                        for (int c = 0; c < TC; c += ROWS1 ? 2 : 1) {  // in pairs as loaded
                            if (ROWS1) {
                                linear::axpy2<false>(&x[r][c], bv[r], cv + c);
                            } else {
                                float pair[2] = {x[r][c], x[r + 1][c]};
                                linear::axpy2<false>(pair, cv[c], bv + r);
                                x[r][c] = pair[0];
                                x[r + 1][c] = pair[1];
                            }
                        }
                }
            }
            if (heads > 1) {
                state_to(start_of(ho * heads + h));
                if (step + 1 < steps) state_from(state_before((step + 1) / heads, ho * heads + (step + 1) % heads));
            }
            share_state();
        }
        add_halves<RI>(acc, 1);
#pragma unroll
        for (int r = 0; r < RI / 2; r++) {
            const int u = out_row(r + (lane & 1) * (RI / 2));
            if (u < m) store_n<4>(out + (size_t)(t0 + (w.reverse ? m - 1 - u : u)) * out_stride + oc, acc[r]);
        }
#pragma unroll
        for (int r = 0; r < RI; r++)
#pragma unroll
            for (int c = 0; c < 4; c++) acc[r][c] = 0.f;
    }
    if (s.nseg == 1 && args.last) state_to(args.last + ((size_t)b * s.Hv + ho) * head_floats);  // heads == 1
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DK, int RS>
cudaError_t summary(const LinearSummaryArgs& a, cudaStream_t st) {
    const int bytes = 4 * (2 * LC * (RS + 4) + 2 * LC * (DK + 4) + LC + 1);
    if (cudaError_t e = allow_smem(linear_summary_kernel<DK, RS>, bytes)) return e;
    trace_begin("linear_summary", st);
    linear_summary_kernel<DK, RS><<<dim3(a.s.nseg * (a.s.Dv / RS), a.s.Hv, a.s.B), 256, bytes, st>>>(a);
    trace_end(st);
    return cudaGetLastError();
}

template <int D1, int CS, bool ROWS1>
cudaError_t mix(const LinearMixArgs& a, const MixView& w, int D2, cudaStream_t st) {
    const int bytes = 4 * (3 * LC * (D1 + 4) + 2 * LC * (CS + 4) + D1 * (CS + 4) + LC * (LC + 4) + 2 * (LC + 1));
    auto kernel = linear_mix_kernel<D1, CS, ROWS1>;
    if (cudaError_t e = allow_smem(kernel, bytes)) return e;
    trace_begin("linear_mix", st);
    const cudaError_t e = launch_after(kernel, dim3(a.s.nseg * (D2 / CS), w.ho, a.s.B), 256, bytes, st, a.overlap, a, w);
    trace_end(st);
    return e;
}

template <int CS, bool ROWS1>
cudaError_t mix_d1(const LinearMixArgs& a, const MixView& w, int D1, int D2, cudaStream_t st) {
    switch (D1) {
        case 32: return mix<32, CS, ROWS1>(a, w, D2, st);
        case 64: return mix<64, CS, ROWS1>(a, w, D2, st);
        default: return mix<128, CS, ROWS1>(a, w, D2, st);
    }
}

}  // namespace

// Segments of whole blocks: none where the heads alone give two CTAs per SM, since a second pass over the
// tokens for the segments' sums takes 0.4 of the mix pass's time; else as many as give two CTAs per
// SM, or up to eight if segments stay four blocks long, so that the SMs end together (T = 4096, 32 heads
// of 128: with one round of CTAs a mix pass of 422 us takes 465).
int linear_segments(int B, int T, int Hv, int Dv) {
    const long long blocks = (T + kLinearBlock - 1) / kLinearBlock, units = (long long)B * Hv * (Dv < 64 ? 1 : Dv / 64);
    if (blocks <= 1 || units <= 0 || units >= 304) return 1;
    const long long one = 304 / units, four = 1216 / units, fine = four < blocks / 4 ? four : blocks / 4;
    const long long want = one < fine ? fine : one;
    return (int)(want < blocks ? want : blocks);
}

cudaError_t launch_linear_summary(const LinearSummaryArgs& a, cudaStream_t st) {
    const bool narrow = a.s.Dv == 32;
    switch (a.s.Dk) {
        case 32: return narrow ? summary<32, 32>(a, st) : summary<32, 64>(a, st);
        case 64: return narrow ? summary<64, 32>(a, st) : summary<64, 64>(a, st);
        default: return narrow ? summary<128, 32>(a, st) : summary<128, 64>(a, st);
    }
}

cudaError_t launch_linear_combine(const LinearCombineArgs& a, bool overlap, cudaStream_t st) {
    trace_begin("linear_combine", st);
    const dim3 grid((a.s.Dv * a.s.Dk + 1023) / 1024, a.s.Hv, a.s.B);
    const cudaError_t e = launch_after(linear_combine_kernel, grid, 256, 0, st, overlap, a);
    trace_end(st);
    return e;
}

cudaError_t launch_linear_mix(const LinearMixArgs& a, cudaStream_t st) {
    const LinearShape& s = a.s;
    const int Hk = s.Hk, Hv = s.Hv;
    MixView w;
    switch (a.pass) {
        case LINEAR_O: w = {a.q, a.k, a.v, Hk, Hv, Hv, 0, a.scale, a.scale, 1.f}; break;
        case LINEAR_DQ: w = {a.do_, a.v, a.k, Hv, Hk, Hk, 0, a.scale, a.scale, 1.f}; break;
        case LINEAR_DK: w = {a.v, a.do_, a.q, Hv, Hk, Hk, 1, a.scale, 1.f, a.scale}; break;
        default: w = {a.k, a.q, a.do_, Hk, Hv, Hv, 1, a.scale, 1.f, a.scale}; break;
    }
    const bool rows1 = a.pass == LINEAR_DQ || a.pass == LINEAR_DK;
    const int D1 = rows1 ? s.Dv : s.Dk, D2 = rows1 ? s.Dk : s.Dv;
    if (rows1) return D2 == 32 ? mix_d1<32, true>(a, w, D1, D2, st) : mix_d1<64, true>(a, w, D1, D2, st);
    return D2 == 32 ? mix_d1<32, false>(a, w, D1, D2, st) : mix_d1<64, false>(a, w, D1, D2, st);
}

}  // namespace gdr
