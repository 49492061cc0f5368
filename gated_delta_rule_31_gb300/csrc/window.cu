// window.cu - softmax attention with a sliding window and visible first tokens (gdr_window_fwd, gdr_window_bwd): the launches,
// and fp32 problems on the CUDA cores: tiles of 64 queries and 64 keys in shared memory, all arithmetic in fp32.
//
// Forward, a CTA for each (64 queries, head, entry): with the running maximum m and sum l of each row, per tile
//     S = scale Q K^T,  m' = max(m, max S),  P = exp(S - m'),  l <- exp(m - m') l + sum P,  O <- exp(m - m') O + P V.
// VJP from lse = m + log l and delta = sum do o: P = exp(S - lse), dS = P (do V^T - delta),
//     dq = scale dS K over the tiles of keys (a CTA for each 64 queries and head),
//     dv = P^T do, dk = scale dS^T q over the queries that see a tile of keys, of all heads that share it.
// The two walk the pairs separately, 7 products for the 5 that one walk would need, so that neither adds into
// memory that another CTA adds into: the order of every sum is fixed.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention.h"
#include "common.cuh"
#include "kernels.h"
#include "window_host.h"

namespace gdr {

namespace {

constexpr int N = 64, THREADS = 256, LP = N + 4;  // tokens of a tile, row stride of P

__device__ __forceinline__ float4 get4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Rows t0 .. t0 + 63 of one head of x [B, T, H, D] into shared memory; rows from n on are zero.
template <int D>
__device__ __forceinline__ void load_tile(float* to, const void* x, int len, int H, int b, int h, int t0, int n) {
    for (int i = threadIdx.x; i < N * D / 4; i += THREADS) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + r < n) v = get4(static_cast<const float*>(x) + (((size_t)b * len + t0 + r) * H + h) * D + c);
        *reinterpret_cast<float4*>(to + r * (D + 4) + c) = v;
    }
}

// acc[i][j] = a row 4 ty + i . b row tx + 16 j
template <int D>
__device__ __forceinline__ void rows_by_rows(const float* a, const float* b, float (&acc)[4][4]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] = get4(a + (4 * ty + i) * (D + 4) + d);
#pragma unroll
        for (int j = 0; j < 4; j++) y[j] = get4(b + (tx + 16 * j) * (D + 4) + d);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
    }
}

// Columns of an output row that a thread keeps: D / 16 of them, W together.
template <int D>
struct Cols {
    static constexpr int W = D / 16 < 4 ? D / 16 : 4, NW = D / 16 / W;
    static __device__ __forceinline__ int at(int g) { return threadIdx.x % 16 * W + g * 16 * W; }
};

// acc[i][.] += sum over k of p[4 ty + i][k] b[k][columns]
template <int D>
__device__ __forceinline__ void rows_by_cols(const float* p, const float* b, float (&acc)[4][D / 16]) {
    using C = Cols<D>;
    const int ty = threadIdx.x / 16;
#pragma unroll 2
    for (int k = 0; k < N; k += 4) {
        float x[4][4];
#pragma unroll
        for (int i = 0; i < 4; i++) *reinterpret_cast<float4*>(x[i]) = get4(p + (4 * ty + i) * LP + k);
#pragma unroll
        for (int kk = 0; kk < 4; kk++)
#pragma unroll
            for (int g = 0; g < C::NW; g++) {
                float y[C::W];
#pragma unroll
                for (int c = 0; c < C::W; c++) y[c] = b[(k + kk) * (D + 4) + C::at(g) + c];
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int c = 0; c < C::W; c++) acc[i][g * C::W + c] = fmaf(x[i][kk], y[c], acc[i][g * C::W + c]);
            }
    }
}

__device__ __forceinline__ bool sees(const WindowShape& s, int t, int j, int n) {
    return j <= t && t < n && (t - j < s.window || j < s.sinks);
}
__device__ __forceinline__ float over16(float x, bool max) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = max ? fmaxf(x, y) : x + y;
    }
    return x;
}

template <int D>
__device__ __forceinline__ void put_rows(void* x, int len, int H, int b, int h, int t0, const float (&acc)[4][D / 16],
                                         const float* f) {
    using C = Cols<D>;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int t = t0 + threadIdx.x / 16 * 4 + i;
        if (t >= len) continue;
        float* row = static_cast<float*>(x) + (((size_t)b * len + t) * H + h) * D;
#pragma unroll
        for (int g = 0; g < C::NW; g++)
#pragma unroll
            for (int c = 0; c < C::W; c++) row[C::at(g) + c] = f[i] * acc[i][g * C::W + c];
    }
}

template <int D>
constexpr int tile_bytes() { return N * (D + 4) * 4; }

template <int D>
__global__ void __launch_bounds__(THREADS) window_fwd_kernel(WindowArgs a) {
    extern __shared__ __align__(16) float sh[];
    float *Q = sh, *K = Q + tile_bytes<D>() / 4, *V = K + tile_bytes<D>() / 4, *P = V + tile_bytes<D>() / 4;
    const WindowShape& s = a.s;
    const int t0 = (gridDim.x - 1 - blockIdx.x) * N, h = blockIdx.y, b = blockIdx.z, hk = h / (s.Hq / s.Hk), n = s.tokens(b);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    if (blockIdx.x + blockIdx.y + blockIdx.z == 0 && threadIdx.x < 4) a.status[threadIdx.x] = 0;
    const KeyTiles tiles(N, s.window, s.sinks, t0, min(t0 + N, n));
    load_tile<D>(Q, a.q, s.T, s.Hq, b, h, t0, n);
    float m[4], l[4], acc[4][D / 16] = {};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    for (int it = 0; it < tiles.count(); it++) {
        const int j0 = tiles.at(it) * N;
        __syncthreads();
        load_tile<D>(K, a.k, s.T, s.Hk, b, hk, j0, n);
        load_tile<D>(V, a.v, s.T, s.Hk, b, hk, j0, n);
        __syncthreads();
        float S[4][4];
        rows_by_rows<D>(Q, K, S);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int t = t0 + 4 * ty + i;
            float top = m[i], sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                S[i][j] = sees(s, t, j0 + tx + 16 * j, n) ? s.scale * S[i][j] : -INFINITY;
                top = fmaxf(top, S[i][j]);
            }
            top = over16(top, true);
            const float base = top == -INFINITY ? 0.f : top;  // no token seen yet
            const float fade = expf(m[i] - base);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                S[i][j] = expf(S[i][j] - base);
                sum += S[i][j];
                P[(4 * ty + i) * LP + tx + 16 * j] = S[i][j];
            }
            m[i] = top;
            l[i] = fade * l[i] + over16(sum, false);
#pragma unroll
            for (int c = 0; c < D / 16; c++) acc[i][c] *= fade;
        }
        __syncthreads();
        rows_by_cols<D>(P, V, acc);
    }
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
    put_rows<D>(a.o, s.T, s.Hq, b, h, t0, acc, f);
    if (a.lse && tx == 0)
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (t0 + 4 * ty + i < s.T)
                a.lse[((size_t)b * s.Hq + h) * s.T + t0 + 4 * ty + i] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
}

// delta [B, Hq, T]: 8 lanes a row.
__global__ void __launch_bounds__(256) window_delta_kernel(WindowArgs a) {
    const WindowShape& s = a.s;
    const size_t row = ((size_t)blockIdx.x * 256 + threadIdx.x) / 8, rows = (size_t)s.B * s.T * s.Hq;
    if (blockIdx.x == 0 && threadIdx.x < 4) a.status[threadIdx.x] = 0;
    if (row >= rows) return;  // whole groups of 8 lanes
    const int h = row % s.Hq, lane = threadIdx.x % 8;
    const size_t bt = row / s.Hq;
    const int t = bt % s.T, b = bt / s.T;
    float x = 0.f;
    if (t < s.tokens(b))
        for (int d = 4 * lane; d < s.D; d += 32) {
            const float4 u = get4(static_cast<const float*>(a.do_) + row * s.D + d), v = get4(static_cast<const float*>(a.o) + row * s.D + d);
            x += u.x * v.x + u.y * v.y + u.z * v.z + u.w * v.w;
        }
    const uint32_t group = 0xffu << (threadIdx.x & 24);
    for (int m = 4; m > 0; m >>= 1) x += __shfl_xor_sync(group, x, m);
    if (lane == 0) a.delta[((size_t)b * s.Hq + h) * s.T + t] = x;
}

template <int D>
__global__ void __launch_bounds__(THREADS) window_dq_kernel(WindowArgs a) {
    extern __shared__ __align__(16) float sh[];
    constexpr int TILE = tile_bytes<D>() / 4;
    float *Q = sh, *G = Q + TILE, *K = G + TILE, *V = K + TILE, *P = V + TILE;
    const WindowShape& s = a.s;
    const int t0 = (gridDim.x - 1 - blockIdx.x) * N, h = blockIdx.y, b = blockIdx.z, hk = h / (s.Hq / s.Hk), n = s.tokens(b);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const KeyTiles tiles(N, s.window, s.sinks, t0, min(t0 + N, n));
    load_tile<D>(Q, a.q, s.T, s.Hq, b, h, t0, n);
    load_tile<D>(G, a.do_, s.T, s.Hq, b, h, t0, n);
    float lse[4], delta[4], acc[4][D / 16] = {};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int t = t0 + 4 * ty + i;
        const size_t at = ((size_t)b * s.Hq + h) * s.T + t;
        lse[i] = t < n ? a.lse[at] : 0.f;
        delta[i] = t < n ? a.delta[at] : 0.f;
    }
    for (int it = 0; it < tiles.count(); it++) {
        const int j0 = tiles.at(it) * N;
        __syncthreads();
        load_tile<D>(K, a.k, s.T, s.Hk, b, hk, j0, n);
        load_tile<D>(V, a.v, s.T, s.Hk, b, hk, j0, n);
        __syncthreads();
        float S[4][4], dP[4][4];
        rows_by_rows<D>(Q, K, S);
        rows_by_rows<D>(G, V, dP);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bool on = sees(s, t0 + 4 * ty + i, j0 + tx + 16 * j, n);
                P[(4 * ty + i) * LP + tx + 16 * j] = on ? expf(s.scale * S[i][j] - lse[i]) * (dP[i][j] - delta[i]) : 0.f;
            }
        __syncthreads();
        rows_by_cols<D>(P, K, acc);
    }
    const float f[4] = {s.scale, s.scale, s.scale, s.scale};
    put_rows<D>(a.dq, s.T, s.Hq, b, h, t0, acc, f);
}

template <int D>
__global__ void __launch_bounds__(THREADS) window_dkv_kernel(WindowArgs a) {
    extern __shared__ __align__(16) float sh[];
    constexpr int TILE = tile_bytes<D>() / 4;
    float *Q = sh, *G = Q + TILE, *K = G + TILE, *V = K + TILE, *P = V + TILE, *dS = P + N * LP;
    const WindowShape& s = a.s;
    const int j0 = blockIdx.x * N, hk = blockIdx.y, b = blockIdx.z, group = s.Hq / s.Hk, n = s.tokens(b);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    load_tile<D>(K, a.k, s.T, s.Hk, b, hk, j0, n);
    load_tile<D>(V, a.v, s.T, s.Hk, b, hk, j0, n);
    float dk[4][D / 16] = {}, dv[4][D / 16] = {};
    const int end = j0 < n ? queries_end(N, s.window, s.sinks, j0, n) : 0;
    for (int h = hk * group; h < (hk + 1) * group; h++)
        for (int t0 = j0; t0 < end; t0 += N) {
            __syncthreads();
            load_tile<D>(Q, a.q, s.T, s.Hq, b, h, t0, n);
            load_tile<D>(G, a.do_, s.T, s.Hq, b, h, t0, n);
            __syncthreads();
            float S[4][4], dP[4][4];  // rows: keys, columns: queries
            rows_by_rows<D>(K, Q, S);
            rows_by_rows<D>(V, G, dP);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int t = t0 + tx + 16 * j;
                const size_t at = ((size_t)b * s.Hq + h) * s.T + t;
                const float lse = t < n ? a.lse[at] : 0.f, delta = t < n ? a.delta[at] : 0.f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const bool on = sees(s, t, j0 + 4 * ty + i, n);
                    const float p = on ? expf(s.scale * S[i][j] - lse) : 0.f;
                    P[(4 * ty + i) * LP + tx + 16 * j] = p;
                    dS[(4 * ty + i) * LP + tx + 16 * j] = on ? p * (dP[i][j] - delta) : 0.f;
                }
            }
            __syncthreads();
            rows_by_cols<D>(P, G, dv);
            rows_by_cols<D>(dS, Q, dk);
        }
    const float f[4] = {s.scale, s.scale, s.scale, s.scale}, one[4] = {1.f, 1.f, 1.f, 1.f};
    put_rows<D>(a.dk, s.T, s.Hk, b, hk, j0, dk, f);
    put_rows<D>(a.dv, s.T, s.Hk, b, hk, j0, dv, one);
}

template <typename K>
cudaError_t launch(K kernel, const char* name, int heads, int smem, const WindowArgs& a, cudaStream_t st) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
    trace_begin(name, st);
    kernel<<<dim3((a.s.T + N - 1) / N, heads, a.s.B), THREADS, smem, st>>>(a);
    trace_end(st);
    return cudaGetLastError();
}
template <int D>
cudaError_t fwd(const WindowArgs& a, cudaStream_t st) {
    return launch(window_fwd_kernel<D>, "window_fwd", a.s.Hq, 3 * tile_bytes<D>() + N * LP * 4, a, st);
}
cudaError_t delta(const WindowArgs& a, cudaStream_t st) {
    const size_t rows = (size_t)a.s.B * a.s.T * a.s.Hq;
    trace_begin("window_delta", st);
    window_delta_kernel<<<(unsigned)((rows + 31) / 32), 256, 0, st>>>(a);
    trace_end(st);
    return cudaGetLastError();
}
template <int D>
cudaError_t bwd(const WindowArgs& a, cudaStream_t st) {
    if (cudaError_t e = launch(window_dq_kernel<D>, "window_dq", a.s.Hq, 4 * tile_bytes<D>() + N * LP * 4, a, st)) return e;
    return launch(window_dkv_kernel<D>, "window_dkv", a.s.Hk, 4 * tile_bytes<D>() + 2 * N * LP * 4, a, st);
}

}  // namespace

cudaError_t launch_window_fwd(const WindowArgs& a, cudaStream_t st) {
    if (a.s.bf16) return launch_window_fwd_tc(a, st);
    return a.s.D == 32 ? fwd<32>(a, st) : a.s.D == 64 ? fwd<64>(a, st) : fwd<128>(a, st);
}

cudaError_t launch_window_bwd(const WindowArgs& a, cudaStream_t st) {
    if (a.s.bf16) return launch_window_bwd_tc(a, st);
    if (cudaError_t e = delta(a, st)) return e;
    return a.s.D == 32 ? bwd<32>(a, st) : a.s.D == 64 ? bwd<64>(a, st) : bwd<128>(a, st);
}

}  // namespace gdr
