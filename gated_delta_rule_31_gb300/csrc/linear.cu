// linear.cu - linear attention with a constant decay per head on the CUDA cores, in fp32: the
// segment summary, the combine step and the mix pass (linear.h).
//
// A chunk holds up to 64 tokens in processing order (u = 0 is the first token of the chunk, or
// its last one in reverse), so both directions run the same sums over j <= r:
//     P_rj = f l^(r-j) (a_r . b_j),   out_r = f' l^(r+1-s) a_r X + sum_{j<=r} P_rj c_j,
//     X <- l^m X + f'' sum_j l^(m-1-j+s) b_j c_j^T          (m tokens in the chunk; s = reverse)
// with f = scale, and (f', f'') = (scale, 1) forwards, (1, scale) in reverse: in reverse X is the
// adjoint of the state after the chunk, which reaches token 0 (the last one) undecayed. Every
// power of l has an exponent >= 0, so no decay overflows, and l^0 = 1 also where l = 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "linear.h"
#include "linear_dev.cuh"

namespace gdr {

namespace {

constexpr int LC = 64;  // tokens of a chunk

using linear::power;

__device__ __forceinline__ int valid_tokens(const LinearShape& s, int b) {
    return s.lengths ? min(max(s.lengths[b], 0), s.T) : s.T;
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

// Columns [c0, c0 + D) of a chunk's tokens of one head, in processing order, as fp32 rows of
// stride D + 4; rows m .. 63 are zero.
template <int D, typename T>
__device__ __forceinline__ void load_tile(float* dst, const T* src, size_t token0, size_t token_stride, int c0, int m,
                                          int reverse) {
    constexpr int V = D / 4;
    for (int i = threadIdx.x; i < LC * V; i += blockDim.x) {
        const int u = i / V, c = 4 * (i % V);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u < m) x = load4(src + (token0 + (reverse ? m - 1 - u : u)) * token_stride + c0 + c);
        *reinterpret_cast<float4*>(dst + u * (D + 4) + c) = x;
    }
}

__device__ __forceinline__ float at(const float4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// grid (nseg * Dv / RS, Hv, B): rows [RS * i, ...) of the state's sum over one segment.
template <int DK, int RS, typename T>
__global__ void __launch_bounds__(256) linear_summary_kernel(LinearSummaryArgs a) {
    extern __shared__ float sm[];
    float* X = sm;                      // [64][RS + 4]
    float* Y = X + LC * (RS + 4);       // [64][DK + 4]
    float* pw = Y + LC * (DK + 4);      // l^0 .. l^64
    const LinearShape& s = a.s;
    const int nr = s.Dv / RS, seg = blockIdx.x / nr, r0 = (blockIdx.x % nr) * RS;
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / (s.Hv / s.Hk);
    constexpr int TR = RS / 16, TC = DK / 16;  // rows and columns of a thread
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    if (threadIdx.x <= LC) pw[threadIdx.x] = power(s.g[hv], threadIdx.x);
    const int first = min(seg * s.seg_tokens, valid_tokens(s, b));
    const int last = min(first + s.seg_tokens, valid_tokens(s, b));
    const int nc = (last - first + LC - 1) / LC;
    const T* rows = static_cast<const T*>(a.rows) + ((size_t)b * s.T * s.Hv + hv) * s.Dv;
    const T* cols = static_cast<const T*>(a.cols) + ((size_t)b * s.T * s.Hk + hk) * s.Dk;
    float z[TR][TC] = {};
    for (int i = 0; i < nc; i++) {
        const int t0 = first + (a.reverse ? nc - 1 - i : i) * LC, m = min(LC, last - t0);
        __syncthreads();
        load_tile<RS>(X, rows, t0, (size_t)s.Hv * s.Dv, r0, m, a.reverse);
        load_tile<DK>(Y, cols, t0, (size_t)s.Hk * s.Dk, 0, m, a.reverse);
        __syncthreads();
        const float over = pw[m];
#pragma unroll
        for (int r = 0; r < TR; r++)
#pragma unroll
            for (int c = 0; c < TC; c++) z[r][c] *= over;
        for (int u = 0; u < m; u++) {
            const float w = a.factor * pw[m - 1 - u + a.reverse];
            float y[TC];
#pragma unroll
            for (int c = 0; c < TC; c++) y[c] = Y[u * (DK + 4) + tx + 16 * c];
#pragma unroll
            for (int r = 0; r < TR; r++) {
                const float x = w * X[u * (RS + 4) + ty + 16 * r];
#pragma unroll
                for (int c = 0; c < TC; c++) z[r][c] += x * y[c];
            }
        }
    }
    float* out = a.z + ((((size_t)b * s.Hv + hv) * s.nseg + seg) * s.Dv + r0) * s.Dk;
#pragma unroll
    for (int r = 0; r < TR; r++)
#pragma unroll
        for (int c = 0; c < TC; c++) out[(size_t)(ty + 16 * r) * s.Dk + tx + 16 * c] = z[r][c];
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

struct MixView {  // the roles of a pass (linear.h)
    const void *a, *b, *c;
    int ha, hc, ho;  // heads of a and b, of c, and of the output
    int reverse;
    float fp, fx, fu;  // factors of P, of a X and of the state's update
};

// grid (nseg * D2 / CS, output heads, B). D1: width of a and b; a CTA forms CS of the D2 output columns.
// ROWS1: the state's rows (Dv) run along D1 (dq, dk), else along D2 (o, dv).
template <int D1, int CS, bool ROWS1, typename T>
__global__ void __launch_bounds__(256) linear_mix_kernel(LinearMixArgs args, MixView w) {
    extern __shared__ float sm[];
    float* A = sm;                         // [64][D1 + 4]
    float* Bm = A + LC * (D1 + 4);         // [64][D1 + 4]
    float* Cm = Bm + LC * (D1 + 4);        // [64][CS + 4]
    float* X = Cm + LC * (CS + 4);         // [D1][CS + 4]
    float* P = X + D1 * (CS + 4);          // [64][68]
    float* pw = P + LC * (LC + 4);         // l^0 .. l^64
    const LinearShape& s = args.s;
    const int D2 = ROWS1 ? s.Dk : s.Dv;
    const int ns = D2 / CS, seg = blockIdx.x / ns, c0 = (blockIdx.x % ns) * CS;
    const int ho = blockIdx.y, b = blockIdx.z, heads = s.Hv / w.ho;  // value heads summed into this output
    const int G = s.Hv / s.Hk;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    constexpr int TC = CS / 16, TK = D1 / 16;
    const int n = valid_tokens(s, b);
    const int begin = seg * s.seg_tokens, end = min(begin + s.seg_tokens, s.T);
    const int first = min(begin, n), last = min(end, n), nc = (last - first + LC - 1) / LC;
    T* out = static_cast<T*>(args.out) + ((size_t)b * s.T * w.ho + ho) * D2 + c0;
    const size_t out_stride = (size_t)w.ho * D2;
    for (int i = threadIdx.x; i < (end - max(begin, n)) * (CS / 4); i += 256)  // past the length: zero
        store4(out + (size_t)(max(begin, n) + i / (CS / 4)) * out_stride + 4 * (i % (CS / 4)),
               make_float4(0.f, 0.f, 0.f, 0.f));
    const size_t head_floats = (size_t)s.Dv * s.Dk;
    auto start_of = [&](int hv) { return args.starts + (((size_t)b * s.Hv + hv) * s.nseg + seg) * head_floats; };
    auto move_state = [&](float* p, bool load) {
        for (int i = threadIdx.x; i < D1 * CS; i += 256) {
            // along the state's rows in memory, so that neighbouring threads touch neighbouring floats
            const int d1 = ROWS1 ? i / CS : i % D1, d2 = ROWS1 ? i % CS : i / D1;
            float* q = ROWS1 ? p + (size_t)d1 * s.Dk + c0 + d2 : p + (size_t)(c0 + d2) * s.Dk + d1;
            if (load) X[d1 * (CS + 4) + d2] = *q;
            else *q = X[d1 * (CS + 4) + d2];
        }
    };
    if (heads == 1 && nc > 0) move_state(start_of(ho), true);
    for (int i = 0; i < nc; i++) {
        const int t0 = first + (w.reverse ? nc - 1 - i : i) * LC, m = min(LC, last - t0);
        float acc[4][TC] = {};
        for (int h = 0; h < heads; h++) {
            const int hv = ho * heads + h, hk = hv / G;
            const int ia = w.ha == s.Hv ? hv : hk, ic = w.hc == s.Hv ? hv : hk;
            __syncthreads();
            if (heads > 1) move_state(start_of(hv), true);
            if (threadIdx.x <= LC) pw[threadIdx.x] = power(s.g[hv], threadIdx.x);
            load_tile<D1>(A, static_cast<const T*>(w.a) + ((size_t)b * s.T * w.ha + ia) * D1, t0, (size_t)w.ha * D1, 0, m,
                          w.reverse);
            load_tile<D1>(Bm, static_cast<const T*>(w.b) + ((size_t)b * s.T * w.ha + ia) * D1, t0, (size_t)w.ha * D1, 0,
                          m, w.reverse);
            load_tile<CS>(Cm, static_cast<const T*>(w.c) + ((size_t)b * s.T * w.hc + ic) * D2, t0, (size_t)w.hc * D2, c0,
                          m, w.reverse);
            __syncthreads();
            {  // P: rows ty + 16 i, columns tx + 16 j
                float p[4][4] = {};
                for (int k = 0; k < D1; k += 4) {
                    float4 x[4], y[4];
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        x[r] = load4(A + (ty + 16 * r) * (D1 + 4) + k);
                        y[r] = load4(Bm + (tx + 16 * r) * (D1 + 4) + k);
                    }
#pragma unroll
                    for (int r = 0; r < 4; r++)
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            p[r][j] += x[r].x * y[j].x + x[r].y * y[j].y + x[r].z * y[j].z + x[r].w * y[j].w;
                }
#pragma unroll
                for (int r = 0; r < 4; r++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int u = ty + 16 * r, v = tx + 16 * j;
                        P[u * (LC + 4) + v] = v <= u ? w.fp * pw[u - v] * p[r][j] : 0.f;
                    }
            }
            {  // a X
                float x[4][TC] = {};
                for (int k = 0; k < D1; k += 4) {
                    float4 av[4];
#pragma unroll
                    for (int r = 0; r < 4; r++) av[r] = load4(A + (ty + 16 * r) * (D1 + 4) + k);
#pragma unroll
                    for (int e = 0; e < 4; e++)
#pragma unroll
                        for (int c = 0; c < TC; c++) {
                            const float xv = X[(k + e) * (CS + 4) + tx + 16 * c];
#pragma unroll
                            for (int r = 0; r < 4; r++) x[r][c] += at(av[r], e) * xv;
                        }
                }
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const float f = w.fx * pw[ty + 16 * r + 1 - w.reverse];
#pragma unroll
                    for (int c = 0; c < TC; c++) acc[r][c] += f * x[r][c];
                }
            }
            __syncthreads();  // P is written, X is read
            for (int k = 0; k < m; k += 4) {  // P c
                float4 pv[4];
#pragma unroll
                for (int r = 0; r < 4; r++) pv[r] = load4(P + (ty + 16 * r) * (LC + 4) + k);
#pragma unroll
                for (int e = 0; e < 4; e++)
#pragma unroll
                    for (int c = 0; c < TC; c++) {
                        const float cv = Cm[(k + e) * (CS + 4) + tx + 16 * c];
#pragma unroll
                        for (int r = 0; r < 4; r++) acc[r][c] += at(pv[r], e) * cv;
                    }
            }
            {  // the state over this chunk: rows ty + 16 r, columns tx + 16 c
                float x[TK][TC];
                const float over = pw[m];
#pragma unroll
                for (int r = 0; r < TK; r++)
#pragma unroll
                    for (int c = 0; c < TC; c++) x[r][c] = over * X[(ty + 16 * r) * (CS + 4) + tx + 16 * c];
                for (int u = 0; u < m; u++) {
                    const float f = w.fu * pw[m - 1 - u + w.reverse];
                    float cv[TC];
#pragma unroll
                    for (int c = 0; c < TC; c++) cv[c] = f * Cm[u * (CS + 4) + tx + 16 * c];
#pragma unroll
                    for (int r = 0; r < TK; r++) {
                        const float bv = Bm[u * (D1 + 4) + ty + 16 * r];
#pragma unroll
                        for (int c = 0; c < TC; c++) x[r][c] += bv * cv[c];
                    }
                }
#pragma unroll
                for (int r = 0; r < TK; r++)
#pragma unroll
                    for (int c = 0; c < TC; c++) X[(ty + 16 * r) * (CS + 4) + tx + 16 * c] = x[r][c];
            }
            if (heads > 1) {
                __syncthreads();
                move_state(start_of(hv), false);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int u = ty + 16 * r;
            if (u >= m) continue;
            T* row = out + (size_t)(t0 + (w.reverse ? m - 1 - u : u)) * out_stride;
#pragma unroll
            for (int c = 0; c < TC; c++) {
                if constexpr (sizeof(T) == 4) row[tx + 16 * c] = acc[r][c];
                else row[tx + 16 * c] = __float2bfloat16_rn(acc[r][c]);
            }
        }
    }
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DK, int RS, typename T>
cudaError_t summary(const LinearSummaryArgs& a, cudaStream_t st) {
    const int bytes = 4 * (LC * (RS + 4) + LC * (DK + 4) + LC + 1);
    auto kernel = linear_summary_kernel<DK, RS, T>;
    if (cudaError_t e = allow_smem(kernel, bytes)) return e;
    trace_begin("linear_summary", st);
    kernel<<<dim3(a.s.nseg * (a.s.Dv / RS), a.s.Hv, a.s.B), 256, bytes, st>>>(a);
    trace_end(st);
    return cudaGetLastError();
}

template <typename T>
cudaError_t summary_of(const LinearSummaryArgs& a, cudaStream_t st) {
    const bool narrow = a.s.Dv == 32;
    switch (a.s.Dk) {
        case 32: return narrow ? summary<32, 32, T>(a, st) : summary<32, 64, T>(a, st);
        case 64: return narrow ? summary<64, 32, T>(a, st) : summary<64, 64, T>(a, st);
        default: return narrow ? summary<128, 32, T>(a, st) : summary<128, 64, T>(a, st);
    }
}

template <int D1, int CS, bool ROWS1, typename T>
cudaError_t mix(const LinearMixArgs& a, const MixView& w, int D2, cudaStream_t st) {
    const int bytes = 4 * (2 * LC * (D1 + 4) + LC * (CS + 4) + D1 * (CS + 4) + LC * (LC + 4) + LC + 1);
    auto kernel = linear_mix_kernel<D1, CS, ROWS1, T>;
    if (cudaError_t e = allow_smem(kernel, bytes)) return e;
    trace_begin("linear_mix", st);
    kernel<<<dim3(a.s.nseg * (D2 / CS), w.ho, a.s.B), 256, bytes, st>>>(a, w);
    trace_end(st);
    return cudaGetLastError();
}

template <int CS, bool ROWS1, typename T>
cudaError_t mix_d1(const LinearMixArgs& a, const MixView& w, int D1, int D2, cudaStream_t st) {
    switch (D1) {
        case 32: return mix<32, CS, ROWS1, T>(a, w, D2, st);
        case 64: return mix<64, CS, ROWS1, T>(a, w, D2, st);
        default: return mix<128, CS, ROWS1, T>(a, w, D2, st);
    }
}

template <typename T>
cudaError_t mix_of(const LinearMixArgs& a, cudaStream_t st) {
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
    if (rows1)
        return D2 == 32 ? mix_d1<32, true, T>(a, w, D1, D2, st) : mix_d1<64, true, T>(a, w, D1, D2, st);
    return D2 == 32 ? mix_d1<32, false, T>(a, w, D1, D2, st) : mix_d1<64, false, T>(a, w, D1, D2, st);
}

}  // namespace

// Segments: enough CTAs for two per SM, each of whole chunks.
int linear_segments(int B, int T, int Hv, int Dv) {
    const long long chunks = (T + LC - 1) / LC, units = (long long)B * Hv * (Dv < 64 ? 1 : Dv / 64);
    if (chunks <= 1 || units <= 0) return 1;
    const long long want = (2 * 152 + units - 1) / units;
    return (int)(want < chunks ? want : chunks);
}

cudaError_t launch_linear_summary(const LinearSummaryArgs& a, cudaStream_t st) {
    return a.s.bf16 ? summary_of<__nv_bfloat16>(a, st) : summary_of<float>(a, st);
}

cudaError_t launch_linear_combine(const LinearCombineArgs& a, bool overlap, cudaStream_t st) {
    trace_begin("linear_combine", st);
    const dim3 grid((a.s.Dv * a.s.Dk + 1023) / 1024, a.s.Hv, a.s.B);
    const cudaError_t e = launch_after(linear_combine_kernel, grid, 256, 0, st, overlap, a);
    trace_end(st);
    return e;
}

cudaError_t launch_linear_mix(const LinearMixArgs& a, cudaStream_t st) {
    return a.s.bf16 ? mix_of<__nv_bfloat16>(a, st) : mix_of<float>(a, st);
}

}  // namespace gdr
