// paged.cu - attention of one new token of each sequence over a paged cache (gdr_paged_decode_step).
//
// Entry b with n tokens sees tokens j >= n - window and j < sinks: a list of `first` tokens from the start and those
// from lo on, cut into tiles of 64. The tiles of all entries and key heads in a row (entries outermost) are dealt
// out evenly, a run of neighbouring tiles to each CTA, whatever the lengths, which only the device knows. A CTA
// walks its run with the running maximum m and sum l of a softmax and the sum O of exp(s - m) v for the heads that share a key
// head; a head whose tiles lie in one run is written at once, of one that is cut each run leaves (m, l, O), and a second
// kernel joins them, runs in order: o = sum exp(m_i - m) O_i / sum exp(m_i - m) l_i.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention.h"
#include "common.cuh"
#include "kernels.h"
#include "linear.h"
#include "linear_dev.cuh"

namespace gdr {

namespace {

constexpr int TILE = 64, THREADS = 128, HEADS = 8;  // tokens of a tile, heads that share a walk
constexpr int RUNS = 2 * 152;                        // CTAs

__device__ __forceinline__ float4 get4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 get4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y));
}
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The tokens that entry b sees.
struct Seen {
    int first, lo, count;
    __device__ Seen(const PagedArgs& a, int b) {
        const long long most = (long long)a.table_pages * a.page_size;
        const int n = (int)min((long long)max(a.lengths[b], 0), most);
        lo = a.window > 0 ? max(n - a.window, 0) : 0;
        first = min(a.sinks, lo);
        count = first + n - lo;
    }
    __device__ int at(int i) const { return i < first ? i : lo + (i - first); }
    __device__ int tiles() const { return (count + TILE - 1) / TILE; }
};

// Which entry and how far into it: entry, tiles before it per walk (a walk is a key head's block of heads).
struct Place {
    int b;
    long long before;
};

// Tiles of all entries, per walk, and the places of two tiles (numbered over all entries and walks), by all threads of a CTA of THREADS.
__device__ long long find(const PagedArgs& a, int walks, int run, int runs, Place& from, long long& begin, long long& end) {
    __shared__ long long total_sh, part[THREADS / 32];
    __shared__ Place from_sh;
    const int tid = threadIdx.x, per = (a.B + THREADS - 1) / THREADS;
    long long mine = 0;
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); b++) mine += Seen(a, b).tiles();
    long long scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, scan, o);
        if ((tid & 31) >= o) scan += y;
    }
    if ((tid & 31) == 31) part[tid >> 5] = scan;
    __syncthreads();
    long long before = scan - mine;
    for (int w = 0; w < tid >> 5; w++) before += part[w];
    if (tid == THREADS - 1) total_sh = before + mine;
    __syncthreads();
    const long long total = total_sh * walks;
    begin = total * run / runs;
    end = total * (run + 1) / runs;
    if (before * walks <= begin && begin < (before + mine) * walks)
        for (int b = tid * per; b < min(a.B, (tid + 1) * per); b++) {
            const long long t = Seen(a, b).tiles();
            if (begin < (before + t) * walks) {
                from_sh = Place{b, before};
                break;
            }
            before += t;
        }
    __syncthreads();
    from = from_sh;
    return total;
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS) paged_kernel(PagedArgs a, int blocks) {
    extern __shared__ __align__(16) float sh[];
    constexpr int LD = D + 4;
    float *K = sh, *V = K + TILE * LD, *Q = V + TILE * LD, *P = Q + HEADS * LD;
    __shared__ float m_sh[HEADS], l_sh[HEADS], fade_sh[HEADS];
    linear::next_kernel_may_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = a.Hq / a.Hk, walks = a.Hk * blocks;
    Place at;
    long long begin, end;
    find(a, walks, blockIdx.x, gridDim.x, at, begin, end);
    long long tile = begin;
    int segment = 0;
    while (tile < end) {
        const Seen seen(a, at.b);
        const int tiles = seen.tiles();
        if (tile >= (at.before + tiles) * walks) {
            at.before += tiles;
            at.b++;
            continue;
        }
        const int walk = (int)((tile - at.before * walks) / tiles), t0 = (int)(tile - at.before * walks - (long long)walk * tiles);
        const int t1 = (int)min((long long)tiles, t0 + end - tile);
        const int hk = walk / blocks, g0 = walk % blocks * HEADS, ng = min(HEADS, group - g0);
        const size_t q0 = (size_t)at.b * a.Hq + hk * group + g0;
        __syncthreads();
        for (int i = tid; i < HEADS * D; i += THREADS)
            Q[i / D * LD + i % D] = i / D < ng ? a.scale * as_float(static_cast<const T*>(a.q)[q0 * D + i]) : 0.f;
        if (tid < HEADS) {
            m_sh[tid] = -INFINITY;
            l_sh[tid] = 0.f;
        }
        float acc[HEADS * D / THREADS];  // heads tid / D + (THREADS / D) i, channel tid % D
#pragma unroll
        for (int i = 0; i < HEADS * D / THREADS; i++) acc[i] = 0.f;
        for (int t = t0; t < t1; t++) {
            __syncthreads();
            for (int i = tid; i < TILE * D / 4; i += THREADS) {
                const int r = i / (D / 4), c = i % (D / 4) * 4, x = t * TILE + r;
                float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
                bool on = x < seen.count;
                if (on) {
                    const int j = seen.at(x), page = a.table[(size_t)at.b * a.table_pages + j / a.page_size];
                    on = (unsigned)page < (unsigned)a.pages;
                    if (on) {
                        const size_t row = (((size_t)page * a.page_size + j % a.page_size) * a.Hk + hk) * D + c;
                        k = get4(static_cast<const T*>(a.k) + row);
                        v = get4(static_cast<const T*>(a.v) + row);
                    }
                }
                *reinterpret_cast<float4*>(K + r * LD + c) = k;
                *reinterpret_cast<float4*>(V + r * LD + c) = v;
                if (c == 0) K[r * LD + D] = on ? 0.f : -INFINITY;  // whether the token is there
            }
            __syncthreads();
            for (int g = warp; g < ng; g += THREADS / 32) {  // a warp per head, two tokens a lane
                float s[TILE / 32];
                float top = m_sh[g], sum = 0.f;
#pragma unroll
                for (int i = 0; i < TILE / 32; i++) {
                    const float* k = K + (lane + 32 * i) * LD;
                    float x = 0.f;
#pragma unroll 8
                    for (int d = 0; d < D; d += 4) {
                        const float4 u = get4(k + d), w = get4(Q + g * LD + d);
                        x += u.x * w.x + u.y * w.y + u.z * w.z + u.w * w.w;
                    }
                    s[i] = k[D] == 0.f ? x : -INFINITY;
                    top = fmaxf(top, s[i]);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int i = 0; i < TILE / 32; i++) {
                    const float p = expf(s[i] - base);
                    P[g * TILE + lane + 32 * i] = p;
                    sum += p;
                }
                sum = warp_sum(sum);
                if (lane == 0) {
                    fade_sh[g] = expf(m_sh[g] - base);
                    l_sh[g] = fade_sh[g] * l_sh[g] + sum;
                    m_sh[g] = top;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < HEADS * D / THREADS; i++) {
                const int g = tid / D + THREADS / D * i;
                if (g >= ng) continue;
                float x = fade_sh[g] * acc[i];
#pragma unroll 8
                for (int j = 0; j < TILE; j++) x = fmaf(P[g * TILE + j], V[j * LD + tid % D], x);
                acc[i] = x;
            }
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == tiles;
        float* part = a.parts + (size_t)(2 * blockIdx.x + (segment > 0)) * HEADS * (D + 2);
#pragma unroll
        for (int i = 0; i < HEADS * D / THREADS; i++) {
            const int g = tid / D + THREADS / D * i;
            if (g >= ng) continue;
            if (whole) put(static_cast<T*>(a.o) + (q0 + g) * D + tid % D, l_sh[g] > 0.f ? acc[i] / l_sh[g] : 0.f);
            else part[g * (D + 2) + tid % D] = acc[i];
        }
        if (!whole && tid < ng) {
            part[tid * (D + 2) + D] = m_sh[tid];
            part[tid * (D + 2) + D + 1] = l_sh[tid];
        }
        tile += t1 - t0;
        segment++;
    }
    // entries without a token: zero
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (Seen(a, b).count == 0)
            for (int i = tid; i < a.Hq * D; i += THREADS) put(static_cast<T*>(a.o) + (size_t)b * a.Hq * D + i, 0.f);
}

// Joins the walk that the border before run blockIdx.x + 1 cuts, if that border is the first in it.
template <int D, typename T>
__global__ void __launch_bounds__(THREADS) paged_join_kernel(PagedArgs a, int blocks) {
    linear::next_kernel_may_start();
    const int tid = threadIdx.x, group = a.Hq / a.Hk, walks = a.Hk * blocks, run = blockIdx.x + 1, runs = gridDim.x + 1;
    Place at;
    long long begin, end;
    const long long total = find(a, walks, run, runs, at, begin, end);
    linear::wait_kernel_before();
    if (begin >= total) return;
    const long long tiles = Seen(a, at.b).tiles(), start = at.before * walks;
    const int walk = (int)((begin - start) / tiles);
    const long long w0 = start + walk * tiles, w1 = w0 + tiles;
    if (w0 == begin || total * (run - 1) / runs > w0) return;
    const int hk = walk / blocks, g0 = walk % blocks * HEADS, ng = min(HEADS, group - g0);
    const size_t q0 = (size_t)at.b * a.Hq + hk * group + g0;
    for (int i = tid; i < ng * D; i += THREADS) {
        const int g = i / D, d = i % D;
        float m = -INFINITY, l = 0.f, x = 0.f;
        for (int r = run - 1; r < runs; r++) {
            const long long rb = total * r / runs, re = total * (r + 1) / runs;
            if (rb >= w1) break;
            if (rb == re) continue;
            const float* part = a.parts + (size_t)(2 * r + (rb < w0)) * HEADS * (D + 2) + g * (D + 2);
            const float mr = part[D], top = fmaxf(m, mr);
            if (mr == -INFINITY) continue;
            const float f0 = expf(m - top), f1 = expf(mr - top);
            x = f0 * x + f1 * part[d];
            l = f0 * l + f1 * part[D + 1];
            m = top;
        }
        put(static_cast<T*>(a.o) + (q0 + g) * D + d, l > 0.f ? x / l : 0.f);
    }
}

template <int D, typename T>
cudaError_t step(const PagedArgs& a, cudaStream_t st) {
    const int blocks = (a.Hq / a.Hk + HEADS - 1) / HEADS, smem = (2 * TILE * (D + 4) + HEADS * (D + 4) + HEADS * TILE) * 4;
    if (cudaError_t e = cudaFuncSetAttribute(paged_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
    trace_begin("paged_step", st);
    cudaError_t e = launch_after(paged_kernel<D, T>, dim3(RUNS), THREADS, smem, st, false, a, blocks);
    trace_end(st);
    if (e != cudaSuccess) return e;
    trace_begin("paged_join", st);
    e = launch_after(paged_join_kernel<D, T>, dim3(RUNS - 1), THREADS, 0, st, true, a, blocks);
    trace_end(st);
    return e;
}
template <typename T>
cudaError_t step_of(const PagedArgs& a, cudaStream_t st) {
    return a.D == 32 ? step<32, T>(a, st) : a.D == 64 ? step<64, T>(a, st) : step<128, T>(a, st);
}

}  // namespace

size_t paged_parts_bytes(int, int, int, int D) { return (size_t)2 * RUNS * HEADS * (D + 2) * sizeof(float); }

cudaError_t launch_paged_step(const PagedArgs& a, cudaStream_t st) {
    return a.bf16 ? step_of<__nv_bfloat16>(a, st) : step_of<float>(a, st);
}

}  // namespace gdr
