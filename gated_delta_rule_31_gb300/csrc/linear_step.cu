// linear_step.cu - one token of linear attention with a constant decay per head
// (gdr_linear_decode_step): S <- exp(g) S + v k^T in place, o = scale S q.
//
// The state is read and written once, 8 bytes an element against 4 operations, so HBM bounds a
// batch and latency a single sequence. Neighbouring CTAs take neighbouring rows of the state: B = 128 of 32
// heads, 128 x 128, 540 MB, in 80.0 us, the rate of a plain copy, against 89.7 with the heads
// fastest. A warp has ROWS state rows in flight (2: 83.6, 8: 88.7 us), and their dot products with q
// are reduced together: each exchange halves the rows a lane still holds. A step is launched so that it may start
// while the kernel before it on the stream ends (programmatic dependent launch), and reads and writes only
// after that kernel is complete.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "linear.h"
#include "linear_dev.cuh"

namespace gdr {

namespace {

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// grid (Dv / (4 ROWS), Hv, B), 4 warps of ROWS (4 or 2) state rows; a row is DK / 32 floats a lane.
template <int DK, int ROWS, typename T>
__global__ void __launch_bounds__(128) linear_step_kernel(LinearStepArgs a) {
    constexpr int EL = DK / 32;
    using Vec = typename std::conditional<EL == 4, float4, typename std::conditional<EL == 2, float2, float>::type>::type;
    linear::next_kernel_may_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / (a.Hv / a.Hk);
    const size_t bh = (size_t)b * a.Hv + hv;
    const int r0 = (blockIdx.x * 4 + warp) * ROWS;
    const T* q = static_cast<const T*>(a.q) + ((size_t)b * a.Hk + hk) * DK + lane * EL;
    const T* k = static_cast<const T*>(a.k) + ((size_t)b * a.Hk + hk) * DK + lane * EL;
    const T* v = static_cast<const T*>(a.v) + bh * a.Dv + r0;
    T* o = static_cast<T*>(a.o) + bh * a.Dv + r0;
    Vec* S = reinterpret_cast<Vec*>(a.state + (bh * a.Dv + r0) * DK) + lane;
    linear::wait_kernel_before();
    __align__(16) float x[ROWS][EL];
#pragma unroll
    for (int r = 0; r < ROWS; r++) *reinterpret_cast<Vec*>(x[r]) = __ldcs(S + r * 32);
    float kf[EL], qf[EL];
#pragma unroll
    for (int e = 0; e < EL; e++) {
        kf[e] = as_float(k[e]);
        qf[e] = as_float(q[e]);
    }
    const float l = expf(a.g[hv]);
    float acc[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; r++) {
        const float vr = as_float(v[r]);
        acc[r] = 0.f;
#pragma unroll
        for (int e = 0; e < EL; e++) {
            x[r][e] = l * x[r][e] + vr * kf[e];
            acc[r] += x[r][e] * qf[e];
        }
        __stcs(S + r * 32, *reinterpret_cast<Vec*>(x[r]));
    }
    int off = 16;
#pragma unroll
    for (int n = ROWS / 2; n > 0; n /= 2, off /= 2) {  // lanes with bit `off` keep the upper half of the rows
        const bool up = lane & off;
#pragma unroll
        for (int r = 0; r < n; r++) {
            const float send = up ? acc[r] : acc[r + n], keep = up ? acc[r + n] : acc[r];
            acc[r] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    constexpr int LEFT = 32 / ROWS;  // lanes that share a row now
#pragma unroll
    for (int m = LEFT / 2; m > 0; m /= 2) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], m);
    if (lane % LEFT == 0) put(o + lane / LEFT, a.scale * acc[0]);
}

template <int DK, int ROWS, typename T>
cudaError_t step(const LinearStepArgs& a, cudaStream_t st) {
    trace_begin("linear_step", st);
    const cudaError_t e =
        launch_after(linear_step_kernel<DK, ROWS, T>, dim3(a.Dv / (4 * ROWS), a.Hv, a.B), 128, 0, st, true, a);
    trace_end(st);
    return e;
}

// Few states (less than two CTAs per SM) are spread over twice the warps.
template <int DK, typename T>
cudaError_t step_rows(const LinearStepArgs& a, cudaStream_t st) {
    return (long long)a.B * a.Hv * a.Dv < 2 * 152 * 16 ? step<DK, 2, T>(a, st) : step<DK, 4, T>(a, st);
}

template <typename T>
cudaError_t step_of(const LinearStepArgs& a, cudaStream_t st) {
    return a.Dk == 32 ? step_rows<32, T>(a, st) : a.Dk == 64 ? step_rows<64, T>(a, st) : step_rows<128, T>(a, st);
}

}  // namespace

cudaError_t launch_linear_step(const LinearStepArgs& a, cudaStream_t st) {
    return a.bf16 ? step_of<__nv_bfloat16>(a, st) : step_of<float>(a, st);
}

}  // namespace gdr
