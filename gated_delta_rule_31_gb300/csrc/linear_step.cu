// linear_step.cu - one token of linear attention with a constant decay per head
// (gdr_linear_decode_step): S <- exp(g) S + v k^T in place, o = scale S q.
//
// The state is read and written once, 8 bytes an element against 4 operations, so HBM bounds a
// batch and latency a single sequence.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "linear.h"

namespace gdr {

namespace {

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// grid (Hv, B, Dv / (4 WROWS)), 4 warps of WROWS state rows; a row is DK / 32 floats a lane.
template <int DK, int WROWS, typename T>
__global__ void __launch_bounds__(128) linear_step_kernel(LinearStepArgs a) {
    constexpr int EL = DK / 32;
    using Vec = typename std::conditional<EL == 4, float4, typename std::conditional<EL == 2, float2, float>::type>::type;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hv = blockIdx.x, b = blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const size_t bh = (size_t)b * a.Hv + hv;
    const int r0 = (blockIdx.z * 4 + warp) * WROWS;
    const T* q = static_cast<const T*>(a.q) + ((size_t)b * a.Hk + hk) * DK + lane * EL;
    const T* k = static_cast<const T*>(a.k) + ((size_t)b * a.Hk + hk) * DK + lane * EL;
    const T* v = static_cast<const T*>(a.v) + bh * a.Dv;
    T* o = static_cast<T*>(a.o) + bh * a.Dv;
    Vec* S = reinterpret_cast<Vec*>(a.state + (bh * a.Dv + r0) * DK) + lane;
    __align__(16) float x[WROWS][EL];
#pragma unroll
    for (int r = 0; r < WROWS; r++) *reinterpret_cast<Vec*>(x[r]) = S[r * 32];
    float kf[EL], qf[EL];
#pragma unroll
    for (int e = 0; e < EL; e++) {
        kf[e] = as_float(k[e]);
        qf[e] = as_float(q[e]);
    }
    const float l = expf(a.g[hv]);
#pragma unroll
    for (int r = 0; r < WROWS; r++) {
        const float vr = as_float(v[r0 + r]);
        float acc = 0.f;
#pragma unroll
        for (int e = 0; e < EL; e++) {
            x[r][e] = l * x[r][e] + vr * kf[e];
            acc += x[r][e] * qf[e];
        }
        S[r * 32] = *reinterpret_cast<Vec*>(x[r]);
        acc = warp_sum(acc);
        if (lane == 0) put(o + r0 + r, a.scale * acc);
    }
}

template <int DK, typename T>
cudaError_t step(const LinearStepArgs& a, cudaStream_t st) {
    trace_begin("linear_step", st);
    linear_step_kernel<DK, 8, T><<<dim3(a.Hv, a.B, a.Dv / 32), 128, 0, st>>>(a);
    trace_end(st);
    return cudaGetLastError();
}

template <typename T>
cudaError_t step_of(const LinearStepArgs& a, cudaStream_t st) {
    return a.Dk == 32 ? step<32, T>(a, st) : a.Dk == 64 ? step<64, T>(a, st) : step<128, T>(a, st);
}

}  // namespace

cudaError_t launch_linear_step(const LinearStepArgs& a, cudaStream_t st) {
    return a.bf16 ? step_of<__nv_bfloat16>(a, st) : step_of<float>(a, st);
}

}  // namespace gdr
