// linear_step.cu - one token of linear attention with a constant decay per head
// (gdr_linear_decode_step): S <- exp(g) S + v k^T in place, o = scale S q.
//
// The state is read and written once, 8 bytes an element against 4 operations, so HBM bounds a
// batch and latency a single sequence. Neighbouring CTAs take neighbouring parts of the state: B = 128 of 32
// heads, 128 x 128, 540 MB, in 80.0 us, the rate of a plain copy, against 89.7 with the heads
// fastest. A warp reads 512 contiguous bytes at a time, one to four state rows, LINES of them in flight
// (eight: 88.7 us; for heads of 64 x 64 a row at a time, 256 bytes, takes 20.1 us at B = 128 in L2 instead
// of 16.0), and the rows' dot products with q are reduced together: each exchange halves
// those that a lane still holds. A step is launched so that it may start while the kernel before it on the
// stream ends (programmatic dependent launch), and reads and writes only after that kernel is complete.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "linear.h"
#include "linear_dev.cuh"

namespace gdr {

namespace {

__device__ __forceinline__ void get4(const float* p, float* x) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void get4(const __nv_bfloat16* p, float* x) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = bf16lo(v.x); x[1] = bf16hi(v.x); x[2] = bf16lo(v.y); x[3] = bf16hi(v.y);
}
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// 4 warps, each LINES (4 or 2) lines of 128 floats: 128 / DK state rows of one head in a line, LANES lanes a row.
template <int DK, int LINES, typename T>
__global__ void __launch_bounds__(128) linear_step_kernel(LinearStepArgs a) {
    constexpr int LANES = DK / 4, PER = 32 / LANES;
    linear::next_kernel_may_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned row0 = (blockIdx.x * 4 + warp) * (LINES * PER), rows = (unsigned)a.B * a.Hv * a.Dv;
    if (row0 >= rows) return;  // a head has whole warps of rows, not whole CTAs
    float4* S = reinterpret_cast<float4*>(a.state + (size_t)row0 * DK) + lane;
    const unsigned bh = row0 / a.Dv, b = bh / a.Hv, hv = bh - b * a.Hv, hk = hv / ((unsigned)a.Hv / a.Hk);
    const size_t at = ((size_t)b * a.Hk + hk) * DK + lane % LANES * 4, row = row0 + lane / LANES;  // and every PER-th row
    linear::wait_kernel_before();
    float4 x[LINES];
#pragma unroll
    for (int r = 0; r < LINES; r++) x[r] = __ldcs(S + r * 32);
    float kf[4], qf[4];
    get4(static_cast<const T*>(a.k) + at, kf);
    get4(static_cast<const T*>(a.q) + at, qf);
    const float l = expf(a.g[hv]);
    float acc[LINES];
#pragma unroll
    for (int r = 0; r < LINES; r++) {
        const float vr = as_float(static_cast<const T*>(a.v)[row + r * PER]);
        x[r].x = l * x[r].x + vr * kf[0];
        x[r].y = l * x[r].y + vr * kf[1];
        x[r].z = l * x[r].z + vr * kf[2];
        x[r].w = l * x[r].w + vr * kf[3];
        acc[r] = x[r].x * qf[0] + x[r].y * qf[1] + x[r].z * qf[2] + x[r].w * qf[3];
        __stcs(S + r * 32, x[r]);
    }
    int off = LANES / 2;
#pragma unroll
    for (int n = LINES / 2; n > 0; n /= 2, off /= 2) {  // lanes with bit `off` keep the upper half of the rows
        const bool up = lane & off;
#pragma unroll
        for (int r = 0; r < n; r++) {
            const float send = up ? acc[r] : acc[r + n], keep = up ? acc[r + n] : acc[r];
            acc[r] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    constexpr int LEFT = LANES / LINES;  // lanes that share a row now
#pragma unroll
    for (int m = LEFT / 2; m > 0; m /= 2) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], m);
    if (lane % LEFT == 0) put(static_cast<T*>(a.o) + row + lane % LANES / LEFT * PER, a.scale * acc[0]);
}

template <int DK, int LINES, typename T>
cudaError_t step(const LinearStepArgs& a, cudaStream_t st) {
    constexpr int ROWS = 4 * LINES * 128 / DK;  // of a CTA
    const long long rows = (long long)a.B * a.Hv * a.Dv;
    trace_begin("linear_step", st);
    const cudaError_t e =
        launch_after(linear_step_kernel<DK, LINES, T>, dim3((unsigned)((rows + ROWS - 1) / ROWS)), 128, 0, st, true, a);
    trace_end(st);
    return e;
}

// Two lines a warp while that gives no more than two rounds of 16 CTAs per SM (32 heads of 128 x 128, states
// in L2: B = 1 2.7 us with either, B = 4 3.2 with two, 4.6 with four; from HBM: B = 8 7.2 and 7.6), else
// four (in L2: B = 16 9.9 with two, 8.6 with four; B = 128 82.6 and 79.8).
template <int DK, typename T>
cudaError_t step_lines(const LinearStepArgs& a, cudaStream_t st) {
    return (long long)a.B * a.Hv * a.Dv * DK / 128 < 2 * 152 * 128 ? step<DK, 2, T>(a, st) : step<DK, 4, T>(a, st);
}

template <typename T>
cudaError_t step_of(const LinearStepArgs& a, cudaStream_t st) {
    return a.Dk == 32 ? step_lines<32, T>(a, st) : a.Dk == 64 ? step_lines<64, T>(a, st) : step_lines<128, T>(a, st);
}

}  // namespace

cudaError_t launch_linear_step(const LinearStepArgs& a, cudaStream_t st) {
    return a.bf16 ? step_of<__nv_bfloat16>(a, st) : step_of<float>(a, st);
}

}  // namespace gdr
