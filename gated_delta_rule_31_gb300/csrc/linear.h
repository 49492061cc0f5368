// linear.h - launch interface of the linear attention with a constant decay per head
// (gdr_linear_*), shared by its C ABI (api_linear.cu) and its kernels.
//
// Per (b, hv) the state S [Dv x Dk] evolves as S_t = l S_{t-1} + v_t k_t^T with l = exp(g[hv]),
// and its adjoint D_t = l D_{t+1} + scale do_t q_t^T. The forward and each gradient are one
// "mix" pass over the tokens,
//
//     out_t = sum_{j <= t} l^(t-j) (a_t . b_j) c_j + (decayed) a_t X,
//
// in token order for o (a, b, c = q, k, v; X = S) and dq (do, v, k; S), in reverse order for
// dk (v, do, q; D) and dv (k, q, do; D). The tokens are cut into segments that run in parallel:
// a summary pass forms what each segment adds to the state, a combine step the state that
// enters each segment, and the mix pass starts from it.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr {

struct LinearShape {
    int B, T, Hk, Hv, Dk, Dv, bf16;
    int nseg, seg_tokens;  // tokens of batch entry b in segment s: [s * seg_tokens, ...) below its length
    const float* g;        // [Hv] log-decay
    const int* lengths;    // [B] valid tokens, or null (T)
};

// What the segments add to the state (reverse == 0: sum of w v k^T; reverse == 1: of w do q^T).
struct LinearSummaryArgs {
    LinearShape s;
    const void* rows;  // v or do [B, T, Hv, Dv]
    const void* cols;  // k or q  [B, T, Hk, Dk]
    float factor;      // 1, or scale in reverse
    int reverse;
    float* z;  // [B, Hv, nseg, Dv, Dk]
    int* clear;  // fp32: the call's status word, which its first kernel clears, or null
};

// z -> the state entering each segment (in place), and the state after all of them (with last null
// the z of the segment processed last is not read).
struct LinearCombineArgs {
    LinearShape s;
    const float* init;  // [B, Hv, Dv, Dk] or null (zero)
    int reverse;
    float* z;
    float* last;  // [B, Hv, Dv, Dk] or null
};

enum LinearPass { LINEAR_O = 0, LINEAR_DQ = 1, LINEAR_DK = 2, LINEAR_DV = 3 };

struct LinearMixArgs {
    LinearShape s;
    int pass;  // LinearPass
    const void *q, *k, *v, *do_;
    float scale;
    float* starts;  // state entering each segment (scratch: passes that sum value heads update it)
    void* out;
    const float* init;  // fp32, one segment: the state before all tokens, or null (zero); and
    float* last;        // o and dv: the state after them, or null
    void* images;   // bf16 o and dv: the state that each 128-token chunk starts from (dv: the adjoint of
                    // the one it ends in) is kept there as a swizzled bf16 tile, 32 KB for each
                    // (b, hv, chunk), for launch_linear_tc_grad; or null
    bool overlap;   // fp32: the kernel before it on the stream is the combine step of its call (launch_after)
    int* clear;     // fp32: as LinearSummaryArgs
};

// A launch that, with `overlap`, may begin while the kernel before it on the stream still runs; that kernel
// lets it (griddepcontrol.launch_dependents), and the new one waits before it reads its results
// (linear_dev.cuh). Of a call's kernels the first is launched without, but for the decode step.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, bool overlap, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = overlap ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr int kLinearBlock = 64, kLinearBlockTc = 128;  // tokens that segments are made of: fp32, bf16
int linear_segments(int B, int T, int Hv, int Dv);
cudaError_t launch_linear_summary(const LinearSummaryArgs& a, cudaStream_t st);
cudaError_t launch_linear_combine(const LinearCombineArgs& a, bool overlap, cudaStream_t st);
cudaError_t launch_linear_mix(const LinearMixArgs& a, cudaStream_t st);

// bf16 on the tensor cores (linear_tc.cu): the summary of the segments (all of them, or all but the
// last in processing order), and the mix passes of o and dv. start: the state entering each
// segment (start_segs = nseg), or before all of them (1; may be null: zero). last: the state after
// the last segment, or null. status: status word, cleared by the kernel if `clear`. overlap: the kernel
// before it on the stream is of the same call (launch_after).
int linear_tc_segments(int B, int T, int Hv);
cudaError_t launch_linear_tc_summary(const LinearSummaryArgs& a, bool all, int* status, bool clear, cudaStream_t st);
cudaError_t launch_linear_tc_mix(const LinearMixArgs& a, const float* start, int start_segs, float* last, int* status,
                                 bool clear, bool overlap, cudaStream_t st);

// dq and dk of bf16 problems from the kept states (linear_grad.cu).
struct LinearGradArgs {
    LinearShape s;
    const void *q, *k, *v, *do_;
    float scale;
    const void *states, *adjoints;  // images of the o and dv passes
    void *dq, *dk;
    int* status;
};
cudaError_t launch_linear_tc_grad(const LinearGradArgs& a, cudaStream_t st);

struct LinearStepArgs {
    int B, Hk, Hv, Dk, Dv, bf16;
    float scale;
    const void *q, *k, *v;
    const float* g;
    float* state;
    void* o;
};
cudaError_t launch_linear_step(const LinearStepArgs& a, cudaStream_t st);

}  // namespace gdr
