// group_norm.h - launch interface of the per-token group norm (gdr_group_norm_*), shared by its C
// ABI (api_linear.cu) and its kernels.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

#include "gdr.h"

namespace gdr {

struct GroupNormArgs {
    long long rows;
    int groups, D, bf16, act, center;
    float eps;
    const void *x, *gate;        // [rows, groups D]; gate may be null
    const float *weight, *bias;  // [groups D] or null
    void* y;                     // forward
    const void* dy;              // backward
    void *dx, *dgate;
    float *dweight, *dbias;  // or null
};

cudaError_t launch_group_norm_fwd(const GroupNormArgs& a, cudaStream_t st);
cudaError_t launch_group_norm_bwd(const GroupNormArgs& a, float* part, cudaStream_t st);
// Bytes of the partial sums of dweight and dbias.
size_t group_norm_bwd_partials(const GroupNormArgs& a);

}  // namespace gdr
