// window_host.h - host helpers of the tensor-core kernels of window attention.
#pragma once
#include "attention.h"
#include "tma_host.h"

namespace gdr {

// Tiles of one 64-channel panel and 128 tokens of one head of a [B, T, H, D] tensor.
inline bool rows_map(CUtensorMap* m, const void* p, const WindowShape& s, int H) {
    return make_map_4d_bf16(m, p, s.D, H, s.T, s.B, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t launch_window_fwd_tc(const WindowArgs& a, cudaStream_t st);
size_t window_parts_bytes_tc(const WindowShape& s);
cudaError_t launch_window_bwd_tc(const WindowArgs& a, cudaStream_t st);

}  // namespace gdr
