// linear_host.h - host helpers of the tensor-core kernels of linear attention.
#pragma once
#include "linear.h"
#include "tma_host.h"

namespace gdr {

// Tiles of one 64-channel panel and 128 tokens of a [B, T, H, D] tensor.
inline bool tile_map(CUtensorMap* m, const void* p, const LinearShape& s, int H, int D) {
    return make_map_4d_bf16(m, p, D, H, s.T, s.B, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
}

inline int panels(int d) { return d > 64 ? 2 : 1; }

}  // namespace gdr
