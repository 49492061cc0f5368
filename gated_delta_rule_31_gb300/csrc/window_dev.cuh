// window_dev.cuh - device helpers of the tensor-core kernels of window attention: which pairs of a tile are seen, the
// exponentials, zeroing of rows past the end, and arithmetic on fp32 pairs.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "attention.h"
#include "linear_dev.cuh"

namespace gdr {
namespace window {

using namespace linear;  // C = 128 tokens of a tile, TILE, PANEL, products and waits

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Four products in a row with one election: both operands in shared memory, 16 channels on each time (d accumulates but for
// the first with begin); and the left one in TMEM, 8 columns on, against 16 rows of b on each time.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, bool begin) {
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b64 x, y;\n\t.reg .b32 u, v;\n\t"
        "setp.eq.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t"
        "add.u32 u, %1, 2;\n\tadd.u32 v, %2, 2;\n\tmov.b64 x, {u, %5};\n\tmov.b64 y, {v, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
        "add.u32 u, %1, 4;\n\tadd.u32 v, %2, 4;\n\tmov.b64 x, {u, %5};\n\tmov.b64 y, {v, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
        "add.u32 u, %1, 6;\n\tadd.u32 v, %2, 6;\n\tmov.b64 x, {u, %5};\n\tmov.b64 y, {v, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"((uint32_t)begin), "r"(DESC_HI)
        : "memory");
}
template <int STEP>
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint32_t blo, uint32_t idesc, bool begin) {
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b64 y;\n\t.reg .b32 u, v;\n\t"
        "setp.eq.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t"
        "add.u32 u, %1, 8;\n\tadd.u32 v, %2, %6;\n\tmov.b64 y, {v, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t"
        "add.u32 u, %1, 16;\n\tadd.u32 v, %2, %7;\n\tmov.b64 y, {v, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t"
        "add.u32 u, %1, 24;\n\tadd.u32 v, %2, %8;\n\tmov.b64 y, {v, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t}" ::"r"(d),
        "r"(a), "r"(blo), "r"(idesc), "r"((uint32_t)begin), "r"(DESC_HI), "n"(STEP), "n"(2 * STEP), "n"(3 * STEP)
        : "memory");
}
// d = a b^T over `channels` channels, of the rows that the instruction's shape says, tiles in shared memory (a: or in TMEM).
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, int channels) {
    if (channels < 64) {
        mma_ss(d, alo, blo, idesc, 0);
        mma_ss(d, alo + 2, blo + 2, idesc, 1);
    } else {
#pragma unroll 1
        for (int c = 0; c < channels; c += 64, alo += PANEL >> 4, blo += PANEL >> 4) mma_ss4(d, alo, blo, idesc, c == 0);
    }
}
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t idesc, int channels) {
    if (channels < 64) {
        mma_ts(d, a, blo, idesc, 0);
        mma_ts(d, a + 8, blo + 2, idesc, 1);
    } else {
#pragma unroll 1
        for (int c = 0; c < channels; c += 64, a += 32, blo += PANEL >> 4) mma_ts4<2>(d, a, blo, idesc, c == 0);
    }
}
// d (+)= p b over 64 rows of b (blo: MN-major), p in TMEM; the first `rows` are enough, the others weigh nothing
__device__ __forceinline__ void product_sum64(uint32_t d, uint32_t p, uint32_t blo, uint32_t idesc, int rows, bool begin) {
    if (rows > 48) {
        mma_ts4<step_mnmajor(1)>(d, p, blo, idesc, begin);
    } else {
#pragma unroll 1
        for (int r = 0; r < rows; r += 16, p += 8, blo += step_mnmajor(1)) mma_ts(d, p, blo, idesc, r > 0 || !begin);
    }
}

// Whether every query of t0 .. t0 + 127 sees every key of j0 .. j0 + 127.
__device__ __forceinline__ bool all_seen(const WindowShape& s, int t0, int j0, int n) {
    return j0 + C - 1 <= t0 && t0 + C <= n && (t0 + C - 1 - j0 < s.window || j0 + C <= s.sinks);
}
__device__ __forceinline__ uint32_t below(int c) { return c <= 0 ? 0u : c >= 32 ? 0xffffffffu : (1u << c) - 1; }
// Which of keys j .. j + 31 query t sees, as bits.
__device__ __forceinline__ uint32_t keys_seen(const WindowShape& s, int t, int j, int n) {
    const uint32_t upto = t < n ? below(t + 1 - j) : 0u;
    return upto & (~below(t - s.window + 1 - j) | below(s.sinks - j));
}
// Which of queries t .. t + 31 see key j.
__device__ __forceinline__ uint32_t seen_by(const WindowShape& s, int t, int j, int n) {
    const uint32_t from = j < n ? below(n - t) & ~below(j - t) : 0u;
    return j < s.sinks ? from : from & below(j + s.window - t);
}

// Rows m .. 127 of a 128-token tile in shared memory to zero, by a whole warp: operands of products must be finite there.
__device__ __forceinline__ void zero_rows(uint32_t tile, int m, int panels, int lane) {
    const int ch = lane & 15;
    if (ch < 8 * panels)
#pragma unroll 1
        for (int z = m + (lane >> 4); z < C; z += 2) st_shared_v4(tile + sw128_chunk(z, ch, C), 0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

}  // namespace window
}  // namespace gdr
