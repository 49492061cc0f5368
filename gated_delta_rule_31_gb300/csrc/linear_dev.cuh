// linear_dev.cuh - device helpers of the tensor-core kernels of linear attention: decays, the issue of
// products by a converged warp, TMEM stores, pairwise arithmetic and the bounded wait of a warp.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "chunk_dev.cuh"
#include "common.cuh"

namespace gdr {
namespace linear {

constexpr int C = 128;                                  // tokens of a chunk
constexpr uint32_t TILE = 32768, PANEL = TILE / 2;      // bf16 [128 x 128] and its 64-channel halves

// l^n of the head with log-decay g; l^0 = 1 also where l = 0.
__device__ __forceinline__ float power(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }

// Products are issued by the elected lane of a converged warp, which keeps their operands in uniform
// registers: the issue is what paces them. A descriptor is a fixed high word and a low word that
// advances by a constant per 16-wide step. (Issued by a lone thread with descriptors built for
// each step, a product took 140 to 240 cycles, not 70.)
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1024, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t lo_kmajor(uint32_t tile) { return (tile >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t lo_mnmajor(uint32_t tile) { return (tile >> 4) | ((PANEL >> 4) << 16); }
__device__ constexpr uint32_t step_mnmajor(int k) { return k * (2048 >> 4); }

__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.u32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
        "setp.ne.u32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\tmov.b64 y, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(blo), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Products and sums of two values at once: fp32 pairs, and bf16 pairs with one rounding.
__device__ __forceinline__ void scale2(float* x, float f) {
    uint64_t v, w;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x[0]), "f"(x[1]));
    asm("mov.b64 %0, {%1, %1};" : "=l"(w) : "f"(f));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x[0]), "=f"(x[1]) : "l"(v));
}
template <bool FADE>  // s <- f s + d, or s + f d
__device__ __forceinline__ void axpy2(float* s, float f, const float* d) {
    uint64_t v, w, u;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(s[0]), "f"(s[1]));
    asm("mov.b64 %0, {%1, %1};" : "=l"(w) : "f"(f));
    asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(d[0]), "f"(d[1]));
    if (FADE) asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(w), "l"(u));
    else asm("fma.rn.f32x2 %0, %2, %1, %0;" : "+l"(v) : "l"(w), "l"(u));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(s[0]), "=f"(s[1]) : "l"(v));
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_neg(uint32_t a) {
    uint32_t d;
    asm("neg.bf16x2 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Programmatic dependent launch: a kernel lets the next one on the stream begin at once, and one launched to
// do so (launch_after) waits for the kernel before it ahead of its first access to memory that another kernel
// of the same call writes, or reads and it writes. A call's first kernel starts when all work before the call is
// complete, so its kernels may read the call's inputs, and write outputs that are theirs alone, before they
// wait; the decode steps, each a call's only kernel, wait first of all. What follows a call can begin
// early as well, so whatever kernel is launched that way as a call's first has to wait first of all.
__device__ __forceinline__ void next_kernel_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Bounded wait of a whole warp for phase `parity`, in few instructions, since the warps' roles share the
// instruction caches: the warp is parked in the barrier unit for up to a millisecond at a time. Gives
// up after about a second, leaving the site in *failed, or as soon as another warp has.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* failed, int site) {
    auto parked = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
            : "memory");
        return __all_sync(0xffffffffu, ok) != 0;
    };
    bool ok = parked();
    if (!ok) {
        const long long t0 = clock64();
        while (!(ok = parked())) {
            if (clock64() - t0 > kWaitCycles) *failed = site;
            if (__any_sync(0xffffffffu, *failed)) break;
        }
    }
    return ok;
}

}  // namespace linear
}  // namespace gdr
