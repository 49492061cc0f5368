// group_norm.cu - group norm over the channels of each token, with an activation of the result or
// of a gate beside it (gdr_group_norm_fwd, gdr_group_norm_bwd).
//
//   h = (x - mean) r, r = 1 / sqrt(var + eps) over the D channels of a token's group (mean = 0 if
//   not centered, var = the mean of h's squares before scaling), n = w h + b,
//   y = act(n), or n act(z) with a gate z.
//   dn = dy act'(n) or dy act(z);  dz = dy n act'(z);  dw = sum dn h, db = sum dn over tokens;
//   dh = w dn;  dx = r (dh - mean(dh) - h mean(dh h)), without mean(dh) if not centered.
//
// HBM bounds both directions, so a group's values are read once and stay in registers: LPG lanes
// share a group, each with NV vectors of VEC values, and the statistics are sums over those lanes
// (two passes over the registers: the mean, then the squares about it). The backward forms the
// statistics again from x, which it needs anyway, so the forward stores none. A lane keeps its
// channels for all the tokens it works on: w and b are read once, and dw and db are sums in
// registers, written as one partial row for each (block row, lane row) and added up in a fixed
// order by a second kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "common.cuh"
#include "group_norm.h"
#include "kernels.h"

namespace gdr {

namespace {

constexpr int THREADS = 256;

// VEC values as loaded: 16 bytes, or a single value.
template <int VEC, typename T>
struct RawOf { using type = T; };
template <>
struct RawOf<8, __nv_bfloat16> { using type = uint4; };
template <>
struct RawOf<4, float> { using type = float4; };

template <int VEC, typename T>
__device__ __forceinline__ typename RawOf<VEC, T>::type load_raw(const T* p) {
    return *reinterpret_cast<const typename RawOf<VEC, T>::type*>(p);
}
__device__ __forceinline__ void values(const uint4& u, float* x) {
    x[0] = bf16lo(u.x); x[1] = bf16hi(u.x); x[2] = bf16lo(u.y); x[3] = bf16hi(u.y);
    x[4] = bf16lo(u.z); x[5] = bf16hi(u.z); x[6] = bf16lo(u.w); x[7] = bf16hi(u.w);
}
__device__ __forceinline__ void values(const float4& u, float* x) {
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
}
__device__ __forceinline__ void values(const __nv_bfloat16& u, float* x) { x[0] = __bfloat162float(u); }
__device__ __forceinline__ void values(const float& u, float* x) { x[0] = u; }
template <int VEC, typename T>
__device__ __forceinline__ void store_vec(T* p, const float* x) {
    if constexpr (VEC == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                                  pack_bf16(x[6], x[7]));
    else if constexpr (VEC == 4)
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else if constexpr (sizeof(T) == 2)
        *p = __float2bfloat16_rn(x[0]);
    else
        *p = x[0];
}
template <int VEC>
__device__ __forceinline__ void load_param(const float* p, float* x) {
    if constexpr (VEC == 1) {
        x[0] = *p;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) values(*reinterpret_cast<const float4*>(p + i), x + i);
    }
}
template <int VEC>
__device__ __forceinline__ void store_param(float* p, const float* x) {
    if constexpr (VEC == 8) {
        store_vec<4>(p, x);
        store_vec<4>(p + 4, x + 4);
    } else {
        store_vec<VEC>(p, x);
    }
}

// Sums of two values over the LPG lanes of a group. Groups wider than a warp go through shared memory.
template <int LPG>
__device__ __forceinline__ void group_sum2(float& a, float& b, float2* red) {
#pragma unroll
    for (int o = (LPG < 32 ? LPG : 32) / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (LPG > 32) {
        constexpr int W = LPG / 32;
        const int warp = threadIdx.x >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < W; w++) {
            const float2 v = red[warp / W * W + w];
            a += v.x;
            b += v.y;
        }
    }
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float activate(float x, int act) {
    return act == GDR_ACT_NONE ? x : act == GDR_ACT_SILU ? x * sigmoid(x) : sigmoid(x);
}
// act(x) and act'(x)
__device__ __forceinline__ float2 activate2(float x, int act) {
    if (act == GDR_ACT_NONE) return make_float2(x, 1.f);
    const float s = sigmoid(x);
    if (act == GDR_ACT_SIGMOID) return make_float2(s, s * (1.f - s));
    return make_float2(x * s, s * (1.f + x * (1.f - s)));
}

// Which token rows and group a lane works on. A block covers `per` groups (blockIdx.x) and `rl` token
// rows at a time, LPG lanes each; lanes past the last row or group only join the sums.
struct Place {
    int group, lane, slot_row;
    long long row0, row_step;
    bool live;
};
template <int LPG>
__device__ __forceinline__ Place place(int groups, int per) {
    Place p;
    const int slot = threadIdx.x / LPG, rl = blockDim.x / (LPG * per);
    p.lane = threadIdx.x % LPG;
    p.group = blockIdx.x * per + slot % per;
    p.slot_row = slot / per;
    p.live = p.group < groups && p.slot_row < rl;
    p.row0 = (long long)blockIdx.y * rl + p.slot_row;
    p.row_step = (long long)gridDim.y * rl;
    return p;
}

// A lane asks for its next row before it works on the current one: a row a lane in flight is too little
// to keep HBM busy (T = 32768 rows of 4096 bf16, gated: forward 147 us without).
template <int LPG, int VEC, int NV, typename T>
__global__ void __launch_bounds__(THREADS, NV == 1 ? 4 : 1) group_norm_fwd_kernel(GroupNormArgs a, int per) {
    using Raw = typename RawOf<VEC, T>::type;
    __shared__ float2 red[THREADS / 32];
    const Place at = place<LPG>(a.groups, per);
    const size_t C = (size_t)a.groups * a.D;
    const float inv = 1.f / (float)a.D;
    const T* x = static_cast<const T*>(a.x);
    const T* z = static_cast<const T*>(a.gate);
    T* y = static_cast<T*>(a.y);
    int e[NV];
    bool in[NV];
    float w[NV][VEC], b[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int d = (i * LPG + at.lane) * VEC;
        in[i] = at.live && d < a.D;
        e[i] = at.group * a.D + d;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            w[i][j] = 1.f;
            b[i][j] = 0.f;
        }
        if (in[i] && a.weight) load_param<VEC>(a.weight + e[i], w[i]);
        if (in[i] && a.bias) load_param<VEC>(a.bias + e[i], b[i]);
    }
    Raw nx[NV] = {}, nz[NV] = {};
    auto ask = [&](long long row) {
        if (row >= a.rows) return;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (in[i]) nx[i] = load_raw<VEC>(x + row * C + e[i]);
            if (in[i] && z) nz[i] = load_raw<VEC>(z + row * C + e[i]);
        }
    };
    const long long steps = (a.rows + at.row_step - 1) / at.row_step;
    ask(at.row0);
    for (long long s = 0; s < steps; s++) {
        const long long row = at.row0 + s * at.row_step;
        float v[NV][VEC], u[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            values(nx[i], v[i]);
            values(nz[i], u[i]);
        }
        ask(row + at.row_step);
        float sum = 0.f, none = 0.f;
        if (a.center) {
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int j = 0; j < VEC; j++) sum += v[i][j];
            group_sum2<LPG>(sum, none, red);
        }
        const float mean = sum * inv;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in[i])
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    v[i][j] -= mean;
                    sq += v[i][j] * v[i][j];
                }
        group_sum2<LPG>(sq, none, red);
        const float r = 1.f / sqrtf(sq * inv + a.eps);
        if (row < a.rows)
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (in[i]) {
#pragma unroll
                    for (int j = 0; j < VEC; j++) {
                        const float n = w[i][j] * (v[i][j] * r) + b[i][j];
                        v[i][j] = z ? n * activate(u[i][j], a.act) : activate(n, a.act);
                    }
                    store_vec<VEC>(y + row * C + e[i], v[i]);
                }
    }
}

template <int LPG, int VEC, int NV, typename T>
__global__ void __launch_bounds__(THREADS, NV == 1 ? 3 : 1) group_norm_bwd_kernel(GroupNormArgs a, int per, float* part) {
    using Raw = typename RawOf<VEC, T>::type;
    __shared__ float2 red[THREADS / 32];
    const Place at = place<LPG>(a.groups, per);
    const size_t C = (size_t)a.groups * a.D;
    const float inv = 1.f / (float)a.D;
    const T* x = static_cast<const T*>(a.x);
    const T* z = static_cast<const T*>(a.gate);
    const T* dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.dx);
    T* dz = static_cast<T*>(a.dgate);
    int e[NV];
    bool in[NV];
    float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int d = (i * LPG + at.lane) * VEC;
        in[i] = at.live && d < a.D;
        e[i] = at.group * a.D + d;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            w[i][j] = 1.f;
            b[i][j] = dw[i][j] = db[i][j] = 0.f;
        }
        if (in[i] && a.weight) load_param<VEC>(a.weight + e[i], w[i]);
        if (in[i] && a.bias) load_param<VEC>(a.bias + e[i], b[i]);
    }
    Raw nx[NV] = {}, nz[NV] = {}, ng[NV] = {};
    auto ask = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const bool use = in[i] && row < a.rows;
            if (use) nx[i] = load_raw<VEC>(x + row * C + e[i]);
            if (use && z) nz[i] = load_raw<VEC>(z + row * C + e[i]);
            ng[i] = use ? load_raw<VEC>(dy + row * C + e[i]) : Raw{};  // no row adds nothing to dw and db
        }
    };
    const long long steps = (a.rows + at.row_step - 1) / at.row_step;
    ask(at.row0);
    for (long long s = 0; s < steps; s++) {
        const long long row = at.row0 + s * at.row_step;
        float h[NV][VEC], u[NV][VEC], g[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            values(nx[i], h[i]);
            values(nz[i], u[i]);
            values(ng[i], g[i]);
        }
        ask(row + at.row_step);
        float sum = 0.f, none = 0.f;
        if (a.center) {
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int j = 0; j < VEC; j++) sum += h[i][j];
            group_sum2<LPG>(sum, none, red);
        }
        const float mean = sum * inv;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in[i])
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    h[i][j] -= mean;
                    sq += h[i][j] * h[i][j];
                }
        group_sum2<LPG>(sq, none, red);
        const float r = 1.f / sqrtf(sq * inv + a.eps);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in[i]) {
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    h[i][j] *= r;
                    const float n = w[i][j] * h[i][j] + b[i][j];
                    const float2 f = activate2(z ? u[i][j] : n, a.act);
                    u[i][j] = g[i][j] * n * f.y;  // dz
                    const float dn = g[i][j] * (z ? f.x : f.y);
                    dw[i][j] += dn * h[i][j];
                    db[i][j] += dn;
                    g[i][j] = dn * w[i][j];
                    s1 += g[i][j];
                    s2 += g[i][j] * h[i][j];
                }
                if (z && row < a.rows) store_vec<VEC>(dz + row * C + e[i], u[i]);
            }
        group_sum2<LPG>(s1, s2, red);
        const float m1 = a.center ? s1 * inv : 0.f, m2 = s2 * inv;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in[i] && row < a.rows) {
#pragma unroll
                for (int j = 0; j < VEC; j++) g[i][j] = r * (g[i][j] - m1 - h[i][j] * m2);
                store_vec<VEC>(dx + row * C + e[i], g[i]);
            }
    }
    if (!part) return;
    const int rl = blockDim.x / (LPG * per);
    float* pw = part + ((size_t)blockIdx.y * rl + at.slot_row) * 2 * C;
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (in[i]) {
            store_param<VEC>(pw + e[i], dw[i]);
            store_param<VEC>(pw + C + e[i], db[i]);
        }
}

// grid ceil(2 C / 32): 32 columns a block, 32 threads a column over the partial rows, joined in order.
__global__ void __launch_bounds__(1024) group_norm_params_kernel(const float* part, int n, int C, float* dw, float* db) {
    __shared__ float sh[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float s = 0.f;
    if (c < 2 * C)
#pragma unroll 8
        for (int i = y; i < n; i += 32) s += part[(size_t)i * 2 * C + c];
    sh[y][x] = s;
    __syncthreads();
    s = warp_sum(sh[x][y]);  // column y of this block
    const int d = blockIdx.x * 32 + y;
    if (x == 0 && d < 2 * C) {
        float* out = d < C ? dw : db;
        if (out) out[d < C ? d : d - C] = s;
    }
}

struct Grid {
    int per, rl, threads, x, y;
};
// A block takes as many whole groups as THREADS lanes hold, then several token rows at a time; the
// rows are spread evenly over about as many blocks as run at once.
Grid grid_of(const GroupNormArgs& a, int lpg, int blocks_per_sm) {
    Grid g;
    const int slots = THREADS / lpg;
    g.per = a.groups < slots ? a.groups : slots;
    g.rl = slots / g.per;
    g.threads = (g.per * g.rl * lpg + 31) / 32 * 32;
    g.x = (a.groups + g.per - 1) / g.per;
    const long long rows = (a.rows + g.rl - 1) / g.rl;
    long long y = (152LL * blocks_per_sm * THREADS / g.threads + g.x - 1) / g.x;
    if (y > rows) y = rows;
    if (y > 65535) y = 65535;
    const long long each = (rows + y - 1) / y;  // row steps of a block
    g.y = (int)((rows + each - 1) / each);
    return g;
}

constexpr int kFwdBlocks = 4, kBwdBlocks = 3;  // blocks of THREADS per SM that run at once

// Lanes and vectors for a group of D values: 16-byte vectors where every row of every tensor starts
// on 16 bytes (D a multiple of the vector and aligned pointers), else single values.
template <typename F>
cudaError_t with_shape(const GroupNormArgs& a, bool vectors, F f) {
    const int D = a.D;
    if (a.bf16 && vectors) {
        if (D <= 64) return f.template run<8, 8, 1, __nv_bfloat16>();
        if (D <= 128) return f.template run<16, 8, 1, __nv_bfloat16>();
        if (D <= 256) return f.template run<32, 8, 1, __nv_bfloat16>();
        if (D <= 1024) return f.template run<128, 8, 1, __nv_bfloat16>();
        return f.template run<256, 8, 4, __nv_bfloat16>();
    }
    if (vectors) {
        if (D <= 32) return f.template run<8, 4, 1, float>();
        if (D <= 64) return f.template run<16, 4, 1, float>();
        if (D <= 128) return f.template run<32, 4, 1, float>();
        if (D <= 512) return f.template run<128, 4, 1, float>();
        return f.template run<256, 4, 8, float>();
    }
    if (a.bf16) {
        if (D <= 128) return f.template run<32, 1, 4, __nv_bfloat16>();
        if (D <= 1024) return f.template run<128, 1, 8, __nv_bfloat16>();
        return f.template run<256, 1, 32, __nv_bfloat16>();
    }
    if (D <= 128) return f.template run<32, 1, 4, float>();
    if (D <= 1024) return f.template run<128, 1, 8, float>();
    return f.template run<256, 1, 32, float>();
}

bool aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    return true;
}
bool fits_vectors(const GroupNormArgs& a) {
    return a.D % (a.bf16 ? 8 : 4) == 0 && aligned({a.x, a.gate, a.weight, a.bias, a.y, a.dy, a.dx, a.dgate});
}

struct Forward {
    const GroupNormArgs& a;
    cudaStream_t st;
    template <int LPG, int VEC, int NV, typename T>
    cudaError_t run() const {
        const Grid g = grid_of(a, LPG, kFwdBlocks);
        trace_begin("group_norm_fwd", st);
        group_norm_fwd_kernel<LPG, VEC, NV, T><<<dim3(g.x, g.y), g.threads, 0, st>>>(a, g.per);
        trace_end(st);
        return cudaGetLastError();
    }
};
struct Backward {
    const GroupNormArgs& a;
    float* part;
    cudaStream_t st;
    template <int LPG, int VEC, int NV, typename T>
    cudaError_t run() const {
        const Grid g = grid_of(a, LPG, kBwdBlocks);
        float* p = a.dweight || a.dbias ? part : nullptr;
        trace_begin("group_norm_bwd", st);
        group_norm_bwd_kernel<LPG, VEC, NV, T><<<dim3(g.x, g.y), g.threads, 0, st>>>(a, g.per, p);
        trace_end(st);
        if (cudaError_t e = cudaGetLastError()) return e;
        if (!p) return cudaSuccess;
        const int C = a.groups * a.D;
        trace_begin("group_norm_params", st);
        group_norm_params_kernel<<<(2 * C + 31) / 32, 1024, 0, st>>>(p, g.y * g.rl, C, a.dweight, a.dbias);
        trace_end(st);
        return cudaGetLastError();
    }
};
struct Partials {
    const GroupNormArgs& a;
    size_t* rows;
    template <int LPG, int VEC, int NV, typename T>
    cudaError_t run() const {
        const Grid g = grid_of(a, LPG, kBwdBlocks);
        *rows = (size_t)g.y * g.rl;
        return cudaSuccess;
    }
};

}  // namespace

cudaError_t launch_group_norm_fwd(const GroupNormArgs& a, cudaStream_t st) {
    return with_shape(a, fits_vectors(a), Forward{a, st});
}
cudaError_t launch_group_norm_bwd(const GroupNormArgs& a, float* part, cudaStream_t st) {
    return with_shape(a, fits_vectors(a), Backward{a, part, st});
}
// The larger of the two shapes' needs: pointers, which choose between them, are not known here.
size_t group_norm_bwd_partials(const GroupNormArgs& a) {
    size_t v = 0, s = 0;
    if (a.D % (a.bf16 ? 8 : 4) == 0) with_shape(a, true, Partials{a, &v});
    with_shape(a, false, Partials{a, &s});
    return (v > s ? v : s) * 2 * (size_t)a.groups * a.D * sizeof(float);
}

}  // namespace gdr
