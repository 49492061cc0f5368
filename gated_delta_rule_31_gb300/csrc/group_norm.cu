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
// order by a second kernel. 32768 rows of 32 groups of 128, bf16, gated: forward 123 us (805 MB, 96% of a
// plain copy's rate; centered, with offsets, 128), backward 233 + 6 us (1.34 GB, 85%).
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
// Values are worked on in pairs, one instruction for two (fp32 pairs), or singly where VEC is 1.
struct Pair {
    uint64_t v;
};
__device__ __forceinline__ Pair pair(float a, float b) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ float2 split(Pair p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p.v));
    return f;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ float total(Pair p) {
    const float2 f = split(p);
    return f.x + f.y;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float total(float x) { return x; }
__device__ __forceinline__ void fill(Pair& p, float x) { p = pair(x, x); }
__device__ __forceinline__ void fill(float& p, float x) { p = x; }
template <typename V>
__device__ __forceinline__ V all(float x) {
    V v;
    fill(v, x);
    return v;
}

template <int VEC>
struct Lanes {  // VEC values as N units of type V
    using V = Pair;
    static constexpr int N = VEC / 2;
};
template <>
struct Lanes<1> {
    using V = float;
    static constexpr int N = 1;
};

__device__ __forceinline__ Pair bf16_pair(uint32_t u) { return pair(bf16lo(u), bf16hi(u)); }
__device__ __forceinline__ void values(const uint4& u, Pair* x) {
    x[0] = bf16_pair(u.x); x[1] = bf16_pair(u.y); x[2] = bf16_pair(u.z); x[3] = bf16_pair(u.w);
}
__device__ __forceinline__ void values(const float4& u, Pair* x) {
    x[0] = pair(u.x, u.y); x[1] = pair(u.z, u.w);
}
__device__ __forceinline__ void values(const __nv_bfloat16& u, float* x) { x[0] = __bfloat162float(u); }
__device__ __forceinline__ void values(const float& u, float* x) { x[0] = u; }
__device__ __forceinline__ uint32_t pack(Pair p) {
    const float2 f = split(p);
    return pack_bf16(f.x, f.y);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const Pair (&x)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack(x[0]), pack(x[1]), pack(x[2]), pack(x[3]));
}
__device__ __forceinline__ void store_vec(float* p, const Pair (&x)[2]) {
    const float2 a = split(x[0]), b = split(x[1]);
    *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_vec(float* p, const Pair (&x)[4]) {
    const float2 a = split(x[0]), b = split(x[1]), c = split(x[2]), d = split(x[3]);
    *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<float4*>(p + 4) = make_float4(c.x, c.y, d.x, d.y);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[1]) { *p = __float2bfloat16_rn(x[0]); }
__device__ __forceinline__ void store_vec(float* p, const float (&x)[1]) { *p = x[0]; }
__device__ __forceinline__ void load_param(const float* p, Pair (&x)[4]) {
    values(*reinterpret_cast<const float4*>(p), x);
    values(*reinterpret_cast<const float4*>(p + 4), x + 2);
}
__device__ __forceinline__ void load_param(const float* p, Pair (&x)[2]) { values(*reinterpret_cast<const float4*>(p), x); }
__device__ __forceinline__ void load_param(const float* p, float (&x)[1]) { x[0] = *p; }

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

// The sum of one value.
template <int LPG>
__device__ __forceinline__ float group_sum(float a, float2* red) {
    float none = 0.f;
    if constexpr (LPG > 32) {
        group_sum2<LPG>(a, none, red);
    } else {
#pragma unroll
        for (int o = LPG / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    }
    return a;
}

// 1 / (1 + 2^(-x log2 e)) by the hardware's approximate power of two and reciprocal, each good to a few units
// in the last place; results below the smallest normal number are zero. (Through __expf and
// __fdividef, which look after those, the backward was bound by its 462 instructions for each 8 values.)
__device__ __forceinline__ float sigmoid(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
__device__ __forceinline__ Pair sigmoid(Pair x) {
    const float2 f = split(x);
    return pair(sigmoid(f.x), sigmoid(f.y));
}
// x <- act(x)
template <typename V, int N>
__device__ __forceinline__ void activate(V (&x)[N], int act) {
    if (act == GDR_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; j++) x[j] = mul(x[j], sigmoid(x[j]));
    } else if (act == GDR_ACT_SIGMOID) {
#pragma unroll
        for (int j = 0; j < N; j++) x[j] = sigmoid(x[j]);
    }
}
// x <- act(x), d = act'(x)
template <typename V, int N>
__device__ __forceinline__ void activate2(V (&x)[N], V (&d)[N], int act) {
    const V one = all<V>(1.f), minus = all<V>(-1.f);
    if (act == GDR_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; j++) {
            const V s = sigmoid(x[j]), f = mul(x[j], s);
            d[j] = fma(f, fma(s, minus, one), s);  // s + x s (1 - s)
            x[j] = f;
        }
    } else if (act == GDR_ACT_SIGMOID) {
#pragma unroll
        for (int j = 0; j < N; j++) {
            const V s = sigmoid(x[j]);
            d[j] = mul(s, fma(s, minus, one));
            x[j] = s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) d[j] = one;
    }
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
// to keep HBM busy (32768 rows of 4096 bf16, gated: forward 147 us without).
template <int LPG, int VEC, int NV, typename T>
__global__ void __launch_bounds__(THREADS, NV == 1 ? 4 : 1) group_norm_fwd_kernel(GroupNormArgs a, int per) {
    using Raw = typename RawOf<VEC, T>::type;
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    __shared__ float2 red[THREADS / 32];
    const Place at = place<LPG>(a.groups, per);
    const size_t C = (size_t)a.groups * a.D;
    const float inv = 1.f / (float)a.D;
    const T* x = static_cast<const T*>(a.x);
    const T* z = static_cast<const T*>(a.gate);
    T* y = static_cast<T*>(a.y);
    int e[NV];
    bool in[NV];
    V w[NV][N], b[NV][N];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int d = (i * LPG + at.lane) * VEC;
        in[i] = at.live && d < a.D;
        e[i] = at.group * a.D + d;
#pragma unroll
        for (int j = 0; j < N; j++) {
            w[i][j] = all<V>(1.f);
            b[i][j] = all<V>(0.f);
        }
        if (in[i] && a.weight) load_param(a.weight + e[i], w[i]);
        if (in[i] && a.bias) load_param(a.bias + e[i], b[i]);
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
        V v[NV][N], u[NV][N];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            values(nx[i], v[i]);
            values(nz[i], u[i]);
        }
        ask(row + at.row_step);
        if (a.center) {
            V sum = all<V>(0.f);
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int j = 0; j < N; j++) sum = add(sum, v[i][j]);
            const V mean = all<V>(-inv * group_sum<LPG>(total(sum), red));
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (in[i])
#pragma unroll
                    for (int j = 0; j < N; j++) v[i][j] = add(v[i][j], mean);
        }
        V sq = all<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < N; j++) sq = fma(v[i][j], v[i][j], sq);
        const V r = all<V>(rsqrtf(group_sum<LPG>(total(sq), red) * inv + a.eps));
        if (row < a.rows)
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (in[i]) {
#pragma unroll
                    for (int j = 0; j < N; j++) v[i][j] = fma(w[i][j], mul(v[i][j], r), b[i][j]);
                    activate(z ? u[i] : v[i], a.act);
                    if (z)
#pragma unroll
                        for (int j = 0; j < N; j++) v[i][j] = mul(v[i][j], u[i][j]);
                    store_vec(y + row * C + e[i], v[i]);
                }
    }
}

template <int LPG, int VEC, int NV, typename T>
__global__ void __launch_bounds__(THREADS, NV == 1 ? 2 : 1) group_norm_bwd_kernel(GroupNormArgs a, int per, float* part) {
    using Raw = typename RawOf<VEC, T>::type;
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
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
    V w[NV][N], b[NV][N], dw[NV][N], db[NV][N];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int d = (i * LPG + at.lane) * VEC;
        in[i] = at.live && d < a.D;
        e[i] = at.group * a.D + d;
#pragma unroll
        for (int j = 0; j < N; j++) {
            w[i][j] = all<V>(1.f);
            b[i][j] = dw[i][j] = db[i][j] = all<V>(0.f);
        }
        if (in[i] && a.weight) load_param(a.weight + e[i], w[i]);
        if (in[i] && a.bias) load_param(a.bias + e[i], b[i]);
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
        V h[NV][N], u[NV][N], g[NV][N];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            values(nx[i], h[i]);
            values(nz[i], u[i]);
            values(ng[i], g[i]);
        }
        ask(row + at.row_step);
        if (a.center) {
            V sum = all<V>(0.f);
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int j = 0; j < N; j++) sum = add(sum, h[i][j]);
            const V mean = all<V>(-inv * group_sum<LPG>(total(sum), red));
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (in[i])
#pragma unroll
                    for (int j = 0; j < N; j++) h[i][j] = add(h[i][j], mean);
        }
        V sq = all<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < N; j++) sq = fma(h[i][j], h[i][j], sq);
        const float r = rsqrtf(group_sum<LPG>(total(sq), red) * inv + a.eps);
        V s1 = all<V>(0.f), s2 = all<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in[i]) {
                V n[N], d[N];
#pragma unroll
                for (int j = 0; j < N; j++) {
                    h[i][j] = mul(h[i][j], all<V>(r));
                    n[j] = fma(w[i][j], h[i][j], b[i][j]);
                }
                if (z) {  // u: act(z), then dz = dy n act'(z); g: dn = dy act(z)
                    activate2(u[i], d, a.act);
#pragma unroll
                    for (int j = 0; j < N; j++) {
                        const V dy1 = g[i][j];
                        g[i][j] = mul(dy1, u[i][j]);
                        u[i][j] = mul(mul(dy1, n[j]), d[j]);
                    }
                } else {  // dn = dy act'(n)
                    activate2(n, d, a.act);
#pragma unroll
                    for (int j = 0; j < N; j++) g[i][j] = mul(g[i][j], d[j]);
                }
#pragma unroll
                for (int j = 0; j < N; j++) {
                    const V dn = g[i][j];
                    dw[i][j] = fma(dn, h[i][j], dw[i][j]);
                    db[i][j] = add(db[i][j], dn);
                    g[i][j] = mul(dn, w[i][j]);
                    s1 = add(s1, g[i][j]);
                    s2 = fma(g[i][j], h[i][j], s2);
                }
                if (z && row < a.rows) store_vec(dz + row * C + e[i], u[i]);
            }
        float t1 = total(s1), t2 = total(s2);
        group_sum2<LPG>(t1, t2, red);
        // dx = r g - r m1 - h r m2
        const V vr = all<V>(r), m1 = all<V>(a.center ? -t1 * inv * r : 0.f), m2 = all<V>(-t2 * inv * r);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in[i] && row < a.rows) {
#pragma unroll
                for (int j = 0; j < N; j++) g[i][j] = fma(g[i][j], vr, fma(h[i][j], m2, m1));
                store_vec(dx + row * C + e[i], g[i]);
            }
    }
    if (!part) return;
    const int rl = blockDim.x / (LPG * per);
    float* pw = part + ((size_t)blockIdx.y * rl + at.slot_row) * 2 * C;
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (in[i]) {
            store_vec(pw + e[i], dw[i]);
            store_vec(pw + C + e[i], db[i]);
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

constexpr int kFwdBlocks = 4, kBwdBlocks = 2;  // blocks of THREADS per SM that run at once

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
