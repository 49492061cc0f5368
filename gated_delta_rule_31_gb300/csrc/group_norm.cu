// group_norm.cu - group norm over the channels of each token, with an activation of the result or
// of a gate beside it (gdr_group_norm_fwd, gdr_group_norm_bwd).
//
//   h = (x - mean) r, r = 1 / sqrt(var + eps) over the D channels of a token's group (mean = 0 if
//   not centered, var = the mean of h's squares before scaling), n = w h + b,
//   y = act(n), or n act(z) with a gate z.
//   dn = dy act'(n) or dy act(z);  dz = dy n act'(z);  dw = sum dn h, db = sum dn over tokens;
//   dh = w dn;  dx = r (dh - mean(dh) - h mean(dh h)), without mean(dh) if not centered.
//
// HBM bounds both directions, so a group's values are read once and stay in registers: some lanes share a
// group, each with NV vectors of VEC values, and the statistics are sums over those lanes (two passes
// over the registers: the mean, then the squares about it). The backward forms the statistics again from
// x, which it needs anyway, so the forward stores none. A lane keeps its channels for all the tokens it
// works on: w and b are read once, and dw and db are sums in registers, written as one partial row for
// each (block row, lane row) and added up in a fixed order by a second kernel. Groups that start between
// vectors are read in the row's vectors all the same, and what a vector holds of a neighbour is masked.
// 32768 rows of 32 groups of 128, bf16, gated: forward 128 us (805 MB, 93% of a plain copy's rate;
// centered, with offsets, 130), backward 235 + 6 us (1.34 GB, 84%). Wider groups wait at a barrier for each
// sum: one group of 4096, 24414 rows: forward 110 us (80%), backward 246 (60%).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "group_norm.h"
#include "kernels.h"

namespace gdr {

namespace {

constexpr int THREADS = 256;

// VEC values as loaded: 16 bytes, a pair, or a single value.
template <int VEC, typename T>
struct RawOf { using type = T; };
template <>
struct RawOf<8, __nv_bfloat16> { using type = uint4; };
template <>
struct RawOf<2, __nv_bfloat16> { using type = uint32_t; };
template <>
struct RawOf<4, float> { using type = float4; };
template <>
struct RawOf<2, float> { using type = float2; };

template <int VEC, typename T>
__device__ __forceinline__ typename RawOf<VEC, T>::type load_raw(const T* p) {
    return *reinterpret_cast<const typename RawOf<VEC, T>::type*>(p);
}
// Sets the values of u whose bit in `valid` is clear to zero, whatever they hold.
__device__ __forceinline__ uint32_t halves(uint32_t u, uint32_t valid) {
    return u & ((valid & 1 ? 0xffffu : 0u) | (valid & 2 ? 0xffff0000u : 0u));
}
__device__ __forceinline__ void keep(uint4& u, uint32_t valid) {
    u = make_uint4(halves(u.x, valid), halves(u.y, valid >> 2), halves(u.z, valid >> 4), halves(u.w, valid >> 6));
}
__device__ __forceinline__ void keep(uint32_t& u, uint32_t valid) { u = halves(u, valid); }
__device__ __forceinline__ void keep(float4& u, uint32_t valid) {
    u = make_float4(valid & 1 ? u.x : 0.f, valid & 2 ? u.y : 0.f, valid & 4 ? u.z : 0.f, valid & 8 ? u.w : 0.f);
}
__device__ __forceinline__ void keep(float2& u, uint32_t valid) { u = make_float2(valid & 1 ? u.x : 0.f, valid & 2 ? u.y : 0.f); }
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
__device__ __forceinline__ void values(const uint32_t& u, Pair* x) { x[0] = bf16_pair(u); }
__device__ __forceinline__ void values(const float2& u, Pair* x) { x[0] = pair(u.x, u.y); }
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
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const Pair (&x)[1]) { *reinterpret_cast<uint32_t*>(p) = pack(x[0]); }
__device__ __forceinline__ void store_vec(float* p, const Pair (&x)[1]) { *reinterpret_cast<float2*>(p) = split(x[0]); }
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[1]) { *p = __float2bfloat16_rn(x[0]); }
__device__ __forceinline__ void store_vec(float* p, const float (&x)[1]) { *p = x[0]; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
template <typename T, int N>
__device__ __forceinline__ void store_some(T* p, const Pair (&x)[N], uint32_t valid) {
#pragma unroll
    for (int j = 0; j < N; j++) {
        const float2 f = split(x[j]);
        if (valid >> (2 * j) & 1) put(p + 2 * j, f.x);
        if (valid >> (2 * j) & 2) put(p + 2 * j + 1, f.y);
    }
}
// The valid values of a vector; all of them unless CUT.
template <bool CUT, typename T, typename V, int N>
__device__ __forceinline__ void store_valid(T* p, const V (&x)[N], uint32_t valid) {
    if constexpr (CUT) {
        if (valid != (1u << (2 * N)) - 1) {
            store_some(p, x, valid);
            return;
        }
    }
    store_vec(p, x);
}
// The valid values of a weight's or offset's vector, which need no alignment; the others stay. (Read for each
// row a value at a time, the backward of groups of 4096 takes 338 us, by 16 bytes 246.)
template <bool CUT, int N>
__device__ __forceinline__ void load_param(const float* p, uint32_t valid, Pair (&x)[N]) {
    if constexpr (!CUT && N % 2 == 0) {
        if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
            for (int j = 0; j < N; j += 2) values(*reinterpret_cast<const float4*>(p + 2 * j), x + j);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < N; j++) {
        float2 f = split(x[j]);
        if (!CUT || valid >> (2 * j) & 1) f.x = p[2 * j];
        if (!CUT || valid >> (2 * j) & 2) f.y = p[2 * j + 1];
        x[j] = pair(f.x, f.y);
    }
}
template <bool CUT>
__device__ __forceinline__ void load_param(const float* p, uint32_t, float (&x)[1]) { x[0] = *p; }

// v where the pair's values are valid (the lowest two bits), else zero.
template <bool CUT>
__device__ __forceinline__ Pair valid_part(Pair v, uint32_t valid) {
    if (!CUT) return v;
    const float2 f = split(v);
    return pair(valid & 1 ? f.x : 0.f, valid & 2 ? f.y : 0.f);
}
template <bool CUT>
__device__ __forceinline__ float valid_part(float v, uint32_t) {
    return v;
}

// Which token rows and group a lane works on. A block covers `per` groups (blockIdx.x) and `rl` token
// rows at a time, `lanes` lanes each; lanes past the last row or group only join the sums.
struct Place {
    int group, lane, lanes, slot_row, rl;
    int warp0, warps;  // of a group wider than a warp
    long long row0, row_step;
    bool live;
};
__device__ __forceinline__ Place place(int groups, int per, int lanes) {
    Place p;
    const int slot = threadIdx.x / lanes;
    p.lanes = lanes;
    p.rl = blockDim.x / (lanes * per);
    p.lane = threadIdx.x - slot * lanes;
    p.slot_row = slot / per;
    p.group = blockIdx.x * per + slot - p.slot_row * per;
    p.warps = lanes / 32;
    p.warp0 = slot * p.warps;
    p.live = p.group < groups && p.slot_row < p.rl;
    p.row0 = (long long)blockIdx.y * p.rl + p.slot_row;
    p.row_step = (long long)gridDim.y * p.rl;
    return p;
}
// The vector that starts at lane index k of the group: its first channel, and a bit for each of its VEC
// channels that is the group's. With CUT the vectors are those of the row, of which the group's first and
// last may begin or end in a neighbouring group.
template <int VEC, bool CUT>
__device__ __forceinline__ uint32_t vector_of(const Place& at, int D, int k, int* first) {
    const int from = at.group * D, c = (CUT ? from / VEC * VEC : from) + k * VEC, end = from + D;
    *first = c;
    if (!at.live || c >= end) return 0;
    uint32_t valid = (1u << VEC) - 1;
    if (CUT && c < from) valid &= valid << (from - c);
    if (CUT && c + VEC > end) valid &= (1u << (end - c)) - 1;
    return valid;
}

// Sums over the lanes of a group: one or two values; groups wider than a warp go through shared memory, two
// buffers in turn (a warp that has passed one sum's barrier has read the sum before).
struct Sums {
    float2 (*red)[THREADS / 32];
    int turn = 0;
};
__device__ __forceinline__ void group_sum2(float& a, float& b, const Place& at, Sums& sums) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < at.lanes) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    if (at.lanes > 32) {
        float2* red = sums.red[sums.turn];
        sums.turn ^= 1;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
        for (int w = 0; w < at.warps; w++) {
            const float2 v = red[at.warp0 + w];
            a += v.x;
            b += v.y;
        }
    }
}
__device__ __forceinline__ float group_sum(float a, const Place& at, Sums& sums) {
    if (at.lanes > 32) {
        float none = 0.f;
        group_sum2(a, none, at, sums);
        return a;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < at.lanes) a += __shfl_xor_sync(0xffffffffu, a, o);
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

// A lane asks for its next row before it works on the current one: a row a lane in flight is too little
// to keep HBM busy (32768 rows of 4096 bf16, gated: forward 147 us without).
// L: the lanes of a group where the kernel is made for them, else 0.
template <int VEC, int NV, int L, bool CUT, typename T>
__global__ void __launch_bounds__(THREADS, VEC == 1 ? 1 : VEC > 2 && VEC * NV <= 8 ? 4 : VEC * NV <= 16 ? 2 : 1)
    group_norm_fwd_kernel(GroupNormArgs a, int per, int lanes_) {
    const int lanes = L ? L : lanes_;
    using Raw = typename RawOf<VEC, T>::type;
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    __shared__ float2 red[2][THREADS / 32];
    Sums sums{red};
    const Place at = place(a.groups, per, lanes);
    const size_t C = (size_t)a.groups * a.D;
    const float inv = 1.f / (float)a.D;
    const T* x = static_cast<const T*>(a.x);
    const T* z = static_cast<const T*>(a.gate);
    T* y = static_cast<T*>(a.y);
    int e[NV];
    typename std::conditional<CUT, uint32_t, bool>::type in[NV];  // valid values
    V w[NV][N], b[NV][N];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        in[i] = vector_of<VEC, CUT>(at, a.D, i * lanes + at.lane, &e[i]);
#pragma unroll
        for (int j = 0; j < N; j++) {
            w[i][j] = all<V>(1.f);
            b[i][j] = all<V>(0.f);
        }
        if (in[i] && a.weight) load_param<CUT>(a.weight + e[i], in[i], w[i]);
        if (in[i] && a.bias) load_param<CUT>(a.bias + e[i], in[i], b[i]);
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
            if constexpr (CUT) keep(nx[i], in[i]);
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
            const V mean = all<V>(-inv * group_sum(total(sum), at, sums));
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (in[i])
#pragma unroll
                    for (int j = 0; j < N; j++) v[i][j] = add(v[i][j], valid_part<CUT>(mean, (uint32_t)in[i] >> (2 * j)));
        }
        V sq = all<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < N; j++) sq = fma(v[i][j], v[i][j], sq);
        const V r = all<V>(rsqrtf(group_sum(total(sq), at, sums) * inv + a.eps));
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
                    store_valid<CUT>(y + row * C + e[i], v[i], in[i]);
                }
    }
}

// With 16 values a lane or more, the sums of dw and db lie in shared memory, in places of the lane's own,
// and w and b are read for each row: registers hold what a row needs (24414 rows of 4096, bf16: 246 us; all
// in registers 395).
template <int VEC, int NV, int L, bool CUT, typename T>
__global__ void __launch_bounds__(THREADS, VEC * NV <= 16 ? 2 : 1)
    group_norm_bwd_kernel(GroupNormArgs a, int per, int lanes_, float* part) {
    const int lanes = L ? L : lanes_;
    using Raw = typename RawOf<VEC, T>::type;
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    constexpr bool WIDE = VEC * NV > 8 && VEC > 1;
    extern __shared__ __align__(16) unsigned char far[];
    __shared__ float2 red[2][THREADS / 32];
    Sums sums{red};
    const Place at = place(a.groups, per, lanes);
    const size_t C = (size_t)a.groups * a.D;
    const float inv = 1.f / (float)a.D;
    const T* x = static_cast<const T*>(a.x);
    const T* z = static_cast<const T*>(a.gate);
    const T* dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.dx);
    T* dz = static_cast<T*>(a.dgate);
    int e[NV];
    typename std::conditional<CUT, uint32_t, bool>::type in[NV];  // valid values
#pragma unroll
    for (int i = 0; i < NV; i++) in[i] = vector_of<VEC, CUT>(at, a.D, i * lanes + at.lane, &e[i]);
    constexpr int KEPT = WIDE ? 1 : NV;
    V w[KEPT][N], b[KEPT][N], dw[KEPT][N], db[KEPT][N];
    auto params = [&](int i) {
        V(&wi)[N] = w[WIDE ? 0 : i], (&bi)[N] = b[WIDE ? 0 : i];
#pragma unroll
        for (int j = 0; j < N; j++) {
            wi[j] = all<V>(1.f);
            bi[j] = all<V>(0.f);
        }
        if (in[i] && a.weight) load_param<CUT>(a.weight + e[i], in[i], wi);
        if (in[i] && a.bias) load_param<CUT>(a.bias + e[i], in[i], bi);
    };
    auto sum_at = [&](int i, int j) { return reinterpret_cast<V*>(far) + ((i * N + j) * 2) * THREADS + threadIdx.x; };
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (!WIDE) params(i);
#pragma unroll
        for (int j = 0; j < N; j++) {
            if (WIDE) {
                sum_at(i, j)[0] = sum_at(i, j)[THREADS] = all<V>(0.f);
            } else {
                dw[WIDE ? 0 : i][j] = db[WIDE ? 0 : i][j] = all<V>(0.f);
            }
        }
    }
    Raw nx[NV] = {}, nz[NV] = {}, ng[NV] = {};
    auto ask = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const bool use = in[i] && row < a.rows;
            if (use) nx[i] = load_raw<VEC>(x + row * C + e[i]);
            if (use && z) nz[i] = load_raw<VEC>(z + row * C + e[i]);
            if (use) ng[i] = load_raw<VEC>(dy + row * C + e[i]);
        }
    };
    const long long steps = (a.rows + at.row_step - 1) / at.row_step;
    ask(at.row0);
    for (long long s = 0; s < steps; s++) {
        const long long row = at.row0 + s * at.row_step;
        V h[NV][N], u[NV][N], g[NV][N];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if constexpr (CUT) keep(nx[i], in[i]), keep(nz[i], in[i]), keep(ng[i], in[i]);
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
            const V mean = all<V>(-inv * group_sum(total(sum), at, sums));
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (in[i])
#pragma unroll
                    for (int j = 0; j < N; j++) h[i][j] = add(h[i][j], valid_part<CUT>(mean, (uint32_t)in[i] >> (2 * j)));
        }
        V sq = all<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < N; j++) sq = fma(h[i][j], h[i][j], sq);
        const float r = rsqrtf(group_sum(total(sq), at, sums) * inv + a.eps);
        V s1 = all<V>(0.f), s2 = all<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in[i] && row < a.rows) {  // no row adds nothing to dw and db: what its registers hold may not be finite
                V n[N], d[N];
                if (WIDE) params(i);
                const int k = WIDE ? 0 : i;
#pragma unroll
                for (int j = 0; j < N; j++) {
                    h[i][j] = mul(h[i][j], all<V>(r));
                    n[j] = fma(w[k][j], h[i][j], b[k][j]);
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
                    if (WIDE) {
                        V* sum = sum_at(i, j);
                        sum[0] = fma(dn, h[i][j], sum[0]);
                        sum[THREADS] = add(sum[THREADS], dn);
                    } else {
                        dw[k][j] = fma(dn, h[i][j], dw[k][j]);
                        db[k][j] = add(db[k][j], dn);
                    }
                    g[i][j] = mul(dn, w[k][j]);
                    s1 = add(s1, g[i][j]);
                    s2 = fma(g[i][j], h[i][j], s2);
                }
                if (z) store_valid<CUT>(dz + row * C + e[i], u[i], in[i]);
            }
        float t1 = total(s1), t2 = total(s2);
        group_sum2(t1, t2, at, sums);
        // dx = r g - r m1 - h r m2
        const V vr = all<V>(r), m1 = all<V>(a.center ? -t1 * inv * r : 0.f), m2 = all<V>(-t2 * inv * r);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in[i] && row < a.rows) {
#pragma unroll
                for (int j = 0; j < N; j++) g[i][j] = fma(g[i][j], vr, fma(h[i][j], m2, m1));
                store_valid<CUT>(dx + row * C + e[i], g[i], in[i]);
            }
    }
    if (!part) return;
    float* pw = part + ((size_t)blockIdx.y * at.rl + at.slot_row) * 2 * C;
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (in[i]) {
            const int k = WIDE ? 0 : i;
            if (WIDE)
#pragma unroll
                for (int j = 0; j < N; j++) {
                    dw[k][j] = sum_at(i, j)[0];
                    db[k][j] = sum_at(i, j)[THREADS];
                }
            store_valid<CUT>(pw + e[i], dw[k], in[i]);
            store_valid<CUT>(pw + C + e[i], db[k], in[i]);
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
// A block takes as many whole groups as THREADS lanes hold, spread evenly over the blocks of a row, then
// several token rows at a time; the rows are spread evenly over about as many blocks as run at once.
Grid grid_of(const GroupNormArgs& a, int lanes, int blocks_per_sm) {
    Grid g;
    const int slots = THREADS / lanes;
    g.x = (a.groups + slots - 1) / slots;
    g.per = (a.groups + g.x - 1) / g.x;
    g.rl = slots / g.per;
    g.threads = (g.per * g.rl * lanes + 31) / 32 * 32;
    const long long rows = (a.rows + g.rl - 1) / g.rl;
    long long y = 152LL * (blocks_per_sm * THREADS / g.threads) / g.x;
    if (y < 1) y = 1;
    if (y > rows) y = rows;
    if (y > 65535) y = 65535;
    const long long each = (rows + y - 1) / y;  // row steps of a block
    g.y = (int)((rows + each - 1) / each);
    return g;
}

// The most vectors that a group touches.
int vectors_of(const GroupNormArgs& a, int vec) {
    int gcd = vec;
    while (a.D % gcd) gcd /= 2;
    return ((a.groups == 1 ? 0 : vec - gcd) + a.D + vec - 1) / vec;
}
// Values of a vector: 16 bytes where every row of every tensor starts on 16 bytes, else two values or one
// (24414 rows of about 4096 in groups of 96, 33 and 99 channels, bf16: 129, 351 and 235 us forward).
bool rows_on(const GroupNormArgs& a, int vec, bool pointers) {
    if ((long long)a.groups * a.D % vec != 0 || vectors_of(a, vec) * vec > GDR_NORM_MAX_D) return false;
    if (pointers)
        for (const void* p : {a.x, a.gate, (const void*)a.y, a.dy, (const void*)a.dx, (const void*)a.dgate})
            if (reinterpret_cast<uintptr_t>(p) % (vec * (a.bf16 ? 2 : 4)) != 0) return false;
    return true;
}
// NV vectors a lane, and as many lanes as hold a group: a power of two within a warp, else whole warps.
// For the powers of two there are kernels made for that number (4 groups of 1024, bf16: forward and backward
// 115 and 204 us, by the general kernel 146 and 252).
template <int VEC, int NV, typename T, typename F>
cudaError_t with_lanes(const GroupNormArgs& a, F f) {
    const int need = (vectors_of(a, VEC) + NV - 1) / NV;
    int lanes = 1;
    while (lanes < need && lanes < 32) lanes *= 2;
    if (need > 32) lanes = (need + 31) / 32 * 32;
    if (a.D % VEC != 0) return f.template run<VEC, NV, 0, true, T>(lanes);
    if constexpr (VEC > 2) {
        if constexpr (NV == 1) {
            if (lanes == 8) return f.template run<VEC, NV, 8, false, T>(lanes);
            if (lanes == 16) return f.template run<VEC, NV, 16, false, T>(lanes);
            if (lanes == 32) return f.template run<VEC, NV, 32, false, T>(lanes);
        }
        if constexpr (VEC * NV == 8) {
            if (lanes == 64) return f.template run<VEC, NV, 64, false, T>(lanes);
            if (lanes == 128) return f.template run<VEC, NV, 128, false, T>(lanes);
        }
        if constexpr (VEC * NV >= 8)
            if (lanes == 256) return f.template run<VEC, NV, 256, false, T>(lanes);
    }
    return f.template run<VEC, NV, 0, false, T>(lanes);
}
// One 16-byte vector a lane while a block has lanes enough, and two, four or eight for the widest groups. fp32
// takes two from 33 vectors on, as many values as bf16's one (8 groups of 512, 24414 rows: 205 and 294 us;
// one vector in 128 lanes 192 and 363). Vectors of two values: four a lane, so that a warp holds 256.
template <typename T, typename F>
cudaError_t with_shape(const GroupNormArgs& a, int vec, F f) {
    constexpr int FULL = 16 / sizeof(T);
    const int v = vectors_of(a, vec);
    if (vec == FULL) {
        if (v <= (FULL == 8 ? 256 : 32)) return with_lanes<FULL, 1, T>(a, f);
        if (v <= 512) return with_lanes<FULL, 2, T>(a, f);
        return with_lanes<FULL, 32 / FULL, T>(a, f);
    }
    if (vec == 2) return v <= 1024 ? with_lanes<2, 4, T>(a, f) : with_lanes<2, 16, T>(a, f);
    // Single values, 32 a lane in the widest groups, whose backward then keeps more than registers hold (spills of 700
    // bytes a thread; one group of 5001, 20000 rows, bf16: 2080 us).
    if (v <= 128) return f.template run<1, 4, 32, false, T>(32);
    if (v <= 1024) return f.template run<1, 8, 0, false, T>((v + 255) / 256 * 32);
    return f.template run<1, 32, 256, false, T>(256);
}
template <typename F>
cudaError_t with_type(const GroupNormArgs& a, int vec, F f) {
    return a.bf16 ? with_shape<__nv_bfloat16>(a, vec, f) : with_shape<float>(a, vec, f);
}
int vec_of(const GroupNormArgs& a, bool pointers) {
    for (int vec : {a.bf16 ? 8 : 4, 2})
        if (rows_on(a, vec, pointers)) return vec;
    return 1;
}

constexpr int kFwdBlocks = 4, kBwdBlocks = 2;  // blocks of THREADS per SM that run at once

struct Forward {
    const GroupNormArgs& a;
    cudaStream_t st;
    template <int VEC, int NV, int L, bool CUT, typename T>
    cudaError_t run(int lanes) const {
        const Grid g = grid_of(a, lanes, kFwdBlocks);
        trace_begin("group_norm_fwd", st);
        group_norm_fwd_kernel<VEC, NV, L, CUT, T><<<dim3(g.x, g.y), g.threads, 0, st>>>(a, g.per, lanes);
        trace_end(st);
        return cudaGetLastError();
    }
};
struct Backward {
    const GroupNormArgs& a;
    float* part;
    cudaStream_t st;
    template <int VEC, int NV, int L, bool CUT, typename T>
    cudaError_t run(int lanes) const {
        const Grid g = grid_of(a, lanes, kBwdBlocks);
        float* p = a.dweight || a.dbias ? part : nullptr;
        const int far = VEC * NV > 8 && VEC > 1 ? 2 * VEC * NV * THREADS * (int)sizeof(float) : 0;
        auto kernel = group_norm_bwd_kernel<VEC, NV, L, CUT, T>;
        if (far)
            if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, far)) return e;
        trace_begin("group_norm_bwd", st);
        kernel<<<dim3(g.x, g.y), g.threads, far, st>>>(a, g.per, lanes, p);
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
    template <int VEC, int NV, int L, bool CUT, typename T>
    cudaError_t run(int lanes) const {
        const Grid g = grid_of(a, lanes, kBwdBlocks);
        if ((size_t)g.y * g.rl > *rows) *rows = (size_t)g.y * g.rl;
        return cudaSuccess;
    }
};

}  // namespace

cudaError_t launch_group_norm_fwd(const GroupNormArgs& a, cudaStream_t st) {
    return with_type(a, vec_of(a, true), Forward{a, st});
}
cudaError_t launch_group_norm_bwd(const GroupNormArgs& a, float* part, cudaStream_t st) {
    return with_type(a, vec_of(a, true), Backward{a, part, st});
}
// The largest of the shapes' needs: pointers, which choose among them, are not known here.
size_t group_norm_bwd_partials(const GroupNormArgs& a) {
    size_t rows = 0;
    for (int vec : {a.bf16 ? 8 : 4, 2, 1})
        if (vec == 1 || rows_on(a, vec, false)) with_type(a, vec, Partials{a, &rows});
    return rows * 2 * (size_t)a.groups * a.D * sizeof(float);
}

}  // namespace gdr
