// api_linear.cu - the C ABI (include/gdr.h) of linear attention with a constant decay per head and
// of the per-token group norm: argument validation, workspace layout and launches. As in api.cu
// nothing here allocates device memory, and every launch goes to the caller's stream.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "gdr.h"
#include "group_norm.h"
#include "linear.h"

using namespace gdr;

namespace {

bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
size_t round_up(size_t x, size_t to) { return (x + to - 1) / to * to; }
bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

gdr_status check_problem(const gdr_linear_problem* p, bool decode) {
    if (!p) return GDR_ERR_INVALID_ARG;
    if (p->B < 0 || p->T < 0 || p->Hk <= 0 || p->Hv <= 0 || p->Dk <= 0 || p->Dv <= 0) return GDR_ERR_INVALID_ARG;
    if (p->Hv % p->Hk != 0) return GDR_ERR_INVALID_ARG;
    if (decode && p->T != 1) return GDR_ERR_INVALID_ARG;
    if (p->dtype != GDR_F32 && p->dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (!isfinite(p->scale)) return GDR_ERR_INVALID_ARG;
    if (!dim_ok(p->Dk) || !dim_ok(p->Dv)) return GDR_ERR_UNSUPPORTED;
    if (p->B > 65535 || p->Hv > 65535) return GDR_ERR_UNSUPPORTED;  // grid y/z limits
    if ((long long)p->B * p->Hv * p->Dv >= 1LL << 32) return GDR_ERR_UNSUPPORTED;  // a state of 512 GB or more
    // Positions past the end of a sequence, by less than a block of tokens for each of up to 1216 segments, are ints.
    if (p->T > GDR_LINEAR_MAX_T) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Required pointers may be null only where the tensors are empty; every pointer is 16-byte aligned.
gdr_status check_ptrs(bool empty, std::initializer_list<const void*> required,
                      std::initializer_list<const void*> optional) {
    for (const void* x : required)
        if ((!x && !empty) || !on(x, 16)) return GDR_ERR_INVALID_ARG;
    for (const void* x : optional)
        if (!on(x, 16)) return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}

LinearShape shape_of(const gdr_linear_problem* p, const float* g, const int* lengths) {
    LinearShape s;
    s.B = p->B; s.T = p->T; s.Hk = p->Hk; s.Hv = p->Hv; s.Dk = p->Dk; s.Dv = p->Dv;
    s.bf16 = p->dtype == GDR_BF16;
    s.nseg = s.bf16 ? linear_tc_segments(p->B, p->T, p->Hv) : linear_segments(p->B, p->T, p->Hv, p->Dv);
    const int block = s.bf16 ? kLinearBlockTc : kLinearBlock;  // segments are whole blocks of tokens
    const int blocks = p->T / block + (p->T % block != 0);
    s.seg_tokens = blocks > 0 ? (blocks + s.nseg - 1) / s.nseg * block : block;
    s.nseg = blocks > 0 ? p->T / s.seg_tokens + (p->T % s.seg_tokens != 0) : 1;
    s.g = g;
    s.lengths = lengths;
    return s;
}

size_t states_bytes(const LinearShape& s) {
    return (size_t)s.B * s.Hv * s.nseg * s.Dv * s.Dk * sizeof(float);
}
// Kept chunk states (bf16 only): a 32 KB tile for each (b, hv, 128-token chunk).
size_t kept_bytes(const LinearShape& s) { return s.bf16 ? (size_t)s.B * s.Hv * ((s.T + 127) / 128) * 32768 : 0; }
size_t tokens_bytes(const LinearShape& s) { return round_up((size_t)s.B * s.T * s.Hv * s.Dv * 2, 256); }
size_t fwd_bytes(const LinearShape& s) { return 256 + states_bytes(s); }
// bf16: segment states, the adjoints of the chunks' states and, unless the forward kept them, their
// states, formed again by an output pass whose output goes nowhere else. fp32: both segment states.
size_t bwd_bytes(const LinearShape& s, bool kept) {
    if (!s.bf16) return 256 + 2 * states_bytes(s);
    return 256 + states_bytes(s) + kept_bytes(s) + (kept ? 0 : kept_bytes(s) + tokens_bytes(s));
}

gdr_status check_ws(const void* ws, size_t have, size_t need) {
    if (!ws || have < need) return GDR_ERR_WORKSPACE;
    return on(ws, 256) ? GDR_OK : GDR_ERR_INVALID_ARG;
}
gdr_status check_kept(const void* kept, size_t have, const LinearShape& s) {
    const size_t need = kept_bytes(s);
    if (need && (!kept || have < need)) return GDR_ERR_WORKSPACE;
    return on(kept, 256) ? GDR_OK : GDR_ERR_INVALID_ARG;
}
gdr_status of(cudaError_t e) { return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }

// The state that enters each segment, forwards (rows = v, cols = k) or in reverse (do, q).
cudaError_t states(const LinearShape& s, const void* rows, const void* cols, float factor, int reverse,
                   const float* init, float* z, float* last, int* clear, cudaStream_t st) {
    LinearSummaryArgs a{s, rows, cols, factor, reverse, z, clear};
    if (cudaError_t e = launch_linear_summary(a, st)) return e;
    LinearCombineArgs c{s, init, reverse, z, last};
    return launch_linear_combine(c, true, st);
}

// A mix pass on the tensor cores from the state `init` before it: with several segments, the states that
// enter them first. The first kernel of a call clears its status word.
cudaError_t mix_tc(const LinearMixArgs& m, const void* rows, const void* cols, float factor, int reverse,
                   const float* init, float* z, float* last, int* status, bool clear, cudaStream_t st) {
    if (m.s.nseg == 1) return launch_linear_tc_mix(m, init, 1, last, status, clear, false, st);
    LinearSummaryArgs a{m.s, rows, cols, factor, reverse, z, nullptr};
    if (cudaError_t e = launch_linear_tc_summary(a, last != nullptr, status, clear, st)) return e;
    LinearCombineArgs c{m.s, init, reverse, z, last};
    if (cudaError_t e = launch_linear_combine(c, true, st)) return e;
    return launch_linear_tc_mix(m, z, m.s.nseg, nullptr, status, false, true, st);
}

// No token or no sequence: nothing can fail, and the state passes through.
gdr_status pass_state(const gdr_linear_problem* p, const float* from, float* to, void* status, cudaStream_t st) {
    if (cudaMemsetAsync(status, 0, 256, st) != cudaSuccess) return GDR_ERR_CUDA;
    if (p->B == 0 || !to) return GDR_OK;
    const size_t bytes = (size_t)p->B * p->Hv * p->Dv * p->Dk * sizeof(float);
    return of(from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, bytes, st));
}

gdr_status check_norm(const gdr_norm_problem* p) {
    if (!p) return GDR_ERR_INVALID_ARG;
    if (p->rows < 0 || p->groups <= 0 || p->D <= 0) return GDR_ERR_INVALID_ARG;
    if (p->dtype != GDR_F32 && p->dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (p->activation != GDR_ACT_NONE && p->activation != GDR_ACT_SILU && p->activation != GDR_ACT_SIGMOID)
        return GDR_ERR_INVALID_ARG;
    if (p->center != 0 && p->center != 1) return GDR_ERR_INVALID_ARG;
    if (!isfinite(p->eps) || p->eps <= 0.f) return GDR_ERR_INVALID_ARG;
    if (p->D > GDR_NORM_MAX_D || (long long)p->groups * p->D > (1 << 24)) return GDR_ERR_UNSUPPORTED;
    if (p->rows > (1LL << 60) / (p->groups * p->D)) return GDR_ERR_UNSUPPORTED;  // sizes in bytes are 64-bit
    return GDR_OK;
}

GroupNormArgs norm_args(const gdr_norm_problem* p) {
    GroupNormArgs a = {};
    a.rows = p->rows; a.groups = p->groups; a.D = p->D;
    a.bf16 = p->dtype == GDR_BF16;
    a.act = p->activation; a.center = p->center; a.eps = p->eps;
    return a;
}

// Pointers of a norm call: required ones may be null only without rows; each aligned to its element.
gdr_status check_norm_ptrs(const gdr_norm_problem* p, std::initializer_list<const void*> required,
                           std::initializer_list<const void*> optional, std::initializer_list<const void*> params) {
    const uintptr_t e = p->dtype == GDR_BF16 ? 2 : 4;
    for (const void* x : required)
        if ((!x && p->rows > 0) || !on(x, e)) return GDR_ERR_INVALID_ARG;
    for (const void* x : optional)
        if (!on(x, e)) return GDR_ERR_INVALID_ARG;
    for (const void* x : params)
        if (!on(x, 4)) return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}

}  // namespace

extern "C" {

size_t gdr_linear_fwd_workspace(const gdr_linear_problem* p) {
    if (check_problem(p, false) != GDR_OK) return 0;
    return fwd_bytes(shape_of(p, nullptr, nullptr));
}

size_t gdr_linear_states_bytes(const gdr_linear_problem* p) {
    if (check_problem(p, false) != GDR_OK) return 0;
    return kept_bytes(shape_of(p, nullptr, nullptr));
}

size_t gdr_linear_bwd_workspace(const gdr_linear_problem* p) {
    if (check_problem(p, false) != GDR_OK) return 0;
    return bwd_bytes(shape_of(p, nullptr, nullptr), false);
}

size_t gdr_linear_bwd_states_workspace(const gdr_linear_problem* p) {
    if (check_problem(p, false) != GDR_OK) return 0;
    return bwd_bytes(shape_of(p, nullptr, nullptr), true);
}

static gdr_status linear_fwd_impl(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                                  const float* g, const float* h0, const int* lengths, void* o, float* ht, bool keep,
                                  void* kept, size_t have, void* ws, size_t ws_bytes, cudaStream_t st) {
    gdr_status r = check_problem(p, false);
    if (r != GDR_OK) return r;
    const bool empty = p->B == 0 || p->T == 0;
    if ((r = check_ptrs(empty, {q, k, v, o}, {h0, ht})) != GDR_OK) return r;
    if (!g || !on(g, 4) || !on(lengths, 4)) return GDR_ERR_INVALID_ARG;
    const LinearShape s = shape_of(p, g, lengths);
    if (keep && (r = check_kept(kept, have, s)) != GDR_OK) return r;
    if ((r = check_ws(ws, ws_bytes, fwd_bytes(s))) != GDR_OK) return r;
    if (empty) return pass_state(p, h0, ht, ws, st);
    int* status = static_cast<int*>(ws);
    float* z = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    LinearMixArgs m{s, LINEAR_O, q, k, v, nullptr, p->scale, z, o, h0, ht, keep ? kept : nullptr,
                    s.nseg > 1, s.nseg > 1 ? nullptr : status};
    if (s.bf16) return of(mix_tc(m, v, k, 1.f, 0, h0, z, ht, status, true, st));
    if (s.nseg > 1 && states(s, v, k, 1.f, 0, h0, z, ht, status, st) != cudaSuccess) return GDR_ERR_CUDA;
    return of(launch_linear_mix(m, st));
}

static gdr_status linear_bwd_impl(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                                  const float* g, const float* h0, const int* lengths, const void* do_,
                                  const float* dht, void* dq, void* dk, void* dv, float* dh0, bool keep,
                                  const void* kept, size_t have, void* ws, size_t ws_bytes, cudaStream_t st) {
    gdr_status r = check_problem(p, false);
    if (r != GDR_OK) return r;
    const bool empty = p->B == 0 || p->T == 0;
    if ((r = check_ptrs(empty, {q, k, v, do_, dq, dk, dv}, {h0, dht, dh0})) != GDR_OK) return r;
    if (!g || !on(g, 4) || !on(lengths, 4)) return GDR_ERR_INVALID_ARG;
    const LinearShape s = shape_of(p, g, lengths);
    if (keep && (r = check_kept(kept, have, s)) != GDR_OK) return r;
    if ((r = check_ws(ws, ws_bytes, bwd_bytes(s, keep))) != GDR_OK) return r;
    if (empty) return pass_state(p, dht, dh0, ws, st);
    int* status = static_cast<int*>(ws);
    uint8_t* w = static_cast<uint8_t*>(ws) + 256;
    float* z = reinterpret_cast<float*>(w);
    if (s.bf16) {
        uint8_t* adjoints = w + states_bytes(s);
        if (!keep) {  // the chunks' states, formed again
            uint8_t* again = adjoints + kept_bytes(s);
            LinearMixArgs m{s, LINEAR_O, q, k, v, nullptr, p->scale, z, again + kept_bytes(s), nullptr, nullptr, again, false, nullptr};
            if (mix_tc(m, v, k, 1.f, 0, h0, z, nullptr, status, true, st) != cudaSuccess) return GDR_ERR_CUDA;
            kept = again;
        }
        LinearMixArgs m{s, LINEAR_DV, q, k, v, do_, p->scale, z, dv, nullptr, nullptr, adjoints, false, nullptr};
        if (mix_tc(m, do_, q, p->scale, 1, dht, z, dh0, status, keep, st) != cudaSuccess) return GDR_ERR_CUDA;
        LinearGradArgs a{s, q, k, v, do_, p->scale, kept, adjoints, dq, dk, status};
        return of(launch_linear_tc_grad(a, st));
    }
    float* zd = reinterpret_cast<float*>(w + states_bytes(s));
    if (s.nseg > 1) {
        if (states(s, v, k, 1.f, 0, h0, z, nullptr, status, st) != cudaSuccess) return GDR_ERR_CUDA;
        if (states(s, do_, q, p->scale, 1, dht, zd, dh0, nullptr, st) != cudaSuccess) return GDR_ERR_CUDA;
    }
    // dv reads the reverse states, which dk, summing over value heads, may update in place: dv first
    const struct { int pass; float* z; void* out; const float* init; float* last; } passes[3] = {
        {LINEAR_DQ, z, dq, h0, nullptr}, {LINEAR_DV, zd, dv, dht, dh0}, {LINEAR_DK, zd, dk, dht, nullptr}};
    for (const auto& x : passes) {
        LinearMixArgs m{s, x.pass, q, k, v, do_, p->scale, x.z, x.out, x.init, x.last, nullptr, false,
                        s.nseg == 1 && x.pass == LINEAR_DQ ? status : nullptr};
        if (launch_linear_mix(m, st) != cudaSuccess) return GDR_ERR_CUDA;
    }
    return GDR_OK;
}

gdr_status gdr_linear_fwd(const gdr_linear_problem* p, const void* q, const void* k, const void* v, const float* g,
                          const float* h0, const int* lengths, void* o, float* ht, void* ws, size_t ws_bytes,
                          gdr_stream_t stream) {
    return linear_fwd_impl(p, q, k, v, g, h0, lengths, o, ht, false, nullptr, 0, ws, ws_bytes, (cudaStream_t)stream);
}

gdr_status gdr_linear_fwd_states(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                                 const float* g, const float* h0, const int* lengths, void* o, float* ht, void* states,
                                 size_t states_bytes, void* ws, size_t ws_bytes, gdr_stream_t stream) {
    return linear_fwd_impl(p, q, k, v, g, h0, lengths, o, ht, true, states, states_bytes, ws, ws_bytes,
                           (cudaStream_t)stream);
}

gdr_status gdr_linear_bwd(const gdr_linear_problem* p, const void* q, const void* k, const void* v, const float* g,
                          const float* h0, const int* lengths, const void* do_, const float* dht, void* dq, void* dk,
                          void* dv, float* dh0, void* ws, size_t ws_bytes, gdr_stream_t stream) {
    return linear_bwd_impl(p, q, k, v, g, h0, lengths, do_, dht, dq, dk, dv, dh0, false, nullptr, 0, ws, ws_bytes,
                           (cudaStream_t)stream);
}

gdr_status gdr_linear_bwd_states(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                                 const float* g, const float* h0, const int* lengths, const void* states,
                                 size_t states_bytes, const void* do_, const float* dht, void* dq, void* dk, void* dv,
                                 float* dh0, void* ws, size_t ws_bytes, gdr_stream_t stream) {
    return linear_bwd_impl(p, q, k, v, g, h0, lengths, do_, dht, dq, dk, dv, dh0, true, states, states_bytes, ws,
                           ws_bytes, (cudaStream_t)stream);
}

gdr_status gdr_linear_decode_step(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                                  const float* g, float* state, void* o, gdr_stream_t stream) {
    gdr_status r = check_problem(p, true);
    if (r != GDR_OK) return r;
    if ((r = check_ptrs(p->B == 0, {q, k, v, state, o}, {})) != GDR_OK) return r;
    if (!g || !on(g, 4)) return GDR_ERR_INVALID_ARG;
    if (p->B == 0) return GDR_OK;
    LinearStepArgs a{p->B, p->Hk, p->Hv, p->Dk, p->Dv, p->dtype == GDR_BF16, p->scale, q, k, v, g, state, o};
    return of(launch_linear_step(a, (cudaStream_t)stream));
}

gdr_status gdr_group_norm_fwd(const gdr_norm_problem* p, const void* x, const void* gate, const float* weight,
                              const float* bias, void* y, gdr_stream_t stream) {
    gdr_status r = check_norm(p);
    if (r != GDR_OK) return r;
    if ((r = check_norm_ptrs(p, {x, y}, {gate}, {weight, bias})) != GDR_OK) return r;
    if (p->rows == 0) return GDR_OK;
    GroupNormArgs a = norm_args(p);
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.y = y;
    return of(launch_group_norm_fwd(a, (cudaStream_t)stream));
}

size_t gdr_group_norm_bwd_workspace(const gdr_norm_problem* p) {
    if (check_norm(p) != GDR_OK) return 0;
    return 256 + (p->rows ? group_norm_bwd_partials(norm_args(p)) : 0);
}

gdr_status gdr_group_norm_bwd(const gdr_norm_problem* p, const void* x, const void* gate, const float* weight,
                              const float* bias, const void* dy, void* dx, void* dgate, float* dweight, float* dbias,
                              void* ws, size_t ws_bytes, gdr_stream_t stream) {
    gdr_status r = check_norm(p);
    if (r != GDR_OK) return r;
    if ((r = check_norm_ptrs(p, {x, dy, dx}, {gate, dgate}, {weight, bias, dweight, dbias})) != GDR_OK) return r;
    if (p->rows > 0 && (gate != nullptr) != (dgate != nullptr)) return GDR_ERR_INVALID_ARG;
    if ((r = check_ws(ws, ws_bytes, gdr_group_norm_bwd_workspace(p))) != GDR_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    if (p->rows == 0) {  // empty sums
        const size_t bytes = (size_t)p->groups * p->D * sizeof(float);
        if (dweight && cudaMemsetAsync(dweight, 0, bytes, st) != cudaSuccess) return GDR_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, bytes, st) != cudaSuccess) return GDR_ERR_CUDA;
        return GDR_OK;
    }
    GroupNormArgs a = norm_args(p);
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.dy = dy;
    a.dx = dx; a.dgate = dgate; a.dweight = dweight; a.dbias = dbias;
    return of(launch_group_norm_bwd(a, reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256), st));
}

}  // extern "C"
