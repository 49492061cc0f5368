// api_attention.cu - the C ABI (include/gdr.h) of the softmax attention layer: window attention and its VJP, rotary
// positions, the append to a paged cache and the decode step over it. Argument validation, workspace layout and
// launches; as in api.cu nothing here allocates device memory, and every launch goes to the caller's stream.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "attention.h"
#include "gdr.h"

using namespace gdr;

namespace {

bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
size_t round_up(size_t x, size_t to) { return (x + to - 1) / to * to; }
gdr_status of(cudaError_t e) { return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }
bool dtype_ok(int d) { return d == GDR_F32 || d == GDR_BF16; }

// Required pointers may be null only where the tensors are empty; all are aligned to `bytes`.
gdr_status check_ptrs(bool empty, uintptr_t bytes, std::initializer_list<const void*> required,
                      std::initializer_list<const void*> optional) {
    for (const void* x : required)
        if ((!x && !empty) || !on(x, bytes)) return GDR_ERR_INVALID_ARG;
    for (const void* x : optional)
        if (!on(x, bytes)) return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}
gdr_status check_ws(const void* ws, size_t have, size_t need) {
    if (!ws || have < need) return GDR_ERR_WORKSPACE;
    return on(ws, 256) ? GDR_OK : GDR_ERR_INVALID_ARG;
}

// Heads, masks and scale of either attention.
gdr_status check_heads(int Hq, int Hk, int D, int window, int sinks, int dtype, float scale) {
    if (Hq <= 0 || Hk <= 0 || D <= 0 || Hq % Hk != 0 || window < 0 || sinks < 0) return GDR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !isfinite(scale) || !(scale > 0.f)) return GDR_ERR_INVALID_ARG;
    if ((D != 32 && D != 64 && D != 128) || Hq > 65535) return GDR_ERR_UNSUPPORTED;  // grid y limit
    return GDR_OK;
}

gdr_status check_window(const gdr_window_problem* p) {
    if (!p || p->B < 0 || p->T < 0) return GDR_ERR_INVALID_ARG;
    const gdr_status r = check_heads(p->Hq, p->Hk, p->D, p->window, p->sinks, p->dtype, p->scale);
    if (r != GDR_OK) return r;
    if (p->B > 65535 || p->T > GDR_WINDOW_MAX_T) return GDR_ERR_UNSUPPORTED;        // grid z limit
    // units of 128 queries (or keys and their pieces, few more than that) of a head are counted in ints
    if ((long long)p->B * p->Hq * ((p->T + 127) / 128) > 1 << 29) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}
WindowArgs window_args(const gdr_window_problem* p, const int* lengths) {
    WindowArgs a = {};
    a.s.B = p->B; a.s.T = p->T; a.s.Hq = p->Hq; a.s.Hk = p->Hk; a.s.D = p->D;
    a.s.bf16 = p->dtype == GDR_BF16;
    a.s.window = p->window == 0 || p->window > p->T ? p->T : p->window;
    a.s.sinks = p->sinks > p->T ? p->T : p->sinks;
    a.s.scale = p->scale;
    a.s.lengths = lengths;
    return a;
}
size_t rows_bytes(const gdr_window_problem* p) { return round_up((size_t)p->B * p->Hq * p->T * sizeof(float), 256); }

gdr_status check_turn(int B, int T, int D, int pairs, int axes, const int* sections, int interleaved) {
    if (B < 0 || T < 0 || D <= 0 || pairs < 0 || (interleaved != 0 && interleaved != 1)) return GDR_ERR_INVALID_ARG;
    if (2LL * pairs > D) return GDR_ERR_INVALID_ARG;
    if (pairs > 0) {
        if (axes < 1 || axes > 4) return GDR_ERR_INVALID_ARG;
        long long sum = 0;
        for (int i = 0; i < axes; i++) {
            if (sections[i] < 0) return GDR_ERR_INVALID_ARG;
            sum += sections[i];
        }
        if (sum != pairs) return GDR_ERR_INVALID_ARG;
    }
    if (D % 2 != 0 || D > 65536) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * T > (1LL << 32) / D) return GDR_ERR_UNSUPPORTED;  // 2^31 pairs of a head
    return GDR_OK;
}
void set_sections(TurnArgs& a, int pairs, int axes, const int* sections, int interleaved) {
    a.pairs = pairs;
    a.axes = axes;
    for (int i = 0; i < 4; i++) a.sections[i] = pairs > 0 && i < axes ? sections[i] : 0;
    a.interleaved = interleaved;
}

gdr_status check_paged(const gdr_paged_problem* p) {
    if (!p || p->B < 0 || p->pages < 0 || p->page_size <= 0 || p->table_pages < 0) return GDR_ERR_INVALID_ARG;
    const gdr_status r = check_heads(p->Hq, p->Hk, p->D, p->window, p->sinks, p->dtype, p->scale);
    if (r != GDR_OK) return r;
    if (p->B > 65535) return GDR_ERR_UNSUPPORTED;
    if ((long long)p->pages * p->page_size >= 0xffffffffLL) return GDR_ERR_UNSUPPORTED;  // rows are counted in 32 bits
    if ((long long)p->table_pages * p->page_size > 0x7fff0000LL) return GDR_ERR_UNSUPPORTED;    // tokens, and a tile more, in 31
    return GDR_OK;
}

}  // namespace

extern "C" {

size_t gdr_window_fwd_workspace(const gdr_window_problem* p) { return check_window(p) == GDR_OK ? 256 : 0; }

gdr_status gdr_window_fwd(const gdr_window_problem* p, const void* q, const void* k, const void* v, const int* lengths,
                          void* o, float* lse, void* rest, void* ws, size_t ws_bytes, gdr_stream_t stream) {
    gdr_status r = check_window(p);
    if (r != GDR_OK) return r;
    const bool empty = p->B == 0 || p->T == 0;
    if ((r = check_ptrs(empty, 16, {q, k, v, o}, {rest})) != GDR_OK) return r;
    if (rest && p->dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (!on(lse, 4) || !on(lengths, 4)) return GDR_ERR_INVALID_ARG;
    if ((r = check_ws(ws, ws_bytes, gdr_window_fwd_workspace(p))) != GDR_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    if (empty) return of(cudaMemsetAsync(ws, 0, 256, st));
    WindowArgs a = window_args(p, lengths);
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse; a.rest = rest;
    a.status = static_cast<int*>(ws);
    return of(launch_window_fwd(a, st));
}

size_t gdr_window_bwd_workspace(const gdr_window_problem* p) {
    return check_window(p) == GDR_OK ? 256 + rows_bytes(p) + window_parts_bytes(window_args(p, nullptr).s) : 0;
}

gdr_status gdr_window_bwd(const gdr_window_problem* p, const void* q, const void* k, const void* v, const int* lengths,
                          const void* o, const float* lse, const void* rest, const void* do_, void* dq, void* dk,
                          void* dv, void* ws, size_t ws_bytes, gdr_stream_t stream) {
    gdr_status r = check_window(p);
    if (r != GDR_OK) return r;
    const bool empty = p->B == 0 || p->T == 0;
    if ((r = check_ptrs(empty, 16, {q, k, v, o, do_, dq, dk, dv}, {rest})) != GDR_OK) return r;
    if (rest && p->dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if ((!lse && !empty) || !on(lse, 4) || !on(lengths, 4)) return GDR_ERR_INVALID_ARG;
    if ((r = check_ws(ws, ws_bytes, gdr_window_bwd_workspace(p))) != GDR_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    if (empty) return of(cudaMemsetAsync(ws, 0, 256, st));
    WindowArgs a = window_args(p, lengths);
    a.q = q; a.k = k; a.v = v; a.o = const_cast<void*>(o); a.lse = const_cast<float*>(lse); a.rest = const_cast<void*>(rest);
    a.do_ = do_; a.dq = dq; a.dk = dk; a.dv = dv;
    a.status = static_cast<int*>(ws);
    a.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256 + rows_bytes(p));
    return of(launch_window_bwd(a, st));
}

gdr_status gdr_rotary(const gdr_rotary_problem* p, const void* x, const int* positions, const float* inv_freq, void* y,
                      gdr_stream_t stream) {
    if (!p) return GDR_ERR_INVALID_ARG;
    if (p->H <= 0 || !dtype_ok(p->dtype) || (p->inverse != 0 && p->inverse != 1)) return GDR_ERR_INVALID_ARG;
    gdr_status r = check_turn(p->B, p->T, p->D, p->pairs, p->axes, p->sections, p->interleaved);
    if (r != GDR_OK) return r;
    if (p->H > 65535) return GDR_ERR_UNSUPPORTED;
    const bool empty = p->B == 0 || p->T == 0;
    if ((r = check_ptrs(empty, p->dtype == GDR_BF16 ? 2 : 4, {x, y}, {})) != GDR_OK) return r;
    if ((r = check_ptrs(empty || p->pairs == 0, 4, {positions, inv_freq}, {})) != GDR_OK) return r;
    if (empty) return GDR_OK;
    TurnArgs a = {};
    a.part[0] = {x, y, p->H, 1, 0};
    a.parts = 1;
    a.B = p->B; a.T = p->T; a.D = p->D; a.bf16 = p->dtype == GDR_BF16;
    set_sections(a, p->pairs, p->axes, p->sections, p->interleaved);
    a.inverse = p->inverse;
    a.inv_freq = inv_freq;
    a.positions = positions;
    return of(launch_turn(a, (cudaStream_t)stream));
}

gdr_status gdr_kv_append(const gdr_append_problem* p, const void* q, const void* k, const void* v, const int* positions,
                         const float* inv_freq, const int* lengths, const int* counts, const int* page_table,
                         void* q_out, void* k_cache, void* v_cache, gdr_stream_t stream) {
    if (!p) return GDR_ERR_INVALID_ARG;
    if (p->Hq < 0 || p->Hk <= 0 || !dtype_ok(p->dtype)) return GDR_ERR_INVALID_ARG;
    if (p->pages < 0 || p->page_size <= 0 || p->table_pages < 0) return GDR_ERR_INVALID_ARG;
    gdr_status r = check_turn(p->B, p->T, p->D, p->pairs, p->axes, p->sections, p->interleaved);
    if (r != GDR_OK) return r;
    if (p->pairs > 0 && !positions && p->axes != 1) return GDR_ERR_INVALID_ARG;  // the place in the sequence is one axis
    if (p->Hq > 65535 || p->Hk > 65535) return GDR_ERR_UNSUPPORTED;
    const bool empty = p->B == 0 || p->T == 0;
    const uintptr_t e = p->dtype == GDR_BF16 ? 2 : 4;
    if ((r = check_ptrs(empty, e, {k, v}, {q, q_out})) != GDR_OK) return r;
    if ((r = check_ptrs(empty || p->pages == 0, e, {k_cache, v_cache}, {})) != GDR_OK) return r;
    if (!empty && p->Hq > 0 && (!q || !q_out)) return GDR_ERR_INVALID_ARG;
    if ((r = check_ptrs(empty, 4, {lengths}, {positions, counts})) != GDR_OK) return r;
    if ((r = check_ptrs(empty || p->table_pages == 0, 4, {page_table}, {})) != GDR_OK) return r;
    if ((r = check_ptrs(empty || p->pairs == 0, 4, {inv_freq}, {})) != GDR_OK) return r;
    if (empty) return GDR_OK;
    TurnArgs a = {};
    if (p->Hq > 0) a.part[a.parts++] = {q, q_out, p->Hq, 1, 0};
    if (p->pages > 0 && p->table_pages > 0) {
        a.part[a.parts++] = {k, k_cache, p->Hk, 1, 1};
        a.part[a.parts++] = {v, v_cache, p->Hk, 0, 1};
    }
    if (a.parts == 0) return GDR_OK;
    a.B = p->B; a.T = p->T; a.D = p->D; a.bf16 = p->dtype == GDR_BF16;
    set_sections(a, p->pairs, p->axes, p->sections, p->interleaved);
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.counts = counts;
    a.lengths = lengths;
    a.table = page_table;
    a.table_pages = p->table_pages; a.page_size = p->page_size; a.pages = p->pages;
    return of(launch_turn(a, (cudaStream_t)stream));
}

size_t gdr_paged_decode_workspace(const gdr_paged_problem* p) {
    return check_paged(p) == GDR_OK ? 256 + paged_parts_bytes(p->D) : 0;
}

gdr_status gdr_paged_decode_step(const gdr_paged_problem* p, const void* q, const void* k_cache, const void* v_cache,
                                 const int* page_table, const int* lengths, void* o, void* ws, size_t ws_bytes,
                                 gdr_stream_t stream) {
    gdr_status r = check_paged(p);
    if (r != GDR_OK) return r;
    const bool empty = p->B == 0;
    if ((r = check_ptrs(empty, 16, {q, o}, {})) != GDR_OK) return r;
    if ((r = check_ptrs(empty || p->pages == 0, 16, {k_cache, v_cache}, {})) != GDR_OK) return r;
    if ((r = check_ptrs(empty || p->table_pages == 0, 4, {page_table}, {})) != GDR_OK) return r;
    if ((r = check_ptrs(empty, 4, {lengths}, {})) != GDR_OK) return r;
    if ((r = check_ws(ws, ws_bytes, gdr_paged_decode_workspace(p))) != GDR_OK) return r;
    if (empty) return GDR_OK;
    PagedArgs a = {p->B, p->Hq, p->Hk, p->D, p->dtype == GDR_BF16, p->pages, p->page_size, p->table_pages, p->window, p->sinks,
                   p->scale, q, k_cache, v_cache, page_table, lengths, o,
                   reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256)};
    return of(launch_paged_step(a, (cudaStream_t)stream));
}

}  // extern "C"
