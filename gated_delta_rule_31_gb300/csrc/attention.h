// attention.h - launch interface of the softmax attention layer (gdr_window_*, gdr_rotary, gdr_kv_append,
// gdr_paged_*), shared by its C ABI (api_attention.cu) and its kernels.
//
// Token t of a batch entry with n tokens sees token j if j <= t, j < n, and t - j < window or
// j < sinks; s = scale q_t . k_j, o_t = sum_j p_j v_j with p the softmax of s over the seen tokens.
// Kernels go over tiles of keys: those that hold first tokens, then those that the window reaches.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr {

struct WindowShape {
    int B, T, Hq, Hk, D, bf16;
    int window, sinks;   // window in 1 .. T (T: every earlier token), sinks in 0 .. T
    float scale;         // > 0
    const int* lengths;  // [B] valid tokens, or null (T)
#ifdef __CUDACC__
    __device__ int tokens(int b) const { return lengths ? min(max(lengths[b], 0), T) : T; }
#endif
};

// Tiles of N keys that queries [t0, t1) (t1 at most the entry's tokens) see: `first` tiles from the start, then
// lo .. hi - 1. And the queries that see keys [j0, j0 + N): from j0 to the end below.
struct KeyTiles {
    int first, lo, hi;
    __host__ __device__ KeyTiles() : first(0), lo(0), hi(0) {}
    __host__ __device__ KeyTiles(int N, int window, int sinks, int t0, int t1) {
        if (t0 >= t1) {
            first = lo = hi = 0;
            return;
        }
        hi = (t1 + N - 1) / N;
        lo = t0 >= window ? (t0 - window + 1) / N : 0;
        const int s = (sinks + N - 1) / N;
        first = s < lo ? s : lo;
    }
    __host__ __device__ int count() const { return first + hi - lo; }
    __host__ __device__ int at(int i) const { return i < first ? i : lo + i - first; }
    __host__ __device__ bool has(int tile) const { return tile < first || (tile >= lo && tile < hi); }
};
__host__ __device__ inline int queries_end(int N, int window, int sinks, int j0, int n) {
    if (j0 < sinks) return n;
    const long long e = (long long)j0 + N - 1 + window;
    return e < n ? (int)e : n;
}

struct WindowArgs {
    WindowShape s;
    const void *q, *k, *v;
    void* o;
    float* lse;   // [B, Hq, T], or null (forward)
    void* rest;   // bf16: what the rounding of o left [B, T, Hq, D], or null
    // VJP
    const void *do_;
    float* delta;  // [B, Hq, T] sum of do o over the channels
    void *dq, *dk, *dv;
    float* parts;  // sums of dk and dv over parts of the queries (window_parts_bytes)
    int* status;
};
cudaError_t launch_window_fwd(const WindowArgs& a, cudaStream_t st);
size_t window_parts_bytes(const WindowShape& s);
cudaError_t launch_window_bwd(const WindowArgs& a, cudaStream_t st);

// Rows of heads: q (and k) with their first 2 `pairs` channels turned, v as it is.
struct TurnPart {
    const void* src;  // [B, T, H, D]
    void* dst;        // [B, T, H, D], or a cache [pages, page_size, H, D]
    int H, turned, cached;
};
struct TurnArgs {
    TurnPart part[3];
    int parts;
    int B, T, D, bf16;
    int pairs, axes, sections[4], interleaved, inverse;
    const float* inv_freq;  // [pairs]
    int freq16;             // set by launch_turn: inv_freq is 16-byte aligned
    const int* positions;   // [B, T, axes], or null: lengths[b] + t
    const int* counts;      // [B] tokens of each entry, or null (T)
    const int* lengths;     // [B] tokens in the cache before, or null
    const int* table;       // [B, table_pages]
    int table_pages, page_size, pages;
};
cudaError_t launch_turn(const TurnArgs& a, cudaStream_t st);

struct PagedArgs {
    int B, Hq, Hk, D, bf16;
    int pages, page_size, table_pages, window, sinks;  // window 0: every token
    float scale;
    const void *q, *k, *v;
    const int *table, *lengths;
    void* o;
    float* parts;
};
size_t paged_parts_bytes(int D);
cudaError_t launch_paged_step(const PagedArgs& a, cudaStream_t st);

}  // namespace gdr
