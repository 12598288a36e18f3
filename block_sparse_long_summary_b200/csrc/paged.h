// Host-side derived sizes and launchers of the paged-cache calls (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/cobs.h"

namespace cobs {

// Whether a kernel's attributes (one flag array per kernel) have still to be set on the current device.
// Setting them twice, by two threads at once, does no harm.
struct OncePerDevice {
    std::atomic<bool> done[64] = {};
    template <typename F> cudaError_t run(F&& set) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
        e = set();
        if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
        return e;
    }
};

constexpr int kMaxKeys = 1 << 30;    // keys of a request, and token rows
constexpr int kMaxRequests = 16384;  // the kernels keep one int per request in shared memory

struct PagedDims {
    int R, Hq, Hkv, G, d;
    int page, page_shift;  // tokens per page (a power of two)
    int n_pages, max_pages, n_tokens, max_new;
    int W, S;              // window (0: none) and sinks
    int dtype;
    long long q_stride, kv_stride;  // elements between token rows
    size_t elem() const { return dtype == COBS_BF16 ? 2 : 4; }
};

inline PagedDims make_paged_dims(const cobs_paged_params& p) {
    PagedDims m;
    m.R = p.R; m.Hq = p.Hq; m.Hkv = p.Hkv; m.G = p.Hkv ? p.Hq / p.Hkv : 0; m.d = p.d;
    m.page = p.page;
    m.page_shift = 0;
    while ((1 << m.page_shift) < p.page) ++m.page_shift;
    m.n_pages = p.n_pages; m.max_pages = p.max_pages; m.n_tokens = p.n_tokens; m.max_new = p.max_new;
    // positions are below 2^30: longer windows are no windows, and sums of both stay in 32 bits
    m.W = p.window < kMaxKeys ? p.window : kMaxKeys;
    m.S = p.sinks < kMaxKeys ? p.sinks : kMaxKeys;
    m.dtype = p.dtype;
    m.q_stride = p.q_stride ? p.q_stride : (long long)p.Hq * p.d;
    m.kv_stride = p.kv_stride ? p.kv_stride : (long long)p.Hkv * p.d;
    return m;
}

cudaError_t launch_paged_tables(const PagedDims& m, const int32_t* cached_len, const int32_t* new_len,
                                const int32_t* free_pages, int n_free, const int32_t* free_count,
                                int32_t* block_table, int32_t* cu_new, int32_t* kv_len, int32_t* slot_map,
                                int32_t* counts, cudaStream_t s, int* err);

cudaError_t launch_paged_append(const PagedDims& m, const void* K, const void* V, const int32_t* slot_map,
                                void* k_cache, void* v_cache, cudaStream_t s, int* err);

size_t paged_attn_workspace_bytes(const PagedDims& m);
cudaError_t launch_paged_attn(const PagedDims& m, const void* Q, const void* k_cache, const void* v_cache,
                              const int32_t* block_table, const int32_t* cu_new, const int32_t* kv_len, void* O,
                              float* lse, void* ws, cudaStream_t s, int* err);

}  // namespace cobs
