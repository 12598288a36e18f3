// Attention of new tokens over a paged cache: workspace layout and choice of kernel.
#include <math.h>

#include "paged.h"
#include "paged_kernels.h"
#include "paged_plan.cuh"

namespace cobs {
namespace {

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// float32 stays on the CUDA cores. One token per request has at most 16 rows against each key
// and is a matter of reading the cache: warps with mma.sync take 8 x 32k keys in 171 us where the
// 128-row tcgen05 tiles take 195 us, one request at 4k keys 10.4 against 15.9 us (on the GPU), 62 ragged ones 69
// against 95 us. Everything else takes the 128-row tiles.
enum Kernel { kSimt, kChunk, kDecode };
Kernel kernel_of(const PagedDims& m) { return m.max_new == 1 ? kDecode : m.dtype == COBS_BF16 ? kChunk : kSimt; }

struct Layout {
    int workers, rec_rows;
    size_t seg_bytes, rec_bytes;
};

Layout layout_of(const PagedDims& m) {
    Layout l;
    switch (kernel_of(m)) {
        case kSimt: l.workers = paged_simt_workers(m); l.rec_rows = paged_simt_rec_rows(m); break;
        case kDecode: l.workers = paged_decode_workers(m); l.rec_rows = paged_decode_rec_rows(m); break;
        default: l.workers = paged_chunk_workers(m); l.rec_rows = paged_chunk_rec_rows(m);
    }
    l.seg_bytes = al256((size_t)l.workers * sizeof(PagedSeg));
    l.rec_bytes = (size_t)l.workers * 2 * l.rec_rows * (m.d + 2) * sizeof(float);
    return l;
}

}  // namespace

// [workers] ranges, then two records per worker (the first and the last unit of its range may be
// pieces): rec_rows x (d + 2) float32.
size_t paged_attn_workspace_bytes(const PagedDims& m) {
    const Layout l = layout_of(m);
    return l.seg_bytes + l.rec_bytes;
}

cudaError_t launch_paged_attn(const PagedDims& m, const void* Q, const void* k_cache, const void* v_cache,
                              const int32_t* block_table, const int32_t* cu_new, const int32_t* kv_len, void* O,
                              float* lse, void* ws, cudaStream_t s, int* err) {
    const Layout l = layout_of(m);
    PagedArgs a{};
    a.table = block_table; a.cu = cu_new; a.kv_len = kv_len; a.lse = lse; a.O = O; a.err = err;
    a.seg = static_cast<PagedSeg*>(ws);
    a.rec_rows = l.rec_rows;
    a.rec = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + l.seg_bytes);
    a.R = m.R; a.Hq = m.Hq; a.Hkv = m.Hkv; a.G = m.G; a.page = m.page; a.page_shift = m.page_shift;
    a.n_pages = m.n_pages; a.max_pages = m.max_pages; a.n_tokens = m.n_tokens; a.max_new = m.max_new;
    a.W = m.W; a.S = m.S;
    a.sl2 = (float)(1.4426950408889634 / sqrt((double)m.d));
    switch (kernel_of(m)) {
        case kChunk: a.lead_one = 2; a.lead_two = 3; return launch_paged_chunk(m, a, Q, k_cache, v_cache, s);
        case kDecode:
            a.lead_one = a.lead_two = 2;
            if (m.dtype == COBS_BF16) return launch_paged_decode(m, a, Q, k_cache, v_cache, s);
            return launch_paged_decode_f32(m, a, static_cast<const float*>(Q), static_cast<const float*>(k_cache),
                                           static_cast<const float*>(v_cache), s);
        default: a.lead_one = a.lead_two = 1;
    }
    return launch_paged_simt(m, a, static_cast<const float*>(Q), static_cast<const float*>(k_cache), static_cast<const float*>(v_cache), s);
}

}  // namespace cobs
