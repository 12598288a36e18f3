// Block tables and slot maps from request lengths, and the append of new keys and values.
#include <algorithm>

#include "common.cuh"
#include "dims.h"
#include "paged.h"
#include "paged_plan.cuh"
#include "tma.h"

namespace cobs {
namespace {

constexpr int kTT = 512;
constexpr int tables_smem(int R) { return (2 * R + 1) * (int)sizeof(int); }

struct TableArgs {
    const int32_t *cached, *fresh, *free_pages, *free_count;
    int32_t *table, *cu, *kv_len, *slots, *counts;
    int* err;
    int R, n_free, n_pages, max_pages, page_shift, n_tokens, max_new;
};

// Every block scans the requests' new tokens and new pages (two running sums, kept in shared
// memory), then takes every gridDim.x-th run of token rows: a row finds its request by bisection,
// its page in the table (pages that were open before) or on the free stack (pages this call
// hands out, whose number is the request's running sum plus the page's place), and the row that
// opens a page writes its table entry. So no block reads what another writes and one launch does.
// Launch-latency bound: one round trip for the lengths, the scan, one for the pages (3.8 us for 256
// requests as for 32768 token rows).
__global__ void __launch_bounds__(kTT) paged_tables_kernel(TableArgs a) {
    extern __shared__ int sh[];
    int* s_tok = sh;               // [R + 1] tokens before each request
    int* s_pg = sh + a.R + 1;      // [R] pages handed out before each request, less its open pages
    __shared__ long long tmp[2][kTT / 32];
    const int tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    const int P = 1 << a.page_shift;
    const int have = min(max(*a.free_count, 0), a.n_free);
    long long tok = 0, pages = 0;
    for (int r0 = 0; r0 < a.R; r0 += kTT) {
        const int r = r0 + tid;
        int c = 0, n = 0;
        if (r < a.R) {
            c = a.cached[r];
            n = a.fresh[r];
            if (c < 0 || n < 0 || n > a.max_new || (long long)c + n > (long long)a.max_pages * P) {
                if (lead) report_error(a.err, kErrBadLength);
                c = n = 0;
            }
        }
        // tokens before each request, then the pages taken before it, which depend on how many of the tokens have a
        // row; a request counts at most one token more than there are rows
        n = min(n, a.n_tokens + 1);
        long long all;
        long long inc = block_scan<kTT>(n, tmp[0], all);
        const long long before = tok + inc - n;
        const int fit = (int)min((long long)n, max(0ll, a.n_tokens - before));  // more tokens than rows: cut off
        if (fit < n && lead) report_error(a.err, kErrBadLength);
        const int open = (c + P - 1) >> a.page_shift, end = (int)(((long long)c + fit + P - 1) >> a.page_shift);
        long long taken;
        const long long pinc = block_scan<kTT>(end - open, tmp[1], taken);
        if (r < a.R) {
            s_tok[r] = (int)min(before, (long long)a.n_tokens);
            s_pg[r] = (int)(pages + pinc - (end - open)) - open;
            if (lead) {
                a.cu[r] = s_tok[r];
                a.kv_len[r] = c + fit;
            }
        }
        tok += all;
        pages += taken;
    }
    const int total = (int)min(tok, (long long)a.n_tokens);
    if (lead && tid == 0) {
        a.cu[a.R] = total;
        a.counts[0] = total;
        a.counts[1] = (int)pages;
        a.counts[2] = (int)max(0ll, have - pages);
        a.counts[3] = (int)max(0ll, pages - have);
    }
    __syncthreads();
    for (int t = blockIdx.x * kTT + tid; t < a.n_tokens; t += gridDim.x * kTT) {
        int slot = -1;
        if (t < total) {
            int lo = 0, hi = a.R - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_tok[mid] <= t) lo = mid; else hi = mid - 1;
            }
            const int c = a.cached[lo], pos = c + t - s_tok[lo], j = pos >> a.page_shift;
            const int open = (c + P - 1) >> a.page_shift;
            int32_t* entry = a.table + (size_t)lo * a.max_pages + j;
            int page;
            if (j < open) {
                page = *entry;
            } else {
                const int at = have - 1 - (s_pg[lo] + j);
                page = at >= 0 ? a.free_pages[at] : -1;
            }
            if (page < -1 || page >= a.n_pages) {
                report_error(a.err, kErrBadIndex);
                page = -1;
            }
            if (j >= open && (pos & (P - 1)) == 0) *entry = page;
            if (page >= 0) slot = (page << a.page_shift) + (pos & (P - 1));
        }
        a.slots[t] = slot;
    }
}

// HBM-bound for long prompts (20000 tokens x 8 heads of 128: 164 MB in 30.7 us a call, 0.81 of the copy rate), one
// launch for single tokens (2.0 us). One 16-byte chunk of K and of V per thread and step, so that a head's
// row is one run on both sides; `per` chunks in a token's row of all heads.
__global__ void __launch_bounds__(256) paged_append_kernel(const uint4* K, const uint4* V, const int32_t* slots,
                                                           uint4* kc, uint4* vc, long long stride, int per, int per_head,
                                                           int page_shift, int Hkv, int n_tokens, long long n_slots,
                                                           int* err) {
    const long long n = (long long)n_tokens * per;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const int t = (int)(i / per), c = (int)(i - (long long)t * per);
        const int slot = slots[t];
        if (slot < 0) continue;
        if (slot >= n_slots) {
            if (c == 0) report_error(err, kErrBadIndex);
            continue;
        }
        const int h = c / per_head, page = slot >> page_shift, off = slot & ((1 << page_shift) - 1);
        const size_t dst = ((((size_t)page * Hkv + h) << page_shift) + off) * per_head + (c - h * per_head);
        const uint4 k = K[(size_t)t * stride + c], v = V[(size_t)t * stride + c];
        kc[dst] = k;
        vc[dst] = v;
    }
}

}  // namespace

cudaError_t launch_paged_tables(const PagedDims& m, const int32_t* cached_len, const int32_t* new_len,
                                const int32_t* free_pages, int n_free, const int32_t* free_count,
                                int32_t* block_table, int32_t* cu_new, int32_t* kv_len, int32_t* slot_map,
                                int32_t* counts, cudaStream_t s, int* err) {
    TableArgs a{};
    a.cached = cached_len; a.fresh = new_len; a.free_pages = free_pages; a.free_count = free_count;
    a.table = block_table; a.cu = cu_new; a.kv_len = kv_len; a.slots = slot_map; a.counts = counts; a.err = err;
    a.R = m.R; a.n_free = n_free; a.n_pages = m.n_pages; a.max_pages = m.max_pages; a.page_shift = m.page_shift;
    a.n_tokens = m.n_tokens; a.max_new = m.max_new;
    static OncePerDevice once;  // (the largest call's limit: a call's own would be lowered by another thread's)
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tables_smem(kMaxRequests));
    });
    if (e != cudaSuccess) return e;
    const int blocks = std::max(1, std::min((m.n_tokens + kTT - 1) / kTT, sm_count()));
    count_launch();
    paged_tables_kernel<<<blocks, kTT, tables_smem(m.R), s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedDims& m, const void* K, const void* V, const int32_t* slot_map,
                                void* k_cache, void* v_cache, cudaStream_t s, int* err) {
    const int per_head = (int)(m.d * m.elem() / 16), per = per_head * m.Hkv;
    const long long n = (long long)m.n_tokens * per;
    const int blocks = (int)std::min<long long>((n + 255) / 256, (long long)sm_count() * 8);
    count_launch();
    paged_append_kernel<<<blocks, 256, 0, s>>>(
        static_cast<const uint4*>(K), static_cast<const uint4*>(V), slot_map, static_cast<uint4*>(k_cache),
        static_cast<uint4*>(v_cache), m.kv_stride * (long long)m.elem() / 16, per, per_head, m.page_shift, m.Hkv,
        m.n_tokens, (long long)m.n_pages * m.page, err);
    return cudaGetLastError();
}

}  // namespace cobs
