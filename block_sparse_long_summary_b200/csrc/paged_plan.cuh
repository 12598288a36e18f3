// The division of a ragged batch's attention over workers, shared by the paged attention kernels.
//
// An entry is one tile of TQ consecutive new tokens of a request; a unit is an entry with one KV
// head. A unit's keys are walked in tiles of KT keys: the tiles that hold sinks, then the tiles
// from the first row's window start (or 0) to the last row's own position. All units' tiles, one
// unit after the other (entry by entry, heads within an entry), form one sequence that is cut
// into equal contiguous ranges, one per worker, so every worker walks the same number of tiles
// whatever the lengths are. The lengths live on the device, so every block finds its own range
// (one scan over the requests, one over the entries) instead of the host or a separate launch.
// A unit cut by a range boundary leaves one record per piece (the running maximum, sum and
// unnormalised output of each row), joined by the merge kernel.
#pragma once

#include <math.h>

#include "common.cuh"
#include "dims.h"

namespace cobs {

constexpr int kErrBadLength = 3;  // lengths that contradict each other, the token rows or the table

// What a worker leaves for the merge: its range in the sequence of tiles and the unit it begins in.
struct alignas(16) PagedSeg {
    long long b0, total;         // first tile, tiles in all
    int count, head, t0, nt;     // tiles walked; the first unit's head, first tile and tiles
    int row0, n, pos0, unused;   // the first unit's first token row, tokens, first position
};

struct PagedArgs {
    const int32_t* table;   // [R, max_pages]
    const int32_t* cu;      // [R + 1]
    const int32_t* kv_len;  // [R]
    float* lse;             // [n_tokens, Hq] or null
    void* O;                // [n_tokens, Hq, d]
    float* rec;             // [workers][2] records: [d / 4][rec_rows][4] output (a warp's rows are contiguous),
                            // then [rec_rows][2] running maximum (log2 units) and sum
    PagedSeg* seg;          // [workers]
    int rec_rows;
    int* err;
    int R, Hq, Hkv, G, page, page_shift, n_pages, max_pages, n_tokens, max_new, W, S;
    float sl2;              // log2(e) / sqrt(d)
};

// Request r: first token row, new tokens, keys. A request whose lengths cannot be right is left out.
__device__ __forceinline__ void request_of(const PagedArgs& a, int r, int& row0, int& n, int& L, bool& bad) {
    row0 = __ldg(a.cu + r);
    n = __ldg(a.cu + r + 1) - row0;
    L = __ldg(a.kv_len + r);
    bad = row0 < 0 || n < 0 || row0 > a.n_tokens || n > a.n_tokens - row0 || n > a.max_new || L < 0 ||
          (long long)L > (long long)a.max_pages * a.page;
    if (bad) n = 0;
}

// One entry: its token rows, positions and key tiles.
struct PagedEntry {
    int r, i;         // request, tile of tokens
    int row0, n;      // first token row, tokens
    int pos0;         // position of the first token (negative: keys shorter than the new tokens)
    int nt;           // key tiles (at least 1: a tile that no row sees still writes the empty result)
    int sT, loT;      // leading sink tiles, first window tile
    int lo;           // first key of the first row's window
    __device__ __forceinline__ int key_tile(int k) const { return k < sT ? k : loT + (k - sT); }
    __device__ __forceinline__ int last_pos() const { return pos0 + n - 1; }
};

template <int KT>
__device__ __forceinline__ void entry_tiles(const PagedArgs& a, PagedEntry& e) {
    const int hi = e.last_pos();
    e.lo = a.W > 0 ? max(0, e.pos0 - a.W + 1) : 0;
    e.loT = e.lo / KT;
    e.sT = min((min(a.S, e.lo) + KT - 1) / KT, e.loT);
    e.nt = hi < 0 ? 1 : e.sT + hi / KT - e.loT + 1;
}

template <int KT>
__device__ __forceinline__ PagedEntry make_entry(const PagedArgs& a, int r, int i, int TQ, int row0, int n, int L) {
    PagedEntry e;
    e.r = r;
    e.i = i;
    e.row0 = row0 + i * TQ;
    e.n = min(TQ, n - i * TQ);
    e.pos0 = L - n + i * TQ;
    entry_tiles<KT>(a, e);
    return e;
}

// Whether key j is visible at position t.
__device__ __forceinline__ bool visible(int j, int t, int W, int S) {
    return j <= t && (W <= 0 || t - j < W || j < S);
}

// A worker's range: its first unit and tile, and how many tiles it walks.
struct PagedRange {
    int r, i;          // entry
    int off;           // tiles of the entry before it: head * nt + tile
    int count;
    long long b0, total;
};

// total * w / n without a 64-bit division where the product is small
__device__ __forceinline__ long long share_of(long long total, int w, int n) {
    const unsigned long long x = (unsigned long long)total * (unsigned)w;
    return x >> 32 ? (long long)(x / (unsigned)n) : (long long)((uint32_t)x / (uint32_t)n);
}
// the worker whose range holds tile x: ceil((x + 1) n / total) - 1
__device__ __forceinline__ int worker_of(long long total, long long x, int n) {
    const unsigned long long y = (unsigned long long)(x + 1) * (unsigned)n + (unsigned long long)total - 1;
    return (int)((y | (unsigned long long)total) >> 32 ? y / (unsigned long long)total : (uint32_t)y / (uint32_t)total) - 1;
}

// Block-wide inclusive scan of one value per thread (T threads); tmp: T / 32 values, not the ones of the
// scan just before.
template <int T>
__device__ __forceinline__ long long block_scan(long long v, long long* tmp, long long& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) tmp[w] = v;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < T / 32; ++k) {
        const long long x = tmp[k];
        if (k < w) before += x;
        all += x;
    }
    total = all;
    return v + before;
}

// Worker w's range where every one of at most 32 requests is one entry: lane r of each warp looks after
// request r, so no warp waits for another (a small call spends most of its time on such steps).
// Returns whether the case is that one.
template <int KT>
__device__ __forceinline__ bool plan_small(const PagedArgs& a, int TQ, int w, int n_workers, PagedRange& out) {
    if (a.R > 32) return false;
    const int lane = threadIdx.x & 31;
    int row0 = 0, n = 0, L = 0;
    bool bad = false;
    if (lane < a.R) request_of(a, lane, row0, n, L, bad);
    if (__any_sync(kFull, n > TQ)) return false;
    if (bad && w == 0) report_error(a.err, kErrBadLength);
    const long long cost = n > 0 ? (long long)make_entry<KT>(a, lane, 0, TQ, row0, n, L).nt * a.Hkv : 0;
    long long inc = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += u;
    }
    const long long total = __shfl_sync(kFull, inc, 31);
    const long long b0 = share_of(total, w, n_workers), b1 = share_of(total, w + 1, n_workers);
    const unsigned at = __ballot_sync(kFull, b0 >= inc - cost && b0 < inc);
    out = PagedRange{0, 0, 0, 0, b0, total};
    if (b1 > b0) {
        out.r = __ffs(at) - 1;
        out.off = (int)(b0 - __shfl_sync(kFull, inc - cost, out.r));
        out.count = (int)(b1 - b0);
    }
    return true;
}

// Worker w's range, by all T threads of the block. scratch: R + 1 ints; tmp: 2 T / 32 values.
template <int T, int KT>
__device__ __forceinline__ void plan_range(const PagedArgs& a, int TQ, int w, int n_workers, int* scratch,
                                           long long* tmp, PagedRange* out) {
    PagedRange small;
    if (plan_small<KT>(a, TQ, w, n_workers, small)) {
        if (threadIdx.x == 0) *out = small;
        __syncthreads();
        return;
    }
    const int tid = threadIdx.x;
    int turn = 0;  // the scans' halves of tmp
    auto scan = [&](long long v, long long& tot) { return block_scan<T>(v, tmp + (turn ^= 1) * (T / 32), tot); };
    // entries before each request
    long long base = 0;
    for (int r0 = 0; r0 < a.R; r0 += T) {
        const int r = r0 + tid;
        int row0, n = 0, L;
        bool bad = false;
        if (r < a.R) request_of(a, r, row0, n, L, bad);
        if (bad && w == 0) report_error(a.err, kErrBadLength);
        long long tot;
        const long long inc = scan((n + TQ - 1) / TQ, tot);
        if (r < a.R) scratch[r + 1] = (int)(base + inc);
        base += tot;
    }
    if (tid == 0) {
        scratch[0] = 0;
        *out = PagedRange{0, 0, 0, 0, 0, 0};
    }
    __syncthreads();
    const int E = (int)base;
    auto cost_of = [&](int e, int& r, int& i) -> int {
        int lo = 0, hi = a.R - 1;  // the last request whose first entry is <= e
        while (lo < hi) {          // (requests without entries share their successor's number)
            const int mid = (lo + hi + 1) >> 1;
            if (scratch[mid] <= e) lo = mid; else hi = mid - 1;
        }
        int row0, n, L;
        bool bad;
        request_of(a, lo, row0, n, L, bad);
        r = lo;
        i = e - scratch[lo];
        return make_entry<KT>(a, r, i, TQ, row0, n, L).nt * a.Hkv;
    };
    long long total = 0;
    int r = 0, i = 0, cost = 0;
    long long inc = 0;
    for (int e0 = 0; e0 < E; e0 += T) {
        cost = e0 + tid < E ? cost_of(e0 + tid, r, i) : 0;
        long long tot;
        inc = scan(cost, tot);
        total += tot;
    }
    const long long b0 = share_of(total, w, n_workers), b1 = share_of(total, w + 1, n_workers);
    long long before = 0;
    for (int e0 = 0; e0 < E; e0 += T) {
        if (E > T) {  // else the values of the only round above still stand
            cost = e0 + tid < E ? cost_of(e0 + tid, r, i) : 0;
            long long tot;
            inc = scan(cost, tot) + before;
            before += tot;
        }
        if (b1 > b0 && b0 >= inc - cost && b0 < inc)
            *out = PagedRange{r, i, (int)(b0 - (inc - cost)), (int)(b1 - b0), b0, total};
    }
    __syncthreads();
}

// A worker's walk over the units of its range.
template <int KT>
struct PagedWalk {
    PagedEntry e;
    int h, t0, t1;    // head and tiles [t0, t1) of the unit in hand
    int left;         // tiles after this unit's
    int row_r, n_r, L_r;
    __device__ __forceinline__ void set(const PagedArgs& a, int TQ) {
        e = make_entry<KT>(a, e.r, e.i, TQ, row_r, n_r, L_r);
    }
    __device__ __forceinline__ bool first(const PagedArgs& a, int TQ, const PagedRange& g) {
        if (g.count == 0) return false;
        bool bad;
        e.r = g.r;
        e.i = g.i;
        request_of(a, g.r, row_r, n_r, L_r, bad);
        set(a, TQ);
        h = g.off / e.nt;
        t0 = g.off - h * e.nt;
        t1 = min(e.nt, t0 + g.count);
        left = g.count - (t1 - t0);
        return true;
    }
    __device__ __forceinline__ bool next(const PagedArgs& a, int TQ) {
        if (left == 0) return false;
        if (++h == a.Hkv) {
            h = 0;
            ++e.i;
            while (e.i * TQ >= n_r) {
                bool bad;
                e.i = 0;
                if (++e.r >= a.R) return false;  // cannot happen: the ranges end with the last entry
                request_of(a, e.r, row_r, n_r, L_r, bad);
            }
            set(a, TQ);
        }
        t0 = 0;
        t1 = min(e.nt, left);
        left -= t1;
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == e.nt; }
    // what the merge has to know (after first(); count 0: no range)
    __device__ __forceinline__ PagedSeg seg(const PagedRange& g) const {
        if (g.count == 0) return PagedSeg{g.b0, g.total, 0, 0, 0, 0, 0, 0, 0, 0};
        return PagedSeg{g.b0, g.total, g.count, h, t0, e.nt, e.row0, e.n, e.pos0, 0};
    }
};

// Page that holds key tokens [j, j + page): -1 behind the table, or (reported) outside the cache.
__device__ __forceinline__ int page_of(const PagedArgs& a, int r, int slot, bool needed) {
    if (slot >= a.max_pages) return -1;
    const int p = __ldg(a.table + (size_t)r * a.max_pages + slot);
    if (p < 0 || p >= a.n_pages) {
        if (needed) report_error(a.err, kErrBadIndex);
        return -1;
    }
    return p;
}

// Joins the records of every unit that range boundaries cut. Block (c, y): boundary c (the start of
// worker c's range) if it is the first one inside its unit, and the unit's rows 8 y .. 8 y + 7.
// Which workers hold the pieces follows from the equal division alone, so after the segment's one
// round trip come the pieces' maxima and sums, then their outputs without waiting on one another.
// Pieces are added in the order of the workers.
constexpr int kMaxWorkers = 512;

template <typename T, int D, int KT>
__global__ void __launch_bounds__(128) paged_merge_kernel(PagedArgs a, int n_workers) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float2 ml[kMaxWorkers][8];
    const int c = blockIdx.x + 1, tid = threadIdx.x;
    const PagedSeg s = a.seg[c];
    const int row = blockIdx.y * 8 + (tid & 7), q = tid >> 3;
    if (s.count == 0 || s.t0 == 0 || blockIdx.y * 8 >= s.n * a.G) return;
    const long long U0 = s.b0 - s.t0, U1 = U0 + s.nt;
    const int f = worker_of(s.total, U0, n_workers), l = worker_of(s.total, U1 - 1, n_workers);
    if (worker_of(s.total, s.b0 - 1, n_workers) != f) return;  // an earlier boundary inside this unit
    const bool begins = share_of(s.total, f, n_workers) == U0;  // the first piece begins its worker's range
    const int rows = a.rec_rows;
    const size_t size = (size_t)rows * (D + 2);
    auto record = [&](int w) { return a.rec + ((size_t)w * 2 + (w == f && !begins ? 1 : 0)) * size; };
    for (int w = f + q; w <= l; w += 16) {
        const bool some = share_of(s.total, w + 1, n_workers) > share_of(s.total, w, n_workers);
        ml[w - f][tid & 7] = some && row < s.n * a.G ? reinterpret_cast<const float2*>(record(w) + (size_t)rows * D)[row]
                                                    : make_float2(-INFINITY, 0.0f);
    }
    __syncthreads();
    if (row >= s.n * a.G) return;
    float M = -INFINITY;
    for (int w = 0; w <= l - f; ++w) M = fmaxf(M, ml[w][tid & 7].x);
    constexpr int C = D / 64;  // float4 columns per thread
    float sum = 0.0f;
    float4 o[C];
#pragma unroll
    for (int k = 0; k < C; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int w = 0; w <= l - f; ++w) {
        const float2 x = ml[w][tid & 7];
        if (x.x == -INFINITY && x.y == 0.0f) continue;
        const float g = exp2f(x.x - M);  // (a piece of NaN scores alone has a sum and no maximum: NaN)
        sum = fmaf(x.y, g, sum);
        const float4* v = reinterpret_cast<const float4*>(record(f + w)) + row;
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const float4 y = v[(size_t)(q + 16 * k) * rows];
            o[k].x = fmaf(y.x, g, o[k].x);
            o[k].y = fmaf(y.y, g, o[k].y);
            o[k].z = fmaf(y.z, g, o[k].z);
            o[k].w = fmaf(y.w, g, o[k].w);
        }
    }
    const int tok = row / a.G;
    const size_t orow = (size_t)(s.row0 + tok) * a.Hq + s.head * a.G + row - tok * a.G;
    const bool empty = s.pos0 + tok < 0;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int k = 0; k < C; ++k) {
        T* out = static_cast<T*>(a.O) + orow * D + 4 * (q + 16 * k);
        float v[4] = {o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv};
        if (empty) v[0] = v[1] = v[2] = v[3] = 0.0f;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        } else {
            *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    if (a.lse && q == 0) a.lse[orow] = empty ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

// The merge after an attention grid of `workers` ranges whose units have at most `rows` rows, as its
// programmatic dependent (its launch overlaps the grid's tail).
template <typename T, int D, int KT>
cudaError_t launch_paged_merge(const PagedArgs& a, int workers, int rows, cudaStream_t s) {
    if (workers < 2) return cudaSuccess;
    if (workers > kMaxWorkers) return cudaErrorInvalidValue;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(workers - 1, (rows + 7) / 8);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D, KT>, a, workers);
}

}  // namespace cobs
