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

struct PagedArgs {
    const int32_t* table;   // [R, max_pages]
    const int32_t* cu;      // [R + 1]
    const int32_t* kv_len;  // [R]
    float* lse;             // [n_tokens, Hq] or null
    void* O;                // [n_tokens, Hq, d]
    float* rec;             // [workers][2][rec_rows][d + 4]: output, then running maximum (log2 units) and sum
    int4* seg;              // [workers]: entry (request, tile of tokens), offset in the entry, tiles walked
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
};

// Block-wide inclusive scan of one value per thread (T threads); tmp: T / 32 + 1 values.
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
    __syncthreads();
    return v + before;
}

// The ranges of workers w0 .. w0 + NW - 1 of n_workers, by all T threads of the block.
// scratch: R + 1 ints; tmp: T / 32 long long; out: NW ranges (shared memory).
template <int T, int KT, int NW>
__device__ __forceinline__ void plan_ranges(const PagedArgs& a, int TQ, int w0, int n_workers, int* scratch,
                                            long long* tmp, PagedRange* out) {
    const int tid = threadIdx.x;
    // entries before each request
    long long base = 0;
    for (int r0 = 0; r0 < a.R; r0 += T) {
        const int r = r0 + tid;
        int row0, n = 0, L;
        bool bad = false;
        if (r < a.R) request_of(a, r, row0, n, L, bad);
        if (bad && w0 == 0) report_error(a.err, kErrBadLength);
        long long tot;
        const long long inc = block_scan<T>((n + TQ - 1) / TQ, tmp, tot);
        if (r < a.R) scratch[r + 1] = (int)(base + inc);
        base += tot;
    }
    if (tid == 0) scratch[0] = 0;
    if (tid < NW) out[tid] = PagedRange{0, 0, 0, 0};
    __syncthreads();
    const int E = (int)base;
    auto cost_of = [&](int e, int& r, int& i) -> int {
        int lo = 0, hi = a.R - 1;  // the last request whose first entry is <= e
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (scratch[mid] <= e) lo = mid; else hi = mid - 1;
        }
        // (requests without entries share their successor's prefix: the last one of equals holds e)
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
        inc = block_scan<T>(cost, tmp, tot);
        total += tot;
    }
    long long before = 0;
    for (int e0 = 0; e0 < E; e0 += T) {
        if (E > T) {  // else the values of the only round above still stand
            cost = e0 + tid < E ? cost_of(e0 + tid, r, i) : 0;
            long long tot;
            inc = block_scan<T>(cost, tmp, tot) + before;
            before += tot;
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const long long b0 = total * (w0 + w) / n_workers, b1 = total * (w0 + w + 1) / n_workers;
            if (b1 > b0 && b0 >= inc - cost && b0 < inc)
                out[w] = PagedRange{r, i, (int)(b0 - (inc - cost)), (int)(b1 - b0)};
        }
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
// worker c's range) if it is the first one inside its unit; the unit's rows 4 y + warp, then every
// 4 gridDim.y, one warp each. Lane i looks after piece i (32 at a time): the pieces' tile counts,
// maxima and sums come in one round trip each, then the outputs without waiting on one another.
// Pieces lie in the order of the workers, so the order of the sums is fixed.
template <typename T, int D, int KT>
__global__ void __launch_bounds__(128) paged_merge_kernel(PagedArgs a, int TQ, int n_workers, int rec_rows) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 s = a.seg[c], before = a.seg[c - 1];
    if (s.w == 0) return;
    int row_r, n_r, L_r;
    bool bad;
    request_of(a, s.x, row_r, n_r, L_r, bad);
    const PagedEntry e = make_entry<KT>(a, s.x, s.y, TQ, row_r, n_r, L_r);
    const int h = s.z / e.nt, t0 = s.z - h * e.nt;
    if (t0 == 0) return;
    // the last worker before with tiles (some have none where there are fewer tiles than workers)
    int p = c - 1;
    int4 q = before;
    while (p > 0 && q.w == 0) q = a.seg[--p];
    const bool same = q.x == s.x && q.y == s.y && q.z / e.nt == h;
    if (same && q.z - h * e.nt > 0) return;  // an earlier boundary inside this unit
    constexpr int C = D / 32;
    for (int row = blockIdx.y * 4 + warp; row < e.n * a.G; row += gridDim.y * 4) {
        float M = -INFINITY, l = 0.0f, o[C];
#pragma unroll
        for (int k = 0; k < C; ++k) o[k] = 0.0f;
        int covered = t0;      // tiles of the unit in the pieces up to worker w0 - 1 (the first one's end at t0)
        for (int w0 = p; w0 < n_workers; w0 += 32) {
            const int w = w0 + lane;
            const int tiles = w > p && w < n_workers ? a.seg[w].w : 0;
            int inc = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(kFull, inc, d);
                if (lane >= d) inc += u;
            }
            // a piece: the first worker, and those whose range begins before the unit's end
            const bool piece = w == p || (tiles > 0 && covered + inc - tiles < e.nt);
            const float* rec = a.rec + (((size_t)w * 2 + (w == p && !same ? 1 : 0)) * rec_rows + row) * (D + 4);
            const float m1 = piece ? rec[D] : -INFINITY, l1 = piece ? rec[D + 1] : 0.0f;
            float nm = m1;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(kFull, nm, d));
            nm = fmaxf(nm, M);
            const float f0 = M == -INFINITY ? 0.0f : exp2f(M - nm);
            // (a piece of NaN scores alone has a sum and no maximum: NaN then)
            const float f1 = m1 == -INFINITY && l1 == 0.0f ? 0.0f : exp2f(m1 - nm);
            float sum = l1 * f1;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
            l = l * f0 + sum;
#pragma unroll
            for (int k = 0; k < C; ++k) o[k] *= f0;
            M = nm;
            const unsigned who = __ballot_sync(kFull, piece && f1 != 0.0f);  // (NaN counts)
            const int first = __ffs(who) - 1, last = 31 - __clz(who);
            if (who) {
#pragma unroll 8
                for (int i = first; i <= last; ++i) {
                    const float f = __shfl_sync(kFull, f1, i);
                    if (!(who >> i & 1u)) continue;
                    const float* src = a.rec + (((size_t)(w0 + i) * 2 + (w0 + i == p && !same ? 1 : 0)) * rec_rows + row) * (D + 4) + lane * C;
                    float v[C];
                    if constexpr (C == 4) {
                        *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
                    } else {
                        *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
                    }
#pragma unroll
                    for (int k = 0; k < C; ++k) o[k] = fmaf(v[k], f, o[k]);
                }
            }
            covered += __shfl_sync(kFull, inc, 31);
            if (covered >= e.nt) break;
        }
        const int tok = row / a.G;
        const size_t orow = (size_t)(e.row0 + tok) * a.Hq + h * a.G + row % a.G;
        const bool empty = e.pos0 + tok < 0;
        const float inv = 1.0f / l;
#pragma unroll
        for (int k = 0; k < C; ++k)
            Elem<T>::store(static_cast<T*>(a.O) + orow * D + lane * C + k, empty ? 0.0f : o[k] * inv);
        if (a.lse && lane == 0) a.lse[orow] = empty ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
    }
}

// The merge after an attention grid of `workers` ranges, as its programmatic dependent (its launch
// overlaps the grid's tail).
template <typename T, int D, int KT>
cudaError_t launch_paged_merge(const PagedArgs& a, int TQ, int workers, int rec_rows, cudaStream_t s) {
    if (workers < 2) return cudaSuccess;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(workers - 1, (rec_rows + 15) / 16);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D, KT>, a, TQ, workers, rec_rows);
}

}  // namespace cobs
