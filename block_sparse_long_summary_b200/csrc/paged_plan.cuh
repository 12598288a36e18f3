// The division of a ragged batch's attention over workers, shared by the paged attention kernels.
//
// An entry is one tile of TQ consecutive new tokens of a request; a unit is an entry with one KV
// head. A unit's keys are walked in tiles of KT keys: the tiles that hold sinks, then the tiles
// from the first row's window start (or 0) to the last row's own position. All units' tiles, one
// unit after the other (entry by entry, heads within an entry), form one sequence that is cut
// into equal contiguous ranges, one per worker, so every worker has the same work whatever the
// lengths are. A unit counts `lead` tiles more than it has, in front of its own, for its start and
// end: without, a batch of many short requests beside long ones left some workers with ten times the
// units of others (62 single tokens at 1 to 16k keys on the 128-row tiles: 182 us without, 92 us with).
// The lengths live on the device, so every block finds its own range (one scan over the requests, one
// over the entries) instead of the host or a separate launch.
// A unit cut by a range boundary leaves one record per piece (the running maximum, sum and
// unnormalised output of each row), joined by the merge kernel.
#pragma once

#include <math.h>

#include "common.cuh"
#include "dims.h"
#include "paged.h"

namespace cobs {

constexpr int kErrBadLength = 3;  // lengths that contradict each other, the token rows or the table

// What a worker leaves for the merge about the boundary at which its range begins: the unit that the
// boundary cuts, if it is the first one to, and the workers whose ranges hold its pieces.
struct alignas(16) PagedSeg {
    int rows;               // rows of the unit (0: nothing to join at this boundary)
    int first, last, slot;  // workers of the pieces, and the first one's record (0 or 1)
    int row0, pos0, head, unused;  // the unit's first token row and position, its head
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
    // a unit's start and end in tiles, for one and two row tiles. us per call at (one, two):
    //   bf16 chunks     (1, 1)  (1, 2)  (2, 2)  (2, 3)  (3, 4)  (4, 6)
    //   mixed            238.0   229.4   229.8   231.4   234.6   239.9
    //   with a window    162.9   160.1   160.1   157.7   156.9   155.1     (a long chunk: 2.20 ms at each)
    //   single tokens        1       2       3       4       6
    //   62 ragged         74.9    69.0    70.8    74.1    79.4             (8 x 32k keys: 171-173 at each)
    //   with a window     24.6    23.0    23.5    24.4    24.7
    //   float32 chunks   147.8   151.5   150.1
    int lead_one, lead_two;
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
    int lead;         // a unit's start and end, in tiles
    __device__ __forceinline__ int key_tile(int k) const { return k < sT ? k : loT + (k - sT); }
    __device__ __forceinline__ int cost() const { return nt + lead; }  // places of a unit
    __device__ __forceinline__ int last_pos() const { return pos0 + n - 1; }
};

template <int KT>
__device__ __forceinline__ void entry_tiles(const PagedArgs& a, int TQ, PagedEntry& e) {
    e.lead = 2 * e.n > TQ ? a.lead_two : a.lead_one;
    const int hi = e.last_pos();
    e.lo = a.W > 0 && e.pos0 >= a.W ? e.pos0 - a.W + 1 : 0;
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
    entry_tiles<KT>(a, TQ, e);
    return e;
}

// Whether key j is visible at position t.
__device__ __forceinline__ bool visible(int j, int t, int W, int S) {
    return j <= t && (W <= 0 || t - j < W || j < S);
}

// A worker's range: its first unit and tile, and how many tiles it walks.
struct PagedRange {
    int r, i;          // entry
    int off;           // place in the entry: head * (nt + lead) + place in the unit
    int count;
    long long b0, total;  // first place, places in all
    int workers;       // that have a range: at most one per place
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

// 2^x on the special-function unit (approximate, flush-to-zero)
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// A worker's walk over the units of its range that have tiles in it.
template <int KT>
struct PagedWalk {
    PagedEntry e;
    int h, t0, t1;    // head and tiles [t0, t1) of the unit in hand
    int left;         // places after this unit's
    int row_r, n_r, L_r;
    __device__ __forceinline__ bool first(const PagedArgs& a, int TQ, const PagedRange& g) {
        left = 0;
        if (g.count == 0) return false;
        bool bad;
        request_of(a, g.r, row_r, n_r, L_r, bad);
        e = make_entry<KT>(a, g.r, g.i, TQ, row_r, n_r, L_r);
        const int unit = e.cost();
        h = g.off / unit;
        const int x = g.off - h * unit, take = min(unit - x, g.count);
        t0 = max(0, x - e.lead);
        t1 = max(0, x + take - e.lead);
        left = g.count - take;
        return t1 > t0 || next(a, TQ);
    }
    __device__ __forceinline__ bool next(const PagedArgs& a, int TQ) {
        if (left == 0) return false;
        if (++h == a.Hkv) {
            h = 0;
            int i = e.i + 1, r = e.r;
            while (i * TQ >= n_r) {
                bool bad;
                i = 0;
                if (++r >= a.R) return false;  // cannot happen: the ranges end with the last entry
                request_of(a, r, row_r, n_r, L_r, bad);
            }
            e = make_entry<KT>(a, r, i, TQ, row_r, n_r, L_r);
        }
        t0 = 0;
        t1 = min(e.nt, left - e.lead);
        left -= min(e.cost(), left);
        return t1 > 0;  // (else the range ends before the unit's tiles)
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == e.nt; }
    // what the merge has to know (after first()): the unit that worker w's boundary cuts, if it cuts one
    __device__ __forceinline__ PagedSeg seg(const PagedArgs& a, const PagedRange& g, int w) const {
        PagedSeg s{};
        if (g.count == 0 || t0 == 0 || t1 <= t0) return s;
        const long long U0 = g.b0 - t0;  // place of the unit's first tile
        s.first = worker_of(g.total, U0, g.workers);
        if (s.first != w - 1) return s;  // an earlier boundary inside this unit
        s.last = worker_of(g.total, U0 + e.nt - 1, g.workers);
        s.slot = share_of(g.total, s.first, g.workers) >= U0 - e.lead ? 0 : 1;  // the unit is that worker's first
        s.rows = e.n * a.G;
        s.row0 = e.row0;
        s.pos0 = e.pos0;
        s.head = h;
        return s;
    }
};

// What a worker starts from: its range, and its walk at the first unit.
template <int KT>
struct PagedStart {
    PagedRange range;
    PagedWalk<KT> walk;
    int more;      // whether there is a unit
    int ready;     // of the warp's attempt below
    __device__ __forceinline__ void set(const PagedArgs& a, int TQ, const PagedRange& g) {  // by one thread
        range = g;
        more = walk.first(a, TQ, g);
    }
};

// Worker w's start where there are at most 32 requests with at most kWarpEntries entries, by one warp: lane
// r looks after request r, then lane i after entries i, i + 32, ... A small call waits for these steps, and
// the warps beside it only add to what its scheduler has to issue. Returns whether the case is that one.
constexpr int kWarpEntries = 256;

template <int KT>
__device__ __forceinline__ bool plan_warp(const PagedArgs& a, int TQ, int w, int n_workers, PagedStart<KT>* out) {
    const int lane = threadIdx.x & 31;
    int row0 = 0, n = 0, L = 0;
    bool bad = false;
    if (lane < a.R) request_of(a, lane, row0, n, L, bad);
    if (bad && w == 0) report_error(a.err, kErrBadLength);
    const int mine = (n + TQ - 1) / TQ;
    int ends = mine;  // entries up to and with this request's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, ends, o);
        if (lane >= o) ends += u;
    }
    const int E = __shfl_sync(kFull, ends, 31);
    if (E > kWarpEntries) return false;
    const int begins = ends - mine;
    int r = 0, i = 0;
    long long cost = 0, inc = 0;
    auto costs = [&](int e0) {  // this lane's entry of the 32 from e0 on, and the sum up to it
        const int e = e0 + lane;
        int lo = 0;  // requests that end at or before e
#pragma unroll
        for (int step = 16; step > 0; step >>= 1) {
            const int x = __shfl_sync(kFull, ends, lo + step - 1);
            if (x <= e) lo += step;
        }
        r = min(lo, 31);
        i = e - __shfl_sync(kFull, begins, r);
        const int rr = __shfl_sync(kFull, row0, r), rn = __shfl_sync(kFull, n, r), rL = __shfl_sync(kFull, L, r);
        cost = e < E ? (long long)make_entry<KT>(a, r, i, TQ, rr, rn, rL).cost() * a.Hkv : 0;
        inc = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += u;
        }
        return __shfl_sync(kFull, inc, 31);
    };
    long long total = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += 32) total += costs(e0);
    const int n_eff = (int)min((long long)n_workers, total);
    if (w >= n_eff) {
        if (lane == 0) out->set(a, TQ, PagedRange{0, 0, 0, 0, 0, 0, 0});
        return true;
    }
    const long long b0 = share_of(total, w, n_eff), b1 = share_of(total, w + 1, n_eff);
    long long before = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += 32) {
        const long long sum = E > 32 ? costs(e0) : total;  // (the values of the only round above still stand)
        const long long at = b0 - before;
        if (at >= inc - cost && at < inc)
            out->set(a, TQ, PagedRange{r, i, (int)(at - (inc - cost)), (int)(b1 - b0), b0, total, n_eff});
        before += sum;
        if (before > b0) break;
    }
    return true;
}

// Worker w's start, for all T threads of the block; `planner` is the warp that tries alone. scratch: R + 1
// ints; tmp: 2 T / 32 values; out: shared memory, to be read after the call.
template <int T, int KT>
__device__ __forceinline__ void plan_start(const PagedArgs& a, int TQ, int w, int n_workers, int planner, int* scratch,
                                           long long* tmp, PagedStart<KT>* out) {
    const int tid = threadIdx.x;
    if (a.R <= 32) {
        if (tid >> 5 == planner) {
            const bool ok = plan_warp<KT>(a, TQ, w, n_workers, out);
            if ((tid & 31) == 0) out->ready = ok;
        }
        __syncthreads();
        if (out->ready) return;
    }
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
    if (tid == 0) scratch[0] = 0;
    __syncthreads();
    const int E = (int)base;
    auto cost_of = [&](int e, int& r, int& i) -> long long {
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
        return (long long)make_entry<KT>(a, r, i, TQ, row0, n, L).cost() * a.Hkv;
    };
    long long total = 0, cost = 0, inc = 0;
    int r = 0, i = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += T) {
        cost = e0 + tid < E ? cost_of(e0 + tid, r, i) : 0;
        long long tot;
        inc = scan(cost, tot);
        total += tot;
    }
    const int n_eff = (int)min((long long)n_workers, total);
    if (w >= n_eff) {
        if (tid == 0) out->set(a, TQ, PagedRange{0, 0, 0, 0, 0, 0, 0});
        __syncthreads();
        return;
    }
    const long long b0 = share_of(total, w, n_eff), b1 = share_of(total, w + 1, n_eff);
    long long before = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += T) {
        if (E > T) {  // else the values of the only round above still stand
            cost = e0 + tid < E ? cost_of(e0 + tid, r, i) : 0;
            long long tot;
            inc = scan(cost, tot) + before;
            before += tot;
        }
        if (b0 >= inc - cost && b0 < inc)
            out->set(a, TQ, PagedRange{r, i, (int)(b0 - (inc - cost)), (int)(b1 - b0), b0, total, n_eff});
    }
    __syncthreads();
}

// The merge may be launched (it waits for this grid's end by itself).
__device__ __forceinline__ void allow_merge() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
// worker c's range), if it is the first one inside its unit, and the unit's rows 8 y .. 8 y + 7. After
// the segment's one round trip come the pieces' maxima and sums, then their outputs without waiting on
// one another. Pieces are added in the order of the workers, 16 at a time. A small call waits for this
// kernel's every instruction (cold code and one warp per scheduler: about 20 cycles each), so what can
// be known before is left by the attention kernel.
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedSeg* seg, const float* recs, T* O, float* lse, int rec_rows,
                                                          int Hq, int G) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float2 ml[2][16][8];
    const int tid = threadIdx.x, col = tid & 7, q = tid >> 3;
    const PagedSeg s = seg[blockIdx.x + 1];
    const int row = blockIdx.y * 8 + col;
    if (blockIdx.y * 8 >= s.rows) return;
    const bool in = row < s.rows;
    constexpr int C = D / 64;  // float4 columns per thread
    const size_t size = (size_t)rec_rows * (D + 2);  // of a record
    const float* rec = recs + (size_t)s.first * 2 * size;  // the pieces' workers are neighbours
    const size_t first = s.slot ? size : 0;
    float M = -INFINITY, sum = 0.0f;
    float4 o[C];
#pragma unroll
    for (int k = 0; k < C; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int pieces = s.last - s.first + 1;
    const float* mine = rec + (in ? row * 4 : 0) + (size_t)q * 4 * rec_rows;  // this thread's first float4
    constexpr int N = 8;  // pieces in flight
    float4 v[N][C];
    auto fetch = [&](int p0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int p = min(p0 + i, pieces - 1);
#pragma unroll
            for (int k = 0; k < C; ++k)
                v[i][k] = *reinterpret_cast<const float4*>(mine + (size_t)p * 2 * size + (p ? 0 : first) + (size_t)(64 * k) * rec_rows);
        }
    };
    for (int p0 = 0, turn = 0; p0 < pieces; p0 += 16, turn ^= 1) {
        const int p = p0 + q;
        float2 x = make_float2(-INFINITY, 0.0f);
        if (in && p < pieces)
            x = reinterpret_cast<const float2*>(rec + (size_t)p * 2 * size + (p ? 0 : first) + (size_t)rec_rows * D)[row];
        fetch(p0);  // on their way with the maxima
        ml[turn][q][col] = x;
        __syncthreads();
        float nm = M;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) nm = fmaxf(nm, ml[turn][i][col].x);
        const float f0 = M == -INFINITY ? 0.0f : exp2_fast(M - nm);
        M = nm;
        sum *= f0;
#pragma unroll
        for (int k = 0; k < C; ++k) o[k] = make_float4(o[k].x * f0, o[k].y * f0, o[k].z * f0, o[k].w * f0);
        const int n = min(16, pieces - p0);
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += N) {
            if (i0 > 0) fetch(p0 + i0);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 y = ml[turn][i0 + i][col];
                // (nothing seen, or no piece: neither maximum nor sum; NaN scores alone: a sum and no maximum)
                const bool use = y.x != -INFINITY || y.y != 0.0f;
                const float g = use ? exp2_fast(y.x - M) : 0.0f;
                sum = fmaf(y.y, g, sum);
#pragma unroll
                for (int k = 0; k < C; ++k)
                    if (use) {
                        o[k].x = fmaf(v[i][k].x, g, o[k].x);
                        o[k].y = fmaf(v[i][k].y, g, o[k].y);
                        o[k].z = fmaf(v[i][k].z, g, o[k].z);
                        o[k].w = fmaf(v[i][k].w, g, o[k].w);
                    }
            }
        }
    }
    if (!in) return;
    const int tok = row / G;
    const size_t orow = (size_t)(s.row0 + tok) * Hq + s.head * G + row - tok * G;
    const bool empty = s.pos0 + tok < 0;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int k = 0; k < C; ++k) {
        T* out = O + orow * D + 4 * (q + 16 * k);
        float v[4] = {o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv};
        if (empty) v[0] = v[1] = v[2] = v[3] = 0.0f;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        } else {
            *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    if (lse && q == 0) lse[orow] = empty ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

// The merge after an attention grid of `workers` ranges whose units have at most `rows` rows, as its
// programmatic dependent: that grid allows it from its own start, so that the launch is over with when
// the records are complete (one token at 4k keys 14.3 -> 12.3 us per call; allowed at the grid's end it
// was slower than a plain launch). It asks for the attention grid's division of the SM's memory, so that
// an SM need not change it between the two.
template <typename T, int D>
cudaError_t launch_paged_merge(const PagedArgs& a, int workers, int rows, cudaStream_t s) {
    if (workers < 2) return cudaSuccess;
    static OncePerDevice once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(paged_merge_kernel<T, D>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    count_launch();
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(workers - 1, (rows + 7) / 8);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D>, (const PagedSeg*)a.seg, (const float*)a.rec, static_cast<T*>(a.O), a.lse,
                              a.rec_rows, a.Hq, a.G);
}

}  // namespace cobs
