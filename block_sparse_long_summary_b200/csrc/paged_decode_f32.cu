// Attention of single new tokens over a paged cache, float32: the cache's bytes bound it, or the latency of
// one pass through the kernel; the products stay on the CUDA cores, which a matter of reading the cache
// leaves enough of.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(q . k_j / sqrt(d)),  over the keys j <= t visible at the
//   token's position t (all of them, or the last W and the first S).
//
// One CTA per SM walks its range of (unit, 64-key tile) pairs (paged_plan.cuh); a unit is one request and KV
// head, its rows the G heads of the group. Warp w takes keys 8 w .. + 7 of every tile, by itself: it copies
// them (cp.async) two tiles ahead (one for more than 8 heads), over the ends of units, and needs no barrier until the unit's
// end, where the eight warps' maxima, sums and outputs are joined through shared memory. Rows that the
// token does not see are filled with zeros by the copy. For the scores lane 4 r + q takes key r of the
// slice and every fourth 16 bytes of its row, for P V every lane takes d / 32 columns.
// 4 x 2000 keys of 8 heads, groups of 4: 29 us per call, against 55 us as a 16-row case of the chunk kernel; 8 x 32768
// keys 467 us, 0.70 of the copy bandwidth. With groups of 16 the products bound it (2 heads of 8 x 32768 keys: 325 us,
// 0.25): the heads come one after another, and each reads the slice's V from shared memory and Q through L1 again.
#include <algorithm>

#include "paged.h"
#include "paged_kernels.h"
#include "paged_plan.cuh"
#include "tma.h"

namespace cobs {
namespace {

constexpr int kWarps = 8, kT = 32 * kWarps;

constexpr int kSlice = 8, kKT = kSlice * kWarps;  // keys of a warp's slice and of a tile

template <int D, int NT>  // NT: heads, in eights
struct Cfg {
    static constexpr int kStages = NT == 1 ? 3 : 2;
    static constexpr int kTensor = kSlice * D * 4;  // a slice of K or V
    static constexpr int kStage = 2 * kTensor;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kRow = D + 4;                     // row stride of the joined outputs (no bank conflicts)
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kJoin = kWarps * kHeads * (kRow + 2) * 4;
    static constexpr size_t kSmem = kRing + kJoin;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// A warp's copies: it walks the range's units and tiles ahead of the computation.
template <int D, int NT>
struct Slices {
    using C = Cfg<D, NT>;
    const PagedArgs& a;
    const float *kc, *vc;
    PagedWalk<kKT> f;    // the unit whose slices are being copied
    bool fetching, looked;  // looked: the slice looked up last is to be copied
    int tile;               // to look up next
    int page, j;            // table entry (any value) and first key of the slice looked up last
    uint32_t ring, put;     // this warp's ring, next stage
    int warp, lane;

    __device__ __forceinline__ Slices(const PagedArgs& a_, const float* k, const float* v, const PagedStart<kKT>& s, uint32_t ring_)
        : a(a_), kc(k), vc(v), f(s.walk), fetching(s.more), looked(false), tile(s.walk.t0), page(-1), j(0), ring(ring_), put(0),
          warp(threadIdx.x >> 5), lane(threadIdx.x & 31) {}
    // the table entry of the next slice: asked for a tile before it is used
    __device__ __forceinline__ void look_up() {
        looked = false;
        if (!fetching) return;
        const int pos = f.e.pos0;
        j = f.e.key_tile(tile) * kKT + warp * kSlice;
        looked = j <= pos && (j + kSlice > f.e.lo || j < a.S) && (j >> a.page_shift) < a.max_pages;
        if (looked) page = __ldg(a.table + (size_t)f.e.r * a.max_pages + (j >> a.page_shift));
    }
    __device__ __forceinline__ void advance() {
        if (fetching && ++tile == f.t1) {
            fetching = f.next(a, 1);
            tile = f.t0;
        }
    }
    // The slice looked up, into the next stage: whole rows, the 16-byte chunks of odd rows in the other half of
    // each 128 bytes (two rows are read at once); rows the token does not see are zero.
    __device__ __forceinline__ void fetch() {
        if (looked) {
            const bool in = page >= 0 && page < a.n_pages;
            if (!in && lane == 0) report_error(a.err, kErrBadIndex);
            constexpr int kChunks = D / 4, kRows = 32 / kChunks;  // 16-byte chunks of a row, rows a warp copies at once
            const int row = lane / kChunks, col = lane % kChunks;
            const int pos = f.e.pos0, off = j & (a.page - 1);
            const size_t at = ((((size_t)(in ? page : 0) * a.Hkv + f.h) << a.page_shift) + off + row) * D + col * 4;
            const uint32_t dst = ring + put * C::kStage;
#pragma unroll
            for (int i = 0; i < kSlice; i += kRows) {
                const int r = i + row;
                const bool ok = in && visible(j + r, pos, a.W, a.S);
                const uint32_t o = dst + r * D * 4 + ((col ^ ((r & 1) << 2)) << 4);
                copy16(o, kc + at + (size_t)i * D, ok);
                copy16(o + C::kTensor, vc + at + (size_t)i * D, ok);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == C::kStages ? 0 : put + 1;
    }
    __device__ __forceinline__ void step() {
        fetch();
        advance();
        look_up();
    }
};

// The unit's result from its warps' outputs (join: [warp][head][kRow]), maxima and sums (ml: [warp][head]).
template <int D, int NT>
__device__ __forceinline__ void join_warps(const PagedArgs& a, const PagedWalk<kKT>& w, int piece, const float* join,
                                           const float2* ml) {
    using C = Cfg<D, NT>;
    const bool whole = w.whole(), empty = w.e.pos0 < 0;
    float* rec = a.rec + ((size_t)blockIdx.x * 2 + (piece == 0 ? 0 : 1)) * a.rec_rows * (D + 2);
    for (int i = threadIdx.x; i < a.G * (D / 4); i += kT) {
        const int h = i / (D / 4), c = i % (D / 4);
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) M = fmaxf(M, ml[v * C::kHeads + h].x);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            const float2 z = ml[v * C::kHeads + h];
            // (a slice of NaN scores alone has a sum and no maximum: NaN)
            const float fac = z.x == -INFINITY && z.y == 0.0f ? 0.0f : exp2_fast(z.x - M);
            const float4 x = *reinterpret_cast<const float4*>(join + (v * C::kHeads + h) * C::kRow + 4 * c);
            L = fmaf(z.y, fac, L);
            y.x = fmaf(x.x, fac, y.x);
            y.y = fmaf(x.y, fac, y.y);
            y.z = fmaf(x.z, fac, y.z);
            y.w = fmaf(x.w, fac, y.w);
        }
        if (whole) {
            const size_t orow = (size_t)w.e.row0 * a.Hq + w.h * a.G + h;
            const float inv = 1.0f / L;
            *reinterpret_cast<float4*>(static_cast<float*>(a.O) + orow * D + 4 * c) =
                empty ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
            if (a.lse && c == 0) a.lse[orow] = empty ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        } else {
            reinterpret_cast<float4*>(rec)[(size_t)c * a.rec_rows + h] = y;
            if (c == 0) reinterpret_cast<float2*>(rec + (size_t)a.rec_rows * D)[h] = make_float2(M, L);
        }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(kT, 1) paged_decode_f32_kernel(PagedArgs a, const float* Q, long long q_stride, const float* kc,
                                                                 const float* vc) {
    using C = Cfg<D, NT>;
    constexpr int CW = D / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long tmp[2 * kT / 32];
    __shared__ PagedStart<kKT> start;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    allow_merge();
    plan_start<kT, kKT>(a, 1, blockIdx.x, gridDim.x, 0, reinterpret_cast<int*>(smem), tmp, &start);
    unsigned char* ring = smem + warp * C::kStages * C::kStage;
    float* join = reinterpret_cast<float*>(smem + C::kRing);
    float2* ml = reinterpret_cast<float2*>(join + kWarps * C::kHeads * C::kRow);
    PagedWalk<kKT> w = start.walk;
    bool more = start.more;
    if (tid == 0) a.seg[blockIdx.x] = w.seg(a, start.range, blockIdx.x);
    Slices<D, NT> slices(a, kc, vc, start, smem_addr(ring));
    slices.look_up();
#pragma unroll 1
    for (int s = 0; s < C::kStages - 1; ++s) slices.step();

    uint32_t get = 0;
    int piece = 0;
    const int r = lane >> 2, q = lane & 3;
    for (; more; more = w.next(a, 1), ++piece) {
        const PagedEntry& e = w.e;
        const int pos = e.pos0;
        const float* qrow = Q + (size_t)e.row0 * q_stride + (size_t)w.h * a.G * D + 4 * q;
        float m[C::kHeads], l[C::kHeads], o[C::kHeads][CW];  // l: this lane's keys
#pragma unroll
        for (int h = 0; h < C::kHeads; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.0f;
#pragma unroll
            for (int c = 0; c < CW; ++c) o[h][c] = 0.0f;
        }
#pragma unroll 1
        for (int k = w.t0; k < w.t1; ++k) {
            slices.step();
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
            __syncwarp();
            const unsigned char* sK = ring + get * C::kStage;
            const unsigned char* sV = sK + C::kTensor;
            get = get + 1 == C::kStages ? 0 : get + 1;
            const bool see = visible(e.key_tile(k) * kKT + warp * kSlice + r, pos, a.W, a.S);
            const unsigned seen = __ballot_sync(kFull, see);
            if (seen) {
                float4 kv[D / 16];
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    kv[c] = *reinterpret_cast<const float4*>(sK + r * D * 4 + (((4 * c + q) ^ ((r & 1) << 2)) << 4));
#pragma unroll
                for (int h = 0; h < C::kHeads; ++h) {
                    if (h >= a.G) break;  // (uniform)
                    float s = 0.0f;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const float4 x = __ldg(reinterpret_cast<const float4*>(qrow + (size_t)h * D + 16 * c));
                        s = fmaf(x.w, kv[c].w, fmaf(x.z, kv[c].z, fmaf(x.y, kv[c].y, fmaf(x.x, kv[c].x, s))));
                    }
                    s += __shfl_xor_sync(kFull, s, 1);
                    s += __shfl_xor_sync(kFull, s, 2);
                    s = see ? s * a.sl2 : -INFINITY;
                    float mx = s;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                    if (mx > m[h]) {  // (uniform: every lane has the maximum)
                        const float fac = exp2_fast(m[h] - mx);
                        m[h] = mx;
                        l[h] *= fac;
#pragma unroll
                        for (int c = 0; c < CW; ++c) o[h][c] *= fac;
                    }
                    const float p = exp2_fast(s - (m[h] == -INFINITY ? 0.0f : m[h]));
                    l[h] += p;
#pragma unroll
                    for (int y = 0; y < kSlice; ++y) {
                        const float py = __shfl_sync(kFull, p, 4 * y);
                        const unsigned char* v = sV + y * D * 4;
                        if constexpr (CW == 4) {
                            const float4 x = *reinterpret_cast<const float4*>(v + ((lane ^ ((y & 1) << 2)) << 4));
                            o[h][0] = fmaf(py, x.x, o[h][0]);
                            o[h][1] = fmaf(py, x.y, o[h][1]);
                            o[h][2] = fmaf(py, x.z, o[h][2]);
                            o[h][3] = fmaf(py, x.w, o[h][3]);
                        } else {
                            const float2 x = *reinterpret_cast<const float2*>(v + (((lane >> 1) ^ ((y & 1) << 2)) << 4) + (lane & 1) * 8);
                            o[h][0] = fmaf(py, x.x, o[h][0]);
                            o[h][1] = fmaf(py, x.y, o[h][1]);
                        }
                    }
                }
            }
            __syncwarp();  // the stage has been read
        }
#pragma unroll
        for (int h = 0; h < C::kHeads; ++h) {
            float sum = l[h];  // the four lanes of a key hold the same
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(kFull, sum, d);
            float* row = join + (warp * C::kHeads + h) * C::kRow + CW * lane;
#pragma unroll
            for (int c = 0; c < CW; ++c) row[c] = o[h][c];
            if (lane == 0) ml[warp * C::kHeads + h] = make_float2(m[h], sum);
        }
        __syncthreads();
        join_warps<D, NT>(a, w, piece, join, ml);
        __syncthreads();  // before the next unit's outputs
    }
}

template <int D, int NT>
cudaError_t run(const PagedDims& m, const PagedArgs& a, const float* Q, const float* kc, const float* vc, cudaStream_t s) {
    using C = Cfg<D, NT>;
    static_assert(C::kSmem + 1024 <= 227 * 1024, "shared memory");
    static_assert((kMaxRequests + 1) * 4 <= C::kSmem, "the plan's scratch");
    static OncePerDevice once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(paged_decode_f32_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    });
    if (e != cudaSuccess) return e;
    const int workers = sm_count();
    count_launch();
    paged_decode_f32_kernel<D, NT><<<workers, kT, C::kSmem, s>>>(a, Q, m.q_stride, kc, vc);
    const cudaError_t f = cudaGetLastError();
    if (f != cudaSuccess) return f;
    return launch_paged_merge<float, D>(a, workers, m.G, s);
}

}  // namespace

cudaError_t launch_paged_decode_f32(const PagedDims& m, const PagedArgs& a, const float* Q, const float* kc, const float* vc,
                                    cudaStream_t s) {
    if (m.d == 64) return m.G <= 8 ? run<64, 1>(m, a, Q, kc, vc, s) : run<64, 2>(m, a, Q, kc, vc, s);
    return m.G <= 8 ? run<128, 1>(m, a, Q, kc, vc, s) : run<128, 2>(m, a, Q, kc, vc, s);
}

}  // namespace cobs
