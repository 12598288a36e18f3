// Attention of single new tokens over a paged cache, bf16: every visible key and value is read once, so
// the cache's bytes bound it (long contexts), or the latency of one pass through the kernel (short ones).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(q . k_j / sqrt(d)),  over the keys j <= t visible at the
//   token's position t (all of them, or the last W and the first S).
//
// One CTA per SM walks its range of (unit, 128-key tile) pairs (paged_plan.cuh); a unit is one request
// and KV head, its rows the G heads of the group. Warp w takes keys 16 w .. + 15 of every tile, by
// itself: it copies them (cp.async, 16 bytes a lane, into the 128-byte swizzle) two tiles ahead (one for
// more than 8 heads a group), over the ends of units, and needs no barrier until the unit's end, where the eight warps'
// maxima, sums and outputs are joined through shared memory. Rows that the token does not see are
// filled with zeros by the copy, so nothing they hold gets in.
// A warp's step is transposed: S^T = K Q^T with the keys as the 16 rows of mma.sync m16n8k16 and the
// heads as its columns, then O^T += V^T P^T. With at most 16 heads there are not the 128 rows of a
// tcgen05 tile, and the tensor pipe is far from being the bound: a 64 KB tile takes the eight warps
// about a third of the time its bytes take to arrive.
#include <algorithm>

#include "paged.h"
#include "paged_kernels.h"
#include "paged_plan.cuh"
#include "tma.h"

namespace cobs {
namespace {

constexpr int kWarps = 8, kT = 32 * kWarps;
constexpr int kKT = 128, kSlice = kKT / kWarps;  // keys of a tile and of a warp's slice of it

template <int D, int NT>  // NT: 8-head columns
struct Cfg {
    static constexpr int kStages = NT == 1 ? 3 : 2;
    static constexpr int kHalf = kSlice * 128;             // 16 rows of 64 columns
    static constexpr int kTensor = D / 64 * kHalf;         // a slice of K or V
    static constexpr int kStage = 2 * kTensor;
    static constexpr int kRow = D + 4;                     // row stride of the joined outputs (no bank conflicts)
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kJoin = kWarps * 8 * NT * (kRow + 2) * 4;
    static constexpr size_t kSmem = kRing + kJoin;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// The two parts of p >= 0 (see the use): the upper 16 bits of two, packed, and what they leave.
__device__ __forceinline__ uint32_t high_parts(float x, float y) {
    return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}
__device__ __forceinline__ float low_part(float x) {
    return fmaxf(x - __uint_as_float(__float_as_uint(x) & 0xffff0000u), 1.17549435e-38f);
}

template <int D, int NT>
__global__ void __launch_bounds__(kT, 1) paged_decode_kernel(PagedArgs a, const __nv_bfloat16* Q, long long q_stride,
                                                             const __nv_bfloat16* kc, const __nv_bfloat16* vc) {
    using C = Cfg<D, NT>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long tmp[2 * kT / 32];
    __shared__ PagedStart<kKT> start;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    allow_merge();
    plan_start<kT, kKT>(a, 1, blockIdx.x, gridDim.x, 0, reinterpret_cast<int*>(smem), tmp, &start);
    unsigned char* ring = smem + warp * C::kStages * C::kStage;
    float* join = reinterpret_cast<float*>(smem + C::kRing);  // [warp][head][kRow]
    float2* ml = reinterpret_cast<float2*>(join + kWarps * 8 * NT * C::kRow);  // [warp][head]

    PagedWalk<kKT> w = start.walk, f = w;  // the unit in hand, and the one whose tiles are being fetched
    bool more = start.more;
    if (tid == 0) a.seg[blockIdx.x] = w.seg(a, start.range, blockIdx.x);
    bool fetching = more;
    int ft = f.t0;          // tile to look up next
    int page = -1, j = 0;   // table entry (any value) and first key of the slice looked up last
    bool looked = false;    // whether it is to be copied
    // the table entry of the next slice: asked for a tile before it is used
    auto look_up = [&] {
        looked = false;
        if (!fetching) return;
        const int pos = f.e.pos0;
        j = f.e.key_tile(ft) * kKT + warp * kSlice;
        looked = j <= pos && (j + kSlice > f.e.lo || j < a.S) && (j >> a.page_shift) < a.max_pages;
        if (looked) page = __ldg(a.table + (size_t)f.e.r * a.max_pages + (j >> a.page_shift));
    };
    auto advance = [&] {
        if (fetching && ++ft == f.t1) {
            fetching = f.next(a, 1);
            ft = f.t0;
        }
    };
    uint32_t put = 0;  // stage
    const uint32_t lane_row = lane / (D / 8), lane_col = lane % (D / 8);
    auto fetch = [&] {  // the slice looked up, into the next stage
        if (looked) {
            const bool in = page >= 0 && page < a.n_pages;
            if (!in && lane == 0) report_error(a.err, kErrBadIndex);
            const int pos = f.e.pos0, off = j & (a.page - 1);
            const size_t at = ((((size_t)(in ? page : 0) * a.Hkv + f.h) << a.page_shift) + off + lane_row) * D + lane_col * 8;
            const uint32_t dst = smem_addr(ring) + put * C::kStage + (lane_col >> 3) * C::kHalf;
            constexpr int kRows = 256 / D;  // rows a warp copies at once
#pragma unroll
            for (int i = 0; i < kSlice; i += kRows) {
                const int r = i + lane_row, key = j + r;
                const bool ok = in && visible(key, pos, a.W, a.S);
                const uint32_t o = dst + r * 128 + (((lane_col & 7) ^ (r & 7)) << 4);
                copy16(o, kc + at + (size_t)i * D, ok);
                copy16(o + C::kTensor, vc + at + (size_t)i * D, ok);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == C::kStages ? 0 : put + 1;
    };
    look_up();
#pragma unroll 1
    for (int s = 0; s < C::kStages - 1; ++s) {
        fetch();
        advance();
        look_up();
    }

    uint32_t get = 0;
    int piece = 0;
    const int g = lane >> 2, h0 = 2 * (lane & 3), mi = lane >> 3;
    for (; more; more = w.next(a, 1), ++piece) {
        const PagedEntry& e = w.e;
        const int pos = e.pos0;
        // Q^T as the B operand: heads past G are zero
        uint32_t qb[NT][D / 16][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool in = 8 * n + g < a.G;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(Q + (size_t)e.row0 * q_stride + (size_t)(w.h * a.G + (in ? 8 * n + g : 0)) * D + h0);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                qb[n][ks][0] = in ? q[ks * 8] : 0u;
                qb[n][ks][1] = in ? q[ks * 8 + 4] : 0u;
            }
        }
        float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.0f;
        }
#pragma unroll 1
        for (int k = w.t0; k < w.t1; ++k) {
            fetch();  // (the stage read in the last step; its readers are this warp's own)
            advance();
            look_up();
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
            __syncwarp();
            const unsigned char* sK = ring + get * C::kStage;
            const unsigned char* sV = sK + C::kTensor;
            get = get + 1 == C::kStages ? 0 : get + 1;
            const int j0 = e.key_tile(k) * kKT + warp * kSlice;
            // keys of the slice that the token sees
            const bool see0 = visible(j0 + g, pos, a.W, a.S), see1 = visible(j0 + g + 8, pos, a.W, a.S);
            if (__any_sync(kFull, see0 || see1)) {
                float s[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const int r = (lane & 7) + ((mi & 1) << 3), cc = (ks & 3) * 2 + (mi >> 1);
                    uint32_t ak[4];
                    ldmatrix_x4(ak[0], ak[1], ak[2], ak[3], sK + (ks >> 2) * C::kHalf + r * 128 + ((cc ^ (r & 7)) << 4));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_bf16_16816(s[n], ak, qb[n][ks][0], qb[n][ks][1]);
                }
                float mx[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        s[n][x] = see0 ? s[n][x] * a.sl2 : -INFINITY;
                        s[n][2 + x] = see1 ? s[n][2 + x] * a.sl2 : -INFINITY;
                        mx[n][x] = fmaxf(s[n][x], s[n][2 + x]);
                    }
                }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mx[n][0] = fmaxf(mx[n][0], __shfl_xor_sync(kFull, mx[n][0], d));
                        mx[n][1] = fmaxf(mx[n][1], __shfl_xor_sync(kFull, mx[n][1], d));
                    }
                // the reference maxima move only when a head's maximum passes them by more than 2^8
                bool grow = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) grow |= mx[n][0] > m[n][0] + 8.0f || mx[n][1] > m[n][1] + 8.0f;
                if (__any_sync(kFull, grow)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (mx[n][x] > m[n][x]) {
                                const float fac = exp2_fast(m[n][x] - mx[n][x]);
                                m[n][x] = mx[n][x];
                                l[n][x] *= fac;
#pragma unroll
                                for (int t = 0; t < D / 16; ++t) {
                                    o[n][t][x] *= fac;
                                    o[n][t][2 + x] *= fac;
                                }
                            }
                }
                // p in two bf16 parts, the first one cut to 8 bits and the second (under 2^-7 of p) rounded: p is off by
                // 2^-15, next to nothing beside o's rounding (with one part the error against 64 bits was 1.4 times that
                // of o's rounding; the time is the same). Neither part of a visible key's p is negative, and the second
                // is at least 2^-126, the smallest normal: an infinite value then gives that infinity in both products,
                // where a second part of 0 or below would make it NaN. (A hidden key's value is zero in the ring.)
                uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float u0 = m[n][0] == -INFINITY ? 0.0f : m[n][0], u1 = m[n][1] == -INFINITY ? 0.0f : m[n][1];
                    const float p0 = exp2_fast(s[n][0] - u0), p1 = exp2_fast(s[n][1] - u1);
                    const float p2 = exp2_fast(s[n][2] - u0), p3 = exp2_fast(s[n][3] - u1);
                    l[n][0] += p0 + p2;
                    l[n][1] += p1 + p3;
                    pb[n][0] = movmatrix_trans(high_parts(p0, p1));
                    pb[n][1] = movmatrix_trans(high_parts(p2, p3));
                    pl[n][0] = movmatrix_trans(pack_bf16(low_part(p0), low_part(p1)));
                    pl[n][1] = movmatrix_trans(pack_bf16(low_part(p2), low_part(p3)));
                }
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    const int r = (lane & 7) + ((mi >> 1) << 3), cc = (t & 3) * 2 + (mi & 1);
                    uint32_t av[4];
                    ldmatrix_x4_trans(av[0], av[1], av[2], av[3], sV + (t >> 2) * C::kHalf + r * 128 + ((cc ^ (r & 7)) << 4));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_bf16_16816(o[n][t], av, pb[n][0], pb[n][1]);
                        mma_bf16_16816(o[n][t], av, pl[n][0], pl[n][1]);
                    }
                }
            }
            __syncwarp();  // the stage has been read
        }
        // ---- join the warps
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][x] += __shfl_xor_sync(kFull, l[n][x], d);
                float* row = join + (warp * 8 * NT + 8 * n + h0 + x) * C::kRow + g;
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    row[t * 16] = o[n][t][x];
                    row[t * 16 + 8] = o[n][t][2 + x];
                }
                if (g == 0) ml[warp * 8 * NT + 8 * n + h0 + x] = make_float2(m[n][x], l[n][x]);
            }
        }
        __syncthreads();
        const bool whole = w.whole(), empty = pos < 0;
        float* rec = a.rec + ((size_t)blockIdx.x * 2 + (piece == 0 ? 0 : 1)) * a.rec_rows * (D + 2);
        for (int i = tid; i < a.G * (D / 4); i += kT) {
            const int h = i / (D / 4), c = i % (D / 4);
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) M = fmaxf(M, ml[v * 8 * NT + h].x);
            float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                const float2 z = ml[v * 8 * NT + h];
                // (a slice of NaN scores alone has a sum and no maximum: NaN)
                const float fac = z.x == -INFINITY && z.y == 0.0f ? 0.0f : exp2_fast(z.x - M);
                const float4 x = *reinterpret_cast<const float4*>(join + (v * 8 * NT + h) * C::kRow + 4 * c);
                L = fmaf(z.y, fac, L);
                y.x = fmaf(x.x, fac, y.x);
                y.y = fmaf(x.y, fac, y.y);
                y.z = fmaf(x.z, fac, y.z);
                y.w = fmaf(x.w, fac, y.w);
            }
            if (whole) {
                const size_t orow = (size_t)e.row0 * a.Hq + w.h * a.G + h;
                const float inv = 1.0f / L;
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + orow * D + 4 * c) =
                    empty ? make_uint2(0u, 0u) : make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
                if (a.lse && c == 0) a.lse[orow] = empty ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
            } else {
                reinterpret_cast<float4*>(rec)[(size_t)c * a.rec_rows + h] = y;
                if (c == 0) reinterpret_cast<float2*>(rec + (size_t)a.rec_rows * D)[h] = make_float2(M, L);
            }
        }
        __syncthreads();  // before the next unit's outputs
    }
}

template <int D, int NT>
cudaError_t run(const PagedDims& m, const PagedArgs& a, const void* Q, const void* kc, const void* vc, cudaStream_t s) {
    using C = Cfg<D, NT>;
    static_assert(C::kSmem + 1024 <= 227 * 1024, "shared memory");
    static_assert((kMaxRequests + 1) * 4 <= C::kSmem, "the plan's scratch");
    static OncePerDevice once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(paged_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    });
    if (e != cudaSuccess) return e;
    const int workers = sm_count();
    count_launch();
    paged_decode_kernel<D, NT><<<workers, kT, C::kSmem, s>>>(a, static_cast<const __nv_bfloat16*>(Q), m.q_stride,
                                                             static_cast<const __nv_bfloat16*>(kc), static_cast<const __nv_bfloat16*>(vc));
    const cudaError_t f = cudaGetLastError();
    if (f != cudaSuccess) return f;
    return launch_paged_merge<__nv_bfloat16, D>(a, workers, m.G, s);
}

}  // namespace

// an even number: a row's d + 2 floats are a multiple of 8 bytes, and records start at multiples of 16
int paged_decode_rec_rows(const PagedDims& m) { return (m.G + 1) & ~1; }
int paged_decode_workers(const PagedDims&) { return sm_count(); }

cudaError_t launch_paged_decode(const PagedDims& m, const PagedArgs& a, const void* Q, const void* kc, const void* vc,
                                cudaStream_t s) {
    if (m.d == 64) return m.G <= 8 ? run<64, 1>(m, a, Q, kc, vc, s) : run<64, 2>(m, a, Q, kc, vc, s);
    return m.G <= 8 ? run<128, 1>(m, a, Q, kc, vc, s) : run<128, 2>(m, a, Q, kc, vc, s);
}

}  // namespace cobs
