// Attention of new tokens over a paged cache on the CUDA cores: float32.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(q . k_j / sqrt(d)),  over the keys j <= t visible at
//   the row's position t (all of them, or the last W and the first S).
//
// A block of 256 threads walks its range of (unit, 64-key tile) pairs. The unit's rows (tokens x
// the G heads of the group) are M = 64 or 16 rows; thread (ty, tx) of 16 x 16 holds M / 16 rows x
// 4 keys of the scores and M / 16 rows x d / 16 columns of the output in registers, and each row's
// running maximum and sum. V of a tile is in flight (cp.async) while its scores are formed; P takes K's
// place, so that two blocks fit an SM at d = 128 and one computes while the other waits for K or at a
// barrier. The float32 products stay on the FMA
// pipes: the tensor cores' tf32 would drop 13 bits of each factor.
#include <algorithm>
#include <type_traits>

#include "paged.h"
#include "paged_plan.cuh"
#include "paged_kernels.h"
#include "tma.h"

namespace cobs {
namespace {

constexpr int kT = 256;
constexpr int kKT = 64;      // keys per tile
constexpr int kPS = kKT + 4;  // row stride of P

__device__ __forceinline__ void cp16(void* dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D, int M>
constexpr size_t simt_smem() {
    return sizeof(float) * ((size_t)M * (D + 4) + (size_t)kKT * (D + 4) + (size_t)kKT * D);  // P (M x kPS) in K's place
}

// Blocks resident on an SM (shared memory and registers): one waits for its copies and its barriers, the
// others compute.
constexpr int blocks_per_sm(int d, int m) { return m == 16 ? (d == 64 ? 3 : 2) : 2; }

template <int D, int M>
__global__ void __launch_bounds__(kT, blocks_per_sm(D, M)) paged_simt_kernel(PagedArgs a, const float* Q, long long q_stride,
                                                        const float* kc, const float* vc) {
    extern __shared__ __align__(16) float sm[];
    __shared__ long long tmp[2 * kT / 32];
    __shared__ PagedStart<kKT> start;
    __shared__ int page_sh[2][kKT / 16];
    constexpr int RM = M / 16, CD = D / 16, KS = D + 4;
    float* sQ = sm;               // [M][D + 4]
    float* sK = sQ + M * KS;      // [64][D + 4]
    float* sV = sK + kKT * KS;    // [64][D]
    float* sP = sK;               // [M][68]
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int TQ = M / a.G;
    allow_merge();
    plan_start<kT, kKT>(a, TQ, blockIdx.x, gridDim.x, 0, reinterpret_cast<int*>(sm), tmp, &start);
    PagedWalk<kKT> w = start.walk;
    int piece = 0;
    bool more = start.more;
    if (tid == 0) a.seg[blockIdx.x] = w.seg(a, start.range, blockIdx.x);
    for (; more; more = w.next(a, TQ), ++piece) {
        const PagedEntry& e = w.e;
        const int rows = e.n * a.G, hi = e.last_pos();
        const int ppt = kKT >> a.page_shift;  // pages per tile (0: a page holds two tiles)
        auto fetch_pages = [&](int k) {       // pages of tile k, by the first threads
            if (tid < max(1, ppt) && k < w.t1) {
                const int j0 = e.key_tile(k) * kKT + (tid << a.page_shift);
                page_sh[k & 1][tid] = page_of(a, e.r, j0 >> a.page_shift, j0 <= hi && (j0 + min(a.page, kKT) > e.lo || j0 < a.S));
            }
        };
        // one tile of K or V: rows no position of the unit sees are zero
        auto load = [&](float* dst, int stride, const float* cache, int k) {
            const int j0 = e.key_tile(k) * kKT;
            for (int c = tid; c < kKT * D / 4; c += kT) {
                const int row = c / (D / 4), col = c % (D / 4) * 4, j = j0 + row;
                const int page = page_sh[k & 1][ppt ? row >> a.page_shift : 0];
                const bool ok = page >= 0 && j <= hi && (j >= e.lo || j < a.S);
                const size_t at = (((size_t)(ok ? page : 0) * a.Hkv + w.h) * a.page + (j & (a.page - 1))) * D + col;
                cp16(dst + row * stride + col, cache + at, ok);
            }
        };
        __syncthreads();  // the last unit's (or the plan's) shared memory is free
        fetch_pages(w.t0);
        for (int c = tid; c < M * D / 4; c += kT) {
            const int row = c / (D / 4), col = c % (D / 4) * 4;
            const bool ok = row < rows;
            const float* q = Q + (ok ? (size_t)(e.row0 + row / a.G) * q_stride + (size_t)(w.h * a.G + row % a.G) * D : 0);
            cp16(sQ + row * KS + col, q + col, ok);
        }
        __syncthreads();
        load(sK, KS, kc, w.t0);
        cp_commit();
        float m[RM], l[RM], o[RM][CD];
        int pos[RM];
#pragma unroll
        for (int y = 0; y < RM; ++y) {
            m[y] = -INFINITY;
            l[y] = 0.0f;
            const int row = ty + 16 * y;
            pos[y] = row < rows ? e.pos0 + row / a.G : -1;
#pragma unroll
            for (int x = 0; x < CD; ++x) o[y][x] = 0.0f;
        }
        for (int k = w.t0; k < w.t1; ++k) {
            const int j0 = e.key_tile(k) * kKT;
            load(sV, D, vc, k);
            cp_commit();
            cp_wait<1>();
            fetch_pages(k + 1);
            __syncthreads();
            float s[RM][4];
#pragma unroll
            for (int y = 0; y < RM; ++y) s[y][0] = s[y][1] = s[y][2] = s[y][3] = 0.0f;
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                float4 kv[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) kv[x] = *reinterpret_cast<const float4*>(sK + (tx + 16 * x) * KS + c);
#pragma unroll
                for (int y = 0; y < RM; ++y) {
                    const float4 q = *reinterpret_cast<const float4*>(sQ + (ty + 16 * y) * KS + c);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        s[y][x] = fmaf(q.w, kv[x].w, fmaf(q.z, kv[x].z, fmaf(q.y, kv[x].y, fmaf(q.x, kv[x].x, s[y][x]))));
                }
            }
            __syncthreads();  // K has been read
            // a tile that every row sees in full needs no masks
            const bool full = j0 + kKT - 1 <= e.pos0 && (a.W <= 0 || hi - j0 < a.W);
#pragma unroll
            for (int y = 0; y < RM; ++y) {
                float mx = -INFINITY;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[y][x] *= a.sl2;
                    if (!full && !visible(j0 + tx + 16 * x, pos[y], a.W, a.S)) s[y][x] = -INFINITY;
                    mx = fmaxf(mx, s[y][x]);
                }
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
                const float nm = fmaxf(m[y], mx), use = nm == -INFINITY ? 0.0f : nm;
                const float f = m[y] == nm ? 1.0f : exp2_fast(m[y] - use);
                m[y] = nm;
                float sum = 0.0f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float pv = exp2_fast(s[y][x] - use);
                    sP[(ty + 16 * y) * kPS + tx + 16 * x] = pv;
                    sum += pv;
                }
                l[y] = l[y] * f + sum;  // this thread's keys; joined over tx at the end
#pragma unroll
                for (int x = 0; x < CD; ++x) o[y][x] *= f;
            }
            cp_wait<0>();  // V
            __syncthreads();
            // a hidden key adds nothing, whatever its value holds: tiles with masks test every pair (the test
            // costs as much as the products, so the others do without)
            auto product = [&](auto masked) {
#pragma unroll 2
                for (int j = 0; j < kKT; j += 4) {
                    float4 p4[RM];
#pragma unroll
                    for (int y = 0; y < RM; ++y) p4[y] = *reinterpret_cast<const float4*>(sP + (ty + 16 * y) * kPS + j);
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        float v[CD];
#pragma unroll
                        for (int x = 0; x < CD; x += 4)
                            *reinterpret_cast<float4*>(v + x) =
                                *reinterpret_cast<const float4*>(sV + (j + jj) * D + (x / 4) * 64 + tx * 4);
#pragma unroll
                        for (int y = 0; y < RM; ++y) {
                            const float pv = jj == 0 ? p4[y].x : jj == 1 ? p4[y].y : jj == 2 ? p4[y].z : p4[y].w;
                            if (!decltype(masked)::value || visible(j0 + j + jj, pos[y], a.W, a.S))
#pragma unroll
                                for (int x = 0; x < CD; ++x) o[y][x] = fmaf(pv, v[x], o[y][x]);
                        }
                    }
                }
            };
            if (full) product(std::false_type()); else product(std::true_type());
            __syncthreads();  // V and P have been read
            if (k + 1 < w.t1) load(sK, KS, kc, k + 1);
            cp_commit();
        }
        const bool whole = w.whole();
        const int slot = piece == 0 ? 0 : 1;
#pragma unroll
        for (int y = 0; y < RM; ++y) {
            float sum = l[y];
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
            const int row = ty + 16 * y;
            if (row >= rows) continue;
            float4* dst;
            size_t step = 16;  // float4 from one 64-column group to the next
            float f = 1.0f;
            if (whole) {
                const size_t orow = (size_t)(e.row0 + row / a.G) * a.Hq + w.h * a.G + row % a.G;
                const bool empty = pos[y] < 0;
                dst = reinterpret_cast<float4*>(static_cast<float*>(a.O) + orow * D) + tx;
                f = empty ? 0.0f : 1.0f / sum;
                if (a.lse && tx == 0) a.lse[orow] = empty ? -INFINITY : (m[y] + log2f(sum)) * 0.6931471805599453f;
            } else {
                float* rec = a.rec + ((size_t)blockIdx.x * 2 + slot) * M * (D + 2);
                dst = reinterpret_cast<float4*>(rec) + tx * M + row;
                step = 16 * M;
                if (tx == 0) reinterpret_cast<float2*>(rec + (size_t)M * D)[row] = make_float2(m[y], sum);
            }
#pragma unroll
            for (int x = 0; x < CD; x += 4)
                dst[(x / 4) * step] = make_float4(o[y][x] * f, o[y][x + 1] * f, o[y][x + 2] * f, o[y][x + 3] * f);
        }
    }
}

template <int D, int M>
cudaError_t run(const PagedArgs& a, int workers, const float* Q, long long q_stride, const float* kc, const float* vc,
                cudaStream_t s) {
    constexpr auto smem_of = [](int R) { return std::max(simt_smem<D, M>(), (size_t)(R + 1) * sizeof(int)); };
    const size_t smem = smem_of(a.R);
    static OncePerDevice once;  // (the largest call's limit: a call's own would be lowered by another thread's)
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(paged_simt_kernel<D, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(kMaxRequests));
    });
    if (e != cudaSuccess) return e;
    paged_simt_kernel<D, M><<<workers, kT, smem, s>>>(a, Q, q_stride, kc, vc);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_paged_merge<float, D>(a, workers, std::min(M / a.G, a.max_new) * a.G, s);
}

}  // namespace

// 16 rows where no request has more (a few tokens of few heads): a tile's products are then a quarter.
static int simt_rows(const PagedDims& m) { return (long long)m.max_new * m.G <= 16 ? 16 : 64; }

int paged_simt_rec_rows(const PagedDims& m) { return simt_rows(m); }
int paged_simt_workers(const PagedDims& m) { return sm_count() * blocks_per_sm(m.d, simt_rows(m)); }

cudaError_t launch_paged_simt(const PagedDims& m, const PagedArgs& a, const float* Q, const float* kc,
                              const float* vc, cudaStream_t s) {
    const int n = paged_simt_workers(m);
    const bool few = simt_rows(m) == 16;
    count_launch();
    if (m.d == 64) return few ? run<64, 16>(a, n, Q, m.q_stride, kc, vc, s) : run<64, 64>(a, n, Q, m.q_stride, kc, vc, s);
    return few ? run<128, 16>(a, n, Q, m.q_stride, kc, vc, s) : run<128, 64>(a, n, Q, m.q_stride, kc, vc, s);
}

}  // namespace cobs
