// Attention of new tokens over a paged cache on the fifth-generation tensor cores (tcgen05, TMEM), bf16.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(q . k_j / sqrt(d)),  over the keys j <= t visible at
//   the row's position t (all of them, or the last W and the first S).
//
// One persistent CTA per SM walks its range of (unit, 128-key tile) pairs (paged_plan.cuh). A unit's
// rows are two MMA tiles of 128: each holds floor(128 / G) tokens x the G heads of the group, so K
// and V are read once per group and a tile spans few positions. Per key tile and row tile g:
//   S_g = Q_g K^T           tcgen05.mma, M 128, N 128, K d, into 128 TMEM columns
//   p = 2^(s c - m)         two threads per row, which exchange their maxima; m moves only when a row's
//                           maximum grows by more than 2^8 (then the threads rescale their row of
//                           O, which is seldom)
//   O_g += P_g V            P in bf16 over S's columns (A operand from TMEM), V MN-major. The MMA takes A and B
//                           of one type, and a second product with what the rounding leaves would be half as much
//                           again for the busiest pipe: the error against 64 bits is 2.3e-3, where o's own rounding
//                           alone gives 1.7e-3 (2048 tokens at 32k keys). The sum of p is not rounded.
// The two row tiles alternate: while the tensor pipe runs P V of one and the next Q K^T of it, the
// other one's softmax runs. MMAs are issued by one thread in the order PV_0(k) QK_0(k+1) PV_1(k)
// QK_1(k+1): the pipe runs them in order, so S_g(k+1) arriving means that P_g(k) has been read and
// O_g is up to date, and no barrier is needed for either. A unit of one row tile (single tokens,
// short chunks) gives both halves of the machine to it: the two groups take its key tiles in turn,
// each with an accumulator and maxima of its own, joined at the unit's end.
// Roles: warps 0-15 softmax and epilogue (four for each row tile and half of the columns); warp 16 loads
// K and V (one TMA box per page and 64 columns; pages no row needs come as out-of-range boxes, that is
// zeros); warp 17 issues the MMAs; warps 18 and 19 (the first also loads Q) prepare V of the tiles that
// some row does not see in full: rows of V no row of the unit sees (slots behind the keys, keys before
// the window: any bits) are set to zero, since 0 * NaN would reach O, and the others are looked over
// for infinities and NaN: such a tile's product is formed by the softmax threads, key by key, so that
// only the rows that see them change.
// Every wait is bounded; one that gives up sets the device error flag and the CTA winds down.
//
// What bounds it: the chain of a row tile. 2048 tokens at 32k keys, 64 / 4 heads of 128: 2.17-2.20 ms, 970-980
// TFLOP/s, 0.59 of the measured bf16 peak (1.92 ms and 0.67 on the fastest machine seen); a key tile of both row
// tiles takes some 3.9k cycles, of which the tensor pipe has work for 2.1k and the special-function unit for
// 2.05k. In a trace a row tile's P V and Q K^T take 1.6k cycles with their hand-over, its softmax 2.2k (maxima
// 0.4k, powers 1.5k), and two row tiles are all that tensor memory holds (two S of 128 columns, two O of d). The
// softmax reads its scores twice, in masked tiles three times: 96 registers a thread do not hold them beside the
// rest. Measured and left out: key tiles in
// halves with N = 64 (four streams, but Q K^T is then bound by shared memory: half as fast); powers partly
// on the FMA pipes (7% slower and more); P handed over in halves (3%); scores kept in registers between
// maxima and powers (spills), or read 16 at a time (18%).
#include <stddef.h>

#include <algorithm>

#include "paged.h"
#include "paged_kernels.h"
#include "paged_plan.cuh"
#include "tc.cuh"
#include "tma.h"

namespace cobs {
namespace {

constexpr int kThreads = 640;
constexpr int kKT = 128;      // keys per tile
constexpr int kLoadWarp = 16, kMmaWarp = 17, kFixWarp = 18;
constexpr int kFixDepth = 4;    // tiles whose V may be prepared ahead of their products
constexpr uint32_t kBox = 128 * 128;  // 128 rows of 64 columns
constexpr uint32_t kColO = 256;       // S_g (and P_g) at 128 g, O_g at 256 + 128 g

// Shared memory behind Q and the ring.
template <int STAGES>
struct Misc {
    uint64_t barQ, barQfree, barKV[STAGES], barFree[STAGES], barS[2], barP[2], barO[2], barFix[kFixDepth], barDone;
    long long tmp[2 * kThreads / 32];
    PagedStart<kKT> start;
    int dirty[kFixDepth][2];
    uint32_t tmem;
    float row[2][2][128];  // [group][half of the columns][row]: maxima of a tile, sums and maxima of a unit
};

template <int D>
struct Cfg {
    static constexpr int H = D / 64;                  // 64-column halves
    static constexpr uint32_t kTile = H * kBox;       // a row tile of Q, a key tile of K or V
    static constexpr int kStages = D == 128 ? 5 : 8;  // K and V tiles in flight
    static constexpr uint32_t kSmem = (2 + kStages) * kTile + sizeof(Misc<kStages>);
    static constexpr uint32_t kIdescS = tc::idesc_bf16(128, kKT, 0, 0);
    static constexpr uint32_t kIdescPV = tc::idesc_bf16(128, D, 0, 1);
};

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 32 columns into s, without waiting
__device__ __forceinline__ void ld32_to(uint32_t taddr, float (&s)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(s[0]), "=f"(s[1]), "=f"(s[2]), "=f"(s[3]), "=f"(s[4]), "=f"(s[5]), "=f"(s[6]), "=f"(s[7]), "=f"(s[8]), "=f"(s[9]),
          "=f"(s[10]), "=f"(s[11]), "=f"(s[12]), "=f"(s[13]), "=f"(s[14]), "=f"(s[15]), "=f"(s[16]), "=f"(s[17]), "=f"(s[18]),
          "=f"(s[19]), "=f"(s[20]), "=f"(s[21]), "=f"(s[22]), "=f"(s[23]), "=f"(s[24]), "=f"(s[25]), "=f"(s[26]), "=f"(s[27]),
          "=f"(s[28]), "=f"(s[29]), "=f"(s[30]), "=f"(s[31])
        : "r"(taddr));
}
// The registers of a load are not to be used before the wait for it.
__device__ __forceinline__ void touch32(float (&s)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) asm volatile("" : "+f"(s[j]));
}
__device__ __forceinline__ void wait_ld32(float (&s)[32]) {
    tc::wait_ld();
    touch32(s);
}
__device__ __forceinline__ float ld1(uint32_t taddr) {
    float v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(taddr));
    return v;
}
template <int N> __device__ __forceinline__ void rows_sync(int id) {
    __syncwarp();  // (the barrier is for converged warps)
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}
// shared memory to global, both 16-byte aligned, a multiple of 16 bytes
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
}

// a box of shared memory (128-byte swizzle) to a 3-D tensor
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, const void* src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y), "r"(z),
                 "r"(smem_addr(src))
                 : "memory");
}

// Bounded wait without a suspend hint: with one, a poll of a phase that is already complete costs 46
// cycles, without 15 (clock64 around completed phases), and most waits here find theirs complete. A poll
// of an incomplete one comes back after 4 us: kMaxPolls are a quarter of a second.
constexpr uint32_t kMaxPolls = 1u << 16;
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* err) {
    if (mbar_test(bar, parity)) return true;
#pragma unroll 1
    for (uint32_t i = 0; i < kMaxPolls; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (done) return true;
    }
    report_error(err, kErrWaitTimeout);
    return false;
}
// The same for a whole warp, which goes on together: what follows (tcgen05 loads, named barriers) is for
// converged warps, and the lanes leave the loop above one by one.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* err) {
    return __all_sync(kFull, wait_on(bar, parity, err));
}

// n ones from bit 0 up (none for n <= 0, all for n >= 32)
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)), "l"(reinterpret_cast<uint64_t&>(z)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)));
    return r;
}

// A position in the ring: stage, and parity of its phase.
template <int STAGES>
struct Pos {
    uint32_t s = 0, ph = 0;
    __device__ __forceinline__ Pos plus(uint32_t k) const {  // k <= STAGES
        const uint32_t t = s + k;
        return t >= STAGES ? Pos{t - STAGES, ph ^ 1u} : Pos{t, ph};
    }
    __device__ __forceinline__ void advance(uint32_t k) {
        const uint32_t t = s + k, q = t / STAGES;
        s = t - q * STAGES;
        ph ^= q & 1u;
    }
};

// How a unit runs: one row tile whose key tiles the two groups take in turn, or two; and whether its
// output leaves through the ring (a stage per row tile): a thread's row is 2 d bytes apart from its
// neighbour's, so direct stores of 32 rows touch 32 lines each, which took 7k cycles per unit of 256 rows
// against 1k through the ring. A full row tile leaves as one box per 64 columns (a copy per token is issued
// lane by lane: 3 to 4k cycles for 32 of them), a partial one token by token. One warp's rows and records go
// directly.
template <int KT>
struct Shape {
    bool pair, staged;
    uint32_t stages;  // of the output
    __device__ __forceinline__ Shape(const PagedArgs& a, int n, bool whole, int TM) {
        pair = n <= TM;
        staged = whole && n * a.G > 32;
        stages = staged ? (pair ? 1 : 2) : 0;
    }
    __device__ __forceinline__ Shape(const PagedArgs& a, const PagedWalk<KT>& w, int TM) : Shape(a, w.e.n, w.whole(), TM) {}
};

// A walk in one register of a warp: value k in lane k.
template <int KT>
__device__ __forceinline__ int pack_walk(const PagedWalk<KT>& w, int lane) {
    static_assert(sizeof(PagedWalk<KT>) == 17 * sizeof(int), "17 values");
    const int* f = reinterpret_cast<const int*>(&w);
    int v = 0;
#pragma unroll
    for (int k = 0; k < 17; ++k) v = lane == k ? f[k] : v;
    return v;
}
template <int KT>
__device__ __forceinline__ PagedWalk<KT> unpack_walk(int v) {
    PagedWalk<KT> w;
    int* f = reinterpret_cast<int*>(&w);
#pragma unroll
    for (int k = 0; k < 17; ++k) f[k] = __shfl_sync(kFull, v, k);
    return w;
}

struct ChunkMaps {
    CUtensorMap q, k, v, o;
};

// A tile some row of the unit does not see in full.
__device__ __forceinline__ bool masked_tile(const PagedArgs& a, int pos0, int n, int j0) {
    return !(j0 + kKT - 1 <= pos0 && (a.W <= 0 || pos0 + n - 1 - j0 < a.W));
}
__device__ __forceinline__ bool masked_tile(const PagedArgs& a, const PagedEntry& e, int j0) { return masked_tile(a, e.pos0, e.n, j0); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(const __grid_constant__ ChunkMaps maps, PagedArgs a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char sQ[];  // (no other shared memory: it starts at its first kilobyte)
    unsigned char* sKV = sQ + 2 * C::kTile;
    Misc<C::kStages>& sh_ = *reinterpret_cast<Misc<C::kStages>*>(sKV + C::kStages * C::kTile);
    uint64_t &barQ = sh_.barQ, &barQfree = sh_.barQfree, &barDone = sh_.barDone;
    auto& barKV = sh_.barKV;
    auto& barFree = sh_.barFree;
    auto& barS = sh_.barS;
    auto& barP = sh_.barP;
    auto& barO = sh_.barO;
    auto& barFix = sh_.barFix;
    auto& dirty_sh = sh_.dirty;
    auto& row_sh = sh_.row;
    if (smem_addr(sQ) & 1023u) {  // the swizzled tiles need it
        report_error(a.err, kErrWaitTimeout);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int TM = 128 / a.G, TQ = 2 * TM;  // tokens of a row tile and of a unit
    if (warp == 0) {
        tc::tmem_alloc(&sh_.tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 32) {
        mbar_init(&barQ, 1);
        mbar_init(&barQfree, 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&barKV[s], 1);
            mbar_init(&barFree[s], 3);  // the MMAs that read it, and the two V warps
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&barS[g], 1);
            mbar_init(&barP[g], 8);
            mbar_init(&barO[g], 1);
        }
        for (int f = 0; f < kFixDepth; ++f) mbar_init(&barFix[f], 2);
        mbar_init(&barDone, 1);
        fence_barrier_init();
    }
    allow_merge();
    plan_start<kThreads, kKT>(a, TQ, blockIdx.x, gridDim.x, kLoadWarp, reinterpret_cast<int*>(sKV), sh_.tmp, &sh_.start);
    fence_proxy_async();  // the plan's use of the ring before TMA's
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh_.tmem;
    bool ok = true;
    PagedWalk<kKT> w = sh_.start.walk;
    bool more = sh_.start.more;
    if (tid == kFixWarp * 32 + 32) a.seg[blockIdx.x] = w.seg(a, sh_.start.range, blockIdx.x);

    if (warp < 16) {
        // ------------------------------------------------------------ softmax and epilogue of row tile g
        // (after a wait that gave up these warps go on without waiting: they meet at named barriers)
        const int g = (warp >> 2) & 1, half = warp >> 3, row = tid & 127;  // row tile, half of the columns
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + 128 * g, tO = tmem + lanes + kColO + 128 * g;
        const int tok = row / a.G, hrow = row - tok * a.G;
        const float sl2 = a.sl2;
        uint32_t nS = 0, nO = 0, nFix = 0;
        Pos<C::kStages> at;  // of the unit's first tile
        int piece = 0;
        // Of the walk's 17 values the loop over the tiles needs six. The others wait in one register, value k in
        // lane k (as registers of every lane they were spilled in that loop, and in local memory they did not fit
        // beside the other threads' in what the shared memory leaves of L1: 1.6k cycles per unit).
        int packed = pack_walk(w, lane);
#define PACKED(field) __shfl_sync(kFull, packed, offsetof(PagedWalk<kKT>, field) / sizeof(int))
        for (; more; ++piece) {
            const int pos0 = PACKED(e.pos0), en = PACKED(e.n), t0 = PACKED(t0), t1 = PACKED(t1), sT = PACKED(e.sT), loT = PACKED(e.loT);
            const bool pair = en <= TM;
            const int tok0 = pair ? 0 : g * TM;       // first token of this group's rows
            const int ntok = min(TM, en - tok0);
            const bool live = tok < ntok;
            const bool warp_live = (warp & 3) * 32 < ntok * a.G;
            const int t = pos0 + tok0 + tok;
            float m = -INFINITY, l = 0.0f;
            const int kg = t0 + (pair ? g : 0);  // this group's first tile
            for (int k = t0; k < t1; ++k) {
                const int j0 = (k < sT ? k : loT + (k - sT)) * kKT;
                const bool masked = masked_tile(a, pos0, en, j0);
                const uint32_t fix = nFix;
                nFix += masked;
                if (pair && ((k - t0) & 1) != g) continue;
                if (ok) ok = wait_warp(&barS[g], nS & 1, a.err);
                ++nS;
                int dirty = 0;  // the stage of V (from 1) where this thread forms the product
                tc::fence_after_sync();
                if (warp_live) {
                    const int hi = t - j0, lo = a.W > 0 ? hi - a.W + 1 : 0, sk = a.W > 0 ? a.S - j0 : 0;
                    const uint32_t tH = tS + 64 * half;
                    if (masked) {  // the scores this row does not see: -infinity, in place
#pragma unroll 1
                        for (int c = 64 * half; c < 64 * half + 64; c += 32) {
                            const uint32_t see = bits_below(hi - c + 1) & (~bits_below(lo - c) | bits_below(sk - c));
                            float s[32];
                            ld32_to(tS + c, s);
                            wait_ld32(s);
#pragma unroll
                            for (int j = 0; j < 32; ++j) s[j] = see & (1u << j) ? s[j] : -INFINITY;
                            tc::st32(tS + c, s);
                        }
                        tc::wait_st();
                    }
                    float mx[2] = {-INFINITY, -INFINITY};
                    float s[32];
                    ld32_to(tH, s);
                    wait_ld32(s);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) mx[(j >> 1) & 1] = max3(mx[(j >> 1) & 1], s[j], s[j + 1]);
                    ld32_to(tH + 32, s);
                    wait_ld32(s);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) mx[(j >> 1) & 1] = max3(mx[(j >> 1) & 1], s[j], s[j + 1]);
                    const float mine = fmaxf(mx[0], mx[1]);
                    row_sh[g][half][row] = mine;
                    // the warp with the other half of these rows; its scores stored above may be read below (dirty)
                    if (masked) tc::fence_before_sync();
                    rows_sync<64>(1 + 4 * g + (warp & 3));
                    if (masked) tc::fence_after_sync();
                    const float mt = fmaxf(mine, row_sh[g][half ^ 1][row]) * sl2;
                    const bool grow = mt > m + 8.0f;  // (from -infinity too; never for a row that sees nothing)
                    if (k > kg && __any_sync(kFull, grow && m != -INFINITY)) {
                        const float f = grow ? tc::ex2(m - mt) : 1.0f;
                        l *= f;
#pragma unroll 1
                        for (int c = half * (D / 2); c < half * (D / 2) + D / 2; c += 32) {
                            float o[32];
                            ld32_to(tO + c, o);
                            wait_ld32(o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] *= f;
                            tc::st32(tO + c, o);
                        }
                        tc::wait_st();
                    }
                    if (grow) m = mt;
                    const float neg = m == -INFINITY ? 0.0f : -m;
                    if (masked && ok) {  // (after S: the tiles before this one have then been prepared)
                        ok = wait_warp(&barFix[fix % kFixDepth], (fix / kFixDepth) & 1, a.err);
                        dirty = max(dirty_sh[fix % kFixDepth][0], dirty_sh[fix % kFixDepth][1]);
                    }
                    // p = 2^(s c - m) of 32 keys at a time; P, half as wide, over this half's own scores
                    float2 ps[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    const float2 scale = make_float2(sl2, sl2), shift = make_float2(neg, neg);
#pragma unroll 1
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t pk[16];
                        ld32_to(tH + c, s);
                        wait_ld32(s);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 x = fma2(make_float2(s[2 * j], s[2 * j + 1]), scale, shift);
                            x.x = tc::ex2(x.x);
                            x.y = tc::ex2(x.y);
                            ps[j & 1] = add2(ps[j & 1], x);
                            pk[j] = pack_bf16(x.x, x.y);
                        }
                        if (!dirty) st16(tH + c / 2, pk);
                    }
                    ps[0] = add2(ps[0], ps[1]);
                    l += ps[0].x + ps[0].y;
                    tc::wait_st();
                    if (dirty) {
                        // P V by this row's thread: p again from S (P has not replaced it), rounded to bf16 as the
                        // tensor cores take it, V from the ring
                        const unsigned char* sV = sKV + (size_t)(dirty - 1) * C::kTile;
#pragma unroll 1
                        for (int c = half * (D / 2); c < half * (D / 2) + D / 2; c += 32) {
                            float o[32];
                            if (k > kg) {
                                ld32_to(tO + c, o);
                                wait_ld32(o);
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = 0.0f;
                            }
#pragma unroll 1
                            for (int j = 0; j < kKT; ++j) {
                                float p = ld1(tS + j);
                                tc::wait_ld();
                                asm volatile("" : "+f"(p));
                                p = __bfloat162float(__float2bfloat16_rn(tc::ex2(fmaf(p, sl2, neg))));
                                const bool see = j <= hi && (j >= lo || j < sk);
                                const unsigned char* vr = sV + (c >> 6) * kBox + j * 128;
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(vr + (((((c & 63) >> 3) + q) ^ (j & 7)) << 4));
                                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                    for (int y = 0; y < 4; ++y) {
                                        o[8 * q + 2 * y] = see ? fmaf(p, __uint_as_float(x[y] << 16), o[8 * q + 2 * y]) : o[8 * q + 2 * y];
                                        o[8 * q + 2 * y + 1] =
                                            see ? fmaf(p, __uint_as_float(x[y] & 0xffff0000u), o[8 * q + 2 * y + 1]) : o[8 * q + 2 * y + 1];
                                    }
                                }
                            }
                            tc::st32(tO + c, o);
                        }
                        tc::wait_st();
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&barP[g]);
            }
            const bool any = kg < t1;  // (a pair's second group may have no tile)
            if (any) {
                if (ok) ok = wait_warp(&barO[g], nO & 1, a.err);
                ++nO;
            }
            const bool whole = t0 == 0 && t1 == PACKED(e.nt);
            const Shape<kKT> sh(a, en, whole, TM);
            at.advance(2 * (t1 - t0));  // the output's first stage
            const Pos<C::kStages> mine = at.plus(pair ? 0 : g);
            at.advance(sh.stages);
            if (ok && sh.staged) ok = wait_warp(&barKV[mine.s], mine.ph, a.err);
            tc::fence_after_sync();
            // The threads of one row are in warps of the same TMEM lanes: two of each group, each with a share
            // of the columns, of both accumulators if the unit's tiles went to both groups.
            float f0 = 1.0f, f1 = 0.0f;  // factors of O_0 and O_1 (of O_g alone, if not both)
            const bool both = pair && t1 - t0 > 1, empty = t < 0;
            if (warp_live && any) {
                auto meet = [&] { if (both) rows_sync<128>(9 + (warp & 3)); else rows_sync<64>(1 + 4 * g + (warp & 3)); };
                // (each group has waited for its own accumulator only, and reads the other's behind the meetings)
                if (both) tc::fence_before_sync();
                row_sh[g][half][row] = l;
                meet();
                l = row_sh[g][0][row] + row_sh[g][1][row];
                if (both) {
                    const float l0 = row_sh[0][0][row] + row_sh[0][1][row], l1 = row_sh[1][0][row] + row_sh[1][1][row];
                    meet();
                    row_sh[g][half][row] = m;
                    meet();
                    const float m0 = row_sh[0][0][row], m1 = row_sh[1][0][row];
                    m = fmaxf(m0, m1);
                    // (a group of NaN scores alone has a sum and no maximum: NaN then)
                    f0 = m0 == -INFINITY && l0 == 0.0f ? 0.0f : tc::ex2(m0 - m);
                    f1 = m1 == -INFINITY && l1 == 0.0f ? 0.0f : tc::ex2(m1 - m);
                    l = l0 * f0 + l1 * f1;
                }
                meet();  // before the slots are written again
                if (both) tc::fence_after_sync();
                const int c0 = both ? 32 * (2 * g + half) : half * (D / 2), c1 = both ? min(c0 + 32, D) : c0 + D / 2;
                const size_t orow = (size_t)(PACKED(e.row0) + tok0 + (live ? tok : 0)) * a.Hq + PACKED(h) * a.G + (live ? hrow : 0);
                float* rec = a.rec + ((size_t)blockIdx.x * 2 + (piece == 0 ? 0 : 1)) * a.rec_rows * (D + 2);
                const bool full = ntok == TM;  // a staged tile leaves as swizzled boxes
                const int rrow = live ? (tok0 + tok) * a.G + hrow : 0;
                unsigned char* out = sh.staged ? sKV + (size_t)mine.s * C::kTile + row * (full ? 128 : 2 * D)
                                               : reinterpret_cast<unsigned char*>(static_cast<__nv_bfloat16*>(a.O) + orow * D);
                if (whole) {
                    const float inv = empty ? 0.0f : __fdividef(1.0f, l);  // (2 units in the last place; the result has 8 bits)
                    f0 *= inv;
                    f1 *= inv;
                }
                {
#pragma unroll 1
                    for (int c = c0; c < c1; c += 32) {
                        float o[32];
                        __syncwarp();  // (rows of no token have skipped the stores)
                        ld32_to((both ? tmem + lanes + kColO : tO) + c, o);
                        wait_ld32(o);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] *= f0;  // (a row that sees nothing: 0 * 0)
                        if (both) {
                            float o1[32];
                            ld32_to(tmem + lanes + kColO + 128 + c, o1);
                            wait_ld32(o1);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = fmaf(o1[j], f1, o[j]);
                        }
                        if (whole) {
                            uint4 v[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                v[j] = make_uint4(pack_bf16(o[8 * j], o[8 * j + 1]), pack_bf16(o[8 * j + 2], o[8 * j + 3]),
                                                  pack_bf16(o[8 * j + 4], o[8 * j + 5]), pack_bf16(o[8 * j + 6], o[8 * j + 7]));
                            if (sh.staged && full) {
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    *reinterpret_cast<uint4*>(out + (c >> 6) * kBox + (((((c & 63) >> 3) + j) ^ (row & 7)) << 4)) = v[j];
                            } else if (sh.staged) {
                                // the rows' common pitch puts a chunk of all rows in the same banks: lane r
                                // writes chunk (j + r) % 4 in step j, two steps of exchange
                                const bool r1 = lane & 1, r2 = lane & 2;
                                const uint4 w0 = r1 ? v[1] : v[0], w1 = r1 ? v[2] : v[1], w2 = r1 ? v[3] : v[2], w3 = r1 ? v[0] : v[3];
                                v[0] = r2 ? w2 : w0;
                                v[1] = r2 ? w3 : w1;
                                v[2] = r2 ? w0 : w2;
                                v[3] = r2 ? w1 : w3;
#pragma unroll
                                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(out + 2 * c + 16 * ((j + lane) & 3)) = v[j];
                            } else if (live) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(out + 2 * c + 16 * j) = v[j];
                            }
                        } else if (live) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4)
                                reinterpret_cast<float4*>(rec)[(size_t)((c + j) >> 2) * a.rec_rows + rrow] =
                                    make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                        }
                    }
                }
                if (live && half == 0 && (!both || g == 0)) {
                    if (!whole) {
                        reinterpret_cast<float2*>(rec + (size_t)a.rec_rows * D)[rrow] = make_float2(m, l);
                    } else if (a.lse) {
                        a.lse[orow] = empty ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                    }
                }
            }
            // neither group's accumulator is written again before both have read it
            tc::fence_before_sync();
            const bool copier = sh.staged && (warp & 3) == 0 && half == 0 && (!pair || g == 0);
            if (sh.staged) {
                fence_proxy_async();
                if (pair) rows_sync<512>(15); else rows_sync<256>(13 + g);
                if (copier) {
                    const unsigned char* src = sKV + (size_t)mine.s * C::kTile;
                    const int row0 = PACKED(e.row0) + tok0, head = PACKED(h) * a.G;
                    if (ntok == TM) {
                        if (lane == 0)
                            for (int h = 0; h < C::H; ++h)
                                tma_store_3d(&maps.o, 64 * h, head, row0, src + h * kBox);
                    } else {  // (a box would write the next request's rows) a token's rows are one run of both memories
                        for (int i = lane; i < ntok; i += 32)
                            bulk_s2g(static_cast<__nv_bfloat16*>(a.O) + ((size_t)(row0 + i) * a.Hq + head) * D,
                                     src + (size_t)i * a.G * 2 * D, a.G * 2 * D);
                    }
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            } else if (both && warp_live) {
                rows_sync<128>(9 + (warp & 3));
            }
            {
                PagedWalk<kKT> x = unpack_walk<kKT>(packed);
                more = x.next(a, TQ);
                packed = pack_walk(x, lane);
            }
            if (copier) {
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&barFree[mine.s]);
            }
        }
#undef PACKED
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else {
        if (warp == kLoadWarp) {
            // -------------------------------------------------------- loads
            const int shift = 7 - a.page_shift, ppt = 1 << shift, per = 32 >> shift;  // pages per tile, tiles per look-up
            const int my_tile = lane >> shift, my_key = (lane & (ppt - 1)) << a.page_shift;
            const uint32_t zero_box = (uint32_t)a.n_pages * a.Hkv;
            uint32_t n = 0;
            Pos<C::kStages> at;
            for (; more && ok; more = w.next(a, TQ)) {
                const PagedEntry& e = w.e;
                const int hi = e.last_pos();
                int raw, k0 = w.t0;
                bool needed;
                auto look_up = [&](int k) {  // table entry (any value) of this lane's page of the tiles from k on
                    const int j = k + my_tile < w.t1 ? e.key_tile(k + my_tile) * kKT + my_key : INT_MAX;
                    needed = j <= hi && (j >> a.page_shift) < a.max_pages && (j + a.page > e.lo || j < a.S);
                    raw = needed ? __ldg(a.table + (size_t)e.r * a.max_pages + (j >> a.page_shift)) : -1;
                };
                look_up(w.t0);
                uint32_t z = 0;
                for (int k = w.t0; k < w.t1 && ok; ++k) {
                    if (k == w.t0 || k == k0 + per) {
                        k0 = k;
                        // pages no row needs, and (recorded) those outside the cache, read as zeros
                        const bool in = raw >= 0 && raw < a.n_pages;
                        if (!in && needed) report_error(a.err, kErrBadIndex);
                        z = in ? (uint32_t)raw * a.Hkv + w.h : zero_box;
                        look_up(k0 + per);
                    }
                    const uint32_t zt = __shfl_sync(kFull, z, ((k - k0) << shift) + (lane & (ppt - 1)));
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++n, at = at.plus(1)) {
                        if (ok) ok = wait_warp(&barFree[at.s], at.ph ^ 1, a.err);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&barKV[at.s], C::kTile);
                        __syncwarp();
                        if (lane < ppt) {
                            unsigned char* dst = sKV + (size_t)at.s * C::kTile + my_key * 128;
#pragma unroll
                            for (int h = 0; h < C::H; ++h)
                                tma_load_3d(dst + h * kBox, kv == 0 ? &maps.k : &maps.v, 64 * h, 0, (int)zt, &barKV[at.s]);
                        }
                    }
                }
                for (uint32_t i = Shape<kKT>(a, w, TM).stages; i > 0 && ok; --i, ++n, at = at.plus(1)) {  // the output's
                    ok = wait_warp(&barFree[at.s], at.ph ^ 1, a.err);
                    if (ok && lane == 0) mbar_arrive(&barKV[at.s]);
                }
            }
            // wait for the copies that no one consumed (only after a wait that gave up)
            if (!ok)
                for (uint32_t s = 0; s < C::kStages && s < n; ++s) wait_warp(&barKV[s], ((n - 1 - s) / C::kStages) & 1, a.err);
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------- tensor cores (one thread)
            if (lane == 0) {
                const uint64_t desc = tc::smem_desc_sw128(0, 16, 1024), desc_v = tc::smem_desc_sw128(0, kBox, 1024);
                const uint64_t q_desc = desc + (smem_addr(sQ) >> 4), kv_addr = smem_addr(sKV) >> 4;
                uint32_t u = 0, nFix = 0, nP[2] = {0, 0};
                using Pos = Pos<C::kStages>;
                Pos n;
                auto wait_stage = [&](Pos i) { if (ok) ok = wait_on(&barKV[i.s], i.ph, a.err); };
                auto free_stage = [&](Pos i) { tc::commit(&barFree[i.s]); };
                // S_g = Q_q K^T with K at position i of the ring
                auto qk = [&](int g, int q, Pos i) {
                    const uint64_t kb = desc + kv_addr + i.s * (C::kTile >> 4), qb = q_desc + q * (C::kTile >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint64_t at = ((ks >> 2) * kBox + (ks & 3) * 32) >> 4;
                        tc::mma_f16_ss(tmem + 128 * g, qb + at, kb + at, C::kIdescS, ks > 0);
                    }
                    tc::commit(&barS[g]);
                };
                // O_g (+)= P_g V with V at position i
                auto pv = [&](int g, Pos i, bool add) {
                    const uint64_t vb = desc_v + kv_addr + i.s * (C::kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < kKT / 16; ++kk)
                        mma_f16_ts(tmem + kColO + 128 * g, tmem + 128 * g + 64 * (kk >> 2) + 8 * (kk & 3), vb + kk * (16 * 128 >> 4), C::kIdescPV, add || kk > 0);
                };
                for (; more && ok; more = w.next(a, TQ), ++u) {
                    const PagedEntry& e = w.e;
                    const Shape<kKT> sh(a, w, TM);
                    const bool pair = sh.pair;
                    const int nt = w.t1 - w.t0, ahead = pair ? 2 : 1;  // a group's next tile
                    if (ok) ok = wait_on(&barQ, u & 1, a.err);
                    wait_stage(n);
                    if (!ok) break;
                    tc::fence_after_sync();
                    qk(0, 0, n);
                    if (pair) {
                        free_stage(n);
                        if (nt > 1) {
                            wait_stage(n.plus(2));
                            if (!ok) break;
                            tc::fence_after_sync();
                            qk(1, 0, n.plus(2));
                            free_stage(n.plus(2));
                        }
                    } else {
                        qk(1, 1, n);
                        free_stage(n);
                    }
                    if (nt <= ahead) tc::commit(&barQfree);
                    for (int k = 0; k < nt && ok; ++k, n = n.plus(2)) {
                        const bool more_tiles = k + ahead < nt;
                        const Pos v = n.plus(1), kn = n.plus(2 * ahead);
                        bool dirty = false;
                        wait_stage(v);
                        if (more_tiles) wait_stage(kn);
                        if (masked_tile(a, e, e.key_tile(w.t0 + k) * kKT)) {
                            if (ok) ok = wait_on(&barFix[nFix % kFixDepth], (nFix / kFixDepth) & 1, a.err);
                            dirty = (dirty_sh[nFix % kFixDepth][0] | dirty_sh[nFix % kFixDepth][1]) != 0;
                            ++nFix;
                        }
                        const int ga = pair ? k & 1 : 0, gb = pair ? ga : 1;
                        for (int g = ga; g <= gb && ok; ++g) {
                            ok = wait_on(&barP[g], nP[g] & 1, a.err);
                            ++nP[g];
                            if (!ok) break;
                            tc::fence_after_sync();
                            if (!dirty) pv(g, v, k >= ahead);
                            if (g == gb) free_stage(v);
                            if (more_tiles) {
                                qk(g, pair ? 0 : g, kn);
                                if (g == gb) {
                                    free_stage(kn);
                                    if (k + ahead + 1 == nt) tc::commit(&barQfree);  // the unit's last use of Q
                                }
                            } else {
                                tc::commit(&barO[g]);
                            }
                        }
                    }
                    n = n.plus(sh.stages);
                }
                tc::commit(&barDone);  // the issuing thread stays until its MMAs are done
                wait_on(&barDone, 0, a.err);
            }
        } else {
            // -------------------------------------------------------- V of the masked tiles
            // They pass every stage of the ring (and hand it back with the MMAs), so that they can
            // neither run ahead of it nor fall behind it.
            // The first of them also loads Q, as soon as the last unit's has been read.
            uint32_t u = 0, nFix = 0;
            Pos<C::kStages> at;
            const int f = tid - kFixWarp * 32;  // 0 .. 63
            for (; more && ok; more = w.next(a, TQ), ++u) {
                const PagedEntry& e = w.e;
                const int hi = e.last_pos();
                const Shape<kKT> sh(a, w, TM);
                if (warp == kFixWarp) {
                    if (u > 0) ok = wait_warp(&barQfree, (u - 1) & 1, a.err);
                    if (ok && lane == 0) {
                        const int tiles = sh.pair ? 1 : 2;
                        mbar_arrive_expect_tx(&barQ, tiles * C::H * a.G * TM * 128);
                        for (int g = 0; g < tiles; ++g)
                            for (int h = 0; h < C::H; ++h)
                                tma_load_3d(sQ + g * C::kTile + h * kBox, &maps.q, 64 * h, w.h * a.G, e.row0 + g * TM, &barQ);
                    }
                    __syncwarp();
                }
                for (int k = w.t0; k < w.t1 && ok; ++k) {
                    const int j0 = e.key_tile(k) * kKT;
                    ok = wait_warp(&barKV[at.s], at.ph, a.err);
                    if (ok && lane == 0) mbar_arrive(&barFree[at.s]);
                    at = at.plus(1);
                    if (ok) ok = wait_warp(&barKV[at.s], at.ph, a.err);
                    if (!ok) break;
                    if (masked_tile(a, e, j0)) {
                        unsigned char* sV = sKV + (size_t)at.s * C::kTile;
                        // rows seen by some row of the unit: [0, n_sink) and [n_lo, n_hi)
                        const int n_hi = max(0, min(kKT, hi - j0 + 1)), n_lo = max(0, min(n_hi, e.lo - j0));
                        const int n_sink = a.W > 0 ? max(0, min(n_lo, a.S - j0)) : 0;
                        auto zero = [&](int from, int to) {
                            for (int c = 8 * from + f; c < 8 * to; c += 64)
#pragma unroll
                                for (int h = 0; h < C::H; ++h)
                                    *reinterpret_cast<uint4*>(sV + h * kBox + (size_t)c * 16) = make_uint4(0u, 0u, 0u, 0u);
                        };
                        zero(n_sink, n_lo);
                        zero(n_hi, kKT);
                        fence_proxy_async();
                        uint32_t inf = 0;  // an exponent of all ones carries into its sign bit
                        auto look = [&](int from, int to) {  // (two chunks of each half a turn: little code, run seldom)
#pragma unroll 1
                            for (int c = 8 * from + f; c < 8 * to; c += 128)
#pragma unroll
                                for (int y = 0; y < 2 * C::H; ++y) {
                                    const int at = min(c + 64 * (y & 1), 8 * to - 1);
                                    const uint4 v = *reinterpret_cast<const uint4*>(sV + (y >> 1) * kBox + (size_t)at * 16);
                                    inf |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                                           ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
                                }
                        };
                        if (e.n > 1) {  // (a single token's rows see the same keys)
                            look(0, n_sink);
                            look(n_lo, n_hi);
                        }
                        const bool odd = __any_sync(kFull, (inf & 0x80008000u) != 0);
                        __syncwarp();
                        if (lane == 0) {
                            // (kFixDepth tiles on, the readers of this flag have passed: the ring holds fewer)
                            dirty_sh[nFix % kFixDepth][warp - kFixWarp] = odd ? (int)at.s + 1 : 0;
                            mbar_arrive(&barFix[nFix % kFixDepth]);
                        }
                        ++nFix;
                    }
                    if (lane == 0) mbar_arrive(&barFree[at.s]);
                    at = at.plus(1);
                }
                for (uint32_t i = sh.stages; i > 0 && ok; --i, at = at.plus(1)) {
                    ok = wait_warp(&barKV[at.s], at.ph, a.err);
                    if (ok && lane == 0) mbar_arrive(&barFree[at.s]);
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t run(const PagedDims& m, const PagedArgs& a, const void* Q, const void* kc, const void* vc, cudaStream_t s) {
    using C = Cfg<D>;
    static_assert(C::kSmem <= 227 * 1024, "shared memory");
    static_assert((kMaxRequests + 1) * 4 <= C::kStages * C::kTile, "the plan's scratch");
    const int TM = 128 / m.G, workers = sm_count();
    ChunkMaps maps;
    const uint64_t qd[3] = {(uint64_t)D, (uint64_t)m.Hq, (uint64_t)m.n_tokens}, qs[2] = {(uint64_t)D * 2, (uint64_t)m.q_stride * 2},
                   os[2] = {(uint64_t)D * 2, (uint64_t)m.Hq * D * 2};
    const uint32_t qb[3] = {64, (uint32_t)m.G, (uint32_t)TM};
    const uint64_t cd[3] = {(uint64_t)D, (uint64_t)m.page, (uint64_t)m.n_pages * m.Hkv}, cs[2] = {(uint64_t)D * 2, (uint64_t)m.page * D * 2};
    const uint32_t cb[3] = {64, (uint32_t)m.page, 1};
    if (!encode_tmap_bf16_3d(&maps.q, Q, qd, qs, qb) || !encode_tmap_bf16_3d(&maps.k, kc, cd, cs, cb) ||
        !encode_tmap_bf16_3d(&maps.v, vc, cd, cs, cb) || !encode_tmap_bf16_3d(&maps.o, a.O, qd, os, qb))
        return cudaErrorInvalidValue;
    static OncePerDevice once;
    cudaError_t e = once.run([] { return cudaFuncSetAttribute(paged_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem); });
    if (e != cudaSuccess) return e;
    count_launch();
    paged_chunk_kernel<D><<<workers, kThreads, C::kSmem, s>>>(maps, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_paged_merge<__nv_bfloat16, D>(a, workers, std::min(2 * TM, m.max_new) * m.G, s);
}

}  // namespace

int paged_chunk_rec_rows(const PagedDims& m) { return 128 / m.G * 2 * m.G; }
int paged_chunk_workers(const PagedDims&) { return sm_count(); }

cudaError_t launch_paged_chunk(const PagedDims& m, const PagedArgs& a, const void* Q, const void* kc, const void* vc,
                               cudaStream_t s) {
    return m.d == 64 ? run<64>(m, a, Q, kc, vc, s) : run<128>(m, a, Q, kc, vc, s);
}

}  // namespace cobs
