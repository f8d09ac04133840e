// tb_mx4_gemm.cu -- Y = X W^T of two microscaled 4-bit tensors on the
// block-scaled tensor cores (tcgen05.mma kind::mxf4).
//
//     Y[m][n] = sum over blocks b of 32 k:  Sw[n][b] Sx[m][b] sum_{k in b} w[n][k] x[m][k]
//
// The MMA reads the packed nibbles and the scale bytes as they are stored:
// nothing is decoded, so a small batch streams W at the copy engine's pace
// and a prefill batch runs at the 4-bit rate.  Every product is exact; the
// sums are the MMA's fp32 accumulation.
//
// k_mx4_gemm, small batches and outputs that tensor stores cannot write.  The
// weights are the MMA's A (128 rows of W, so a few batch rows waste no tensor
// rows) and the batch its B (NT = 16 .. 128 rows of X).  A unit is (128 rows
// of W, NT rows of X); K goes by chunks of 256 (128-byte rows, the swizzle
// span).  Units too few for the GPU split their chunks over a cluster of S
// CTAs, which add their partial sums through distributed shared memory in
// rank order (deterministic; no workspace, no spinning on global memory);
// units enough run one after the other in persistent CTAs, S = 1.  Bound by
// W's bytes and, below about 10 us, by the fixed parts (launch, first copy,
// cluster sum, about 3 us): 4096 x 4096, one row, 4.6 us; 17408 x 5120, 61
// rows, 11.5 us (4.1 TB/s of W; the byte floor is 7.6).
// Below 128 rows a unit has all of them: the MMA takes X's scales from the
// first column of a tile of 128 rows, and no unit may begin inside one.
//
// k_mx4_prefill, whole tiles of large batches: below.  17408 x 5120, 4096
// rows: 162 us alone, 4.5 PFLOP/s (2.7 times the measured bf16 rate; the 4-bit
// rate is four times it), the tensor pipe busy 56 % of the time; 183 to 191
// back to back under the power cap.  Where rows of Y are not multiples of 16
// bytes the small-batch kernel runs instead, in blocks of 128 rows: 17407 x
// 5120, 4096 rows, 245 to 258 us.
//
// A CTA: a producer warp (per chunk two tensor copies, W and X, 128-byte
// swizzled, and bulk copies of the scale tiles), an MMA warp (scale tiles
// from shared into tensor memory, four MMAs of k = 64 per chunk; each stage
// has its own scale columns, so they are rewritten only after the MMAs that
// read them) and four or eight epilogue warps.  Every wait is bounded: one that gives up
// is counted, aborts the CTA and leaves NaN in its outputs.
#include "tb_async.cuh"
#include "tb_device.cuh"
#include "tb_internal.h"

#include <algorithm>
#include <cstring>

namespace tb {

__device__ unsigned int g_mx_timeouts = 0;

struct MxArgs {
    CUtensorMap wmap, xmap;  // codes: bytes {K/2, rows}, box {128, 128} / {128, NT}, 128-byte swizzle
    const uint8_t* wsf;      // scale tiles [ceil(N/128)][KT][512]
    const uint8_t* xsf;      // scale tiles [ceil(M/128)][KT][512]
    void* Y;                 // [M][ldy]
    int64_t N, ldy;
    long long wait_cycles;
    int32_t M, K, KC, KT, MB, ydt, stall;
    uint32_t units;
};

namespace {

constexpr int kRows = 128;
constexpr int kChunkK = 256;
constexpr int kABytes = kRows * kChunkK / 2;

template <int NT_, int STAGES_, int EPI_>
struct MxCfg {
    static constexpr int NT = NT_, STAGES = STAGES_, EPI = EPI_;
    static constexpr int kB = NT * kChunkK / 2;
    static constexpr int kStage = kABytes + kB + 2048;
    static constexpr int kSfCols = 16;  // per stage: W's two tiles of 4 columns, X's
    static constexpr int kDCols = NT < 32 ? 32 : NT;
    static constexpr int kCols = kDCols + STAGES * kSfCols;
    static constexpr int kTmem = kCols <= 64 ? 64 : (kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512));
    static constexpr int kThreads = (2 + EPI) * 32;
    static constexpr int smem(int S) { return STAGES * kStage + 1024 + (S > 1 ? NT * kRows * 4 : 0); }
    static constexpr int per_sm(int S) {
        const int a = (227 * 1024) / (smem(S) + 1024 + 512), b = 512 / kTmem;
        return a < b ? a : b;
    }
    static_assert(kCols <= 512 && kStage % 1024 == 0, "tensor memory, swizzle atoms");
};
using Mx16 = MxCfg<16, 4, 4>;
using Mx32 = MxCfg<32, 4, 8>;
using Mx64 = MxCfg<64, 3, 8>;
using Mx64Alone = MxCfg<64, 7, 8>;  // with an SM to itself: 61 rows x 17408 x 5120 14.7 -> 12.8 us
using Mx128 = MxCfg<128, 4, 8>;

constexpr float kMxNaN = __builtin_nanf("");

// K-major operand, 128-byte swizzle: rows of 128 bytes, 8-row atoms of 1 KB
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// a 512-byte scale tile: 32 rows of 16 bytes, 8-row core matrices 128 bytes apart, no swizzle
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}
// kind::mxf4 instruction descriptor: E2M1 A and B, both K-major, UE8M0 scales, M = 128, N = nt; `id` selects the
// scale bytes {id, id + 1} of a 32-bit column
__host__ __device__ constexpr uint32_t mx_idesc(int nt, int id) {
    return ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(nt >> 3) << 17) | (1u << 23) |
           ((uint32_t)(kRows >> 7) << 27) | ((uint32_t)id << 29);
}
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
        : "memory");
}
// a scale tile from shared memory to four columns of all four 32-lane parts of tensor memory
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::per_sm(2)) k_mx4_gemm(const __grid_constant__ MxArgs A, int S) {
    constexpr int NT = C::NT, ST = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[ST], empty[ST], dfull, dfree;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    volatile int* abort = &abort_sh;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = (sm_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t red = base + ST * C::kStage;  // S > 1: partial sums [source rank][column of the slice][row]
    const uint32_t rank = S > 1 ? cluster_rank() : 0u;
    const uint32_t cid = blockIdx.x / (uint32_t)S, ncl = gridDim.x / (uint32_t)S;
    const int c0 = (int)((int64_t)A.KC * rank / S), c1 = (int)((int64_t)A.KC * (rank + 1) / S);

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mb_init(sm_addr(&full[s]), 1);
            mb_init(sm_addr(&empty[s]), 1);
        }
        mb_init(sm_addr(&dfull), 1);
        mb_init(sm_addr(&dfree), C::EPI);
        abort_sh = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    if (S > 1) cluster_arrive();  // every CTA of the cluster has begun before any writes into another
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&tmem_sh)),
                     "r"((uint32_t)C::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc5_fence_before();
    __syncthreads();
    tc5_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_sh, 0);
    pdl_trigger();
    pdl_wait();
    fence_copies();
    int issued = 0, committed = 0;

    if (warp == 0) {
        // ---------------- producer ----------------
        if (lane == 0 && !A.stall) {
            bool ok = true;
            for (uint32_t u = cid; u < A.units && ok; u += ncl) {
                const uint32_t t = u / (uint32_t)A.MB, b = u - t * (uint32_t)A.MB;
                for (int c = c0; c < c1; ++c) {
                    const int s = issued % ST;
                    if (issued >= ST && !mb_wait(sm_addr(&empty[s]), (uint32_t)(issued / ST - 1) & 1u, A.wait_cycles,
                                                 abort, &g_mx_timeouts)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = base + s * C::kStage, bar = sm_addr(&full[s]);
                    const uint32_t sfb = 512u * (uint32_t)min(2, A.KT - 2 * c);  // bytes of a row tile's scales
                    mb_arrive_expect(bar, (uint32_t)(kABytes + C::kB) + 2u * sfb);
                    tma_load_2d(st, &A.wmap, c * (kChunkK / 2), (int)(t * kRows), bar);
                    tma_load_2d(st + kABytes, &A.xmap, c * (kChunkK / 2), (int)(b * NT), bar);
                    bulk_load(st + kABytes + C::kB, A.wsf + ((int64_t)t * A.KT + 2 * c) * 512, sfb, bar);
                    bulk_load(st + kABytes + C::kB + 1024,
                              A.xsf + ((int64_t)b * A.KT + 2 * c) * 512, sfb, bar);
                    ++issued;
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA: one elected lane waits and issues ----------------
        if (elect_one()) {
            bool ok = true;
            int n = 0, s = 0;
            uint32_t phase = 0;
            for (uint32_t u = cid; u < A.units && ok; u += ncl, ++n) {
                if (n > 0 && !mb_wait(sm_addr(&dfree), (uint32_t)(n - 1) & 1u, A.wait_cycles, abort, &g_mx_timeouts))
                    break;
                for (int c = c0; c < c1; ++c) {
                    if (!mb_wait(sm_addr(&full[s]), phase, A.wait_cycles, abort, &g_mx_timeouts)) {
                        ok = false;
                        break;
                    }
                    tc5_fence_after();
                    const uint32_t sa = base + s * C::kStage, sb = sa + kABytes, sf = sb + C::kB;
                    const uint32_t ta = tmem + C::kDCols + s * C::kSfCols, tb = ta + 8;
                    const int left = A.K - c * kChunkK;
                    const int nk = left >= 256 ? 4 : (left + 63) >> 6;
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
                        if (kt * 2 < nk) {
                            cp_scales(ta + kt * 4, desc_scales(sf + kt * 512));
                            cp_scales(tb + kt * 4, desc_scales(sf + 1024 + kt * 512));
                        }
                    const uint64_t da = desc_sw128(sa), db = desc_sw128(sb);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < nk)
                            mma_mx(tmem, da + 2 * j, db + 2 * j, mx_idesc(NT, 2 * (j & 1)), ta + (j >> 1) * 4,
                                   tb + (j >> 1) * 4, (c > c0 || j > 0) ? 1u : 0u);
                    tc5_commit_one(sm_addr(&empty[s]));
                    ++committed;
                    if (++s == ST) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) tc5_commit_one(sm_addr(&dfull));
            }
            // what is in flight ends before the exit (every commit follows the ones before it)
            if (*abort != 0 && committed > 0)
                mb_drain(sm_addr(&empty[(committed - 1) % ST]), (uint32_t)((committed - 1) / ST) & 1u, A.wait_cycles);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: rows 32 (warp % 4) .. + 31, columns EC e .. + EC - 1 ----------------
        constexpr int EC = NT / (C::EPI / 4);
        const int e = (warp - 2) >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t tcol = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(e * EC);
        const int lg = 31 - __clz(NT / S);  // S > 1: columns of a rank's slice, as a shift
        int n = 0;
        bool failed = false;
        for (uint32_t u = cid; u < A.units; u += ncl, ++n) {
            const uint32_t t = u / (uint32_t)A.MB, b = u - t * (uint32_t)A.MB;
            const int64_t row = (int64_t)t * kRows + r;
            const int m0 = (int)b * NT + e * EC, count = min(EC, A.M - m0);  // this warp's columns
            if (!failed)
                failed = !__all_sync(0xffffffffu, mb_wait(sm_addr(&dfull), (uint32_t)n & 1u, A.wait_cycles, abort,
                                                          &g_mx_timeouts));
            tc5_fence_after();
            if (S > 1) cluster_wait();
            const int64_t at = (int64_t)m0 * A.ldy + row;
            float* yf = static_cast<float*>(A.Y) + at;
            __nv_bfloat16* yb = static_cast<__nv_bfloat16*>(A.Y) + at;
#pragma unroll 1
            for (int cc = 0; cc < count; cc += 16) {
                uint32_t v[16];
                if (!failed) {
                    tc5_ld16(tcol + cc, v);
                    tc5_ld_wait();
                    tc5_ld_done(v);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(kMxNaN);
                }
                if (S > 1) {
                    // a column of this rank's partial sums goes to the rank whose slice it is in
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t m = (uint32_t)(e * EC + cc + i), to = m >> lg;
                        if (cc + i < count)
                            st_cluster_f32(map_rank(red + ((((rank - to) << lg) + m) * kRows + (uint32_t)r) * 4, to),
                                           __uint_as_float(v[i]));
                    }
                } else if (row < A.N) {
                    if (A.ydt == kF32) {
#pragma unroll
                        for (int i = 0; i < 16; ++i, yf += A.ldy)
                            if (cc + i < count) *yf = __uint_as_float(v[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i, yb += A.ldy)
                            if (cc + i < count) *yb = __float2bfloat16_rn(__uint_as_float(v[i]));
                    }
                }
            }
            tc5_fence_before();
            __syncwarp();
            if (lane == 0) mb_arrive(sm_addr(&dfree));
        }
    }

    // Tensor memory is given back before the cluster waits for its ranks: no CTA holds columns that another CTA of its SM
    // waits for while it waits itself for one that may be waiting for columns.
    tc5_fence_before();
    __syncthreads();
    tc5_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)C::kTmem)
                     : "memory");

    if (S > 1) {
        // every rank's partial sums have arrived: add this rank's slice of columns in rank order
        __syncwarp();
        if (warp < 2) cluster_wait();  // the first barrier (the epilogue warps waited above)
        cluster_arrive();
        cluster_wait();
        if (warp >= 2) {
            const uint32_t t = cid / (uint32_t)A.MB, b = cid - t * (uint32_t)A.MB;
            const int e = (warp - 2) >> 2, r = 32 * (warp & 3) + lane, cw = NT / S;
            const int64_t row = (int64_t)t * kRows + r, m0 = (int64_t)b * NT + (int64_t)rank * cw;
            const int count = (int)min((int64_t)cw, (int64_t)A.M - m0);
            const float* p = reinterpret_cast<const float*>(smem_raw + (red - sm_addr(smem_raw))) + r;
            if (row < A.N)
                for (int c = e; c < count; c += C::EPI / 4) {
                    float sum = 0.f;
                    for (int q = 0; q < S; ++q) sum += p[(q * cw + c) * kRows];
                    const int64_t at = (m0 + c) * A.ldy + row;
                    if (A.ydt == kF32) static_cast<float*>(A.Y)[at] = sum;
                    else static_cast<__nv_bfloat16*>(A.Y)[at] = __float2bfloat16_rn(sum);
                }
        }
    }

    // ---------------- drain and exit ----------------
    const bool aborted = __syncthreads_or(*abort) != 0;
    if (aborted && warp == 0 && lane == 0)
        for (int k = issued > ST ? issued - ST : 0; k < issued; ++k)
            mb_drain(sm_addr(&full[k % ST]), (uint32_t)(k / ST) & 1u, A.wait_cycles);
    __syncthreads();
}

// ---- prefill: batches of whole tiles -----------------------------------------------------
// The same product with the roles exchanged: X's rows are the MMA's A (128 of them) and W's its B (NW = 128 or 256), so
// a thread of the epilogue holds consecutive outputs of a batch row.  They are rounded into a swizzled tile of shared
// memory and leave by tensor stores while the next unit's MMAs run (the accumulator is free as soon as it has been
// read; its 256 columns and the scales leave no room for a second one).  Y's rows and their used part have to be
// multiples of 16 bytes.
constexpr int kPreEpi = 8;
constexpr int kPreThreads = (2 + kPreEpi) * 32;
constexpr int kPreOut = 65536;  // staged outputs: 128 rows x 256 bf16 or 128 fp32

template <int NW_, int STAGES_>
struct PreCfg {
    static constexpr int NW = NW_, STAGES = STAGES_;
    static constexpr int NB = NW / 128;
    static constexpr int kB = NW * kChunkK / 2;
    static constexpr int kStage = kABytes + kB + 1024 + 1024 * NB;
    static constexpr int kSfCols = 8 + 8 * NB;
    static constexpr int kTmem = NW + STAGES * kSfCols <= 256 ? 256 : 512;
    static constexpr int kOut = NW == 256 ? kPreOut : kPreOut / 2;
    static constexpr int kSmem = STAGES * kStage + kOut + 1024;
    static_assert(NW + STAGES * kSfCols <= 512 && kSmem + 1024 <= 227 * 1024, "tensor and shared memory");
};

struct PreArgs {
    CUtensorMap xmap, wmap;  // codes, boxes {128, 128} and {128, NW}
    CUtensorMap ymap;        // outputs: {N, M}, box {128 bytes, 128 rows}, 128-byte swizzle
    const uint8_t* xsf;
    const uint8_t* wsf;
    long long wait_cycles;
    int64_t N;
    int32_t M, K, KC, KT, TW, ydt, stall;  // TW: tiles of W
    uint32_t units, group;                 // units run over the batch tiles within groups of W tiles
};

template <class C>
__global__ void __launch_bounds__(kPreThreads, 1) k_mx4_prefill(const __grid_constant__ PreArgs A) {
    constexpr int NW = C::NW, ST = C::STAGES, NB = C::NB;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[ST], empty[ST], dfull, dfree;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    volatile int* abort = &abort_sh;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = (sm_addr(smem_raw) + 1023u) & ~1023u, out = base + ST * C::kStage;
    const uint32_t MB = (uint32_t)((A.M + kRows - 1) / kRows);
    // unit u: groups of A.group tiles of W, in a group every batch tile with each of its tiles
    auto place = [&](uint32_t u, uint32_t& m, uint32_t& w) {
        const uint32_t per = A.group * MB, g = u / per, in = u - g * per;
        const uint32_t width = min(A.group, (uint32_t)A.TW - g * A.group);
        m = in / width;
        w = g * A.group + in - m * width;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mb_init(sm_addr(&full[s]), 1);
            mb_init(sm_addr(&empty[s]), 1);
        }
        mb_init(sm_addr(&dfull), 1);
        mb_init(sm_addr(&dfree), kPreEpi);
        abort_sh = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&tmem_sh)),
                     "r"((uint32_t)C::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc5_fence_before();
    __syncthreads();
    tc5_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_sh, 0);
    pdl_trigger();
    pdl_wait();
    fence_copies();
    int issued = 0;

    if (warp == 0) {
        // ---------------- producer ----------------
        if (lane == 0 && !A.stall) {
            bool ok = true;
            for (uint32_t u = blockIdx.x; u < A.units && ok; u += gridDim.x) {
                uint32_t m, w;
                place(u, m, w);
                const bool two = NB == 2 && (int64_t)w * NW + 128 < A.N;
                const uint8_t* xs = A.xsf + (int64_t)m * A.KT * 512;
                const uint8_t* ws = A.wsf + (int64_t)w * NB * A.KT * 512;
                for (int c = 0; c < A.KC; ++c) {
                    const int s = issued % ST;
                    if (issued >= ST && !mb_wait(sm_addr(&empty[s]), (uint32_t)(issued / ST - 1) & 1u, A.wait_cycles,
                                                 abort, &g_mx_timeouts)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = base + s * C::kStage, bar = sm_addr(&full[s]), sf = st + kABytes + C::kB;
                    const uint32_t sfb = 512u * (uint32_t)min(2, A.KT - 2 * c);
                    mb_arrive_expect(bar, (uint32_t)(kABytes + C::kB) + sfb * (two ? 3u : 2u));
                    tma_load_2d(st, &A.xmap, c * (kChunkK / 2), (int)(m * kRows), bar);
                    tma_load_2d(st + kABytes, &A.wmap, c * (kChunkK / 2), (int)(w * NW), bar);
                    bulk_load(sf, xs + (int64_t)c * 1024, sfb, bar);
                    bulk_load(sf + 1024, ws + (int64_t)c * 1024, sfb, bar);
                    if (two) bulk_load(sf + 2048, ws + ((int64_t)A.KT + 2 * c) * 512, sfb, bar);
                    ++issued;
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA ----------------
        if (elect_one()) {
            bool ok = true;
            int n = 0, s = 0, last = -1;
            uint32_t phase = 0;
            for (uint32_t u = blockIdx.x; u < A.units && ok; u += gridDim.x, ++n) {
                if (n > 0 && !mb_wait(sm_addr(&dfree), (uint32_t)(n - 1) & 1u, A.wait_cycles, abort, &g_mx_timeouts))
                    break;
                for (int c = 0; c < A.KC; ++c) {
                    if (!mb_wait(sm_addr(&full[s]), phase, A.wait_cycles, abort, &g_mx_timeouts)) {
                        ok = false;
                        break;
                    }
                    tc5_fence_after();
                    const uint32_t sa = base + s * C::kStage, sb = sa + kABytes, sf = sb + C::kB;
                    const uint32_t ta = tmem + NW + s * C::kSfCols, tb = ta + 8;
                    const int left = A.K - c * kChunkK;
                    const int nk = left >= 256 ? 4 : (left + 63) >> 6;
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
                        if (kt * 2 < nk) {
                            cp_scales(ta + kt * 4, desc_scales(sf + kt * 512));
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                cp_scales(tb + kt * 4 * NB + nb * 4, desc_scales(sf + 1024 + nb * 1024 + kt * 512));
                        }
                    const uint64_t da = desc_sw128(sa), db = desc_sw128(sb);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < nk)
                            mma_mx(tmem, da + 2 * j, db + 2 * j, mx_idesc(NW, 2 * (j & 1)), ta + (j >> 1) * 4,
                                   tb + (j >> 1) * 4 * NB, (c > 0 || j > 0) ? 1u : 0u);
                    tc5_commit_one(sm_addr(&empty[s]));
                    last = s | (int)phase << 8;
                    if (++s == ST) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) tc5_commit_one(sm_addr(&dfull));
            }
            if (*abort != 0 && last >= 0)
                mb_drain(sm_addr(&empty[last & 255]), (uint32_t)last >> 8, A.wait_cycles);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue ----------------
        const int e = (warp - 2) >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const int per = A.ydt == kF32 ? 32 : 64;                  // outputs of a 128-byte row of a box
        const int cp = C::kOut / 128 / (A.ydt == kF32 ? 4 : 2);  // columns staged at once
        const uint32_t rowp = out + (uint32_t)r * 128u;
        const uint32_t sw = (uint32_t)(r & 7);
        int n = 0;
        bool failed = false, pending = false;
        for (uint32_t u = blockIdx.x; u < A.units; u += gridDim.x, ++n) {
            uint32_t m, w;
            place(u, m, w);
            if (!failed)
                failed = !__all_sync(0xffffffffu, mb_wait(sm_addr(&dfull), (uint32_t)n & 1u, A.wait_cycles, abort,
                                                          &g_mx_timeouts));
            tc5_fence_after();
            for (int c0 = 0; c0 < NW; c0 += cp) {
                // the stores of what was staged before have read it
                if (pending && warp == 2 && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                asm volatile("bar.sync 1, %0;" ::"n"(kPreEpi * 32) : "memory");
#pragma unroll 1
                for (int cc = e * (cp / 2); cc < (e + 1) * (cp / 2); cc += 32) {  // columns c0 + cc .. + 31
                    uint32_t v[2][16];
                    if (!failed) {
                        tc5_ld16(lanes + (uint32_t)(c0 + cc), v[0]);
                        tc5_ld16(lanes + (uint32_t)(c0 + cc + 16), v[1]);
                        tc5_ld_wait();
                        tc5_ld_done(v[0]);
                        tc5_ld_done(v[1]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[0][i] = v[1][i] = __float_as_uint(kMxNaN);
                    }
                    const uint32_t box = rowp + (uint32_t)(cc / per) * 16384u;
                    if (A.ydt == kF32) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            st_shared_v4(box + (((uint32_t)q ^ sw) << 4), v[q >> 2][4 * (q & 3)], v[q >> 2][4 * (q & 3) + 1],
                                         v[q >> 2][4 * (q & 3) + 2], v[q >> 2][4 * (q & 3) + 3]);
                    } else {
                        const uint32_t p0 = (uint32_t)(cc & 63) >> 3;  // 16-byte piece of the row: 0 or 4
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t b[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int j = 8 * (q & 1) + 2 * i;
                                const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[q >> 1][j]),
                                                                               __uint_as_float(v[q >> 1][j + 1]));
                                b[i] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            st_shared_v4(box + (((p0 + (uint32_t)q) ^ sw) << 4), b[0], b[1], b[2], b[3]);
                        }
                    }
                }
                if (c0 + cp >= NW) {  // the accumulator has been read
                    tc5_fence_before();
                    __syncwarp();
                    if (lane == 0) mb_arrive(sm_addr(&dfree));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                asm volatile("bar.sync 1, %0;" ::"n"(kPreEpi * 32) : "memory");
                if (warp == 2 && lane == 0) {
                    for (int b = 0; b < cp / per; ++b) {
                        const int64_t x = (int64_t)w * NW + c0 + b * per;
                        if (x < A.N) tma_store_2d(&A.ymap, (int)x, (int)(m * kRows), out + (uint32_t)b * 16384u);
                    }
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
                pending = true;
            }
        }
        if (pending && warp == 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        tc5_fence_before();
    }

    // ---------------- drain and exit ----------------
    const bool aborted = __syncthreads_or(*abort) != 0;
    if (aborted && warp == 0 && lane == 0)
        for (int k = issued > ST ? issued - ST : 0; k < issued; ++k)
            mb_drain(sm_addr(&full[k % ST]), (uint32_t)(k / ST) & 1u, A.wait_cycles);
    tc5_fence_before();
    __syncthreads();
    tc5_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)C::kTmem)
                     : "memory");
}

using Pre256 = PreCfg<256, 3>;
using Pre128 = PreCfg<128, 5>;

bool encode_codes(CUtensorMap* map, const void* codes, int64_t rows, int64_t K, int box_rows) {
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t box[2] = {kChunkK / 2, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Asked how many clusters of k_mx4_gemm the device holds, the runtime answers as for one CTA per SM, since the kernel
// allocates tensor memory: 148 / 74 / 33 / 15 clusters of 1 / 2 / 4 / 8.  By its shared memory and its columns two fit (up to
// 64 batch rows), and two run: 71 clusters of four (71 units of 4096 values of K, one row) take 6.6 us, 72 take 9.3.  This
// kernel has none, and is asked instead.
__global__ void k_mx4_room() {}

// CTAs of S > 1 to a unit: units that run at once
template <class C>
int64_t units_held(int S) {
    struct Room;
    const void* fn = reinterpret_cast<const void*>(&k_mx4_room);
    if (once_per_device<Room>(
            [&] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024); }) != cudaSuccess)
        return 0;
    return clusters_at_once<C>(fn, C::kThreads, (size_t)C::smem(S), S);
}

// CTAs that share a unit's K.  In chunks of one CTA, about 0.32 us: a chunk takes 1.6 times as long for each of two CTAs that
// share an SM; a cluster costs 1 + 0.3 S for its barriers and (0.09 + 0.1 / S) per batch row for adding the partial sums,
// 3.5 for each round after the first.  Measured on 515 products of 1 to 128 rows, from 70 x 128 to 17408 x 17408: within
// 1.2 % of the best of 1, 2, 4 and 8 on average, 22 % at worst.  4096 x 4096, one row: 8.5 / 6.9 / 4.9 / 7.1 us with 1 / 2 /
// 4 / 8 CTAs; 9216 x 4096, one row: 7.7 / 5.9 / 9.3 / 12.0 (72 clusters of four are one too many); 2048 x 5120, 40 rows:
// 8.6 / 9.2 / 6.7 / 10.9 (16 of eight likewise); 17408 x 5120, 61 rows: 11.5 with one, 18.5 with two.
int split_of(int nt, int64_t units, int KC, int sms) {
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= 8 && s <= KC; s *= 2) {
        const bool alone = nt == 128 || (nt == 64 && units * s <= sms);
        const int64_t held = s == 1        ? (int64_t)sms * (alone ? 1 : 2)
                             : nt == 16    ? units_held<Mx16>(s)
                             : nt == 32    ? units_held<Mx32>(s)
                             : nt == 128   ? units_held<Mx128>(s)
                             : alone       ? units_held<Mx64Alone>(s)
                                           : units_held<Mx64>(s);
        if (held < 1 || (s > 1 && units > 4 * held)) continue;  // (of many rounds, whole units are the shortest)
        const double rounds = (double)((units + held - 1) / held);
        const double chunks = ((KC + s - 1) / s) * (units * s > sms && !alone ? 1.6 : 1.0);
        const double cost = s == 1 ? rounds * chunks
                                   : rounds * (chunks + 1 + 0.3 * s + nt * (0.09 + 0.1 / s)) + 3.5 * (rounds - 1);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

template <class C>
cudaError_t launch(MxArgs& A, int64_t units, int S, cudaStream_t st, int sms) {
    const int64_t ctas = S > 1 ? units * S : std::min<int64_t>(units, (int64_t)sms * C::per_sm(1));
    A.units = (uint32_t)units;
    const void* fn = reinterpret_cast<const void*>(&k_mx4_gemm<C>);
    const int smem = C::smem(S);
    const cudaError_t e = once_per_device<C>([&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(2));
    });
    if (e != cudaSuccess) return e;
    void* args[] = {&A, &S};
    return launch_early(fn, ctas, C::kThreads, (size_t)smem, S, args, st);
}

// outputs: rows of N, boxes of 128 bytes x 128 rows
bool encode_out(CUtensorMap* map, void* Y, int ydt, int64_t ldy, int64_t M, int64_t N) {
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    const int es = ydt == kF32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
    const cuuint64_t strides[1] = {(cuuint64_t)(ldy * es)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / es), kRows};
    const cuuint32_t el[2] = {1, 1};
    return enc(map, ydt == kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, Y, dims,
               strides, box, el, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t launch_prefill(PreArgs& A, const void* w, const void* x, int64_t K, cudaStream_t st, int sms) {
    A.TW = (int32_t)((A.N + C::NW - 1) / C::NW);
    const int64_t units = (int64_t)A.TW * ((A.M + kRows - 1) / kRows);
    if (units > 0x7FFFFFFF || !encode_codes(&A.xmap, x, A.M, K, kRows) || !encode_codes(&A.wmap, w, A.N, K, C::NW))
        return cudaErrorInvalidValue;
    A.units = (uint32_t)units;
    // the units that run at once form a block of about sqrt(148) tiles of W by as many of X: what they read from L2
    // and, at long K, from HBM is least
    A.group = 12;
    const cudaError_t e = once_per_device<C>([&] {
        return cudaFuncSetAttribute(k_mx4_prefill<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    void* args[] = {&A};
    return launch_early(reinterpret_cast<const void*>(&k_mx4_prefill<C>), std::min<int64_t>(units, sms), kPreThreads, C::kSmem, 1,
                        args, st);
}

}  // namespace

cudaError_t launch_mx4_gemm(const void* w, const uint8_t* w_scales, const void* x, const uint8_t* x_scales, void* Y,
                            int ydt, int64_t ldy, int64_t M, int64_t N, int64_t K, long long wait_cycles, bool stall,
                            cudaStream_t st) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInitializationError;
    const int64_t T = (N + kRows - 1) / kRows, es = ydt == kF32 ? 4 : 2;
    const int64_t pre = ((M + kRows - 1) / kRows) * T;  // tiles of 128 x 128
    if (M > 128 && pre >= sms / 2 && reinterpret_cast<uintptr_t>(Y) % 16 == 0 && ldy * es % 16 == 0 &&
        N * es % 16 == 0) {  // tensor stores write whole 16-byte pieces of a row
        PreArgs A;
        std::memset(&A, 0, sizeof(A));
        if (!encode_out(&A.ymap, Y, ydt, ldy, M, N)) return cudaErrorInvalidValue;
        A.xsf = x_scales;
        A.wsf = w_scales;
        A.wait_cycles = wait_cycles;
        A.N = N;
        A.M = (int32_t)M;
        A.K = (int32_t)K;
        A.KC = (int32_t)((K + kChunkK - 1) / kChunkK);
        A.KT = (int32_t)((K + 127) / 128);
        A.ydt = ydt;
        A.stall = stall ? 1 : 0;
        if (pre >= 2 * sms) return launch_prefill<Pre256>(A, w, x, K, st, sms);
        return launch_prefill<Pre128>(A, w, x, K, st, sms);
    }
    MxArgs A;
    std::memset(&A, 0, sizeof(A));
    A.wsf = w_scales;
    A.xsf = x_scales;
    A.Y = Y;
    A.N = N;
    A.ldy = ldy;
    A.wait_cycles = wait_cycles;
    A.M = (int32_t)M;
    A.K = (int32_t)K;
    A.KC = (int32_t)((K + kChunkK - 1) / kChunkK);
    A.KT = (int32_t)((K + 127) / 128);
    A.ydt = ydt;
    A.stall = stall ? 1 : 0;
    const int nt = M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128));  // below 128 a unit has all batch rows
    A.MB = (int32_t)((M + nt - 1) / nt);
    const int64_t units = T * A.MB;
    if (units > 0x7FFFFFFF || !encode_codes(&A.wmap, w, N, K, kRows) || !encode_codes(&A.xmap, x, M, K, nt))
        return cudaErrorInvalidValue;
    const int S = split_of(nt, units, A.KC, sms);
    switch (nt) {
        case 16: return launch<Mx16>(A, units, S, st, sms);
        case 32: return launch<Mx32>(A, units, S, st, sms);
        case 64: return units * S <= sms ? launch<Mx64Alone>(A, units, S, st, sms) : launch<Mx64>(A, units, S, st, sms);
        default: return launch<Mx128>(A, units, S, st, sms);
    }
}

unsigned int take_mx_timeouts() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_mx_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    if (v != 0 && cudaMemcpyToSymbol(g_mx_timeouts, &z, sizeof(z)) != cudaSuccess) return 0xFFFFFFFFu;
    return v;
}

}  // namespace tb
