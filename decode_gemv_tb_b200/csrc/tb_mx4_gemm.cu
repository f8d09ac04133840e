// tb_mx4_gemm.cu -- Y = X W^T of two microscaled 4-bit tensors on the
// block-scaled tensor cores (tcgen05.mma kind::mxf4).
//
//     Y[m][n] = sum over blocks b of 32 k:  Sw[n][b] Sx[m][b] sum_{k in b} w[n][k] x[m][k]
//
// The MMA reads the packed nibbles and the scale bytes as they are stored:
// nothing is decoded, so a batch of one streams W at the copy engine's pace
// and a prefill batch runs at the 4-bit rate.  Every product is exact; the
// sums are the MMA's fp32 accumulation.
//
// Work.  The weights are the MMA's A (128 rows of W, so a few batch rows
// waste no tensor rows) and the batch its B (NT = 16 .. 256 rows of X).  A
// unit is (128 rows of W, NT rows of X); K goes by chunks of 256 (128-byte
// rows, the swizzle span).  Units too few for the GPU split their chunks
// over a cluster of S CTAs, which add their partial sums through distributed
// shared memory in rank order (deterministic; no workspace, no spinning on
// global memory); enough units run persistently, S = 1.
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
    static constexpr int NB = NT > 128 ? 2 : 1;  // 128-row scale tiles of X per unit
    static constexpr int kB = NT * kChunkK / 2;
    static constexpr int kStage = kABytes + kB + 1024 + 1024 * NB;
    static constexpr int kSfCols = 8 + 8 * NB;  // per stage: W's two tiles of 4 columns, X's
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
using Mx32 = MxCfg<32, 4, 4>;
using Mx64 = MxCfg<64, 3, 4>;
using Mx128 = MxCfg<128, 4, 4>;
using Mx256 = MxCfg<256, 4, 8>;

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
__global__ void __launch_bounds__(C::kThreads, 1) k_mx4_gemm(const __grid_constant__ MxArgs A, int S) {
    constexpr int NT = C::NT, ST = C::STAGES, NB = C::NB;
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
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&tmem_sh)),
                     "r"((uint32_t)C::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc5_fence_before();
    __syncthreads();
    tc5_fence_after();
    if (S > 1) cluster_arrive();  // every CTA of the cluster has begun before any writes into another
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_sh, 0);
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
                    const bool two = NB == 2 && (int64_t)b * NT + 128 < A.M;
                    mb_arrive_expect(bar, (uint32_t)(kABytes + C::kB) + sfb * (two ? 3u : 2u));
                    tma_load_2d(st, &A.wmap, c * (kChunkK / 2), (int)(t * kRows), bar);
                    tma_load_2d(st + kABytes, &A.xmap, c * (kChunkK / 2), (int)(b * NT), bar);
                    bulk_load(st + kABytes + C::kB, A.wsf + ((int64_t)t * A.KT + 2 * c) * 512, sfb, bar);
                    bulk_load(st + kABytes + C::kB + 1024,
                              A.xsf + ((int64_t)(b * (uint32_t)NT / 128u) * A.KT + 2 * c) * 512, sfb, bar);
                    if (two)
                        bulk_load(st + kABytes + C::kB + 2048,
                                  A.xsf + ((int64_t)(b * (uint32_t)NT / 128u + 1) * A.KT + 2 * c) * 512, sfb, bar);
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
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                cp_scales(tb + kt * 4 * NB + nb * 4, desc_scales(sf + 1024 + nb * 1024 + kt * 512));
                        }
                    const uint64_t da = desc_sw128(sa), db = desc_sw128(sb);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < nk)
                            mma_mx(tmem, da + 2 * j, db + 2 * j, mx_idesc(NT, 2 * (j & 1)), ta + (j >> 1) * 4,
                                   tb + (j >> 1) * 4 * NB, (c > c0 || j > 0) ? 1u : 0u);
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
        int n = 0;
        bool failed = false;
        for (uint32_t u = cid; u < A.units; u += ncl, ++n) {
            const uint32_t t = u / (uint32_t)A.MB, b = u - t * (uint32_t)A.MB;
            const int64_t row = (int64_t)t * kRows + r;
            const int m0 = (int)b * NT, mcount = min(NT, A.M - m0);
            if (!failed)
                failed = !__all_sync(0xffffffffu, mb_wait(sm_addr(&dfull), (uint32_t)n & 1u, A.wait_cycles, abort,
                                                          &g_mx_timeouts));
            tc5_fence_after();
            if (S > 1) cluster_wait();
#pragma unroll 1
            for (int cc = 0; cc < EC; cc += 16) {
                if (e * EC + cc >= mcount) break;
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
                    // column m of this rank's partial sums goes to rank m / (NT / S)
                    const uint32_t cw = (uint32_t)NT / (uint32_t)S;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t m = (uint32_t)(e * EC + cc + i), to = m / cw;
                        if ((int)m < mcount)
                            st_cluster_f32(map_rank(red + (((rank * cw + m - to * cw) * kRows + (uint32_t)r) << 2), to),
                                           __uint_as_float(v[i]));
                    }
                } else if (row < A.N) {
                    const int64_t at = (int64_t)(m0 + e * EC + cc) * A.ldy + row;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (e * EC + cc + i < mcount) {
                            if (A.ydt == kF32) static_cast<float*>(A.Y)[at + i * A.ldy] = __uint_as_float(v[i]);
                            else
                                static_cast<__nv_bfloat16*>(A.Y)[at + i * A.ldy] =
                                    __float2bfloat16_rn(__uint_as_float(v[i]));
                        }
                    }
                }
            }
            tc5_fence_before();
            __syncwarp();
            if (lane == 0) mb_arrive(sm_addr(&dfree));
        }
    }

    if (S > 1) {
        // every rank's partial sums have arrived: add this rank's slice of columns in rank order
        __syncwarp();
        if (warp < 2) cluster_wait();  // the first barrier (the epilogue warps waited above)
        cluster_arrive();
        cluster_wait();
        if (warp >= 2) {
            const uint32_t t = cid / (uint32_t)A.MB, b = cid - t * (uint32_t)A.MB;
            const int r = 32 * (warp & 3) + lane, cw = NT / S;
            const int64_t row = (int64_t)t * kRows + r;
            const float* p = reinterpret_cast<const float*>(smem_raw + (red - sm_addr(smem_raw))) + r;
            for (int c = 0; c < cw; ++c) {
                const int64_t m = (int64_t)b * NT + (int64_t)rank * cw + c;
                if (m >= A.M || row >= A.N) break;
                float sum = 0.f;
                for (int q = 0; q < S; ++q) sum += p[(q * cw + c) * kRows];
                if (A.ydt == kF32) static_cast<float*>(A.Y)[m * A.ldy + row] = sum;
                else static_cast<__nv_bfloat16*>(A.Y)[m * A.ldy + row] = __float2bfloat16_rn(sum);
            }
        }
    }

    // ---------------- drain and exit ----------------
    const bool aborted = __syncthreads_or(*abort) != 0;
    if (aborted) {
        if (warp == 0 && lane == 0)
            for (int k = issued > ST ? issued - ST : 0; k < issued; ++k)
                mb_drain(sm_addr(&full[k % ST]), (uint32_t)(k / ST) & 1u, A.wait_cycles);
    }
    tc5_fence_before();
    __syncthreads();
    tc5_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)C::kTmem)
                     : "memory");
}

int mx_sms() {
    static int sms[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (sms[dev] == 0) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) return 0;
        sms[dev] = v;
    }
    return sms[dev];
}

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

template <class C>
cudaError_t launch(MxArgs& A, int64_t units, cudaStream_t st, int sms) {
    // CTAs per unit: the split whose waves of chunks (plus about three chunks' time to start and finish a
    // CTA) are the shortest
    int S = 1;
    int64_t best = -1;
    for (int s = 1; s <= 8 && s <= A.KC && s <= C::NT / 2; s *= 2) {
        const int64_t slots = (int64_t)sms * C::per_sm(s);
        if (slots == 0 || (s > 1 && units * s > slots)) break;
        const int64_t cost = (units * s + slots - 1) / slots * ((A.KC + s - 1) / s + 3);
        if (best < 0 || cost < best) {
            best = cost;
            S = s;
        }
    }
    const int64_t ctas = S > 1 ? units * S : std::min<int64_t>(units, (int64_t)sms * C::per_sm(1));
    A.units = (uint32_t)units;
    const void* fn = reinterpret_cast<const void*>(&k_mx4_gemm<C>);
    const int smem = C::smem(S);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(2) <= 227 * 1024 ? C::smem(2) : C::smem(1));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    void* args[] = {&A, &S};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_mx4_gemm(const void* w, const uint8_t* w_scales, const void* x, const uint8_t* x_scales, void* Y,
                            int ydt, int64_t ldy, int64_t M, int64_t N, int64_t K, long long wait_cycles, bool stall,
                            cudaStream_t st) {
    const int sms = mx_sms();
    if (sms <= 0) return cudaErrorInitializationError;
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
    const int64_t T = (N + kRows - 1) / kRows;
    int nt = M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128));
    if (M > 128 && T * ((M + 255) / 256) >= sms) nt = 256;
    A.MB = (int32_t)((M + nt - 1) / nt);
    const int64_t units = T * A.MB;
    if (units > 0x7FFFFFFF || !encode_codes(&A.wmap, w, N, K, kRows) || !encode_codes(&A.xmap, x, M, K, nt))
        return cudaErrorInvalidValue;
    switch (nt) {
        case 16: return launch<Mx16>(A, units, st, sms);
        case 32: return launch<Mx32>(A, units, st, sms);
        case 64: return launch<Mx64>(A, units, st, sms);
        case 128: return launch<Mx128>(A, units, st, sms);
        default: return launch<Mx256>(A, units, st, sms);
    }
}

unsigned int take_mx_timeouts() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_mx_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    if (cudaMemcpyToSymbol(g_mx_timeouts, &z, sizeof(z)) != cudaSuccess) return 0xFFFFFFFFu;
    return v;
}

}  // namespace tb
