// tb_moe_route.cu -- the router of a mixture-of-experts layer: logits,
// softmax and the k best experts of every token, in one launch.
//
//     l[t][e] = sum_h x[t][h] R[e][h]      (bf16 inputs, 64-bit sums)
//     ids[t]  = the k largest l[t], the lower index first among equals
//     w[t][j] = exp(l[t][ids[j]] - max l[t]) / (sum over the chosen, or over all, of the same)
//
// The sums are held in 64 bits because they decide an order: two experts'
// logits can be closer than fp32 sums of different order agree, and an expert
// picked by rounding is a different layer.
//
// A bf16 needs no more than the high word of a double (8 exponent and 7
// mantissa bits into 11 and 20), so x is converted once into high words in
// shared memory, and a weight's bits shifted right by 3 are, as the high
// word of a double, w 2^-896 exactly (both exponent fields start at 0, so
// zeros and subnormals map alike); the sums carry that factor.  (Exponent 255
// is mapped as if it were a number's.  A weight that is infinite or no number
// shows in a sum of the weights' products in pairs, one instruction for four
// weights; its row is summed again with the weights as they are.)  A product
// costs one DFMA, two and a half integer operations per weight shared by
// the tokens of the cluster.
//
// Bound by instructions, about 4.8 per DFMA: 64 tokens x 256 experts x 4096 take
// 17.0 us (16.2 without the watch on the weights; the DFMAs alone would take
// 3.7 us, the bytes 0.4); one token x 128 experts x 2048 takes 4.4 us, mostly launch, the
// cluster's barriers and the selection.
//
// A cluster of CTAs handles TB tokens: its warps take two experts
// each at a time (a token's words, the heaviest traffic, are read from shared
// memory once for both) and leave the logits in the shared memory of the CTA that
// selects for the token.  No workspace, no atomics.
#include "tb_async.cuh"
#include "tb_device.cuh"
#include "tb_internal.h"

#include <cstring>

namespace tb {

struct RouteArgs {
    const uint16_t* x;  // [T][ldx]
    const uint16_t* R;  // [E][H]
    int32_t* ids;       // [T][k]
    float* weights;     // [T][k]
    int64_t ldx;
    int32_t T, E, H, k, renorm;
    int32_t C;  // CTAs of a cluster
};

namespace {

constexpr int kRtUnroll = 4;  // 16-byte loads of the router in flight per lane

__device__ __forceinline__ double from_hi(uint32_t hi) { return __hiloint2double((int)hi, 0); }
// high word of w 2^-896 for the bf16 in the upper half of u
__device__ __forceinline__ uint32_t scaled_hi(uint32_t u) { return (uint32_t)((int32_t)u >> 3) & 0x8FFFE000u; }

// A sum of products of pairs of weights, which serves one question: it stops being finite as soon as one of the weights is
// not (an infinity times 0 is no number), and never becomes finite again.  (It may overflow without one: the row is then
// summed again for nothing.)
__device__ __forceinline__ uint32_t watch(uint32_t u0, uint32_t u1, uint32_t before) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(u0), "r"(u1), "r"(before));
    return d;
}
__device__ __forceinline__ bool not_finite(uint32_t pair) {
    return (pair & 0x7F800000u) == 0x7F800000u || (pair & 0x7F80u) == 0x7F80u;
}

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// order of the logits as unsigned integers; NaN below everything but 0, which marks a taken expert
__device__ __forceinline__ uint64_t order_key(double l) {
    if (l != l) return 1;
    const uint64_t b = (uint64_t)__double_as_longlong(l + 0.0);  // -0 equals +0
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// one warp: the k best of E logits, their softmax weights
template <int NPL>
__device__ void select_experts(const double* l, const RouteArgs& A, int64_t t) {
    const int lane = threadIdx.x & 31;
    uint64_t key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < A.E ? order_key(l[e]) : 0;
    }
    int mine = 0;  // the expert of slot `lane`
    double top = 0;
    for (int j = 0; j < A.k; ++j) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
        const uint32_t mhi = __reduce_max_sync(0xffffffffu, hi);
        const uint32_t mlo = __reduce_max_sync(0xffffffffu, hi == mhi ? lo : 0u);
        const uint32_t e = __reduce_min_sync(0xffffffffu, (hi == mhi && lo == mlo) ? (uint32_t)(lane + 32 * at) : ~0u);
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if ((uint32_t)(lane + 32 * i) == e) key[i] = 0;
        if (lane == j) mine = (int)e;
        if (j == 0) top = l[e];
    }
    const float p = lane < A.k ? expf((float)(l[mine] - top)) : 0.f;
    float sum = p;
    if (!A.renorm) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < A.E) sum += expf((float)(l[e] - top));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < A.k) {
        A.ids[t * A.k + lane] = mine;
        A.weights[t * A.k + lane] = p / sum;
    }
}

// The sum of row w over token t's activations, its weights converted as they are: rows with weights that are not finite.
__device__ __noinline__ double plain_sum(const uint4* w, const uint4* x, int H8) {
    double s = 0.0;
    for (int h = threadIdx.x & 31; h < H8; h += 32) {
        const uint4 v = w[h];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint4 a = x[half * H8 + h];
            const uint32_t hi[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s = fma((double)__uint_as_float(j & 1 ? u[2 * half + (j >> 1)] & 0xFFFF0000u : u[2 * half + (j >> 1)] << 16),
                        from_hi(hi[j]), s);
        }
    }
    return s;
}

constexpr int kRtWarps = 16;
constexpr int kRtThreads = kRtWarps * 32;
constexpr int kRtMaxSmem = 224 * 1024;

template <int TB>
__global__ void __launch_bounds__(kRtThreads, 1) k_moe_route(const RouteArgs A) {
    extern __shared__ __align__(16) uint8_t smem[];
    double* logits = reinterpret_cast<double*>(smem);                 // [E]: of this CTA's token
    uint32_t* xs = reinterpret_cast<uint32_t*>(smem + 8 * ((A.E + 1) & ~1));  // [TB][H] high words of x
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int64_t t0 = (int64_t)(blockIdx.x / A.C) * TB;
    const int nt = (int)min((int64_t)TB, A.T - t0);
    cluster_arrive();
    pdl_trigger();
    pdl_wait();
    const int H8 = A.H / 8;  // eights of x: their first four words in one plane, the others in a second
    for (int i0 = threadIdx.x; i0 < TB * H8; i0 += 4 * kRtThreads) {
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + q * kRtThreads, t = i / H8, h = i - t * H8;
            v[q] = make_uint4(0u, 0u, 0u, 0u);
            if (i < TB * H8 && t < nt) v[q] = *reinterpret_cast<const uint4*>(A.x + (t0 + t) * A.ldx + 8 * h);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + q * kRtThreads, t = i / H8, h = i - t * H8;
            if (i >= TB * H8) break;
            const uint32_t u[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
            uint32_t d[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[2 * j] = (uint32_t)__double2hiint((double)__uint_as_float(u[j] << 16));
                d[2 * j + 1] = (uint32_t)__double2hiint((double)__uint_as_float(u[j] & 0xFFFF0000u));
            }
            uint4* p = reinterpret_cast<uint4*>(xs) + t * 2 * H8 + h;
            p[0] = make_uint4(d[0], d[1], d[2], d[3]);
            p[H8] = make_uint4(d[4], d[5], d[6], d[7]);
        }
    }
    __syncthreads();
    cluster_wait();  // every CTA of the cluster has begun
    constexpr int EB = TB > 1 ? 2 : 1;  // experts of a warp's pass
    constexpr int U = kRtUnroll / EB;
    const int step = A.C * kRtWarps;
    uint32_t again = 0u;  // the warp's experts whose rows are not finite
    for (int e0 = (int)rank * kRtWarps + warp; e0 < A.E; e0 += EB * step) {
        const uint4* w[EB];
#pragma unroll
        for (int b = 0; b < EB; ++b)  // a pass without a second expert takes the first again
            w[b] = reinterpret_cast<const uint4*>(A.R + (int64_t)(e0 + b * step < A.E ? e0 + b * step : e0) * A.H);
        double acc[EB][TB];
#pragma unroll
        for (int b = 0; b < EB; ++b)
#pragma unroll
            for (int t = 0; t < TB; ++t) acc[b][t] = 0.0;
        uint32_t odd[EB];  // not finite as soon as a weight of the row is not
#pragma unroll
        for (int b = 0; b < EB; ++b) odd[b] = 0u;
        uint4 next[U][EB];
        auto load = [&](int h0) {
#pragma unroll
            for (int q = 0; q < U; ++q)
#pragma unroll
                for (int b = 0; b < EB; ++b)
                    next[q][b] = h0 + 32 * q < H8 ? w[b][h0 + 32 * q] : make_uint4(0u, 0u, 0u, 0u);
        };
        load(lane);
        for (int h0 = lane; h0 < H8; h0 += 32 * U) {
            uint4 v[U][EB];
#pragma unroll
            for (int q = 0; q < U; ++q)
#pragma unroll
                for (int b = 0; b < EB; ++b) v[q][b] = next[q][b];
            load(h0 + 32 * U);
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const int h = h0 + 32 * q;
                if (h >= H8) break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    double wd[EB][4];
#pragma unroll
                    for (int b = 0; b < EB; ++b) {
                        const uint32_t u0 = half ? v[q][b].z : v[q][b].x, u1 = half ? v[q][b].w : v[q][b].y;
                        wd[b][0] = from_hi(scaled_hi(u0 << 16));
                        wd[b][1] = from_hi(scaled_hi(u0));
                        wd[b][2] = from_hi(scaled_hi(u1 << 16));
                        wd[b][3] = from_hi(scaled_hi(u1));
                        odd[b] = watch(u0, u1, odd[b]);
                    }
#pragma unroll
                    for (int t = 0; t < TB; ++t) {
                        const uint4 a = reinterpret_cast<const uint4*>(xs)[(2 * t + half) * H8 + h];
                        const double x[4] = {from_hi(a.x), from_hi(a.y), from_hi(a.z), from_hi(a.w)};
#pragma unroll
                        for (int b = 0; b < EB; ++b)
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[b][t] = fma(wd[b][j], x[j], acc[b][t]);
                    }
                }
            }
        }
#pragma unroll
        for (int b = 0; b < EB; ++b) {
            const int e = e0 + b * step;
            if (__any_sync(0xffffffffu, not_finite(odd[b]))) again |= 1u << ((uint32_t)e / (uint32_t)step);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                double s = acc[b][t];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                // 2^896: 1023 + 896 in the exponent field
                if (lane == 0 && e < A.E)
                    st_cluster_f64(map_rank(sm_addr(logits + e), (uint32_t)t), s * from_hi(1919u << 20));
            }
        }
    }
    for (; again != 0u; again &= again - 1u) {
        const int e = (int)rank * kRtWarps + warp + (__ffs((int)again) - 1) * step;
        if (e >= A.E) break;  // (the first expert, taken again)
        for (int t = 0; t < TB; ++t) {
            double s = plain_sum(reinterpret_cast<const uint4*>(A.R + (int64_t)e * A.H),
                                 reinterpret_cast<const uint4*>(xs) + t * 2 * H8, H8);
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) st_cluster_f64(map_rank(sm_addr(logits + e), (uint32_t)t), s);
        }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (warp == 0 && (int)rank < nt) {
        if (A.E <= 128) select_experts<4>(logits, A, t0 + rank);
        else if (A.E <= 256) select_experts<8>(logits, A, t0 + rank);
        else select_experts<16>(logits, A, t0 + rank);
    }
}

size_t route_smem(int TB, int E, int H) { return (size_t)8 * ((E + 1) & ~1) + (size_t)TB * H * 4; }

template <int TB>
struct RouteKernel {
    static const void* fn() { return reinterpret_cast<const void*>(&k_moe_route<TB>); }
    static cudaError_t setup() {
        return once_per_device<RouteKernel>(
            [] { return cudaFuncSetAttribute(fn(), cudaFuncAttributeMaxDynamicSharedMemorySize, kRtMaxSmem); });
    }
};

// Cost of a choice: waves of clusters, each about 2.7 us and 3.1, 3.3 or 5.3 per expert of a warp at 4096 columns (TB of 1,
// 2 and 4; two experts share a pass above 1).  Measured without the watch on the weights, us by this choice / by
// one on T alone, 256 experts x 4096: 16 tokens 10.0 / 17.2, 24 tokens 10.1 / 15.3, 64 tokens 16.1 by both (with it 10.6, 10.6
// and 17.0).
template <int TB>
cudaError_t consider(const RouteArgs& A, double* least, int* tb, int* c) {
    const size_t smem = route_smem(TB, A.E, A.H);
    if (smem > kRtMaxSmem) return cudaSuccess;
    const cudaError_t e = RouteKernel<TB>::setup();
    if (e != cudaSuccess) return e;
    constexpr int EB = TB > 1 ? 2 : 1;
    constexpr double per = TB == 1 ? 3.1 : (TB == 2 ? 3.3 : 5.3);
    for (int C = 4; C <= 8; C += 4) {
        // (asked at the largest shared memory: one answer for every shape, whichever is called first)
        const int held = clusters_at_once<RouteKernel<TB>>(RouteKernel<TB>::fn(), kRtThreads, kRtMaxSmem, C);
        if (held < 1) continue;
        const int waves = ((A.T + TB - 1) / TB + held - 1) / held, experts = C * kRtWarps * EB;
        const double cost = waves * (2.7 + (A.E + experts - 1) / experts * EB * per * A.H / 4096);
        if (cost < *least) *least = cost, *tb = TB, *c = C;
    }
    return cudaSuccess;
}

template <int TB>
cudaError_t launch(RouteArgs& A, cudaStream_t st) {
    void* args[] = {&A};
    return launch_early(RouteKernel<TB>::fn(), (int64_t)((A.T + TB - 1) / TB) * A.C, kRtThreads, route_smem(TB, A.E, A.H), A.C,
                        args, st);
}

}  // namespace

bool moe_route_supported(int E, int64_t H) { return H <= INT32_MAX && route_smem(1, E, (int)H) <= kRtMaxSmem; }

cudaError_t launch_moe_route(const uint16_t* x, int64_t ldx, const uint16_t* router, int64_t T, int E, int64_t H, int k,
                             bool renorm, int32_t* ids, float* weights, cudaStream_t st) {
    RouteArgs A;
    std::memset(&A, 0, sizeof(A));
    A.x = x;
    A.R = router;
    A.ids = ids;
    A.weights = weights;
    A.ldx = ldx;
    A.T = (int32_t)T;
    A.E = E;
    A.H = (int32_t)H;
    A.k = k;
    A.renorm = renorm ? 1 : 0;
    double least = 1e300;
    int tb = 1;
    cudaError_t e = consider<1>(A, &least, &tb, &A.C);
    if (e == cudaSuccess && T > 1) e = consider<2>(A, &least, &tb, &A.C);
    if (e == cudaSuccess && T > 2) e = consider<4>(A, &least, &tb, &A.C);
    if (e != cudaSuccess) return e;
    if (A.C == 0) return cudaErrorInvalidConfiguration;  // the device holds no cluster of any of them
    return tb == 1 ? launch<1>(A, st) : (tb == 2 ? launch<2>(A, st) : launch<4>(A, st));
}

}  // namespace tb
