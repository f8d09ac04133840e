// tb_mx4.cu -- microscaled 4-bit floats: quantisation and its inverse.
//
// A block of 32 values along K shares one scale X = 2^(byte - 127); a value
// is stored as the 4-bit float c (sign, two exponent bits, one mantissa bit:
// 0, .5, 1, 1.5, 2, 3, 4, 6) with
//     X = 2^clamp(floor(log2 amax) - 2, -127, 127),   c = rne(w / X), saturating at 6,
// amax over the block's finite values.  All of it is exact: amax's exponent
// field E gives byte = max(E - 2, 0), w 2^(127 - byte) is an exact fp32
// product wherever the result rounds to a nonzero code, and the conversion
// instruction rounds half to even.
//
// Both kernels are bound by HBM: 2 or 4 bytes per weight on the wide side,
// 0.53 on the narrow one (17408 x 5120: fp32 to codes 66.5 us, 6.1 TB/s, codes
// to bf16 36.8 us, 6.1 TB/s; 4096 bf16 values 1.6 us, launch latency).  A warp holds a piece of one row, each lane 16 bytes
// of it per load (contiguous over the lanes), kLoads loads in flight; what is
// addressed after the first load is a constant away.  (With a division and
// 64-bit addresses per load the quantiser was bound by its instructions, 98 us
// on 17408 x 5120 fp32.)
#include "tb_async.cuh"
#include "tb_device.cuh"
#include "tb_internal.h"

#include <algorithm>
#include <cstring>

namespace tb {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;   // quantisation: 16-byte loads of a lane
constexpr int kStores = 8;  // dequantisation: 16-byte stores of a lane

// four values -> two bytes of codes, a in the lowest half-byte
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n .reg .b8 x, y;\n .reg .b16 h;\n cvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 y, %4, %3;\n mov.b16 h, {x, y};\n cvt.u32.u16 %0, h;\n}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

struct QuantArgs {
    const void* W;      // [N][ldw]
    uint8_t* codes;     // [N][K/2]
    uint8_t* scales;    // tiles
    int32_t* bad;       // or null
    int64_t K, ldw, G;  // G: 128-runs of a row
    int64_t warps;      // pieces of all rows
    uint32_t pieces;    // of a row
    int32_t own_bad;    // the only CTA: it writes the count itself
};

// The count that the quantiser adds to, set to 0.
__global__ void k_mx4_zero(int32_t* bad) {
    pdl_trigger();
    pdl_wait();
    *bad = 0;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) k_mx4_quantize(const QuantArgs A) {
    constexpr int V = DT == kF32 ? 4 : 8;   // values of a lane's 16 bytes
    constexpr int S = 32 * V;               // values of a warp's load
    constexpr int B = 32 / V;               // lanes of a block
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    int bad = 0;
    pdl_trigger();
    pdl_wait();
    if (id < A.warps) {
        const int64_t row = A.warps <= 0x7FFFFFFF ? (uint32_t)id / A.pieces : id / A.pieces;
        const int64_t k0 = (id - row * A.pieces) * (S * kLoads) + lane * V;
        const int left = (int)min(A.K - k0, (int64_t)(S * kLoads)), runs = (int)min(A.G * 128 - k0, (int64_t)(S * kLoads));
        const char* src = static_cast<const char*>(A.W) + (row * A.ldw + k0) * (DT == kF32 ? 4 : 2);
        uint4 v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            v[i] = i * S < left ? __ldcs(reinterpret_cast<const uint4*>(src + i * 512)) : make_uint4(0u, 0u, 0u, 0u);
        uint8_t* codes = A.codes + (row * A.K + k0) / 2;
        uint8_t* scale = A.scales + ((row >> 7) * A.G + (k0 >> 7)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
                         ((k0 >> 5) & 3);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            float f[V];
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (DT == kF32) {
                    f[j] = __uint_as_float(u[j]);
                } else {
                    f[2 * j] = __uint_as_float(u[j] << 16);
                    f[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
                }
            }
            float amax = 0.f, odd = 0.f;  // odd: no number as soon as a value is not finite
#pragma unroll
            for (int j = 0; j < V; ++j) {
                amax = fmaxf(amax, fabsf(f[j]));
                odd = fmaf(f[j], 0.f, odd);
            }
            if (odd != 0.f) {
                amax = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const uint32_t a = __float_as_uint(f[j]) & 0x7FFFFFFFu;
                    if (a < 0x7F800000u) {
                        amax = fmaxf(amax, fabsf(f[j]));
                    } else {
                        ++bad;
                        if (a > 0x7F800000u) f[j] = 0.f;  // NaN: code 0; an infinity saturates by itself
                    }
                }
            }
#pragma unroll
            for (int o = 1; o < B; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const uint32_t byte = (uint32_t)max((int)(__float_as_uint(amax) >> 23) - 2, 0);
            const float inv = __uint_as_float((254u - byte) << 23);
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] *= inv;
            if (i * S < left) {
                const uint32_t lo = encode4(f[0], f[1], f[2], f[3]);
                if constexpr (DT == kF32) {
                    *reinterpret_cast<uint16_t*>(codes + i * (S / 2)) = (uint16_t)lo;
                } else {
                    *reinterpret_cast<uint32_t*>(codes + i * (S / 2)) = lo | encode4(f[4], f[5], f[6], f[7]) << 16;
                }
            }
            // one lane of a block; blocks past K in the row's last run write their 0 too
            if ((lane & (B - 1)) == 0 && i * S < runs) scale[i * (S / 128) * 512] = (uint8_t)byte;
        }
    }
    if (A.bad) {
        bad = __reduce_add_sync(0xffffffffu, bad);
        if (A.own_bad) {
            __shared__ int part[kThreads / 32];
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = bad;
            __syncthreads();
            if (threadIdx.x == 0) {
                int t = 0;
                for (int w = 0; w < kThreads / 32; ++w) t += part[w];
                *A.bad = t;
            }
        } else {
            if ((threadIdx.x & 31) == 0 && bad) atomicAdd(A.bad, bad);  // of integers: the order does not matter
        }
    }
}

struct DequantArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    void* W;
    int64_t K, ldw, G, warps;
    uint32_t pieces;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) k_mx4_dequantize(const DequantArgs A) {
    constexpr int V = DT == kF32 ? 4 : 8;  // values of a lane's 16 bytes
    constexpr int S = 32 * V;              // values of a warp's store
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (id >= A.warps) return;
    const int64_t row = A.warps <= 0x7FFFFFFF ? (uint32_t)id / A.pieces : id / A.pieces;
    const int64_t k0 = (id - row * A.pieces) * (S * kStores) + lane * V;
    const int left = (int)min(A.K - k0, (int64_t)(S * kStores));
    const uint8_t* codes = A.codes + (row * A.K + k0) / 2;
    const uint8_t* scale = A.scales + ((row >> 7) * A.G + (k0 >> 7)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
                           ((k0 >> 5) & 3);
    char* out = static_cast<char*>(A.W) + (row * A.ldw + k0) * (DT == kF32 ? 4 : 2);
    uint32_t c[kStores], e[kStores];
#pragma unroll
    for (int i = 0; i < kStores; ++i) {
        const bool in = i * S < left;
        if constexpr (DT == kF32) c[i] = in ? __ldcs(reinterpret_cast<const uint16_t*>(codes + i * (S / 2))) : 0u;
        else c[i] = in ? __ldcs(reinterpret_cast<const uint32_t*>(codes + i * (S / 2))) : 0u;
        e[i] = in ? scale[i * (S / 128) * 512] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kStores; ++i) {
        if (i * S >= left) break;
        // 2^(byte - 127): below the normal range at 0, no number at 255
        const float x = e[i] == 0 ? __uint_as_float(0x00400000u)
                                  : (e[i] == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(e[i] << 23));
        float v[V];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            uint32_t h;
            asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}"
                : "=r"(h)
                : "r"(c[i] >> (8 * j)));
            v[2 * j] = __half2float(__ushort_as_half((unsigned short)h)) * x;
            v[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(h >> 16))) * x;
        }
        if constexpr (DT == kF32) {
            __stcs(reinterpret_cast<float4*>(out + i * 512), make_float4(v[0], v[1], v[2], v[3]));
        } else {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
            __stcs(reinterpret_cast<uint4*>(out + i * 512), make_uint4(u[0], u[1], u[2], u[3]));
        }
    }
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* W, int w_dtype, int64_t ldw, int64_t N, int64_t K, void* codes,
                                uint8_t* scales, int32_t* bad, cudaStream_t st) {
    QuantArgs A;
    A.W = W;
    A.codes = static_cast<uint8_t*>(codes);
    A.scales = scales;
    A.bad = bad;
    A.K = K;
    A.ldw = ldw;
    A.G = (K + 127) / 128;
    const int64_t piece = 32 * (w_dtype == kF32 ? 4 : 8) * kLoads;
    A.pieces = (uint32_t)((K + piece - 1) / piece);
    A.warps = N * A.pieces;
    const int64_t blocks = (A.warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    A.own_bad = blocks == 1;
    if (bad && blocks > 1) {
        void* args[] = {&bad};
        const cudaError_t e = launch_early(reinterpret_cast<const void*>(&k_mx4_zero), 1, 1, 0, 1, args, st);
        if (e != cudaSuccess) return e;
    }
    void* args[] = {&A};
    return launch_early(w_dtype == kF32 ? reinterpret_cast<const void*>(&k_mx4_quantize<kF32>)
                                        : reinterpret_cast<const void*>(&k_mx4_quantize<kBF16>),
                        blocks, kThreads, 0, 1, args, st);
}

cudaError_t launch_mx4_dequantize(const void* codes, const uint8_t* scales, int64_t N, int64_t K, void* W,
                                  int w_dtype, int64_t ldw, cudaStream_t st) {
    DequantArgs A;
    A.codes = static_cast<const uint8_t*>(codes);
    A.scales = scales;
    A.W = W;
    A.K = K;
    A.ldw = ldw;
    A.G = (K + 127) / 128;
    const int64_t piece = 32 * (w_dtype == kF32 ? 4 : 8) * kStores;
    A.pieces = (uint32_t)((K + piece - 1) / piece);
    A.warps = N * A.pieces;
    const int64_t blocks = (A.warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    void* args[] = {&A};
    return launch_early(w_dtype == kF32 ? reinterpret_cast<const void*>(&k_mx4_dequantize<kF32>)
                                        : reinterpret_cast<const void*>(&k_mx4_dequantize<kBF16>),
                        blocks, kThreads, 0, 1, args, st);
}

}  // namespace tb
