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
// 0.53 on the narrow one.  A half-warp holds 128 consecutive k of a row (the
// scale word of a row is then one 4-byte store), a thread 8 of them (one or
// two 16-byte loads), a block of 32 four threads (two shuffles for amax);
// kTasks consecutive 128-runs per half-warp keep that many loads in flight.
#include "tb_async.cuh"
#include "tb_device.cuh"
#include "tb_internal.h"

#include <algorithm>

namespace tb {
namespace {

constexpr int kThreads = 256;
constexpr int kTasks = 4;  // 128-runs per half-warp

// scale word of (row, 128-run): 512-byte tiles of 128 rows x 4 blocks
__device__ __forceinline__ int64_t scale_word(int64_t row, int64_t g, int64_t G) {
    return ((row >> 7) * G + g) * 128 + (row & 31) * 4 + ((row >> 5) & 3);
}

// eight values -> eight codes; w[0] in the lowest nibble
__device__ __forceinline__ uint32_t encode8(const float (&v)[8]) {
    uint32_t d;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

struct QuantArgs {
    const void* W;       // [N][ldw]
    uint32_t* codes;     // [N][K/8] words
    uint32_t* scales;    // tiles
    int32_t* bad;        // or null
    int64_t N, K, ldw, G, tasks;
    int32_t own_bad;     // the only CTA: it writes the count itself
};

template <int DT>
__device__ __forceinline__ void load8(const void* p, float (&v)[8]) {
    if constexpr (DT == kF32) {
        const float4 a = __ldcs(static_cast<const float4*>(p)), b = __ldcs(static_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = __ldcs(static_cast<const uint4*>(p));
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) k_mx4_quantize(const QuantArgs A) {
    const int lane16 = threadIdx.x & 15;
    const int64_t first = ((int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4)) * kTasks;
    int64_t row = first / A.G, g = first - row * A.G;
    float v[kTasks][8];
    int64_t rows[kTasks], gs[kTasks];
    bool in[kTasks];
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
        rows[i] = row;
        gs[i] = g;
        const int64_t k = g * 128 + lane16 * 8;
        in[i] = first + i < A.tasks && k < A.K;
        if (in[i]) {
            load8<DT>(static_cast<const char*>(A.W) + (row * A.ldw + k) * (DT == kF32 ? 4 : 2), v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
        if (++g == A.G) {
            g = 0;
            ++row;
        }
    }
    int bad = 0;
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
        uint32_t amax = 0;  // bits of |w|: ordered like the values
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t a = __float_as_uint(v[i][j]) & 0x7FFFFFFFu;
            if (a < 0x7F800000u) {
                amax = max(amax, a);
            } else {
                ++bad;
                if (a > 0x7F800000u) v[i][j] = 0.f;  // NaN: code 0; an infinity saturates by itself
            }
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = (int)(amax >> 23);
        const uint32_t byte = (uint32_t)max(e - 2, 0);
        const float inv = __uint_as_float((254u - byte) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= inv;
        const uint32_t c = encode8(v[i]);
        // the four blocks' bytes of this 128-run, in the half-warp's first lane
        uint32_t word = byte << (8 * (lane16 >> 2));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if (in[i]) A.codes[(rows[i] * A.K + gs[i] * 128) / 8 + lane16] = c;
        if (lane16 == 0 && first + i < A.tasks) A.scales[scale_word(rows[i], gs[i], A.G)] = word;
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
        } else if ((threadIdx.x & 31) == 0 && bad) {
            atomicAdd(A.bad, bad);  // an integer count: the order does not matter
        }
    }
}

struct DequantArgs {
    const uint32_t* codes;
    const uint32_t* scales;
    void* W;
    int64_t K, ldw, G, tasks;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) k_mx4_dequantize(const DequantArgs A) {
    const int lane16 = threadIdx.x & 15;
    const int64_t first = ((int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4)) * kTasks;
    int64_t row = first / A.G, g = first - row * A.G;
    uint32_t c[kTasks], s[kTasks];
    int64_t at[kTasks];
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
        const int64_t k = g * 128 + lane16 * 8;
        const bool in = first + i < A.tasks && k < A.K;
        at[i] = in ? row * A.ldw + k : -1;
        c[i] = in ? __ldcs(A.codes + (row * A.K + k) / 8) : 0u;
        s[i] = in ? __ldg(A.scales + scale_word(row, g, A.G)) : 0u;
        if (++g == A.G) {
            g = 0;
            ++row;
        }
    }
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
        if (at[i] < 0) continue;
        const uint32_t byte = (s[i] >> (8 * (lane16 >> 2))) & 255u;
        // 2^(byte - 127): below the normal range at 0, no number at 255
        const float x = byte == 0 ? __uint_as_float(0x00400000u)
                                  : (byte == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23));
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h;
            asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}"
                : "=r"(h)
                : "r"(c[i] >> (8 * j)));
            v[2 * j] = __half2float(__ushort_as_half((unsigned short)h)) * x;
            v[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(h >> 16))) * x;
        }
        if constexpr (DT == kF32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(A.W) + at[i]);
            __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
            __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
        } else {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
            __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.W) + at[i]), make_uint4(u[0], u[1], u[2], u[3]));
        }
    }
}

bool blocks_of(int64_t tasks, unsigned* blocks) {
    const int64_t b = (tasks + kThreads / 16 * kTasks - 1) / (kThreads / 16 * kTasks);
    if (b > 0x7FFFFFFF) return false;
    *blocks = (unsigned)b;
    return true;
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* W, int w_dtype, int64_t ldw, int64_t N, int64_t K, void* codes,
                                uint8_t* scales, int32_t* bad, cudaStream_t st) {
    QuantArgs A;
    A.W = W;
    A.codes = static_cast<uint32_t*>(codes);
    A.scales = reinterpret_cast<uint32_t*>(scales);
    A.bad = bad;
    A.N = N;
    A.K = K;
    A.ldw = ldw;
    A.G = (K + 127) / 128;
    A.tasks = N * A.G;
    unsigned blocks;
    if (!blocks_of(A.tasks, &blocks)) return cudaErrorInvalidValue;
    A.own_bad = blocks == 1;
    if (bad && blocks > 1) {
        const cudaError_t e = cudaMemsetAsync(bad, 0, sizeof(int32_t), st);
        if (e != cudaSuccess) return e;
    }
    if (w_dtype == kF32) k_mx4_quantize<kF32><<<blocks, kThreads, 0, st>>>(A);
    else k_mx4_quantize<kBF16><<<blocks, kThreads, 0, st>>>(A);
    return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const void* codes, const uint8_t* scales, int64_t N, int64_t K, void* W,
                                  int w_dtype, int64_t ldw, cudaStream_t st) {
    DequantArgs A;
    A.codes = static_cast<const uint32_t*>(codes);
    A.scales = reinterpret_cast<const uint32_t*>(scales);
    A.W = W;
    A.K = K;
    A.ldw = ldw;
    A.G = (K + 127) / 128;
    A.tasks = N * A.G;
    unsigned blocks;
    if (!blocks_of(A.tasks, &blocks)) return cudaErrorInvalidValue;
    if (w_dtype == kF32) k_mx4_dequantize<kF32><<<blocks, kThreads, 0, st>>>(A);
    else k_mx4_dequantize<kBF16><<<blocks, kThreads, 0, st>>>(A);
    return cudaGetLastError();
}

}  // namespace tb
