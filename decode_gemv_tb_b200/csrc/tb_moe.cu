// tb_moe.cu -- the routed experts of a mixture-of-experts layer for a few
// tokens, straight from the packed codes, in two launches.
//
//     h[t,e] = silu(Wg[e] x[t]) * (Wu[e] x[t]),   y[t] = sum_j w[t,j] Wd[ids[t,j]] h[t,ids[t,j]]
//
// Every expert that some token takes is read once per eight of its tokens:
// with few tokens the layer is bound by the bytes of the experts it touches
// (and, from there, by decoding them).
//
// Both kernels group the (token, choice) pairs by expert themselves, in
// shared memory (a 64-bit token mask per expert, a prefix sum over the
// experts): at most 1024 pairs, no extra launch, no atomics on floats.  A
// block is an expert with up to eight of its tokens -- the MMA's columns.
//
// The products run on mma.sync m16n8k16: 16 weight rows decoded in registers
// to bf16 (tb_device.cuh; exact, 4-bit codes with their power-of-two scale
// too), the tokens' activations as B fragments read as they are.  A lane of a
// quad owns 32 consecutive k of every 128-group in both operands, so a row's
// group is one 8-, 12- or 16-byte read per lane and no code is moved between
// lanes.  Weights stream through a private cp.async ring per warp.
//
// h is kept as two bf16 (high and low part, 16 significant bits together), so
// that the second product sees it as exactly as the fp32 sums it came from
// are worth; with at most four tokens both parts share one MMA (columns 0-3
// and 4-7).
//
// k_moe_up: a unit is (block, 16 rows of gate and of up); S warps of a CTA
// split K when units are few.  k_moe_down: a cluster of C CTAs holds 64 rows
// of H, its CTAs split the blocks; each warp adds its rows' results per
// token in shared memory, the ranks are added in order (deterministic).
#include "tb_async.cuh"
#include "tb_device.cuh"
#include "tb_internal.h"

#include <algorithm>
#include <cstring>

namespace tb {

struct MoeMat {
    const uint8_t* packed;
    const uint8_t* scales;
    int64_t rb;    // bytes of a packed row
    int32_t G;     // 128-groups of a row
    int32_t kind;  // 0: 2 bits, 1: 3 bits, 2: MX4
};

struct MoeArgs {
    MoeMat gate, up, down;
    const uint16_t* x;       // [T][ldx]
    const int32_t* ids;      // [T][k]
    const float* weights;    // [T][k]
    uint16_t *h_hi, *h_lo;   // [slots][I]
    void* y;                 // [T][ldy]
    int64_t ldx, ldy;
    int32_t T, k, E, H, I, ydt;
    int32_t S, C;
};

namespace {

constexpr int kMoeWarps = 4;
constexpr int kMoeThreads = kMoeWarps * 32;
constexpr int kCG = 2;     // 128-groups per step
constexpr int kStages = 3;
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxK;
constexpr int kScaleBytes = 128;  // per matrix and step: 16 rows x 8 bytes

// packed bytes of a row's group, and of a step's row in shared memory (padded: a quad-row read of eight rows
// touches every bank once)
__host__ __device__ constexpr int group_bytes(int kind) { return kind == 0 ? 32 : (kind == 1 ? 48 : 64); }
__host__ __device__ constexpr int row_stride(int kind) { return kind == 0 ? 96 : (kind == 1 ? 112 : 192); }
__host__ __device__ constexpr int mat_bytes(int kind) { return 16 * row_stride(kind) + kScaleBytes; }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 4 bytes, of which the first n (2 or 4) are read
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, uint32_t n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait_groups() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 ldg_plain(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// byte permute whose selector nibbles replicate a byte's sign where their top bit is set
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
// Eight 4-bit codes (nibble j: code j) as four bf16 pairs in order, times the scale pair s: the codes' magnitudes
// index the two bytes of the bf16 values in a byte permute, the sign bits follow as bit 7 of the high bytes.
__device__ __forceinline__ void decode_mx4(uint32_t w, uint32_t s, uint32_t (&r)[4]) {
    constexpr uint32_t kHi0 = 0x3F3F3F00u, kHi1 = 0x40404040u;  // 0 .5 1 1.5 | 2 3 4 6
    constexpr uint32_t kLo0 = 0xC0800000u, kLo1 = 0xC0804000u;
    const uint32_t m = w & 0x77777777u;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint32_t sel = p ? m >> 16 : m, raw = p ? w >> 16 : w;
        // a byte with its top bit set, replicated where the code's sign bit is: 0xFF, else 0x80
        const uint32_t sg = prmt(0x80808080u, 0x80808080u, raw) << 1;
        const uint32_t hi = and_or(sg, 0x80808080u, prmt(kHi0, kHi1, sel));
        const uint32_t lo = prmt(kLo0, kLo1, sel);
        r[2 * p] = mul_bf16x2(prmt(lo, hi, 0x5140), s);
        r[2 * p + 1] = mul_bf16x2(prmt(lo, hi, 0x7362), s);
    }
}
// 2^(byte - 127) as a bf16 pair: below the normal range at 0, no number at 255
__device__ __forceinline__ uint32_t mx4_scale_pair(uint32_t byte) {
    const uint32_t b = byte == 0 ? 0x0040u : (byte == 255 ? 0x7FC0u : byte << 7);
    return b | (b << 16);
}

// One 128-group of 16 rows times the columns in xf (and, with TWO, in xg): acc += s W x.  `row`: shared address of
// row lane/4 of the group, `sc`: of its scales (row r's are 8 r bytes on).
template <bool TWO>
__device__ __forceinline__ void group_product(int kind, uint32_t row, uint32_t sc, int t, const uint32_t (&xf)[16],
                                              const uint32_t (&xg)[16], float (&acc)[4]) {
    if (kind == 2) {
        const uint4 a = lds128(row + 16 * t), b = lds128(row + 8 * row_stride(2) + 16 * t);
        const uint32_t sa = mx4_scale_pair(lds8(sc + t)), sb = mx4_scale_pair(lds8(sc + 64 + t));
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t ra[4], rb[4];
            decode_mx4(wa[i], sa, ra);
            decode_mx4(wb[i], sb, rb);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mma_bf16(acc, ra[2 * j], rb[2 * j], ra[2 * j + 1], rb[2 * j + 1], xf[4 * i + 2 * j],
                         xf[4 * i + 2 * j + 1]);
                if (TWO)
                    mma_bf16(acc, ra[2 * j], rb[2 * j], ra[2 * j + 1], rb[2 * j + 1], xg[4 * i + 2 * j],
                             xg[4 * i + 2 * j + 1]);
            }
        }
        return;
    }
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    if (kind == 0) {
        const uint2 a = lds64(row + 8 * t), b = lds64(row + 8 * row_stride(0) + 8 * t);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t ra[8], rb[8];
            decode2_signed<2>(i ? a.y : a.x, ra);
            decode2_signed<2>(i ? b.y : b.x, rb);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mma_bf16(d, ra[2 * j], rb[2 * j], ra[2 * j + 1], rb[2 * j + 1], xf[8 * i + 2 * j],
                         xf[8 * i + 2 * j + 1]);
                if (TWO)
                    mma_bf16(d, ra[2 * j], rb[2 * j], ra[2 * j + 1], rb[2 * j + 1], xg[8 * i + 2 * j],
                             xg[8 * i + 2 * j + 1]);
            }
        }
    } else {
        uint32_t ra[16], rb[16];
        const uint32_t ar = row + 12 * t, br = ar + 8 * row_stride(1);
        decode3_signed(lds32(ar), lds32(ar + 4), lds32(ar + 8), ra);
        decode3_signed(lds32(br), lds32(br + 4), lds32(br + 8), rb);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            mma_bf16(d, ra[2 * j], rb[2 * j], ra[2 * j + 1], rb[2 * j + 1], xf[2 * j], xf[2 * j + 1]);
            if (TWO) mma_bf16(d, ra[2 * j], rb[2 * j], ra[2 * j + 1], rb[2 * j + 1], xg[2 * j], xg[2 * j + 1]);
        }
    }
    const float s0 = bf16_bits_to_float(lds16(sc)), s1 = bf16_bits_to_float(lds16(sc + 64));
    acc[0] = fmaf(s0, d[0], acc[0]);
    acc[1] = fmaf(s0, d[1], acc[1]);
    acc[2] = fmaf(s1, d[2], acc[2]);
    acc[3] = fmaf(s1, d[3], acc[3]);
}

// Requests rows row0 .. row0 + 15, groups g .. g + n - 1 (n = 1, 2) of a matrix into a stage.
__device__ __forceinline__ void load_step(const MoeMat& m, int64_t row0, int g, int n, uint32_t dst, int lane) {
    const int gb = group_bytes(m.kind), rs = row_stride(m.kind), cpr = kCG * gb / 16;  // 16-byte pieces of a row
    const uint8_t* src = m.packed + row0 * m.rb + (int64_t)g * gb;
    for (int c = lane; c < 16 * cpr; c += 32) {
        const int r = c / cpr, o = (c - r * cpr) * 16;
        if (o < n * gb) cp16(dst + r * rs + o, src + r * m.rb + o);
    }
    const uint32_t sd = dst + 16 * rs;
    if (m.kind == 2) {  // a word per row and group
        const int r = lane >> 1, i = lane & 1;
        const int64_t row = row0 + r;
        if (i < n)
            cp4(sd + r * 8 + i * 4, m.scales + (((row >> 7) * m.G + g + i) * 128 + (row & 31) * 4 + ((row >> 5) & 3)) * 4,
                4);
    } else if (lane < 16) {  // two bytes per row and group: one or two aligned words
        const int64_t at = (row0 + lane) * m.G + g;
        const bool odd = (at & 1) != 0;
        cp4(sd + lane * 8, m.scales + (at & ~(int64_t)1) * 2, odd || n == 2 ? 4 : 2);
        if (odd && n == 2) cp4(sd + lane * 8 + 4, m.scales + (at + 1) * 2, 2);
    }
}
// shared address of the scales of group g + i (i = 0, 1) of row `r` of a stage whose first group is g
__device__ __forceinline__ uint32_t scale_at(const MoeMat& m, int64_t row0, int g, int i, uint32_t dst, int r) {
    const uint32_t sd = dst + 16 * row_stride(m.kind) + r * 8;
    if (m.kind == 2) return sd + i * 4;
    return sd + ((uint32_t)(((row0 + r) * m.G + g) & 1) + i) * 2;
}

// ---- the pairs grouped by expert ---------------------------------------------------
struct MoeList {
    unsigned long long mask[kMoeMaxExperts];  // tokens of each expert
    uint16_t blk_expert[kMaxPairs];
    uint16_t blk_slot[kMaxPairs];  // first slot of a block
    uint8_t blk_count[kMaxPairs];
    uint8_t slot_token[kMaxPairs];
    int scan[2][kMoeWarps];
    int blocks, slots;
};

__device__ void build_list(MoeList& L, const MoeArgs& A) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < A.E; e += kMoeThreads) L.mask[e] = 0ull;
    __syncthreads();
    for (int p = tid; p < A.T * A.k; p += kMoeThreads) {
        const int e = A.ids[p];
        if (e >= 0 && e < A.E) atomicOr(&L.mask[e], 1ull << (p / A.k));  // a set: the order does not matter
    }
    __syncthreads();
    const int per = (A.E + kMoeThreads - 1) / kMoeThreads, e0 = tid * per, e1 = min(A.E, e0 + per);
    int slots = 0, blocks = 0;
    for (int e = e0; e < e1; ++e) {
        const int c = __popcll(L.mask[e]);
        slots += c;
        blocks += (c + 7) >> 3;
    }
    int s = slots, b = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int vs = __shfl_up_sync(0xffffffffu, s, o), vb = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            s += vs;
            b += vb;
        }
    }
    if (lane == 31) {
        L.scan[0][warp] = s;
        L.scan[1][warp] = b;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        s += L.scan[0][w];
        b += L.scan[1][w];
    }
    if (tid == kMoeThreads - 1) {
        L.slots = s;
        L.blocks = b;
    }
    s -= slots;
    b -= blocks;
    for (int e = e0; e < e1; ++e) {
        unsigned long long m = L.mask[e];
        for (int left = __popcll(m); left > 0; left -= 8) {
            L.blk_expert[b] = (uint16_t)e;
            L.blk_slot[b] = (uint16_t)s;
            const int n = min(8, left);
            L.blk_count[b++] = (uint8_t)n;
            for (int i = 0; i < n; ++i) {
                L.slot_token[s++] = (uint8_t)(__ffsll((long long)m) - 1);
                m &= m - 1;
            }
        }
    }
    __syncthreads();
}

// ---- gate and up -----------------------------------------------------------------------
__global__ void __launch_bounds__(kMoeThreads) k_moe_up(const __grid_constant__ MoeArgs A) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ MoeList L;
    __shared__ float part[2][kMoeWarps][256];  // K split: partial sums of gate and up, two units deep
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int gbytes = mat_bytes(A.gate.kind), stage = gbytes + mat_bytes(A.up.kind);
    const uint32_t base = sm_addr(ring) + warp * kStages * stage;
    pdl_wait();
    build_list(L, A);
    pdl_trigger();
    const int S = A.S, s = warp % S, ui = warp / S, per = kMoeWarps / S;
    const int tiles = A.I / 16, units = L.blocks * tiles;
    const int g0 = A.gate.G * s / S, g1 = A.gate.G * (s + 1) / S, steps = (g1 - g0 + kCG - 1) / kCG;
    const int ustep = (int)gridDim.x * per;
    int pu = (int)blockIdx.x * per + ui, ps = 0, issued = 0;  // the next step to request
    auto issue = [&]() {
        if (pu < units) {
            const int blk = pu / tiles, tile = pu - blk * tiles, g = g0 + ps * kCG;
            const int64_t row0 = (int64_t)L.blk_expert[blk] * A.I + tile * 16;
            const uint32_t dst = base + (issued % kStages) * stage;
            const int n = min(kCG, g1 - g);
            load_step(A.gate, row0, g, n, dst, lane);
            load_step(A.up, row0, g, n, dst + gbytes, lane);
            if (++ps == steps) {
                ps = 0;
                pu += ustep;
            }
        }
        ++issued;
        cp_commit_group();
    };
    for (int i = 0; i < kStages - 1; ++i) issue();
    int used = 0, flip = 0;
    for (int u = (int)blockIdx.x * per + ui; u < units; u += ustep, flip ^= 1) {
        const int blk = u / tiles, tile = u - blk * tiles, count = L.blk_count[blk], slot0 = L.blk_slot[blk];
        const int64_t row0 = (int64_t)L.blk_expert[blk] * A.I + tile * 16;
        const uint16_t* xr = A.x + (int64_t)(r < count ? L.slot_token[slot0 + r] : 0) * A.ldx + 32 * t;
        float ag[4] = {0.f, 0.f, 0.f, 0.f}, au[4] = {0.f, 0.f, 0.f, 0.f};
        for (int st = 0; st < steps; ++st) {
            cp_wait_groups<kStages - 2>();
            __syncwarp();
            const int g = g0 + st * kCG, n = min(kCG, g1 - g);
            const uint32_t src = base + (used % kStages) * stage;
#pragma unroll
            for (int i = 0; i < kCG; ++i) {
                if (i >= n) break;
                uint32_t xf[16];
                if (r < count) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 v = ld_act_u4(xr + (int64_t)(g + i) * 128 + 8 * q);
                        xf[4 * q] = v.x, xf[4 * q + 1] = v.y, xf[4 * q + 2] = v.z, xf[4 * q + 3] = v.w;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 16; ++q) xf[q] = 0u;
                }
                group_product<false>(A.gate.kind, src + r * row_stride(A.gate.kind) + i * group_bytes(A.gate.kind),
                                     scale_at(A.gate, row0, g, i, src, r), t, xf, xf, ag);
                group_product<false>(A.up.kind, src + gbytes + r * row_stride(A.up.kind) + i * group_bytes(A.up.kind),
                                     scale_at(A.up, row0, g, i, src + gbytes, r), t, xf, xf, au);
            }
            ++used;
            __syncwarp();
            issue();
        }
        if (S > 1) {
            float* p = part[flip][warp];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i * 32 + lane] = ag[i];
                p[128 + i * 32 + lane] = au[i];
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + ui), "r"(S * 32) : "memory");
            // warp s of the unit finishes registers i = s, s + S, ...
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i % S != s) continue;
                float sg = 0.f, su = 0.f;
                for (int w = 0; w < S; ++w) {
                    sg += part[flip][ui * S + w][i * 32 + lane];
                    su += part[flip][ui * S + w][128 + i * 32 + lane];
                }
                ag[i] = sg;
                au[i] = su;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = 2 * t + (i & 1);
            if ((S > 1 && i % S != s) || col >= count) continue;
            const float h = ag[i] / (1.f + expf(-ag[i])) * au[i];
            const __nv_bfloat16 hi = __float2bfloat16_rn(h);
            const int64_t at = (int64_t)(slot0 + col) * A.I + tile * 16 + r + 8 * (i >> 1);
            A.h_hi[at] = __bfloat16_as_ushort(hi);
            const float rest = h - __bfloat162float(hi);  // no number where hi is infinite
            A.h_lo[at] = fabsf(rest) < INFINITY ? __bfloat16_as_ushort(__float2bfloat16_rn(rest)) : (uint16_t)0;
        }
    }
    cp_wait_groups<0>();
}

// ---- down and the weighted sum ------------------------------------------------------------
constexpr int kDownRows = 16 * kMoeWarps;

__global__ void __launch_bounds__(kMoeThreads) k_moe_down(const __grid_constant__ MoeArgs A) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ MoeList L;
    __shared__ float slot_w[kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int stage = mat_bytes(A.down.kind);
    const uint32_t base = sm_addr(ring) + warp * kStages * stage;
    float* sum = reinterpret_cast<float*>(ring + kMoeWarps * kStages * stage);  // [T][kDownRows]
    const int C = A.C;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int tile = (int)blockIdx.x / C;
    // the kernel before waited for its inputs: ids and weights are final, only h is not
    build_list(L, A);
    for (int b = threadIdx.x; b < L.blocks; b += kMoeThreads)
        for (int i = 0; i < L.blk_count[b]; ++i) {
            const int slot = L.blk_slot[b] + i, tok = L.slot_token[slot];
            float w = 0.f;  // a token may name an expert more than once
            for (int j = 0; j < A.k; ++j)
                if (A.ids[tok * A.k + j] == (int)L.blk_expert[b]) w += A.weights[tok * A.k + j];
            slot_w[slot] = w;
        }
    for (int i = threadIdx.x; i < A.T * kDownRows; i += kMoeThreads) sum[i] = 0.f;
    __syncthreads();
    const int G = A.down.G, steps = (G + kCG - 1) / kCG, blocks = L.blocks;
    const int64_t wrow = (int64_t)tile * kDownRows + warp * 16;
    int pb = rank, ps = 0, issued = 0;
    auto issue = [&]() {
        if (pb < blocks) {
            const int g = ps * kCG;
            load_step(A.down, (int64_t)L.blk_expert[pb] * A.H + wrow, g, min(kCG, G - g),
                      base + (issued % kStages) * stage, lane);
            if (++ps == steps) {
                ps = 0;
                pb += C;
            }
        }
        ++issued;
        cp_commit_group();
    };
    for (int i = 0; i < kStages - 1; ++i) issue();
    pdl_wait();
    int used = 0;
    for (int blk = rank; blk < blocks; blk += C) {
        const int count = L.blk_count[blk], slot0 = L.blk_slot[blk];
        const int64_t row0 = (int64_t)L.blk_expert[blk] * A.H + wrow;
        // with at most four tokens columns 4-7 hold the low parts of columns 0-3
        const bool packed = count <= 4;
        const int col = packed ? r & 3 : r;
        const bool have = col < count;
        const uint16_t* hp = (packed && r >= 4 ? A.h_lo : A.h_hi) + (int64_t)(slot0 + (have ? col : 0)) * A.I + 32 * t;
        const uint16_t* lp = A.h_lo + (int64_t)(slot0 + (have ? col : 0)) * A.I + 32 * t;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int st = 0; st < steps; ++st) {
            cp_wait_groups<kStages - 2>();
            __syncwarp();
            const int g = st * kCG, n = min(kCG, G - g);
            const uint32_t src = base + (used % kStages) * stage;
#pragma unroll
            for (int i = 0; i < kCG; ++i) {
                if (i >= n) break;
                uint32_t xf[16], xg[16];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                    const uint4 v = have ? ldg_plain(hp + (g + i) * 128 + 8 * q) : z;
                    xf[4 * q] = v.x, xf[4 * q + 1] = v.y, xf[4 * q + 2] = v.z, xf[4 * q + 3] = v.w;
                    const uint4 l = have && !packed ? ldg_plain(lp + (g + i) * 128 + 8 * q) : z;
                    xg[4 * q] = l.x, xg[4 * q + 1] = l.y, xg[4 * q + 2] = l.z, xg[4 * q + 3] = l.w;
                }
                const uint32_t row = src + r * row_stride(A.down.kind) + i * group_bytes(A.down.kind);
                const uint32_t sc = scale_at(A.down, row0, g, i, src, r);
                if (packed) group_product<false>(A.down.kind, row, sc, t, xf, xf, acc);
                else group_product<true>(A.down.kind, row, sc, t, xf, xg, acc);
            }
            ++used;
            __syncwarp();
            issue();
        }
        if (packed) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 2);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 2 * t + (i & 1);
            if (c >= count) continue;
            float* p = sum + L.slot_token[slot0 + c] * kDownRows + warp * 16 + r + 8 * (i >> 1);
            *p = fmaf(slot_w[slot0 + c], acc[i], *p);  // this warp's rows: no other writes them
        }
        __syncwarp();
    }
    cp_wait_groups<0>();
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // the ranks' sums in rank order; rank q finishes tokens q, q + C, ...
    const uint32_t sum_s = sm_addr(sum);
    for (int i = threadIdx.x; i < A.T * kDownRows; i += kMoeThreads) {
        const int tok = i / kDownRows, row = i - tok * kDownRows;
        if (tok % C != rank) continue;
        float v = 0.f;
        for (int q = 0; q < C; ++q) {
            float pq;
            if (C > 1)
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pq) : "r"(map_rank(sum_s + 4 * i, (uint32_t)q)) : "memory");
            else
                pq = sum[i];
            v += pq;
        }
        const int64_t at = (int64_t)tok * A.ldy + (int64_t)tile * kDownRows + row;
        if (A.ydt == kF32) static_cast<float*>(A.y)[at] = v;
        else static_cast<__nv_bfloat16*>(A.y)[at] = __float2bfloat16_rn(v);
    }
    if (C > 1) {  // no CTA leaves while another reads its sums
        cluster_arrive();
        cluster_wait();
    }
}

int moe_sms() {
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

MoeMat make_mat(const MoeWeights& w, int64_t K) {
    MoeMat m;
    m.packed = static_cast<const uint8_t*>(w.packed);
    m.scales = static_cast<const uint8_t*>(w.scales);
    m.kind = w.grid == kMx4 ? 2 : (w.grid == kInt3 ? 1 : 0);
    m.G = (int32_t)(K / kGroup);
    m.rb = (int64_t)m.G * group_bytes(m.kind);
    return m;
}

}  // namespace

size_t moe_data_bytes(int64_t T, int k, int64_t I) { return (size_t)((T * k * I * 4 + 255) / 256 * 256); }

cudaError_t launch_moe(const MoeWeights& gate, const MoeWeights& up, const MoeWeights& down, int E, int64_t H, int64_t I,
                       const uint16_t* x, int64_t ldx, const int32_t* ids, const float* weights, int T, int k, void* y,
                       int ydt, int64_t ldy, void* data, cudaStream_t st) {
    const int sms = moe_sms();
    if (sms <= 0) return cudaErrorInitializationError;
    MoeArgs A;
    std::memset(&A, 0, sizeof(A));
    A.gate = make_mat(gate, H);
    A.up = make_mat(up, H);
    A.down = make_mat(down, I);
    A.x = x;
    A.ids = ids;
    A.weights = weights;
    A.h_hi = static_cast<uint16_t*>(data);
    A.h_lo = A.h_hi + (int64_t)T * k * I;
    A.y = y;
    A.ldx = ldx;
    A.ldy = ldy;
    A.T = T;
    A.k = k;
    A.E = E;
    A.H = (int32_t)H;
    A.I = (int32_t)I;
    A.ydt = ydt;
    // units that the pairs can make at most; warps split K while they would leave the GPU's warps idle
    const int64_t units = (int64_t)std::min(T * k, E + T * k / 8) * (I / 16);
    A.S = 1;
    while (A.S < kMoeWarps && units * A.S < (int64_t)sms * 16 && A.gate.G >= 2 * A.S) A.S *= 2;
    A.C = 8;
    const int up_smem = kMoeWarps * kStages * (mat_bytes(A.gate.kind) + mat_bytes(A.up.kind));
    const int down_smem = kMoeWarps * kStages * mat_bytes(A.down.kind) + T * kDownRows * 4;
    cudaError_t e = cudaFuncSetAttribute(k_moe_up, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(k_moe_down, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_moe_up, kMoeThreads, (size_t)up_smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const int64_t ctas = std::min<int64_t>((units * A.S + kMoeWarps - 1) / kMoeWarps, (int64_t)sms * per_sm);

    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[2];
    std::memset(at, 0, sizeof(at));
    cfg.attrs = at;
    cfg.stream = st;
    cfg.blockDim = dim3(kMoeThreads);
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.dynamicSmemBytes = (size_t)up_smem;
    cfg.numAttrs = 0;
    void* args[] = {&A};
    e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&k_moe_up), args);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(H / kDownRows * A.C));
    cfg.dynamicSmemBytes = (size_t)down_smem;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)A.C;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&k_moe_down), args);
}

}  // namespace tb
