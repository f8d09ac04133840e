// tb_moe.cu -- the routed experts of a mixture-of-experts layer for a few
// tokens, straight from the packed codes, in two launches.
//
//     h[t,e] = silu(Wg[e] x[t]) * (Wu[e] x[t]),   y[t] = sum_j w[t,j] Wd[ids[t,j]] h[t,ids[t,j]]
//
// Every expert that some token takes is read once per sixteen of its tokens:
// with few tokens the layer is bound by the bytes of the experts it touches
// and by decoding them.
//
// Both kernels group the (token, choice) pairs by expert themselves, in
// shared memory (a 64-bit token mask per expert, a prefix sum over the
// experts): at most 1024 pairs, no extra launch, no atomics on floats.  A
// block is an expert with up to sixteen of its tokens.
//
// The products run on mma.sync m16n8k16: 16 weight rows decoded in registers
// to bf16 (exact, 4-bit codes with their power-of-two scale too), the
// activations as B fragments read as they are, in sets of eight columns that
// share the decode.  A lane of a quad owns 32 consecutive k of every
// 128-group in both operands, so a row's group is one 8-, 12- or 16-byte read
// per lane, free of bank conflicts, and no code moves between lanes.  Weights
// stream through a private cp.async ring per warp, a group per stage.
//
// h is rounded to bf16 between the two products, as tb_gate_up_silu's is: the
// MMA's operand, and half the activations a second part would cost.
//
// k_moe_up: a unit is (block, 16 rows of gate and of up); S warps of a CTA
// split K when units are few.  k_moe_down: a cluster of C CTAs holds 64 rows
// of H, its CTAs split the blocks; each warp adds its rows' results per
// token in shared memory, the ranks are added in order (deterministic).
#include "tb_async.cuh"
#include "tb_device.cuh"
#include "tb_internal.h"

#include <algorithm>
#include <cmath>
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
    uint16_t* h;             // [slots][I] bf16
    void* y;                 // [T][ldy]
    int64_t ldx, ldy;
    int32_t T, k, E, H, I, ydt;
    int32_t S, C;
    int32_t hperm;  // h in the order of the 4-bit decode's pairs
};

namespace {

constexpr int kMoeWarps = 4;
constexpr int kMoeThreads = kMoeWarps * 32;
constexpr int kStages = 4;
constexpr int kBlockTokens = 16;
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxK;
constexpr int kMaxBlocks = kMoeMaxExperts + kMaxPairs / kBlockTokens;

// packed bytes of a row's group (also its stride in shared memory: with 32, 48 and 64 bytes the reads of eight rows
// by a quad each touch every bank once)
__host__ __device__ constexpr int group_bytes(int kind) { return kind == 0 ? 32 : (kind == 1 ? 48 : 64); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// Eight 4-bit codes (nibble j: code j) as the bf16 pairs (0,4), (1,5), (2,6), (3,7), times f 2^-126: a code's
// exponent and mantissa bits put at the bottom of a bf16's exponent and the top of its mantissa are its magnitude
// times 2^-126 (both formats agree below their normal range), one multiplication by 2^a + 2^b moves them and the
// sign of two codes to their places.
__device__ __forceinline__ void decode_mx4(uint32_t w, uint32_t f, uint32_t (&r)[4]) {
    const uint32_t w8 = w >> 8;
    r[0] = mul_bf16x2(((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, f);
    r[1] = mul_bf16x2(((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, f);
    r[2] = mul_bf16x2(((w8 & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, f);
    r[3] = mul_bf16x2(((w8 & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, f);
}
// eight consecutive activations (four pairs) in the order of those pairs
__device__ __forceinline__ void pair_up(uint32_t (&x)[16], const uint32_t (&v)[16]) {
#pragma unroll
    for (int q = 0; q < 16; q += 4) {
        x[q] = prmt(v[q], v[q + 2], 0x5410);
        x[q + 1] = prmt(v[q], v[q + 2], 0x7632);
        x[q + 2] = prmt(v[q + 1], v[q + 3], 0x5410);
        x[q + 3] = prmt(v[q + 1], v[q + 3], 0x7632);
    }
}

template <int NS, bool BIG>
__device__ __forceinline__ void mx4_product(uint32_t row, int t, uint32_t ba, uint32_t bb,
                                            const uint32_t (&x)[NS][16], float (&acc)[NS][4]) {
    const uint4 a = lds128(row + 16 * t), b = lds128(row + 8 * group_bytes(2) + 16 * t);
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
    // 2^(byte - 1) as a pair; above 2^127 in two factors; 255 is no number
    const uint32_t fa = ((BIG ? min(ba, 128u) : ba) + 126u) * 0x00800080u;
    const uint32_t fb = ((BIG ? min(bb, 128u) : bb) + 126u) * 0x00800080u;
    uint32_t ga = 0, gb = 0;
    if (BIG) {
        ga = ba == 255u ? 0x7FC07FC0u : (max(ba, 128u) - 1u) * 0x00800080u;
        gb = bb == 255u ? 0x7FC07FC0u : (max(bb, 128u) - 1u) * 0x00800080u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t ra[4], rb[4];
        decode_mx4(wa[i], fa, ra);
        decode_mx4(wb[i], fb, rb);
        if (BIG) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ra[j] = mul_bf16x2(ra[j], ga);
                rb[j] = mul_bf16x2(rb[j], gb);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; j += 2)
#pragma unroll
            for (int n = 0; n < NS; ++n)
                mma_bf16(acc[n], ra[j], rb[j], ra[j + 1], rb[j + 1], x[n][4 * i + j], x[n][4 * i + j + 1]);
    }
}

// One 128-group of 16 rows times NS sets of eight columns: acc += s W x.  `row`: shared address of row lane/4 of the
// group, `sc`: of its scale word, `odd`: the scale is the word's upper half.
template <int KIND, int NS>
__device__ __forceinline__ void group_product(uint32_t row, uint32_t sc, bool odd, int t, const uint32_t (&x)[NS][16],
                                              float (&acc)[NS][4]) {
    if constexpr (KIND == 2) {
        const uint32_t ba = lds8(sc + t), bb = lds8(sc + 32 + t);
        if (__builtin_expect(__any_sync(0xffffffffu, max(ba, bb) > 128u), 0)) mx4_product<NS, true>(row, t, ba, bb, x, acc);
        else mx4_product<NS, false>(row, t, ba, bb, x, acc);
    } else {
        float d[NS][4];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[n][i] = 0.f;
        if constexpr (KIND == 0) {
            const uint2 a = lds64(row + 8 * t), b = lds64(row + 8 * group_bytes(0) + 8 * t);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t ra[8], rb[8];
                decode2_signed<2>(i ? a.y : a.x, ra);
                decode2_signed<2>(i ? b.y : b.x, rb);
#pragma unroll
                for (int j = 0; j < 8; j += 2)
#pragma unroll
                    for (int n = 0; n < NS; ++n)
                        mma_bf16(d[n], ra[j], rb[j], ra[j + 1], rb[j + 1], x[n][8 * i + j], x[n][8 * i + j + 1]);
            }
        } else {
            uint32_t ra[16], rb[16];
            const uint32_t ar = row + 12 * t, br = ar + 8 * group_bytes(1);
            decode3_signed(lds32(ar), lds32(ar + 4), lds32(ar + 8), ra);
            decode3_signed(lds32(br), lds32(br + 4), lds32(br + 8), rb);
#pragma unroll
            for (int j = 0; j < 16; j += 2)
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    mma_bf16(d[n], ra[j], rb[j], ra[j + 1], rb[j + 1], x[n][j], x[n][j + 1]);
        }
        const uint32_t w0 = lds32(sc), w1 = lds32(sc + 32);
        const float s0 = __uint_as_float(odd ? w0 & 0xFFFF0000u : w0 << 16);
        const float s1 = __uint_as_float(odd ? w1 & 0xFFFF0000u : w1 << 16);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            acc[n][0] = fmaf(s0, d[n][0], acc[n][0]);
            acc[n][1] = fmaf(s0, d[n][1], acc[n][1]);
            acc[n][2] = fmaf(s1, d[n][2], acc[n][2]);
            acc[n][3] = fmaf(s1, d[n][3], acc[n][3]);
        }
    }
}

// A warp's place in the packed rows of a matrix: group after group of the 16 rows row0 .., each lane with its own
// 16-byte pieces.
template <int KIND>
struct CodeCursor {
    const uint8_t* p;
    uint32_t second;  // from the lane's first piece to its second
    __device__ __forceinline__ void init(const MoeMat& m, int lane) {
        constexpr int P = group_bytes(KIND) / 16;
        const int a = lane, b = lane + 32;
        second = (uint32_t)((b / P - a / P) * m.rb + (b % P - a % P) * 16);
    }
    __device__ __forceinline__ void at(const MoeMat& m, int64_t row0, int g, int lane) {
        constexpr int P = group_bytes(KIND) / 16;
        p = m.packed + (row0 + lane / P) * m.rb + (int64_t)g * group_bytes(KIND) + (lane % P) * 16;
    }
    __device__ __forceinline__ void load(uint32_t dst, int lane) {
        cp16(dst + lane * 16, p);
        if (KIND == 2 || (KIND == 1 && lane < 16)) cp16(dst + (lane + 32) * 16, p + second);
        p += group_bytes(KIND);
    }
};
// The same for a row's scales: two bytes per group, fetched with the aligned word they lie in, or a word per 4-bit
// group.
struct ScaleCursor {
    const uint8_t* p;
    uint32_t step, n;
    template <int KIND>
    __device__ __forceinline__ void at(const MoeMat& m, int64_t row, int g) {
        if constexpr (KIND == 2) {
            p = m.scales + (((row >> 7) * m.G + g) * 128 + (row & 31) * 4 + ((row >> 5) & 3)) * 4;
            step = 512, n = 4;
        } else {
            p = m.scales + (row * m.G + g) * 2;
            step = 2, n = 2;
        }
    }
    __device__ __forceinline__ void load(uint32_t dst) {
        const uintptr_t v = reinterpret_cast<uintptr_t>(p);
        cp4(dst, reinterpret_cast<const void*>(v & ~(uintptr_t)3), (v & 2) ? 4 : n);
        p += step;
    }
};
// the next stage of a ring
__device__ __forceinline__ uint32_t next_stage(uint32_t at, uint32_t base, uint32_t stage) {
    at += stage;
    return at == base + kStages * stage ? base : at;
}

// ---- the pairs grouped by expert ---------------------------------------------------
struct MoeList {
    unsigned long long mask[kMoeMaxExperts];  // tokens of each expert
    uint32_t blk[kMaxBlocks];                 // expert, first slot << 10, tokens << 20
    uint8_t slot_token[kMaxPairs];
    int scan[2][kMoeWarps];
    int blocks, slots;
};
__device__ __forceinline__ int blk_expert(uint32_t b) { return (int)(b & 1023u); }
__device__ __forceinline__ int blk_slot(uint32_t b) { return (int)(b >> 10 & 1023u); }
__device__ __forceinline__ int blk_count(uint32_t b) { return (int)(b >> 20); }

template <int THREADS>
__device__ void build_list(MoeList& L, const MoeArgs& A) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < A.E; e += THREADS) L.mask[e] = 0ull;
    __syncthreads();
    for (int p = tid; p < A.T * A.k; p += THREADS) {
        const int e = A.ids[p];
        if (e >= 0 && e < A.E) atomicOr(&L.mask[e], 1ull << (p / A.k));  // a set: the order does not matter
    }
    __syncthreads();
    const int per = (A.E + THREADS - 1) / THREADS, e0 = tid * per, e1 = min(A.E, e0 + per);
    int slots = 0, blocks = 0;
    for (int e = e0; e < e1; ++e) {
        const int c = __popcll(L.mask[e]);
        slots += c;
        blocks += (c + kBlockTokens - 1) / kBlockTokens;
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
    if (tid == THREADS - 1) {
        L.slots = s;
        L.blocks = b;
    }
    s -= slots;
    b -= blocks;
    for (int e = e0; e < e1; ++e) {
        unsigned long long m = L.mask[e];
        for (int left = __popcll(m); left > 0; left -= kBlockTokens) {
            const int n = min(kBlockTokens, left);
            L.blk[b++] = (uint32_t)e | (uint32_t)s << 10 | (uint32_t)n << 20;
            for (int i = 0; i < n; ++i) {
                L.slot_token[s++] = (uint8_t)(__ffsll((long long)m) - 1);
                m &= m - 1;
            }
        }
    }
    __syncthreads();
}

// ---- gate and up -----------------------------------------------------------------------
template <int KG, int KU>
struct MoeUp {
    static constexpr int kGate = 16 * group_bytes(KG), kUp = 16 * group_bytes(KU);
    static constexpr int kStage = kGate + kUp + 128;  // codes of gate and up, their scale words
    static constexpr int kRing = kMoeWarps * kStages * kStage;

    const MoeArgs& A;
    MoeList& L;
    float* part;    // [2][warps][sets][256]: partial sums of gate and up, two units deep
    uint32_t base;  // this warp's ring
    int lane, warp, r, t, S, s, ui, g0, steps, tiles, units, ustep, sets;
    int pu, ps, flip;
    uint32_t to, from;  // the stages to be filled and read next
    CodeCursor<KG> cg;
    CodeCursor<KU> cu;
    ScaleCursor sc;

    // the first request of unit pu: cursors to its rows
    __device__ __forceinline__ void seek() {
        if (pu >= units) return;
        const int blk = pu / tiles, tile = pu - blk * tiles;
        const int64_t row0 = (int64_t)blk_expert(L.blk[blk]) * A.I + tile * 16;
        cg.at(A.gate, row0, g0, lane);
        cu.at(A.up, row0, g0, lane);
        if (lane < 16) sc.at<KG>(A.gate, row0 + lane, g0);
        else sc.at<KU>(A.up, row0 + lane - 16, g0);
        ps = 0;
    }
    __device__ __forceinline__ void issue() {
        if (pu < units) {
            cg.load(to, lane);
            cu.load(to + kGate, lane);
            sc.load(to + kGate + kUp + 4 * lane);
            if (++ps == steps) {
                pu += ustep;
                seek();
            }
        }
        to = next_stage(to, base, kStage);
        cp_commit_group();
    }

    template <int NS>
    __device__ __forceinline__ void unit(uint32_t block, int tile) {
        const int count = blk_count(block), slot0 = blk_slot(block);
        const int64_t row0 = (int64_t)blk_expert(block) * A.I + tile * 16;
        const uint16_t* xr[NS];
        bool have[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            have[n] = 8 * n + r < count;
            xr[n] = A.x + (int64_t)(have[n] ? L.slot_token[slot0 + 8 * n + r] : 0) * A.ldx + g0 * 128 + 32 * t;
        }
        // parity of the scale's place in its word, for the first group
        const int pg = (int)((row0 + r) * A.gate.G + g0) & 1;
        float ag[NS][4], au[NS][4];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) ag[n][i] = au[n][i] = 0.f;
        uint32_t v[NS][16];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int q = 0; q < 16; ++q) v[n][q] = 0u;
        auto load_x = [&](int st) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (have[n]) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 u = ld_act_u4(xr[n] + st * 128 + 8 * q);
                        v[n][4 * q] = u.x, v[n][4 * q + 1] = u.y, v[n][4 * q + 2] = u.z, v[n][4 * q + 3] = u.w;
                    }
                }
        };
        load_x(0);
        for (int st = 0; st < steps; ++st) {
            // this group's activations in the order of the decoders' pairs; then the next group's are requested
            uint32_t p[NS][16], w[NS][16];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                if constexpr (KG == 2 || KU == 2) pair_up(p[n], v[n]);
                if constexpr (KG != 2 || KU != 2) {
#pragma unroll
                    for (int q = 0; q < 16; ++q) w[n][q] = v[n][q];
                }
            }
            if (NS == 1 && st + 1 < steps) load_x(st + 1);
            cp_wait_groups<kStages - 2>();
            __syncwarp();
            const bool odd = ((pg + st) & 1) != 0;
            group_product<KG, NS>(from + r * group_bytes(KG), from + kGate + kUp + 4 * r, odd, t, KG == 2 ? p : w, ag);
            group_product<KU, NS>(from + kGate + r * group_bytes(KU), from + kGate + kUp + 64 + 4 * r, odd, t,
                                  KU == 2 ? p : w, au);
            if (NS > 1 && st + 1 < steps) load_x(st + 1);
            from = next_stage(from, base, kStage);
            __syncwarp();
            issue();
        }
        if (S > 1) {
            float* mine = part + ((flip * kMoeWarps + warp) * sets) * 256 + lane;
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mine[n * 256 + i * 32] = ag[n][i];
                    mine[n * 256 + 128 + i * 32] = au[n][i];
                }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + ui), "r"(S * 32) : "memory");
            // warp s of the unit finishes registers s, s + S, ... of every set
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((i & (S - 1)) != s) continue;
                    float sg = 0.f, su = 0.f;
                    for (int w = 0; w < S; ++w) {
                        const float* q = part + ((flip * kMoeWarps + ui * S + w) * sets + n) * 256 + i * 32 + lane;
                        sg += q[0];
                        su += q[128];
                    }
                    ag[n][i] = sg;
                    au[n][i] = su;
                }
            flip ^= 1;
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = 8 * n + 2 * t + (i & 1);
                if ((i & (S - 1)) != s || col >= count) continue;
                const float g = ag[n][i], h = g / (1.f + expf(-g)) * au[n][i];
                int c = tile * 16 + r + 8 * (i >> 1);
                if (A.hperm) c = (c & ~7) | (c & 3) << 1 | (c >> 2 & 1);
                A.h[(int64_t)(slot0 + col) * A.I + c] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
            }
    }
};

template <int KG, int KU>
__global__ void __launch_bounds__(kMoeThreads, 4) k_moe_up(const __grid_constant__ MoeArgs A) {
    using Up = MoeUp<KG, KU>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ MoeList L;
    pdl_wait();
    build_list<kMoeThreads>(L, A);
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = A.S, per = kMoeWarps / S;
    Up u{A, L, reinterpret_cast<float*>(ring + Up::kRing), sm_addr(ring) + (uint32_t)(warp * kStages * Up::kStage)};
    u.lane = lane, u.warp = warp, u.r = lane >> 2, u.t = lane & 3;
    u.S = S, u.s = warp & (S - 1), u.ui = warp / S;
    u.g0 = A.gate.G * u.s / S;
    u.steps = A.gate.G * (u.s + 1) / S - u.g0;
    u.tiles = A.I / 16;
    u.units = L.blocks * u.tiles;
    u.ustep = (int)gridDim.x * per;
    u.sets = A.T > 8 ? 2 : 1;
    u.pu = (int)blockIdx.x * per + u.ui;
    u.ps = u.flip = 0;
    u.to = u.from = u.base;
    u.cg.init(A.gate, lane);
    u.cu.init(A.up, lane);
    u.seek();
    for (int i = 0; i < kStages - 1; ++i) u.issue();
    for (int v = (int)blockIdx.x * per + u.ui; v < u.units; v += u.ustep) {
        const int blk = v / u.tiles;
        const uint32_t block = L.blk[blk];
        if (blk_count(block) > 8) u.template unit<2>(block, v - blk * u.tiles);
        else u.template unit<1>(block, v - blk * u.tiles);
    }
    cp_wait_groups<0>();
}

// ---- down and the weighted sum ------------------------------------------------------------
constexpr int kDownRows = 32;    // of a CTA: each warp holds all of them, two tiles that share h's fragments
constexpr int kDownStages = 3;

template <int KIND>
struct MoeDown {
    static constexpr int kCodes = 16 * group_bytes(KIND);
    static constexpr int kStage = 2 * kCodes + 128;
    static constexpr int kRing = kMoeWarps * kDownStages * kStage;

    const MoeArgs& A;
    MoeList& L;
    const float* slot_w;
    float* sum;     // this warp's [T][kDownRows]
    uint32_t base;  // this warp's ring
    int lane, r, t, G, tasks, KS, step;
    int64_t wrow;
    int pq, ps, pend;   // the next request: task, group, end of the task's groups
    uint32_t to, from;  // the stages to be filled and read next
    CodeCursor<KIND> codes;
    int64_t tile2;  // from a piece of the first tile to that of the second
    ScaleCursor sc;

    __device__ __forceinline__ void range(int q, int& b, int& g0, int& g1) const {
        b = q / KS;
        const int k = q - b * KS;
        g0 = G * k / KS;
        g1 = G * (k + 1) / KS;
    }
    __device__ __forceinline__ void seek() {
        if (pq >= tasks) return;
        int b;
        range(pq, b, ps, pend);
        const int64_t row0 = (int64_t)blk_expert(L.blk[b]) * A.H + wrow;
        codes.at(A.down, row0, ps, lane);
        sc.at<KIND>(A.down, row0 + lane, ps);
    }
    __device__ __forceinline__ void issue() {
        if (pq < tasks) {
            CodeCursor<KIND> second = codes;
            second.p += tile2;
            second.load(to + kCodes, lane);
            codes.load(to, lane);
            sc.load(to + 2 * kCodes + 4 * lane);
            if (++ps == pend) {
                pq += step;
                seek();
            }
        }
        to += kStage;
        if (to == base + kDownStages * kStage) to = base;
        cp_commit_group();
    }

    template <int NS>
    __device__ __forceinline__ void block(uint32_t b, int g0, int g1) {
        const int count = blk_count(b), slot0 = blk_slot(b);
        const int64_t row0 = (int64_t)blk_expert(b) * A.H + wrow;
        const int pg = (int)((row0 + r) * A.down.G) & 1;  // 16 rows on it is the same
        const uint16_t* hp[NS];
        bool have[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            have[n] = 8 * n + r < count;
            hp[n] = A.h + (int64_t)(slot0 + (have[n] ? 8 * n + r : 0)) * A.I + 32 * t;
        }
        float acc[2][NS][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
        uint32_t v[NS][16];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int q = 0; q < 16; ++q) v[n][q] = 0u;
        auto load_h = [&](int g) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (have[n]) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 u = ldg_plain(hp[n] + g * 128 + 8 * q);
                        v[n][4 * q] = u.x, v[n][4 * q + 1] = u.y, v[n][4 * q + 2] = u.z, v[n][4 * q + 3] = u.w;
                    }
                }
        };
        load_h(g0);
        for (int g = g0; g < g1; ++g) {
            uint32_t w[NS][16];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int q = 0; q < 16; ++q) w[n][q] = v[n][q];
            if (NS == 1 && g + 1 < g1) load_h(g + 1);
            cp_wait_groups<kDownStages - 2>();
            __syncwarp();
            const bool odd = ((pg + g) & 1) != 0;
            group_product<KIND, NS>(from + r * group_bytes(KIND), from + 2 * kCodes + 4 * r, odd, t, w, acc[0]);
            group_product<KIND, NS>(from + kCodes + r * group_bytes(KIND), from + 2 * kCodes + 64 + 4 * r, odd, t, w,
                                    acc[1]);
            if (NS > 1 && g + 1 < g1) load_h(g + 1);
            from += kStage;
            if (from == base + kDownStages * kStage) from = base;
            __syncwarp();
            issue();
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int tok = 8 * n + 2 * t + j;
                if (tok >= count) continue;
                const float w = slot_w[slot0 + tok];
                float* p = sum + L.slot_token[slot0 + tok] * kDownRows + r;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    p[16 * m] = fmaf(w, acc[m][n][j], p[16 * m]);
                    p[16 * m + 8] = fmaf(w, acc[m][n][2 + j], p[16 * m + 8]);
                }
            }
        __syncwarp();
    }
};

template <int KIND>
__global__ void __launch_bounds__(kMoeThreads, 4) k_moe_down(const __grid_constant__ MoeArgs A) {
    using Down = MoeDown<KIND>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ MoeList L;
    __shared__ float slot_w[kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = A.C;
    const int rank = C > 1 ? (int)cluster_rank() : 0, tile = (int)blockIdx.x / C;
    float* sum = reinterpret_cast<float*>(ring + Down::kRing);  // [warps][T][kDownRows]
    const int sums = A.T * kDownRows;
    // the kernel before waited for its inputs: ids and weights are final, only h is not
    build_list<kMoeThreads>(L, A);
    Down d{A, L, slot_w, sum + warp * sums, sm_addr(ring) + (uint32_t)(warp * kDownStages * Down::kStage)};
    d.lane = lane, d.r = lane >> 2, d.t = lane & 3;
    d.G = A.down.G;
    d.step = C * kMoeWarps;
    // blocks fewer than the warps that share them: their groups are split too
    d.KS = max(1, min(d.G, d.step / max(1, L.blocks)));
    d.tasks = L.blocks * d.KS;
    d.wrow = (int64_t)tile * kDownRows;
    d.tile2 = 16 * A.down.rb;
    const int q0 = rank * kMoeWarps + warp;
    d.pq = q0;
    d.to = d.from = d.base;
    d.codes.init(A.down, lane);
    d.seek();
    for (int i = 0; i < kDownStages - 1; ++i) d.issue();
    for (int b = threadIdx.x; b < L.blocks; b += kMoeThreads) {
        const uint32_t blk = L.blk[b];
        for (int i = 0; i < blk_count(blk); ++i) {
            const int slot = blk_slot(blk) + i, tok = L.slot_token[slot];
            float w = 0.f;  // a token may name an expert more than once
            for (int j = 0; j < A.k; ++j)
                if (A.ids[tok * A.k + j] == blk_expert(blk)) w += A.weights[tok * A.k + j];
            slot_w[slot] = w;
        }
    }
    for (int i = threadIdx.x; i < kMoeWarps * sums; i += kMoeThreads) sum[i] = 0.f;
    __syncthreads();
    pdl_wait();
    for (int q = q0; q < d.tasks; q += d.step) {
        int b, g0, g1;
        d.range(q, b, g0, g1);
        const uint32_t blk = L.blk[b];
        if (blk_count(blk) > 8) d.template block<2>(blk, g0, g1);
        else d.template block<1>(blk, g0, g1);
    }
    cp_wait_groups<0>();
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // the warps' sums, rank by rank; rank q finishes tokens q, q + C, ...
    const uint32_t sum_s = sm_addr(sum);
    for (int i = threadIdx.x; i < sums; i += kMoeThreads) {
        const int tok = i / kDownRows, row = i - tok * kDownRows;
        if (tok % C != rank) continue;
        float v = 0.f;
        for (int q = 0; q < C; ++q)
#pragma unroll
            for (int w = 0; w < kMoeWarps; ++w) {
                const int j = w * sums + i;
                float pq;
                if (C > 1)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(pq)
                                 : "r"(map_rank(sum_s + 4 * j, (uint32_t)q))
                                 : "memory");
                else
                    pq = sum[j];
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

struct KernelOf {
    const void* fn;
    int ring;
};
template <int KG, int KU>
KernelOf up_of() {
    return {reinterpret_cast<const void*>(&k_moe_up<KG, KU>), MoeUp<KG, KU>::kRing};
}
KernelOf up_kernel(int kg, int ku) {
    static const KernelOf table[3][3] = {{up_of<0, 0>(), up_of<0, 1>(), up_of<0, 2>()},
                                         {up_of<1, 0>(), up_of<1, 1>(), up_of<1, 2>()},
                                         {up_of<2, 0>(), up_of<2, 1>(), up_of<2, 2>()}};
    return table[kg][ku];
}
template <int KIND>
KernelOf down_of() {
    return {reinterpret_cast<const void*>(&k_moe_down<KIND>), MoeDown<KIND>::kRing};
}
KernelOf down_kernel(int kind) {
    static const KernelOf table[3] = {down_of<0>(), down_of<1>(), down_of<2>()};
    return table[kind];
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

size_t moe_data_bytes(int64_t T, int k, int64_t I) { return (size_t)((T * k * I * 2 + 255) / 256 * 256); }

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
    A.h = static_cast<uint16_t*>(data);
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
    const int64_t units = (int64_t)std::min(T * k, E + T * k / kBlockTokens) * (I / 16);
    A.S = 1;
    while (A.S < kMoeWarps && units * A.S < (int64_t)sms * 16 && A.gate.G >= 2 * A.S) A.S *= 2;
    A.hperm = A.down.kind == 2 ? 1 : 0;
    const KernelOf ku = up_kernel(A.gate.kind, A.up.kind), kd = down_kernel(A.down.kind);
    const int up_smem = ku.ring + (A.S > 1 ? 2 * kMoeWarps * (T > 8 ? 2 : 1) * 1024 : 0);
    const int down_smem = kd.ring + T * kMoeWarps * kDownRows * 4;
    cudaError_t e = cudaFuncSetAttribute(ku.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kd.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
    int per_sm = 0, down_per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, ku.fn, kMoeThreads, (size_t)up_smem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&down_per_sm, kd.fn, kMoeThreads, (size_t)down_smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1 || down_per_sm < 1) return cudaErrorInvalidConfiguration;
    // CTAs per cluster of the down kernel: the count whose waves, each as long as a warp's share of the blocks that
    // the tokens are expected to fill (in sixteenths of a block), end first
    const double filled = E * (1.0 - std::pow(1.0 - std::min(1.0, (double)k / E), T)) + T * k / (double)(2 * kBlockTokens);
    double best = 0;
    for (int c = 1; c <= 8; ++c) {
        const int64_t waves = (H / kDownRows * c + (int64_t)sms * down_per_sm - 1) / ((int64_t)sms * down_per_sm);
        const double cost = (double)waves * (std::ceil(16 * filled / (c * kMoeWarps)) + 4);
        if (c == 1 || cost < best) {
            best = cost;
            A.C = c;
        }
    }
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
    e = cudaLaunchKernelExC(&cfg, ku.fn, args);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(H / kDownRows * A.C));
    cfg.dynamicSmemBytes = (size_t)down_smem;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)A.C;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, kd.fn, args);
}

}  // namespace tb
