// tb_moe.cu -- the routed experts of a mixture-of-experts layer for a few
// tokens, straight from the packed codes, in two launches.
//
//     h[t,e] = silu(Wg[e] x[t]) * (Wu[e] x[t]),   y[t] = sum_j w[t,j] Wd[ids[t,j]] h[t,ids[t,j]]
//
// Every expert that some token takes is read once per eight or sixteen of its
// tokens:
// with few tokens the layer is bound by the bytes of the experts it touches
// and by decoding them.
//
// Both kernels group the (token, choice) pairs by expert themselves, in
// shared memory (a 64-bit token mask per expert, a prefix sum over the
// experts): at most 1024 pairs, no extra launch, no atomics on floats.  A
// block is an expert with up to eight or sixteen of its tokens.
//
// The products run on mma.sync m16n8k16: 16 weight rows decoded in registers
// to bf16 (exact, 4-bit codes with their power-of-two scale too), the
// activations as B fragments read as they are, in sets of eight columns that
// share the decode.  A lane of a quad owns 32 consecutive k of every
// 128-group in both operands, so a row's group is one 8-, 12- or 16-byte read
// per lane, free of bank conflicts, and no code moves between lanes.  Weights
// stream through a private ring per warp, filled by tensor copies of 16 or 32
// rows x 128 (144) bytes.  (With cp.async, 32 rows' scattered 16- and 4-byte
// pieces per group, both kernels were bound by the L1's request rate: more
// warps changed nothing, 64 tokens x 4-bit experts took 466 us.)
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

__device__ unsigned int g_moe_timeouts = 0;

struct MoeMat {
    CUtensorMap codes;      // packed rows: bytes x rows
    CUtensorMap tiles;      // 4-bit scales: 512 bytes x (row tile, group)
    const uint16_t* scales;  // bf16 [rows][G]
    int32_t G;               // 128-groups of a row
    int32_t kind;            // 0: 2 bits, 1: 3 bits, 2: MX4
};

struct MoeArgs {
    MoeMat gate, up, down;
    const uint16_t* x;       // [T][ldx]
    const int32_t* ids;      // [T][k]
    const float* weights;    // [T][k]
    uint16_t* h;             // [slots][I] bf16
    float* z;                // [H / 32][zrows][32]: weighted results of the slots
    void* y;                 // [T][ldy]
    int64_t ldx, ldy;
    long long wait_cycles;
    int32_t T, k, E, H, I, ydt, stall;
    int32_t S, C, zrows;
    int32_t hperm;  // h in the order of the 4-bit decode's pairs
};

namespace {

constexpr int kMoeWarps = 4;
constexpr int kMoeThreads = kMoeWarps * 32;
constexpr int kStages = 2;  // of a warp's ring
constexpr float kMoeNaN = __builtin_nanf("");
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxK;
constexpr int kMaxBlocks = kMoeMaxExperts + kMaxPairs / 8;

// packed bytes of a row's group; groups of a stage; bytes of a row in it.  The 2-bit and 4-bit stages have 128-byte rows
// in the 128-byte swizzle, the 3-bit ones plain rows of 144 bytes; with a tile's rows taken in bit-reversed order the
// reads of a group (8, 12 or 16 bytes by each lane of a quad, a row per quad) are free of bank conflicts in all three.
__host__ __device__ constexpr int group_bytes(int kind) { return kind == 0 ? 32 : (kind == 1 ? 48 : 64); }
__host__ __device__ constexpr int stage_groups(int kind) { return kind == 0 ? 4 : (kind == 1 ? 3 : 2); }
__host__ __device__ constexpr int row_stride(int kind) { return kind == 1 ? 144 : 128; }
// a unit's bf16 scales are copied whole up to this many groups; longer rows read them one by one
constexpr int kMaxScaleGroups = 64;

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
__device__ __forceinline__ void mx4_product(uint32_t row, uint32_t ba, uint32_t bb,
                                            const uint32_t (&x)[NS][16], float (&acc)[NS][4]) {
    const uint4 a = lds128(row), b = lds128(row + 8 * row_stride(2));
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

// One 128-group of 16 rows times NS sets of eight columns: acc += s W x.  `row`: shared address of the lane's codes in
// the first of its two rows (the second is eight rows on); s0, s1: the rows' scales, or the lane's two scale bytes.
template <int KIND, int NS>
__device__ __forceinline__ void group_product(uint32_t row, uint32_t s0b, uint32_t s1b, const uint32_t (&x)[NS][16],
                                              float (&acc)[NS][4]) {
    if constexpr (KIND == 2) {
        const uint32_t ba = s0b, bb = s1b;
        if (__builtin_expect(__any_sync(0xffffffffu, max(ba, bb) > 128u), 0)) mx4_product<NS, true>(row, ba, bb, x, acc);
        else mx4_product<NS, false>(row, ba, bb, x, acc);
    } else {
        float d[NS][4];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[n][i] = 0.f;
        if constexpr (KIND == 0) {
            const uint2 a = lds64(row), b = lds64(row + 8 * row_stride(0));
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
            const uint32_t br = row + 8 * row_stride(1);
            decode3_signed(lds32(row), lds32(row + 4), lds32(row + 8), ra);
            decode3_signed(lds32(br), lds32(br + 4), lds32(br + 8), rb);
#pragma unroll
            for (int j = 0; j < 16; j += 2)
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    mma_bf16(d[n], ra[j], rb[j], ra[j + 1], rb[j + 1], x[n][j], x[n][j + 1]);
        }
        const float s0 = __uint_as_float(s0b << 16), s1 = __uint_as_float(s1b << 16);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            acc[n][0] = fmaf(s0, d[n][0], acc[n][0]);
            acc[n][1] = fmaf(s0, d[n][1], acc[n][1]);
            acc[n][2] = fmaf(s1, d[n][2], acc[n][2]);
            acc[n][3] = fmaf(s1, d[n][3], acc[n][3]);
        }
    }
}

// ---- a warp's stream of a matrix -------------------------------------------------------
// Units of ROWS consecutive rows and a range of their groups, one after the other, through kStages stages of kGroups
// groups.  The warp refills a stage as soon as it has read it.
template <int KIND, int ROWS>
struct Stream {
    static constexpr int kGroups = stage_groups(KIND);
    static constexpr int kCodes = ROWS * row_stride(KIND);       // of a stage
    static constexpr int kTiles = KIND == 2 ? ROWS * 16 * kGroups : 0;  // a 4-bit stage's scale rows
    static constexpr int kBars = 8 * 2 * kStages;                // per stage; per scale buffer of a unit
    // bytes of a warp's ring (codes first: swizzled stages begin at multiples of 1 KB)
    static constexpr int kRing = (kStages * kCodes + 1023) & ~1023;
    __host__ __device__ static constexpr int side(int G) {
        return (kStages * kTiles + (KIND != 2 && G <= kMaxScaleGroups ? kStages * ROWS * 2 * G : 0) + 127) & ~127;
    }

    const MoeMat& m;
    uint32_t codes, sides, bars;
    long long limit;
    int lane, row, t;  // row: the lane's first row in a 16-row tile
    // requests: the unit's first row, its next group and their end, how many stages and units have been begun
    int64_t prow;
    int pg, pend, pn, pu;
    // reading: stage, its parity, the group in it and how many it holds; the unit's row, number and group
    int stage, gi, left, cu, g;
    uint32_t parity;
    int64_t crow;
    bool dead;

    __device__ __forceinline__ Stream(const MoeMat& m_, uint32_t ring, uint32_t side_, uint32_t bars_, long long limit_)
        : m(m_), codes(ring), sides(side_), bars(bars_), limit(limit_), pn(0), pu(0), stage(0), left(0), cu(0),
          parity(0), dead(false) {
        lane = threadIdx.x & 31;
        row = (lane >> 2 & 1) << 2 | (lane >> 2 & 2) | (lane >> 4);  // lane / 4 with its three bits reversed
        t = lane & 3;
    }
    __device__ __forceinline__ void init_bars() const {
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < 2 * kStages; ++i) mb_init(bars + 8 * i, 1);
    }
    __device__ __forceinline__ bool wide() const { return KIND != 2 && m.G > kMaxScaleGroups; }

    // begins the requests of a unit
    __device__ __forceinline__ void open(int64_t row0, int g0, int g1, bool stall) {
        prow = row0, pg = g0, pend = g1;
        if (KIND != 2 && !wide() && lane == 0 && !stall) {
            const uint32_t bar = bars + 8 * (kStages + (pu % kStages)), n = (uint32_t)(ROWS * 2 * m.G);
            mb_arrive_expect(bar, n);
            bulk_load(sides + (pu % kStages) * n, m.scales + row0 * m.G, n, bar);
        }
        ++pu;
    }
    // requests the next stage of the open unit; false when that was its last
    __device__ __forceinline__ bool request(bool stall) {
        const int s = pn % kStages;
        if (lane == 0 && !stall) {
            const uint32_t bar = bars + 8 * s;
            mb_arrive_expect(bar, (uint32_t)(kCodes + kTiles));
            tma_load_2d(codes + s * kCodes, &m.codes, pg * group_bytes(KIND), (int)prow, bar);
            if constexpr (KIND == 2)
                tma_load_2d(sides + s * kTiles, &m.tiles, (int)(prow & 31) * 16, (int)((prow >> 7) * m.G + pg), bar);
        }
        ++pn;
        pg += kGroups;
        return pg < pend;
    }
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t par) {
        if (!dead) dead = !__all_sync(0xffffffffu, mb_wait_alone(bar, par, limit, &g_moe_timeouts));
        return !dead;
    }
    // begins reading a unit at its group g0
    __device__ __forceinline__ void begin(int64_t row0, int g0) {
        crow = row0, g = g0, left = 0;
        if (KIND != 2 && !wide()) wait(bars + 8 * (kStages + (cu % kStages)), (uint32_t)(cu / kStages) & 1u);
        ++cu;
    }
    // the stage of group g, of which the unit has `more` with the later ones, is there
    __device__ __forceinline__ void arrive(int more) {
        if (left > 0) return;
        wait(bars + 8 * stage, parity);
        gi = 0;
        left = min(kGroups, more);
    }
    // shared address of the lane's codes of the current group in 16-row tile w
    __device__ __forceinline__ uint32_t at(int w) const {
        const uint32_t base = codes + stage * kCodes + (w * 16 + row) * row_stride(KIND);
        if constexpr (KIND == 0) return base + (((uint32_t)(2 * gi + (t >> 1)) ^ (uint32_t)row) << 4) + (t & 1) * 8;
        if constexpr (KIND == 1) return base + gi * 48 + t * 12;
        return base + (((uint32_t)(4 * gi + t) ^ (uint32_t)row) << 4);
    }
    // scale of row `row` + r of the unit at the current group: its bf16 bits, or the lane's byte
    __device__ __forceinline__ uint32_t scale(int r) const {
        if constexpr (KIND == 2) {
            return lds8(sides + stage * kTiles + (gi * ROWS + row + r) * 16 + (int)(crow >> 5 & 3) * 4 + t);
        } else {
            if (wide()) return ld_stream_u16(m.scales + (crow + row + r) * m.G + g);
            return lds16(sides + ((cu - 1) % kStages) * (ROWS * 2 * m.G) + ((row + r) * m.G + g) * 2);
        }
    }
    // the current group has been read; true when its stage has, which then can be requested anew
    __device__ __forceinline__ bool next() {
        ++g, ++gi;
        if (gi < left) return false;
        left = 0;
        if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
        }
        __syncwarp();
        return true;
    }
    // what a wait that gave up left in flight ends, or its own wait does, before the exit
    __device__ __forceinline__ void drain(bool stall) const {
        if (!dead || lane != 0 || stall) return;
        for (int i = pn > kStages ? pn - kStages : 0; i < pn; ++i)
            mb_drain(bars + 8 * (i % kStages), (uint32_t)(i / kStages) & 1u, limit);
        if (KIND != 2 && !wide())
            for (int i = pu > kStages ? pu - kStages : 0; i < pu; ++i)
                mb_drain(bars + 8 * (kStages + i % kStages), (uint32_t)(i / kStages) & 1u, limit);
    }
};

// ---- the pairs grouped by expert ---------------------------------------------------
struct MoeList {
    unsigned long long mask[kMoeMaxExperts];  // tokens of each expert
    uint32_t blk[kMaxBlocks];                 // expert, first slot << 10, tokens << 20
    uint16_t first[kMoeMaxExperts];           // first slot of each expert
    uint8_t slot_token[kMaxPairs];
    int scan[2][kMoeWarps];
    int blocks, slots;
};
__device__ __forceinline__ int blk_expert(uint32_t b) { return (int)(b & 1023u); }
__device__ __forceinline__ int blk_slot(uint32_t b) { return (int)(b >> 10 & 1023u); }
__device__ __forceinline__ int blk_count(uint32_t b) { return (int)(b >> 20); }

// blocks of up to BT tokens
template <int THREADS, int BT>
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
        blocks += (c + BT - 1) / BT;
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
        L.first[e] = (uint16_t)s;
        for (int left = __popcll(m); left > 0; left -= BT) {
            const int n = min(BT, left);
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
template <int KG, int KU, int NS>
struct MoeUp {
    using Gate = Stream<KG, 16>;
    using Up = Stream<KU, 16>;
    static constexpr int kWarpRing = Gate::kRing + Up::kRing;
    static constexpr int kBars = Gate::kBars + Up::kBars;
    __host__ __device__ static int smem(int G, int S) {
        return kMoeWarps * (kWarpRing + Gate::side(G) + Up::side(G) + kBars) +
               (S > 1 ? 2 * kMoeWarps * NS * 1024 : 0) + 1024;
    }
};

template <int KG, int KU, int NS>
__global__ void __launch_bounds__(kMoeThreads, 4) k_moe_up(const __grid_constant__ MoeArgs A) {
    using M = MoeUp<KG, KU, NS>;
    extern __shared__ uint8_t raw[];
    __shared__ MoeList L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int G = A.gate.G, S = A.S, per = kMoeWarps / S, s = warp & (S - 1), ui = warp / S;
    // rings of all warps, then their scales, then partial sums [2][warps][NS][256] (two units deep), then barriers
    const uint32_t base = (sm_addr(raw) + 1023u) & ~1023u;
    const uint32_t ring = base + warp * M::kWarpRing;
    const uint32_t sides = base + kMoeWarps * M::kWarpRing + warp * (M::Gate::side(G) + M::Up::side(G));
    const uint32_t part_s = base + kMoeWarps * (M::kWarpRing + M::Gate::side(G) + M::Up::side(G));
    float* part = reinterpret_cast<float*>(raw + (part_s - sm_addr(raw)));
    const uint32_t bars = part_s + (S > 1 ? 2 * kMoeWarps * NS * 1024 : 0) + warp * M::kBars;
    typename M::Gate gate(A.gate, ring, sides, bars, A.wait_cycles);
    typename M::Up up(A.up, ring + M::Gate::kRing, sides + M::Gate::side(G), bars + M::Gate::kBars, A.wait_cycles);
    gate.init_bars();
    up.init_bars();
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    build_list<kMoeThreads, 8 * NS>(L, A);
    pdl_trigger();

    const int g0 = G * s / S, g1 = G * (s + 1) / S;
    const int tiles = A.I / 16, units = L.blocks * tiles, ustep = (int)gridDim.x * per;
    const bool stall = A.stall != 0;
    auto row_of = [&](int u) {
        const int blk = u / tiles;
        return (int64_t)blk_expert(L.blk[blk]) * A.I + (u - blk * tiles) * 16;
    };
    // each stream's next unit to request
    int gu = (int)blockIdx.x * per + ui, uu = gu;
    auto feed = [&](auto& m, int& u, bool& open) {
        if (u >= units || m.dead) return;
        if (!open) m.open(row_of(u), g0, g1, stall);
        open = m.request(stall);
        if (!open) u += ustep;
    };
    bool gopen = false, uopen = false;
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
        feed(gate, gu, gopen);
        feed(up, uu, uopen);
    }
    int flip = 0;
    for (int u = (int)blockIdx.x * per + ui; u < units; u += ustep) {
        const int blk = u / tiles, tile = u - blk * tiles;
        const uint32_t block = L.blk[blk];
        const int count = blk_count(block), slot0 = blk_slot(block);
        const int64_t row0 = (int64_t)blk_expert(block) * A.I + tile * 16;
        const uint16_t* xr[NS];
        bool have[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            have[n] = 8 * n + r < count;
            xr[n] = A.x + (int64_t)(have[n] ? L.slot_token[slot0 + 8 * n + r] : 0) * A.ldx + 32 * t;
        }
        float ag[NS][4], au[NS][4];
        uint32_t v[NS][16];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ag[n][i] = au[n][i] = 0.f;
#pragma unroll
            for (int q = 0; q < 16; ++q) v[n][q] = 0u;
        }
        gate.begin(row0, g0);
        up.begin(row0, g0);
#pragma unroll 1
        for (int g = g0; g < g1; ++g) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (have[n]) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 w = ld_act_u4(xr[n] + g * 128 + 8 * q);
                        v[n][4 * q] = w.x, v[n][4 * q + 1] = w.y, v[n][4 * q + 2] = w.z, v[n][4 * q + 3] = w.w;
                    }
                }
            // the activations in the order of the 4-bit decoder's pairs, where one is to read them
            uint32_t p[NS][16];
            if constexpr (KG == 2 || KU == 2) {
#pragma unroll
                for (int n = 0; n < NS; ++n) pair_up(p[n], v[n]);
            }
            gate.arrive(g1 - g);
            group_product<KG, NS>(gate.at(0), gate.scale(0), gate.scale(8), KG == 2 ? p : v, ag);
            if (gate.next()) feed(gate, gu, gopen);
            up.arrive(g1 - g);
            group_product<KU, NS>(up.at(0), up.scale(0), up.scale(8), KU == 2 ? p : v, au);
            if (up.next()) feed(up, uu, uopen);
        }
        const bool dead = gate.dead || up.dead;
        if (dead) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) ag[n][i] = au[n][i] = kMoeNaN;
        }
        if (S > 1) {
            float* mine = part + ((flip * kMoeWarps + warp) * NS) * 256 + lane;
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mine[n * 256 + i * 32] = ag[n][i];
                    mine[n * 256 + 128 + i * 32] = au[n][i];
                }
            // (constant barrier numbers: with a variable one a CTA holds all sixteen, and four CTAs fill the SM)
            if (ui == 0) asm volatile("bar.sync 1, %0;" ::"r"(S * 32) : "memory");
            else asm volatile("bar.sync 2, %0;" ::"r"(S * 32) : "memory");
            // warp s of the unit finishes registers s, s + S, ... of every set
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((i & (S - 1)) != s) continue;
                    float sg = 0.f, su = 0.f;
                    for (int w = 0; w < S; ++w) {
                        const float* q = part + ((flip * kMoeWarps + ui * S + w) * NS + n) * 256 + i * 32 + lane;
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
                const float gv = ag[n][i], h = gv / (1.f + expf(-gv)) * au[n][i];
                // h in the order in which the down kernel's lanes read a 128-group: 16-byte pieces (q, t)
                int c = (tile & 7) * 16 + gate.row + 8 * (i >> 1);
                if (A.hperm) c = (c & ~7) | (c & 3) << 1 | (c >> 2 & 1);
                c = ((c >> 3 & 3) << 2 | c >> 5) << 3 | (c & 7);
                A.h[(int64_t)(slot0 + col) * A.I + (tile >> 3) * 128 + c] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
            }
    }
    gate.drain(stall);
    up.drain(stall);
}

// ---- down and the weighted sum ------------------------------------------------------------
constexpr int kDownRows = 32;  // of a CTA: each warp holds all of them, two tiles that share h's fragments

// slices of a block's groups: enough tasks for the warps that share a tile, as far as z holds them
__device__ __forceinline__ int down_slices(int G, int warps, int blocks, int slots, int zrows) {
    if (blocks == 0) return 1;
    return max(1, min(min(G, (3 * warps + blocks - 1) / blocks), zrows / slots));
}

template <int KIND>
struct MoeDown {
    using W = Stream<KIND, kDownRows>;
    __host__ __device__ static int smem(int G) { return kMoeWarps * (W::kRing + W::side(G) + W::kBars) + 1024; }
};

template <int KIND, int NS>
__global__ void __launch_bounds__(kMoeThreads, 4) k_moe_down(const __grid_constant__ MoeArgs A) {
    using M = MoeDown<KIND>;
    extern __shared__ uint8_t raw[];
    __shared__ MoeList L;
    __shared__ float slot_w[kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3, C = A.C, G = A.down.G;
    const int rank = C > 1 ? (int)cluster_rank() : 0, tile = (int)blockIdx.x / C;
    const uint32_t base = (sm_addr(raw) + 1023u) & ~1023u;
    typename M::W w(A.down, base + warp * M::W::kRing, base + kMoeWarps * M::W::kRing + warp * M::W::side(G),
                    base + kMoeWarps * (M::W::kRing + M::W::side(G)) + warp * M::W::kBars, A.wait_cycles);
    w.init_bars();
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // the kernel before waited for its inputs: ids and weights are final, only h is not
    build_list<kMoeThreads, 8 * NS>(L, A);
    float* z = A.z + (int64_t)tile * A.zrows * kDownRows;  // the cluster's [slots][KS][kDownRows]
    // blocks fewer than the warps that share them: their groups are split too
    const int step = C * kMoeWarps, KS = down_slices(G, step, L.blocks, L.slots, A.zrows), tasks = L.blocks * KS;
    const bool stall = A.stall != 0;
    int pq = rank * kMoeWarps + warp;  // the next task to request
    bool open = false;
    auto feed = [&]() {
        if (pq >= tasks || w.dead) return;
        if (!open) {
            const int b = pq / KS, k = pq - b * KS;
            w.open((int64_t)blk_expert(L.blk[b]) * A.H + (int64_t)tile * kDownRows, G * k / KS, G * (k + 1) / KS, stall);
        }
        open = w.request(stall);
        if (!open) pq += step;
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) feed();
    for (int b = threadIdx.x; b < L.blocks; b += kMoeThreads) {
        const uint32_t blk = L.blk[b];
        for (int i = 0; i < blk_count(blk); ++i) {
            const int slot = blk_slot(blk) + i, tok = L.slot_token[slot];
            float v = 0.f;  // a token may name an expert more than once
            for (int j = 0; j < A.k; ++j)
                if (A.ids[tok * A.k + j] == blk_expert(blk)) v += A.weights[tok * A.k + j];
            slot_w[slot] = v;
        }
    }
    __syncthreads();
    pdl_wait();
    for (int q = rank * kMoeWarps + warp; q < tasks; q += step) {
        const int b = q / KS, k = q - b * KS, g0 = G * k / KS, g1 = G * (k + 1) / KS;
        const uint32_t block = L.blk[b];
        const int count = blk_count(block), slot0 = blk_slot(block);
        const uint16_t* hp[NS];
        bool have[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            have[n] = 8 * n + r < count;
            hp[n] = A.h + (int64_t)(slot0 + (have[n] ? 8 * n + r : 0)) * A.I + 8 * t;
        }
        float acc[2][NS][4];
        uint32_t v[NS][16];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][n][i] = acc[1][n][i] = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[n][j] = 0u;
        }
        w.begin((int64_t)blk_expert(block) * A.H + (int64_t)tile * kDownRows, g0);
#pragma unroll 1
        for (int g = g0; g < g1; ++g) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (have[n]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 u = ldg_plain(hp[n] + g * 128 + 32 * j);
                        v[n][4 * j] = u.x, v[n][4 * j + 1] = u.y, v[n][4 * j + 2] = u.z, v[n][4 * j + 3] = u.w;
                    }
                }
            w.arrive(g1 - g);
            group_product<KIND, NS>(w.at(0), w.scale(0), w.scale(8), v, acc[0]);
            group_product<KIND, NS>(w.at(1), w.scale(16), w.scale(24), v, acc[1]);
            if (w.next()) feed();
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int tok = 8 * n + 2 * t + j;
                if (tok >= count) continue;
                const int slot = slot0 + tok;
                float* p = z + ((int64_t)slot * KS + k) * kDownRows + w.row;
                const float f = w.dead ? kMoeNaN : slot_w[slot];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    p[16 * m] = f * acc[m][n][j];
                    p[16 * m + 8] = f * acc[m][n][2 + j];
                }
            }
    }
    w.drain(stall);
    __syncwarp();
    if (C > 1) {  // the cluster's z is complete
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // a token's slots in the order of its choices, a slot's slices in order; rank q finishes tokens q, q + C, ...
    for (int i = threadIdx.x; i < (A.T - rank + C - 1) / C * kDownRows; i += kMoeThreads) {
        const int tok = rank + i / kDownRows * C, row = i % kDownRows;
        float v = 0.f;
        for (int j = 0; j < A.k; ++j) {
            const int e = A.ids[tok * A.k + j];
            if (e < 0 || e >= A.E) continue;
            bool seen = false;
            for (int q = 0; q < j; ++q) seen |= A.ids[tok * A.k + q] == e;
            if (seen) continue;  // its slot holds all its weights
            const int slot = L.first[e] + __popcll(L.mask[e] & ((1ull << tok) - 1));
            const float* p = z + (int64_t)slot * KS * kDownRows + row;
            for (int q = 0; q < KS; ++q) v += __ldcg(p + q * kDownRows);
        }
        const int64_t at = (int64_t)tok * A.ldy + (int64_t)tile * kDownRows + row;
        if (A.ydt == kF32) static_cast<float*>(A.y)[at] = v;
        else static_cast<__nv_bfloat16*>(A.y)[at] = __float2bfloat16_rn(v);
    }
}

struct UpKernel {
    const void* fn;
    int (*smem)(int G, int S);
};
template <int KG, int KU, int NS>
UpKernel up_of() {
    return {reinterpret_cast<const void*>(&k_moe_up<KG, KU, NS>), &MoeUp<KG, KU, NS>::smem};
}
template <int NS>
UpKernel up_kernel(int kg, int ku) {
    static const UpKernel table[3][3] = {{up_of<0, 0, NS>(), up_of<0, 1, NS>(), up_of<0, 2, NS>()},
                                         {up_of<1, 0, NS>(), up_of<1, 1, NS>(), up_of<1, 2, NS>()},
                                         {up_of<2, 0, NS>(), up_of<2, 1, NS>(), up_of<2, 2, NS>()}};
    return table[kg][ku];
}
struct DownKernel {
    const void* fn;
    int (*smem)(int G);
};
template <int KIND, int NS>
DownKernel down_of() {
    return {reinterpret_cast<const void*>(&k_moe_down<KIND, NS>), &MoeDown<KIND>::smem};
}
template <int NS>
DownKernel down_kernel(int kind) {
    static const DownKernel table[3] = {down_of<0, NS>(), down_of<1, NS>(), down_of<2, NS>()};
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

// `rows`: of a unit
bool make_mat(MoeMat* m, const MoeWeights& w, int64_t N, int64_t K, int rows) {
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    m->scales = static_cast<const uint16_t*>(w.scales);
    m->kind = w.grid == kMx4 ? 2 : (w.grid == kInt3 ? 1 : 0);
    m->G = (int32_t)(K / kGroup);
    const cuuint32_t one[2] = {1, 1};
    {
        const cuuint64_t rb = (cuuint64_t)m->G * group_bytes(m->kind);
        const cuuint64_t dims[2] = {rb, (cuuint64_t)N}, strides[1] = {rb};
        const cuuint32_t box[2] = {(cuuint32_t)row_stride(m->kind), (cuuint32_t)rows};
        if (enc(&m->codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(w.packed), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, m->kind == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    if (m->kind == 2) {
        const cuuint64_t dims[2] = {512, (cuuint64_t)((N + 127) / 128 * m->G)}, strides[1] = {512};
        const cuuint32_t box[2] = {(cuuint32_t)(16 * rows), (cuuint32_t)stage_groups(2)};
        if (rows * 16 > 256) {  // a box holds at most 256 elements of a dimension: as 32-bit words
            const cuuint64_t d4[2] = {128, dims[1]};
            const cuuint32_t b4[2] = {(cuuint32_t)(4 * rows), box[1]};
            return enc(&m->tiles, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(w.scales), d4, strides, b4, one,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
        }
        return enc(&m->tiles, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(w.scales), dims, strides, box, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    return true;
}

// One split of the SM's memory for both kernels: with one of its own each, an SM is emptied and set up anew between them.
cudaError_t shape_kernel(const void* fn) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

}  // namespace

namespace {
size_t h_bytes(int64_t T, int k, int64_t I) { return (size_t)((T * k * I * 2 + 255) / 256 * 256); }
// rows of z: a slot's per slice of its groups
int64_t z_rows(int64_t T, int k) { return std::max<int64_t>(T * k, kMoeSliceRows); }
}  // namespace

size_t moe_data_bytes(int64_t T, int k, int64_t H, int64_t I) { return h_bytes(T, k, I) + (size_t)(z_rows(T, k) * H * 4); }

cudaError_t launch_moe(const MoeWeights& gate, const MoeWeights& up, const MoeWeights& down, int E, int64_t H, int64_t I,
                       const uint16_t* x, int64_t ldx, const int32_t* ids, const float* weights, int T, int k, void* y,
                       int ydt, int64_t ldy, void* data, long long wait_cycles, bool stall, cudaStream_t st) {
    const int sms = moe_sms();
    if (sms <= 0) return cudaErrorInitializationError;
    MoeArgs A;
    std::memset(&A, 0, sizeof(A));
    if (!make_mat(&A.gate, gate, E * I, H, 16) || !make_mat(&A.up, up, E * I, H, 16) ||
        !make_mat(&A.down, down, E * H, I, kDownRows))
        return cudaErrorInvalidValue;
    A.wait_cycles = wait_cycles;
    A.stall = stall ? 1 : 0;
    A.x = x;
    A.ids = ids;
    A.weights = weights;
    A.h = static_cast<uint16_t*>(data);
    A.z = reinterpret_cast<float*>(static_cast<char*>(data) + h_bytes(T, k, I));
    A.zrows = (int32_t)z_rows(T, k);
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
    A.hperm = A.down.kind == 2 ? 1 : 0;
    // Sets of eight columns that share a decode: one while an expert's tokens seldom exceed eight, else two (a second
    // set costs about a tenth of a product, a second decode a whole one)
    const int NS = T * k > 5 * E ? 2 : 1;
    const UpKernel ku = NS == 1 ? up_kernel<1>(A.gate.kind, A.up.kind) : up_kernel<2>(A.gate.kind, A.up.kind);
    const DownKernel kd = NS == 1 ? down_kernel<1>(A.down.kind) : down_kernel<2>(A.down.kind);
    const int up_smem = ku.smem(A.gate.G, A.S), down_smem = kd.smem(A.down.G);
    cudaError_t e = shape_kernel(ku.fn);
    if (e != cudaSuccess) return e;
    e = shape_kernel(kd.fn);
    if (e != cudaSuccess) return e;
    int per_sm = 0, down_per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, ku.fn, kMoeThreads, (size_t)up_smem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&down_per_sm, kd.fn, kMoeThreads, (size_t)down_smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1 || down_per_sm < 1) return cudaErrorInvalidConfiguration;
    // CTAs per cluster of the down kernel: the count whose waves, each as long as a warp's share of the blocks that
    // the tokens are expected to fill (in sixteenths of a block), end first
    const double filled = E * (1.0 - std::pow(1.0 - std::min(1.0, (double)k / E), T)) + T * k / (16.0 * NS);
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
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = (size_t)down_smem;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)A.C;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, kd.fn, args);
}

unsigned int take_moe_timeouts() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_moe_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    if (cudaMemcpyToSymbol(g_moe_timeouts, &z, sizeof(z)) != cudaSuccess) return 0xFFFFFFFFu;
    return v;
}

}  // namespace tb
