// tb_moe.cu -- the routed experts of a mixture-of-experts layer for a few
// tokens, straight from the packed codes, in two launches.
//
//     h[t,e] = silu(Wg[e] x[t]) * (Wu[e] x[t]),   y[t] = sum_j w[t,j] Wd[ids[t,j]] h[t,ids[t,j]]
//
// Every expert that some token takes is read once per eight or sixteen of its
// tokens: the layer would be bound by the bytes of the experts it touches, and
// is by the instructions that decode them, at 16 warps per SM (128 registers):
// 64 tokens x 128 experts of 4096 x 1536 in MX4 421 us (3.0 TB/s of codes; byte
// floor 193), issue slots 64 % and the ALU pipe 62 % busy in the up kernel; 16
// tokens x 64 experts of 2048 x 1408 in 2 and 3 bits 64 us (floor 19); one
// token x 8 of 128 experts of 2048 x 768, ternary, 13.5 us (floor 1.5), of
// which two launches, the expert lists and the first copies take about 10.
// A 16 x 128 tile takes a scheduler 153 (2 bits), 178 (3 bits) and 262 cycles
// (MX4), 64 of them its MMAs; HBM delivers one in 93, 137
// and 187.
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
// stream through a private ring per warp, filled by tensor copies of 16 rows
// x 128 (144) bytes.  (With cp.async, 32 rows' scattered 16- and 4-byte
// pieces per group, both kernels were bound by the L1's request rate: more
// warps changed nothing, 64 tokens x 4-bit experts took 466 us when tensor
// copies took 451.)
//
// h is rounded to bf16 between the two products, as tb_gate_up_silu's is: the
// MMA's operand, and half the activations a second part would cost (494 us
// against 416 at 64 tokens of the MX4 layer).
//
// k_moe_up: a unit is (block, 16 rows of gate and of up); S warps of a CTA
// split K where that evens out the warps' shares.  k_moe_down: a cluster of C
// CTAs holds 32 rows of H and deals the blocks, cut into slices of K where
// that evens out the shares, to its warps; each writes its weighted results
// to the workspace, and the cluster adds a token's in order (deterministic).
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
    int32_t C, zrows;
    uint32_t per_k;  // ceil(2^16 / k)
    int32_t hperm;  // h in the order of the 4-bit decode's pairs
};

namespace {

constexpr int kMoeWarps = 8;
constexpr int kMoeThreads = kMoeWarps * 32;
constexpr int kStages = 2;  // of a warp's ring
constexpr int kCtasPerSM = 2;  // of both kernels: 128 registers a thread
constexpr float kMoeNaN = __builtin_nanf("");
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxK;
constexpr int kMaxBlocks = kMoeMaxExperts + kMaxPairs / 8;

// packed bytes of a row's group; groups of a stage; bytes of a row in it.  The 2-bit and 4-bit stages have 128-byte rows
// in the 128-byte swizzle, the 3-bit ones plain rows of 144 bytes; with a tile's rows taken in bit-reversed order the
// reads of a group (8, 12 or 16 bytes by each lane of a quad, a row per quad) are free of bank conflicts in all three.
__host__ __device__ constexpr int group_bytes(int kind) { return kind == 0 ? 32 : (kind == 1 ? 48 : 64); }
__host__ __device__ constexpr int stage_groups(int kind) { return kind == 0 ? 4 : (kind == 1 ? 3 : 2); }
__host__ __device__ constexpr int row_stride(int kind) { return kind == 1 ? 144 : 128; }
// the row of a 16-row tile that a lane holds first (the second is eight on): lane / 4, its three bits reversed
__device__ __forceinline__ int tile_row(int lane) { return (lane >> 2 & 1) << 2 | (lane >> 2 & 2) | lane >> 4; }

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm(
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
__device__ __forceinline__ void mx4_product(const uint4& a, const uint4& b, uint32_t ba, uint32_t bb,
                                            const uint32_t (&x)[NS][16], float (&acc)[NS][4]) {
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

// One 128-group of 16 rows times NS sets of eight columns: acc += s W x.  `row`: the lane's codes in the first of its
// two rows (the second is eight rows on); s0, s1: the rows' scales as bf16 bits, or the lane's two scale bytes.
template <int KIND, int NS>
__device__ __forceinline__ void group_product(const uint8_t* row, uint32_t s0, uint32_t s1, const uint32_t (&x)[NS][16],
                                              float (&acc)[NS][4]) {
    const uint8_t* row8 = row + 8 * row_stride(KIND);
    if constexpr (KIND == 2) {
        const uint4 a = *reinterpret_cast<const uint4*>(row), b = *reinterpret_cast<const uint4*>(row8);
        if (__builtin_expect(__any_sync(0xffffffffu, max(s0, s1) > 128u), 0))
            mx4_product<NS, true>(a, b, s0, s1, x, acc);
        else
            mx4_product<NS, false>(a, b, s0, s1, x, acc);
    } else {
        float d[NS][4];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[n][i] = 0.f;
        if constexpr (KIND == 0) {
            const uint2 a = *reinterpret_cast<const uint2*>(row), b = *reinterpret_cast<const uint2*>(row8);
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
            const uint32_t* a = reinterpret_cast<const uint32_t*>(row);
            const uint32_t* b = reinterpret_cast<const uint32_t*>(row8);
            decode3_signed(a[0], a[1], a[2], ra);
            decode3_signed(b[0], b[1], b[2], rb);
#pragma unroll
            for (int j = 0; j < 16; j += 2)
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    mma_bf16(d[n], ra[j], rb[j], ra[j + 1], rb[j + 1], x[n][j], x[n][j + 1]);
        }
        const float f0 = __uint_as_float(s0 << 16), f1 = __uint_as_float(s1 << 16);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            acc[n][0] = fmaf(f0, d[n][0], acc[n][0]);
            acc[n][1] = fmaf(f0, d[n][1], acc[n][1]);
            acc[n][2] = fmaf(f1, d[n][2], acc[n][2]);
            acc[n][3] = fmaf(f1, d[n][3], acc[n][3]);
        }
    }
}

// ---- a warp's stream of weights -----------------------------------------------------------
// Units (TILES tiles of 16 rows, of one matrix or of two of the same format, and a range of groups), one after the
// other, through kStages stages of kGroups groups.  The warp requests a stage anew as soon as it has read it.
template <int KIND, int TILES>
struct Stream {
    static constexpr int kGroups = stage_groups(KIND);
    static constexpr int kCodes = 16 * row_stride(KIND);                  // of a tile in a stage
    static constexpr int kScales = KIND == 2 ? 256 * kGroups : 0;         // 4-bit: its scale rows
    // (swizzled tiles, 2 KB, begin at multiples of 1 KB)
    static constexpr int kStageCodes = TILES * kCodes;
    static constexpr int kBars = 8 * kStages;
    static constexpr int kRing = kStages * kStageCodes;
    // 4-bit scales beside the ring.  (bf16 scales are read where they are used, two bytes a row and group: copied into
    // shared memory by units they took as long, and the room of a second CTA: 61 tokens x 84 experts of 3584 x 1408,
    // 2- and 3-bit, 237 us against 186.)
    static constexpr int kSide = kStages * TILES * kScales;

    const MoeMat& m0;
    const MoeMat& m1;
    uint8_t *ring, *scl;
    uint32_t bars;
    long long limit;
    int off1;  // rows from tile 0 to tile 1: 0 (two matrices), or 16 from a row0 that is a multiple of 32
    bool stall, dead;
    uint32_t pn, cn;          // stages requested, read
    int64_t prow;             // the open unit's first row, its next group and their end
    int pg, pend;

    __device__ __forceinline__ Stream(const MoeMat& a, const MoeMat& b, int off, uint8_t* ring_, uint8_t* scl_,
                                      uint32_t bars_, const MoeArgs& A)
        : m0(a), m1(b), ring(ring_), scl(scl_), bars(bars_), limit(A.wait_cycles), off1(off), stall(A.stall != 0),
          dead(false), pn(0), cn(0), prow(0), pg(0), pend(0) {
        if (bars != 0 && (threadIdx.x & 31) == 0) {  // (0: a stream that is never used)
#pragma unroll
            for (int i = 0; i < kStages; ++i) mb_init(bars + 8 * i, 1);
            if (threadIdx.x == 0) {
                prefetch_map(&a.codes);
                if (TILES == 2) prefetch_map(&b.codes);
                if (KIND == 2) {
                    prefetch_map(&a.tiles);
                    if (TILES == 2) prefetch_map(&b.tiles);
                }
            }
        }
    }
    __device__ __forceinline__ bool open() const { return pg < pend; }

    // begins the requests of a unit
    __device__ __forceinline__ void start(int64_t row0, int g0, int g1) { prow = row0, pg = g0, pend = g1; }
    // requests the next stage of the open unit
    __device__ __forceinline__ void request() {
        if ((threadIdx.x & 31) == 0 && !stall) {
            const uint32_t s = pn % kStages, bar = bars + 8 * s, dst = sm_addr(ring) + s * kStageCodes;
            mb_arrive_expect(bar, TILES * (kCodes + kScales));
            tma_load_2d(dst, &m0.codes, pg * group_bytes(KIND), (int)prow, bar);
            if (TILES == 2) tma_load_2d(dst + kCodes, &m1.codes, pg * group_bytes(KIND), (int)prow + off1, bar);
            if constexpr (KIND == 2) {
                const uint32_t sd = sm_addr(scl) + s * TILES * kScales;
                tma_load_2d(sd, &m0.tiles, (int)(prow & 31) * 16, (int)((prow >> 7) * m0.G + pg), bar);
                if (TILES == 2) {
                    const int64_t r1 = prow + off1;
                    tma_load_2d(sd + kScales, &m1.tiles, (int)(r1 & 31) * 16, (int)((r1 >> 7) * m0.G + pg), bar);
                }
            }
        }
        ++pn;
        pg += kGroups;
    }
    __device__ __forceinline__ void wait(uint32_t bar, uint32_t parity) {
        if (!dead) dead = !__all_sync(0xffffffffu, mb_wait_alone(bar, parity, limit, &g_moe_timeouts));
    }
    // what is in flight ends, or its own wait does, before the exit
    __device__ __forceinline__ void drain() const {
        if (!dead || (threadIdx.x & 31) != 0 || stall) return;
        for (uint32_t i = pn > kStages ? pn - kStages : 0; i < pn; ++i)
            mb_drain(bars + 8 * (i % kStages), i / kStages & 1u, limit);
    }

    // acc += the unit's rows times the columns that load_x(g, x) gives, groups g0 .. g1 - 1; feed() requests the next
    // stage of this stream.  PAIR: the columns are in natural order and the 4-bit decoder wants its pairs.
    template <int NS, bool PAIR, class LoadX, class Feed>
    __device__ __forceinline__ void multiply(int64_t row0, int g0, int g1, LoadX load_x, Feed feed,
                                             float (&acc)[TILES][NS][4]) {
        const int lane = threadIdx.x & 31, t = lane & 3, row = tile_row(lane), G = m0.G;
        // the lane's codes of a stage's first group, and what the swizzle makes of the others'
        const uint32_t first = KIND == 1 ? row * 144 + t * 12
                                         : row * 128 + (KIND == 0 ? (((t >> 1) ^ row) << 4) + (t & 1) * 8 : (t ^ row) << 4);
        // the lane's first scale: 4-bit of the ring's first stage, else of tile 0 (of tile 1: `beside`)
        const uint8_t* const su = KIND == 2 ? scl + row * 16 + (int)(row0 >> 5 & 3) * 4 + t : nullptr;
        const uint16_t* const sg = KIND == 2 ? nullptr : m0.scales + (row0 + row) * G;
        const uint16_t* const beside = KIND == 2 || TILES == 1 ? nullptr : m1.scales + (row0 + off1 + row) * G;
        constexpr int kBuf = NS == 1 ? 2 : 1;
        uint32_t x[kBuf][NS][16];  // columns without a token stay 0: load_x leaves them alone
#pragma unroll
        for (int i = 0; i < kBuf; ++i)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int q = 0; q < 16; ++q) x[i][n][q] = 0u;
#pragma unroll 1
        for (int g = g0; g < g1; g += kGroups) {
            const uint32_t s = cn % kStages;
            const uint8_t* codes = ring + s * kStageCodes;
            load_x(g, x[0]);
            wait(bars + 8 * s, cn / kStages & 1u);
            ++cn;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                if (i > 0 && g + i >= g1) break;
                // with one set the next group's activations are requested ahead of this one's products
                if (NS == 1 && i + 1 < kGroups && g + i + 1 < g1) load_x(g + i + 1, x[(i + 1) % kBuf]);
                if (NS > 1 && i > 0) load_x(g + i, x[0]);
                uint32_t xp[NS][16];
                if constexpr (PAIR) {
#pragma unroll
                    for (int n = 0; n < NS; ++n) pair_up(xp[n], x[i % kBuf][n]);
                }
#pragma unroll
                for (int w = 0; w < TILES; ++w) {
                    uint32_t s0, s1;
                    if constexpr (KIND == 2) {
                        const uint8_t* p = su + (s * TILES + w) * kScales + i * 256;
                        s0 = p[0], s1 = p[128];
                    } else {
                        const uint16_t* p = (w ? beside : sg) + g + i;
                        s0 = __ldg(p), s1 = __ldg(p + 8 * G);
                    }
                    const uint32_t at = KIND == 1 ? first + i * 48 : first ^ (uint32_t)(i * group_bytes(KIND));
                    if constexpr (PAIR) group_product<KIND, NS>(codes + w * kCodes + at, s0, s1, xp, acc[w]);
                    else group_product<KIND, NS>(codes + w * kCodes + at, s0, s1, x[i % kBuf], acc[w]);
                }
            }
            __syncwarp();
            if (!dead) feed();
        }
    }
};

// ---- the pairs grouped by expert ---------------------------------------------------
struct MoeMasks {
    uint32_t mask[2][kMoeMaxExperts];  // tokens of each expert: the first 32, the others
    uint16_t first[kMoeMaxExperts];    // first slot of each expert
};
struct MoeList {
    uint32_t blk[kMaxBlocks];  // expert, first slot << 10, tokens << 20
    uint8_t slot_token[kMaxPairs];
    int scan[2][kMoeWarps];
    int blocks, slots;
};
__device__ __forceinline__ int blk_expert(uint32_t b) { return (int)(b & 1023u); }
__device__ __forceinline__ int blk_slot(uint32_t b) { return (int)(b >> 10 & 1023u); }
__device__ __forceinline__ int blk_count(uint32_t b) { return (int)(b >> 20); }
// the token of pair p < 1024: p / k by a multiplication (exact, k <= 16)
__device__ __forceinline__ int pair_token(int p, const MoeArgs& A) { return (int)((uint32_t)p * A.per_k >> 16); }

// blocks of up to BT tokens; `pair_expert` (or null): the expert of every pair, -1 for none.  The ids are read past the
// L1: see k_moe_down.
template <int BT>
__device__ void build_list(MoeList& L, MoeMasks& X, int16_t* pair_expert, const MoeArgs& A) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < A.E; e += kMoeThreads) X.mask[0][e] = X.mask[1][e] = 0u;
    __syncthreads();
    for (int p = tid; p < A.T * A.k; p += kMoeThreads) {
        const int id = __ldcg(A.ids + p), t = pair_token(p, A), e = id >= 0 && id < A.E ? id : -1;
        if (e >= 0) atomicOr(&X.mask[t >> 5][e], 1u << (t & 31));  // a set: the order does not matter
        if (pair_expert) pair_expert[p] = (int16_t)e;
    }
    __syncthreads();
    constexpr int kPer = kMoeMaxExperts / kMoeThreads;  // experts of a thread
    int slots = 0, blocks = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        const int c = e < A.E ? __popc(X.mask[0][e]) + __popc(X.mask[1][e]) : 0;
        slots += c;
        blocks += (c + BT - 1) / BT;
    }
    // slots and blocks (below 2^16 each) summed over the threads before this one
    const uint32_t mine = (uint32_t)slots << 16 | (uint32_t)blocks;
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) L.scan[0][warp] = (int)sum;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kMoeWarps; ++w) {
        const uint32_t v = (uint32_t)L.scan[0][w];
        if (w < warp) before += v;
        all += v;
    }
    if (tid == 0) {
        L.slots = (int)(all >> 16);
        L.blocks = (int)(all & 0xFFFFu);
    }
    sum += before - mine;
    int s = (int)(sum >> 16), b = (int)(sum & 0xFFFFu);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        if (e >= A.E) break;
        X.first[e] = (uint16_t)s;
        unsigned long long m = (unsigned long long)X.mask[1][e] << 32 | X.mask[0][e];
        for (int left = __popcll(m); left > 0; left -= BT) {
            const int n = min(BT, left);
            L.blk[b++] = (uint32_t)e | (uint32_t)s << 10 | (uint32_t)n << 20;
            for (int q = 0; q < n; ++q) {
                L.slot_token[s++] = (uint8_t)(__ffsll((long long)m) - 1);
                m &= m - 1;
            }
        }
    }
    __syncthreads();
}

// ---- gate and up -----------------------------------------------------------------------
// Of one format, gate's and up's tiles share the stages and the activations' fragments; else each has a stream.
template <int KG, int KU, int NS>
struct MoeUp {
    static constexpr bool kBoth = KG == KU;
    using Gate = Stream<KG, kBoth ? 2 : 1>;
    using Up = Stream<KU, 1>;
    // a warp's rings: a swizzled one begins at a multiple of 1 KB, so it comes first
    static constexpr bool kUpFirst = !kBoth && KG == 1;
    static constexpr int kGateAt = kUpFirst ? Up::kRing : 0, kUpAt = kBoth || kUpFirst ? 0 : Gate::kRing;
    static constexpr int kRings = Gate::kRing + (kBoth ? 0 : Up::kRing);
    static constexpr int kWarpRing = kBoth && KG == 1 ? kRings : (kRings + 1023) & ~1023;
    static constexpr int kBars = Gate::kBars + (kBoth ? 0 : Up::kBars);
    static constexpr int kPart = kMoeWarps * 1024;  // partial sums of split units, a set at a time; first the masks
    static_assert(sizeof(MoeMasks) <= kPart);
    static constexpr int kSide = Gate::kSide + (kBoth ? 0 : Up::kSide);
    static constexpr int kSmem = kMoeWarps * (kWarpRing + kSide + kBars) + kPart + 1024;
    static_assert(2 * (kSmem + (int)sizeof(MoeList) + 1024) <= 228 * 1024, "two CTAs per SM");
};

// the S warps of unit `ui` of a CTA (constant barrier numbers: with a variable one a CTA holds all sixteen of its SM's)
__device__ __forceinline__ void unit_sync(int ui, int S) {
    if (ui == 0) asm volatile("bar.sync 1, %0;" ::"r"(S * 32) : "memory");
    else if (ui == 1) asm volatile("bar.sync 2, %0;" ::"r"(S * 32) : "memory");
    else if (ui == 2) asm volatile("bar.sync 3, %0;" ::"r"(S * 32) : "memory");
    else asm volatile("bar.sync 4, %0;" ::"r"(S * 32) : "memory");
}

template <int KG, int KU, int NS>
__global__ void __launch_bounds__(kMoeThreads, kCtasPerSM) k_moe_up(const __grid_constant__ MoeArgs A) {
    using M = MoeUp<KG, KU, NS>;
    extern __shared__ uint8_t raw[];
    __shared__ MoeList L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3, G = A.gate.G;
    // rings of all warps, partial sums, the warps' scales, barriers
    uint8_t* const base = raw + ((1024u - (sm_addr(raw) & 1023u)) & 1023u);
    uint8_t* const ring = base + warp * M::kWarpRing;
    float* const part = reinterpret_cast<float*>(base + kMoeWarps * M::kWarpRing);
    uint8_t* const side = base + kMoeWarps * M::kWarpRing + M::kPart + warp * M::kSide;
    const uint32_t bars = sm_addr(base + kMoeWarps * (M::kWarpRing + M::kSide) + M::kPart) + warp * M::kBars;
    typename M::Gate gate(A.gate, M::kBoth ? A.up : A.gate, 0, ring + M::kGateAt, side, bars, A);
    typename M::Up up(A.up, A.up, 0, ring + M::kUpAt, side + M::Gate::kSide,
                      M::kBoth ? 0u : bars + M::Gate::kBars, A);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    fence_copies();
    build_list<8 * NS>(L, *reinterpret_cast<MoeMasks*>(part), nullptr, A);
    pdl_trigger();  // not before pdl_wait: k_moe_down begins with what the kernels before this one wrote

    // warps that share a unit, each a part of K: the number whose rounds over all units end first (in half groups; a unit
    // costs about one to begin and end, two where its parts are added)
    const int tiles = A.I / 16, units = L.blocks * tiles;
    int lg = 0, least = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (1 << i > G) break;
        const int slots = (int)gridDim.x * kMoeWarps >> i, rounds = (units + slots - 1) / slots;
        const int cost = rounds * (2 * (G + (1 << i) - 1 >> i) + (i ? 2 : 1));
        if (cost < least) {
            least = cost;
            lg = i;
        }
    }
    const int S = 1 << lg, per = kMoeWarps >> lg, s = warp & (S - 1), ui = warp >> lg;
    const int g0 = G * s >> lg, g1 = G * (s + 1) >> lg;
    const int ustep = (int)gridDim.x * per, u0 = (int)blockIdx.x * per + ui;
    struct Unit {
        int blk, tile;
    };
    const int sblk = ustep / tiles, stile = ustep - sblk * tiles;
    const Unit first{u0 / tiles, u0 % tiles};
    auto advance = [&](Unit& v) {
        v.blk += sblk;
        v.tile += stile;
        if (v.tile >= tiles) {
            v.tile -= tiles;
            ++v.blk;
        }
    };
    auto row_of = [&](const Unit& v) { return (int64_t)blk_expert(L.blk[v.blk]) * A.I + v.tile * 16; };
    Unit gu = first, uu = first;  // the next units that the streams request
    auto feed_gate = [&]() {
        if (!gate.open()) {
            if (gu.blk >= L.blocks) return;
            gate.start(row_of(gu), g0, g1);
            advance(gu);
        }
        gate.request();
    };
    auto feed_up = [&]() {
        if (!up.open()) {
            if (uu.blk >= L.blocks) return;
            up.start(row_of(uu), g0, g1);
            advance(uu);
        }
        up.request();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
        feed_gate();
        if (!M::kBoth) feed_up();
    }
    for (Unit u = first; u.blk < L.blocks; advance(u)) {
        const int tile = u.tile;
        const uint32_t block = L.blk[u.blk];
        const int count = blk_count(block), slot0 = blk_slot(block);
        const int64_t row0 = row_of(u);
        const uint16_t* xr[NS];
        bool have[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            have[n] = 8 * n + r < count;
            xr[n] = A.x + (int64_t)(have[n] ? L.slot_token[slot0 + 8 * n + r] : 0) * A.ldx + 32 * t;
        }
        auto load = [&](int g, uint32_t (&x)[NS][16]) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (have[n]) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 w = *reinterpret_cast<const uint4*>(xr[n] + g * 128 + 8 * q);
                        x[n][4 * q] = w.x, x[n][4 * q + 1] = w.y, x[n][4 * q + 2] = w.z, x[n][4 * q + 3] = w.w;
                    }
                }
        };
        float acc[2][NS][4];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][n][i] = acc[1][n][i] = 0.f;
        if constexpr (M::kBoth) {
            gate.template multiply<NS, KG == 2>(row0, g0, g1, load, feed_gate, acc);
        } else {
            float one[1][NS][4], two[1][NS][4];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) one[0][n][i] = two[0][n][i] = 0.f;
            gate.template multiply<NS, KG == 2>(row0, g0, g1, load, feed_gate, one);
            up.template multiply<NS, KU == 2>(row0, g0, g1, load, feed_up, two);
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][n][i] = one[0][n][i], acc[1][n][i] = two[0][n][i];
        }
        if (gate.dead || up.dead) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][n][i] = acc[1][n][i] = kMoeNaN;
        }
        if (S > 1) {
            float* mine = part + warp * 256 + lane;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mine[i * 32] = acc[0][n][i];
                    mine[128 + i * 32] = acc[1][n][i];
                }
                unit_sync(ui, S);
                // warp s of the unit finishes registers s, s + S, ... of every set
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((i & (S - 1)) != s) continue;
                    float sg = 0.f, su = 0.f;
                    for (int w = 0; w < S; ++w) {
                        const float* q = part + (ui * S + w) * 256 + i * 32 + lane;
                        sg += q[0];
                        su += q[128];
                    }
                    acc[0][n][i] = sg;
                    acc[1][n][i] = su;
                }
                unit_sync(ui, S);
            }
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = 8 * n + 2 * t + (i & 1);
                if ((i & (S - 1)) != s || col >= count) continue;
                // (the fast functions' errors, at most 2^-16, are far below the rounding of h)
                const float gv = acc[0][n][i], h = __fdividef(gv, 1.f + __expf(-gv)) * acc[1][n][i];
                // h in the order in which the down kernel's lanes read a 128-group: 16-byte pieces (q, t)
                int c = (tile & 7) * 16 + tile_row(lane) + 8 * (i >> 1);
                if (A.hperm) c = (c & ~7) | (c & 3) << 1 | (c >> 2 & 1);
                c = ((c >> 3 & 3) << 2 | c >> 5) << 3 | (c & 7);
                A.h[(int64_t)(slot0 + col) * A.I + (tile >> 3) * 128 + c] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
            }
    }
    gate.drain();
    if (!M::kBoth) up.drain();
}

// ---- down and the weighted sum ------------------------------------------------------------
constexpr int kDownRows = 32;  // of a CTA: each warp holds all of them, two tiles that share h's fragments

// Slices of a block's groups, as far as z holds them: the number whose rounds over the tile's warps end first (in groups;
// a task costs about two more to begin and end).
struct DownSplit {
    int slices, cost;
};
__host__ __device__ __forceinline__ DownSplit down_split(int G, int warps, int blocks, int slots, int zrows) {
    DownSplit best{1, 0x7FFFFFFF};
    for (int k = 1; k <= G && k <= 8 && (k == 1 || k * slots <= zrows); ++k) {
        const int cost = (blocks * k + warps - 1) / warps * ((G + k - 1) / k + 2);
        if (cost < best.cost) best = {k, cost};
    }
    return best;
}

template <int KIND>
struct MoeDown {
    using W = Stream<KIND, 2>;
    static constexpr int kFixed = sizeof(MoeList) + sizeof(MoeMasks) + kMaxPairs * 8;
    static constexpr int kSmem = kMoeWarps * (W::kRing + W::kSide + W::kBars) + 1024;
    static_assert(2 * (kSmem + kFixed + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int KIND, int NS>
__global__ void __launch_bounds__(kMoeThreads, kCtasPerSM) k_moe_down(const __grid_constant__ MoeArgs A) {
    using W = typename MoeDown<KIND>::W;
    extern __shared__ uint8_t raw[];
    __shared__ MoeList L;
    __shared__ MoeMasks X;
    __shared__ float slot_w[kMaxPairs];
    __shared__ int16_t pair_expert[kMaxPairs], pair_slot[kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3, C = A.C, G = A.down.G;
    const int rank = C > 1 ? (int)cluster_rank() : 0, tile = (int)blockIdx.x / C;
    uint8_t* const base = raw + ((1024u - (sm_addr(raw) & 1023u)) & 1023u);
    W w(A.down, A.down, 16, base + warp * W::kRing, base + kMoeWarps * W::kRing + warp * W::kSide,
        sm_addr(base + kMoeWarps * (W::kRing + W::kSide)) + warp * W::kBars, A);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_trigger();
    // Ahead of this kernel's own wait, ids, weights and the experts' codes and scale tiles are read, and nothing else.  They
    // are final: k_moe_up lets this kernel begin only after its own wait, behind which every kernel before it has completed
    // and its writes have reached the L2.  This SM's L1 may still hold older lines (it need not have had a CTA of
    // k_moe_up), so ids and weights are read past it, as the tensor copies read the experts.  bf16 scales, which are read
    // through the L1, and h come after the wait.
    fence_copies();
    build_list<8 * NS>(L, X, pair_expert, A);
    float* z = A.z + (int64_t)tile * A.zrows * kDownRows;  // the cluster's [slots][KS][kDownRows]
    const int step = C * kMoeWarps, KS = down_split(G, step, L.blocks, L.slots, A.zrows).slices, tasks = L.blocks * KS;
    const int q0 = rank * kMoeWarps + warp;
    int pq = q0;  // the next task to request
    auto feed = [&]() {
        if (!w.open()) {
            if (pq >= tasks) return;
            const int b = pq / KS, k = pq - b * KS;
            w.start((int64_t)blk_expert(L.blk[b]) * A.H + (int64_t)tile * kDownRows, G * k / KS, G * (k + 1) / KS);
            pq += step;
        }
        w.request();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) feed();
    // a pair's slot, or -1: none, or its token names the expert before; the slot's weight: that of all such pairs
    for (int p = threadIdx.x; p < A.T * A.k; p += kMoeThreads) {
        const int e = pair_expert[p], tok = pair_token(p, A);
        int slot = -1;
        if (e >= 0) {
            const uint32_t below = (1u << (tok & 31)) - 1u;
            slot = X.first[e] + (tok < 32 ? __popc(X.mask[0][e] & below) : __popc(X.mask[0][e]) + __popc(X.mask[1][e] & below));
            float v = __ldcg(A.weights + p);
            for (int q = tok * A.k; q < (tok + 1) * A.k; ++q)
                if (q != p && pair_expert[q] == e) {
                    if (q < p) slot = -1;
                    v += __ldcg(A.weights + q);
                }
            if (slot >= 0) slot_w[slot] = v;
        }
        pair_slot[p] = (int16_t)slot;
    }
    __syncthreads();
    pdl_wait();
    for (int q = q0; q < tasks; q += step) {
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
        auto load_h = [&](int g, uint32_t (&x)[NS][16]) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (have[n]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 u = *reinterpret_cast<const uint4*>(hp[n] + g * 128 + 32 * j);
                        x[n][4 * j] = u.x, x[n][4 * j + 1] = u.y, x[n][4 * j + 2] = u.z, x[n][4 * j + 3] = u.w;
                    }
                }
        };
        float acc[2][NS][4];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][n][i] = acc[1][n][i] = 0.f;
        w.template multiply<NS, false>((int64_t)blk_expert(block) * A.H + (int64_t)tile * kDownRows, g0, g1, load_h, feed, acc);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int tok = 8 * n + 2 * t + j;
                if (tok >= count) continue;
                const int slot = slot0 + tok;
                float* p = z + ((int64_t)slot * KS + k) * kDownRows + tile_row(lane);
                const float f = w.dead ? kMoeNaN : slot_w[slot];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    p[16 * m] = f * acc[m][n][j];
                    p[16 * m + 8] = f * acc[m][n][2 + j];
                }
            }
    }
    w.drain();
    __syncwarp();
    if (C > 1) {  // the cluster's z is complete
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // Rank q finishes tokens q, q + C, ...: eight lanes an output, each adding every eighth of the token's (choice,
    // slice) results, then one another's.
    const int part = threadIdx.x & 7, items = A.k * KS, outs = (A.T - rank + C - 1) / C * kDownRows;
    for (int i = threadIdx.x >> 3; i < (outs + 3 & ~3); i += kMoeThreads / 8) {  // (a warp's four outputs together)
        const int tok = rank + i / kDownRows * C, row = i % kDownRows;
        float v = 0.f;
        if (i < outs) {
            int j = part / KS, q = part - j * KS;
            const int dj = 8 / KS, dq = 8 - dj * KS;
#pragma unroll 4
            for (int n = part; n < items; n += 8) {
                const int slot = pair_slot[tok * A.k + j];
                if (slot >= 0) v += __ldcg(z + ((int64_t)slot * KS + q) * kDownRows + row);
                j += dj;
                q += dq;
                if (q >= KS) {
                    q -= KS;
                    ++j;
                }
            }
        }
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        if (part == 0 && i < outs) {
            const int64_t at = (int64_t)tok * A.ldy + (int64_t)tile * kDownRows + row;
            if (A.ydt == kF32) static_cast<float*>(A.y)[at] = v;
            else static_cast<__nv_bfloat16*>(A.y)[at] = __float2bfloat16_rn(v);
        }
    }
}

// One split of the SM's memory for both kernels: with one of its own each, an SM is emptied and set up anew between them.
cudaError_t shape_kernel(const void* fn, int smem) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

// A kernel, its shared memory and its setup on the current device.
struct MoeKernel {
    const void* fn;
    int smem;
    cudaError_t (*setup)();
    int (*held)(int c);  // k_moe_down: clusters of c CTAs at once
};
template <int KG, int KU, int NS>
cudaError_t up_setup() {
    return once_per_device<MoeUp<KG, KU, NS>>([] { return shape_kernel(reinterpret_cast<const void*>(&k_moe_up<KG, KU, NS>), MoeUp<KG, KU, NS>::kSmem); });
}
template <int KG, int KU, int NS>
MoeKernel up_of() {
    return {reinterpret_cast<const void*>(&k_moe_up<KG, KU, NS>), MoeUp<KG, KU, NS>::kSmem, &up_setup<KG, KU, NS>, nullptr};
}
template <int NS>
MoeKernel up_kernel(int kg, int ku) {
    static const MoeKernel table[3][3] = {{up_of<0, 0, NS>(), up_of<0, 1, NS>(), up_of<0, 2, NS>()},
                                          {up_of<1, 0, NS>(), up_of<1, 1, NS>(), up_of<1, 2, NS>()},
                                          {up_of<2, 0, NS>(), up_of<2, 1, NS>(), up_of<2, 2, NS>()}};
    return table[kg][ku];
}
template <int KIND, int NS>
struct DownOf;  // names a kernel
template <int KIND, int NS>
cudaError_t down_setup() {
    return once_per_device<DownOf<KIND, NS>>([] { return shape_kernel(reinterpret_cast<const void*>(&k_moe_down<KIND, NS>), MoeDown<KIND>::kSmem); });
}
template <int KIND, int NS>
int down_held(int c) {
    return clusters_at_once<DownOf<KIND, NS>>(reinterpret_cast<const void*>(&k_moe_down<KIND, NS>), kMoeThreads,
                                              (size_t)MoeDown<KIND>::kSmem, c);
}
template <int KIND, int NS>
MoeKernel down_of() {
    return {reinterpret_cast<const void*>(&k_moe_down<KIND, NS>), MoeDown<KIND>::kSmem, &down_setup<KIND, NS>,
            &down_held<KIND, NS>};
}
template <int NS>
MoeKernel down_kernel(int kind) {
    static const MoeKernel table[3] = {down_of<0, NS>(), down_of<1, NS>(), down_of<2, NS>()};
    return table[kind];
}
bool make_mat(MoeMat* m, const MoeWeights& w, int64_t N, int64_t K) {
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    m->scales = static_cast<const uint16_t*>(w.scales);
    m->kind = w.grid == kMx4 ? 2 : (w.grid == kInt3 ? 1 : 0);
    m->G = (int32_t)(K / kGroup);
    const cuuint32_t one[2] = {1, 1};
    {
        const cuuint64_t rb = (cuuint64_t)m->G * group_bytes(m->kind);
        const cuuint64_t dims[2] = {rb, (cuuint64_t)N}, strides[1] = {rb};
        const cuuint32_t box[2] = {(cuuint32_t)row_stride(m->kind), 16};
        if (enc(&m->codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(w.packed), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, m->kind == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    if (m->kind == 2) {
        const cuuint64_t dims[2] = {512, (cuuint64_t)((N + 127) / 128 * m->G)}, strides[1] = {512};
        const cuuint32_t box[2] = {256, (cuuint32_t)stage_groups(2)};
        return enc(&m->tiles, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(w.scales), dims, strides, box, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    return true;
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
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInitializationError;
    MoeArgs A;
    std::memset(&A, 0, sizeof(A));
    if (!make_mat(&A.gate, gate, E * I, H) || !make_mat(&A.up, up, E * I, H) || !make_mat(&A.down, down, E * H, I))
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
    A.per_k = (65536u + (uint32_t)k - 1) / (uint32_t)k;
    A.E = E;
    A.H = (int32_t)H;
    A.I = (int32_t)I;
    A.ydt = ydt;
    A.hperm = A.down.kind == 2 ? 1 : 0;
    // Sets of eight columns that share a decode: one up to ten pairs per expert, then two.  (The second set's activations
    // take the registers of the prefetch, so it pays late: over 130 layers of the supported range two are 5 to 25 %
    // slower below six pairs per expert, even at nine, 5 to 20 % faster above twenty.)
    const int NS = T * k > 10 * E ? 2 : 1;
    const MoeKernel ku = NS == 1 ? up_kernel<1>(A.gate.kind, A.up.kind) : up_kernel<2>(A.gate.kind, A.up.kind);
    const MoeKernel kd = NS == 1 ? down_kernel<1>(A.down.kind) : down_kernel<2>(A.down.kind);
    cudaError_t e = ku.setup();
    if (e != cudaSuccess) return e;
    e = kd.setup();
    if (e != cudaSuccess) return e;
    // CTAs per cluster of the down kernel: the count whose waves end first (in groups of a warp, about 0.6 us: a wave costs
    // its warps' share of the blocks that the tokens are expected to fill and four more, a cluster's barrier three, each
    // of its CTAs a half).  Over 120 layers of the supported range within 2.4 % of the best count of each; always two
    // loses 8 %, always four 13 %.
    const double taken = E * (1.0 - std::pow(1.0 - std::min(1.0, (double)k / E), T));  // experts
    const double filled = taken + std::max(0.0, (T * k - taken * 4 * NS) / (8 * NS));  // blocks: more from half of one on
    int64_t best = INT64_MAX;
    for (int c = 1; c <= 8; ++c) {
        const int64_t held = c == 1 ? (int64_t)sms * kCtasPerSM : kd.held(c);
        if (held < 1) continue;
        const int64_t waves = (H / kDownRows + held - 1) / held;
        const int share = down_split((int)(I / kGroup), c * kMoeWarps, std::max(1, (int)(filled + 0.5)), T * k, A.zrows).cost;
        const int64_t cost = 2 * waves * (share + 4) + (c > 1 ? 6 : 0) + c;
        if (cost < best) {
            best = cost;
            A.C = c;
        }
    }
    // no more CTAs than the units that the pairs can make at most
    const int64_t ctas = std::min<int64_t>((int64_t)std::min(T * k, E + T * k / 8) * (I / 16), (int64_t)sms * kCtasPerSM);

    void* args[] = {&A};
    e = launch_early(ku.fn, ctas, kMoeThreads, (size_t)ku.smem, 1, args, st);
    if (e != cudaSuccess) return e;
    return launch_early(kd.fn, H / kDownRows * A.C, kMoeThreads, (size_t)kd.smem, A.C, args, st);
}

unsigned int take_moe_timeouts() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_moe_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    if (v != 0 && cudaMemcpyToSymbol(g_moe_timeouts, &z, sizeof(z)) != cudaSuccess) return 0xFFFFFFFFu;
    return v;
}

}  // namespace tb
