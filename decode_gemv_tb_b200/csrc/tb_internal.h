// tb_internal.h -- launchers behind the C interface (host side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace tb {

struct Launch;

// The ternary grid in the optional 5-trits-per-byte layout (include/tb.h):
// 26 bytes per 128-group, rows padded to 16 bytes.
constexpr int kTernaryB3 = 3;
constexpr int64_t kB3GroupBytes = 26;
__host__ __device__ inline int64_t b3_row_bytes(int64_t K) { return 16 * ((kB3GroupBytes * (K / 128) + 15) / 16); }

cudaError_t launch_scales(const void* W, int w_dtype, int64_t N, int64_t K, int grid, uint16_t* scales,
                          cudaStream_t st);
cudaError_t launch_pack(const void* W, int w_dtype, int64_t N, int64_t K, int grid, const uint16_t* scales,
                        void* packed, int32_t* bad_count, cudaStream_t st);
cudaError_t launch_unpack(const void* packed, int grid, int64_t N, int64_t K, int8_t* codes, cudaStream_t st);

// Small-batch launch (2 <= M <= 16 batch rows per item): one kernel, no
// workspace.  `nt` is the number of 8-wide column tiles (1 or 2), `ctas`
// the grid.
cudaError_t launch_linear(const Launch& L, int nt, int ctas, cudaStream_t st);
// dynamic shared memory of the main kernel
size_t linear_smem_bytes(int nt, int scl_stride);

struct G8Launch;
// Batch-1 GEMV on the integer tensor path (tb_gemv8.cu): one kernel,
// k_gemv8.  `overlap` launches it as a programmatic dependent of the
// previous work (it streams weights before that work has finished).
// `two`: the layout of two CTAs per SM (calls of many chunks per SM), else
// one CTA per SM.
cudaError_t launch_gemv8(const G8Launch& L, bool two, bool overlap, cudaStream_t st);
// weights of one matrix (box: one chunk x 256 rows) / its scales [N][G] (G % 8 == 0)
bool encode_g8_wmap(CUtensorMap* map, const void* packed, int grid, int64_t N, int64_t K);
bool encode_g8_smap(CUtensorMap* map, const uint16_t* scales, int64_t N, int64_t Gp);
// groups per chunk (4 for the 2-bit container, 2 for 3 bits)
int g8_chunk_groups(int grid);
// CTAs of k_gemv8 resident at once on the current device in the layout
// `two` (0 on error)
int gemv8_ctas(bool two);
// bounded waits of k_gemv8 that gave up since the last call (clears)
unsigned int take_g8_timeouts();

// Batch-1 GEMV in one launch, one warp per output row, no workspace: the
// 5-trits-per-byte layout, and small problems in the other layouts.  The
// activations are staged in shared memory, which bounds K
// (gemv_rowwarp_supported).
bool gemv_rowwarp_supported(int grid, int64_t K);
cudaError_t launch_gemv_rowwarp(const void* packed, int grid, const uint16_t* scales, const uint16_t* x, void* y,
                                int ydt, int64_t N, int64_t K, cudaStream_t st);

// Small-batch GEMM on the tcgen05 tensor cores (2 <= M <= 64): preparation
// kernel + main kernel.  Workspace: gemm_tc_workspace_bytes(M, N, K) bytes,
// 256-byte aligned (device independent).
size_t gemm_tc_workspace_bytes(int64_t M, int64_t N, int64_t K);
cudaError_t launch_gemm_tc(const void* packed, int grid, const uint16_t* scales, const uint16_t* X, int64_t ldx,
                           void* Y, int ydt, int64_t ldy, int M, int64_t N, int64_t K, void* ws, cudaStream_t st);
// Prefill GEMM with both MMA operands in shared memory (tb_gemm_ss.cu): one
// kernel, M > 64 batch rows in blocks of 128.  Its workspace (ws_bytes,
// 256-byte aligned) holds space.control bytes of flags at the front (zero
// before the call and left zero by it) and space.data bytes of partial sums
// at the back.
struct SSSpace {
    size_t control, data;
};
int gemm_ss_np(int64_t M);
SSSpace gemm_ss_space(int64_t M, int64_t N, int64_t K);
cudaError_t launch_gemm_ss(const void* packed, int grid, const uint16_t* scales, const uint16_t* X, int64_t ldx,
                           void* Y, int ydt, int64_t ldy, int64_t M, int64_t N, int64_t K, void* ws,
                           size_t ws_bytes, long long wait_cycles, cudaStream_t st);
unsigned int take_ss_timeouts();

// ---- microscaled 4-bit floats (tb_mx4.cu, tb_mx4_gemm.cu) ----
cudaError_t launch_mx4_quantize(const void* W, int w_dtype, int64_t ldw, int64_t N, int64_t K, void* codes,
                                uint8_t* scales, int32_t* bad, cudaStream_t st);
cudaError_t launch_mx4_dequantize(const void* codes, const uint8_t* scales, int64_t N, int64_t K, void* W,
                                  int w_dtype, int64_t ldw, cudaStream_t st);
// `stall`: test hook, nothing is copied and every wait gives up
cudaError_t launch_mx4_gemm(const void* w, const uint8_t* w_scales, const void* x, const uint8_t* x_scales, void* Y,
                            int ydt, int64_t ldy, int64_t M, int64_t N, int64_t K, long long wait_cycles, bool stall,
                            cudaStream_t st);
unsigned int take_mx_timeouts();

// ---- mixture-of-experts layer (tb_moe_route.cu, tb_moe.cu) ----
constexpr int kMx4 = 4;  // TB_GRID_MX4
constexpr int kMoeMaxTokens = 64, kMoeMaxK = 16, kMoeMaxExperts = 512;
bool moe_route_supported(int E, int64_t H);  // the activations of a token fit in shared memory
cudaError_t launch_moe_route(const uint16_t* x, int64_t ldx, const uint16_t* router, int64_t T, int E, int64_t H, int k,
                             bool renorm, int32_t* ids, float* weights, cudaStream_t st);
struct MoeWeights {
    const void* packed;
    const void* scales;
    int grid;
};
constexpr int kMoeSliceRows = 128;  // of the results, at least: room to split K when pairs are few
// bytes of the gated activations and of the pairs' results (both written before they are read)
size_t moe_data_bytes(int64_t T, int k, int64_t H, int64_t I);
cudaError_t launch_moe(const MoeWeights& gate, const MoeWeights& up, const MoeWeights& down, int E, int64_t H, int64_t I,
                       const uint16_t* x, int64_t ldx, const int32_t* ids, const float* weights, int T, int k, void* y,
                       int ydt, int64_t ldy, void* data, long long wait_cycles, bool stall, cudaStream_t st);
unsigned int take_moe_timeouts();

// bounded device waits that gave up since the last call (clears the count;
// synchronous); 0xFFFFFFFF if the count cannot be read
unsigned int take_wait_timeouts();

}  // namespace tb
