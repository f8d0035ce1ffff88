// Declarations of the ragged-product kernel (grouped products, their weight
// gradient, the symmetric products of the orthogonalised update) and of the
// host helpers that the expert-layer entry points share (not part of the ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gemm.h"
#include "internal.h"

namespace dg {

// What a tile of the ragged kernel is (see ragged_kernel.cuh).
enum : int { RG_ROWS = 0, RG_WGRAD = 1, RG_SYM = 2 };
constexpr int RG_BAND = 8;  // column tiles of a band (see rg_band)

// n / d for 0 <= n < 2^31 as one multiplication (d fixed at the launch).
struct RgDiv {
    uint32_t m, s;
};

// Output D[col][lane]: the lane operand's rows are the output's contiguous
// dimension, the column operand's rows its rows.
struct RgParams {
    CUtensorMap tmap_a;      // lane operand, (inner, outer, z: group or 0)
    CUtensorMap tmap_b;      // column operand, whole-tile boxes
    CUtensorMap tmap_b32;    // column operand, K-major: (K, rows, z), boxes of 64 x 32;
                             // RG_WGRAD: boxes of 64 x 16 rows of the contraction
    CUtensorMap tmap_a16;    // RG_WGRAD: the lane operand's
    CUtensorMap tmap_c;      // RG_WGRAD: output, where c_tma
    const int32_t* offsets;  // [groups + 1] on the device, or null: equal groups
    int32_t groups;
    int32_t rows;            // T: rows that the offsets index (RG_ROWS, RG_WGRAD)
    int32_t n_lane;          // output columns
    int32_t n_col;           // output rows of a group where all groups have as many
    int32_t K;               // contraction extent (RG_ROWS, RG_SYM)
    int32_t lane_tiles;      // ceil(n_lane / lanes of a tile)
    int32_t col_tile;        // columns of a tile at most (a multiple of 32)
    int32_t total_tiles;     // equal groups and RG_WGRAD; else 0 (found on the device)
    int32_t per_group;       // ... of one group
    int32_t chunks;          // ... column tiles of one group
    RgDiv div_group;         // by per_group
    RgDiv div_band;          // by RG_BAND * lane_tiles
    int32_t a_mn, b_mn;      // 1: operand stored with its rows contiguous (MN-major)
    int32_t a_k4, b_k4;      // 1: K-major map is (64 K, rows, K blocks, z): two blocks a load
    int32_t a_z, b_z;        // 1: the operand's z coordinate is the group
    int32_t maps;            // 1: the tensor maps are set (some contraction is not empty)
    uint32_t idesc;          // instruction descriptor without its N field
    void* C;                 // output
    const void* Cin;         // beta's input, same type and shape as C
    int64_t ldc, stride_c, ldcin, stride_cin;
    int32_t c_dtype, cin_dtype;  // types of one size
    int32_t c_tma;           // RG_WGRAD: C leaves by TMA (its base and strides allow)
    int32_t c_vec;           // C (and Cin) rows start on 16-byte boundaries
    float alpha, beta;
    float diag;              // RG_SYM: added on the diagonal
    // RG_SYM, where set: n_col floats a group, stride_resid apart.  resid_in 0: what the
    // diagonal lost by its rounding, times twice the rounded value, goes there; 1: alpha
    // times that is added on the diagonal.
    float* resid;
    int64_t stride_resid;
    int32_t resid_in;
    const float* bias;       // [groups][n_lane] with stride_bias, or null
    int64_t stride_bias;
    int32_t act;
    int32_t test_stall;      // test only: leave one stage unfilled
    // 1: launched as the programmatic dependent of the kernel that prepares an operand
    // (a copy, or weights made from 4-bit ones): set up while it runs, then wait for it
    int32_t pdl;
    int* status;
    uint64_t timeout_ns;
#if DG_DEBUG
    int64_t dbg_c_elems;     // elements of C from C that the call may touch
#endif
};

// Kernel variants: CTAs per tile (1, or 2 with cta_group::2 MMAs) and columns
// of a tile at most; lanes are 128 per CTA.
cudaError_t rg_launch_rows(int cg, int bt, const RgParams& p, int grid, cudaStream_t stream);
cudaError_t rg_launch_wgrad(int cg, int bt, const RgParams& p, int grid, cudaStream_t stream);
cudaError_t rg_prepare_rows();   // kernel attributes (once per device)
cudaError_t rg_prepare_wgrad();

// A sequence of products in one cooperative launch, each waiting for the one before
// matrix by matrix: `steps` times the three products of a Newton-Schulz step.  ph[0..2]
// serve even steps, ph[3..5] odd ones (the state alternates between two buffers),
// ph[6] is the last step's third product.
struct RgSeq {
    RgParams ph[7];
    int32_t steps;
    unsigned int* arrived;   // a word per matrix, zero at the start: epilogue warps that
                             // finished a tile of it
};
cudaError_t rg_launch_seq(int cg, int bt, const RgSeq& q, int grid, cudaStream_t stream);
cudaError_t rg_prepare_seq();

// ---- host helpers (gemm_api.cu)
struct DeviceInfo {
    int sm_count;      // CTAs a launch may have: one per SM, or the cap of GEMM_OPT_MAX_CTAS
    int max_pairs;     // two-CTA clusters resident at once, under the cap (0: none)
    int* status;       // device error word
    bool i8;           // gemm_i8's kernels are ready
};
gemm_status_t device_info(DeviceInfo* out);   // the current device
uint64_t option_timeout_ns();
bool option_w4_exact();       // no 16-bit weights
bool option_overlap_copy();   // a product may start while its operand is prepared
int take_test_stall();

// Three-dimensional tensor map of 16-bit elements (inner, outer, depth), 128-byte
// swizzled; strides in bytes.  False on failure.
bool encode_map16(CUtensorMap* map, int dt, const void* ptr, int64_t inner, int64_t outer,
                  int64_t depth, int64_t outer_stride, int64_t depth_stride, uint32_t box_inner,
                  uint32_t box_outer);
// Output of 32-column boxes: 32 rows of 64 bytes, swizzled by 64 bytes, or 16 rows of
// fp32.
bool encode_map_out(CUtensorMap* map, int dt, const void* ptr, int64_t cols, int64_t rows,
                    int64_t depth, int64_t row_stride, int64_t depth_stride);
// K-major matrix with a whole number of 64-wide K blocks as (64, rows, K blocks,
// depth), in boxes of 64 x box_rows x 2 blocks.
bool encode_map16_k4(CUtensorMap* map, int dt, const void* ptr, int64_t k, int64_t rows,
                     int64_t depth, int64_t row_stride, int64_t depth_stride, uint32_t box_rows);
// Bytes in 128-byte blocks: (128, rows, blocks, depth) in boxes of `box_blocks`
// blocks, or (bytes, rows, depth) with box_blocks == 0.
bool encode_map8(CUtensorMap* map, const void* ptr, int64_t inner, int64_t rows, int64_t depth,
                 uint32_t box_rows, uint32_t box_blocks);
// int8 matrices in boxes of 128 bytes x box_rows; ld and stride in bytes.
bool encode_map8_rows(CUtensorMap* map, const void* ptr, int64_t inner, int64_t rows, int64_t depth,
                      int64_t ld, int64_t stride, uint32_t box_rows);
// 16-bit rows in 64-wide blocks: (64, rows, blocks) in boxes of `box_blocks` blocks.
bool encode_map16_blocks(CUtensorMap* map, int dt, const void* ptr, int64_t k, int64_t rows,
                         int64_t row_stride, uint32_t box_rows, uint32_t box_blocks);

// One ragged product, from checked arguments (experts_api.cu): the lane
// operand `a` and the column operand `b` as stored matrices.
struct RgOperand {
    const void* ptr;
    int64_t ld;        // elements, a multiple of 8
    int64_t stride;    // elements between groups (0: one matrix)
    bool mn;           // stored with its rows contiguous
    int64_t rows;      // rows in its role (lanes or columns)
    int64_t k;         // contraction extent as stored
};
struct RgProblem {
    int form;
    int dt;            // DT_BF16 or DT_F16 operands
    int64_t groups, T, n_lane, n_col, K;
    const int32_t* offsets;
    RgOperand a, b;
    void* C;
    const void* Cin;
    int64_t ldc, stride_c, ldcin, stride_cin;
    int c_dtype, cin_dtype;  // cin_dtype: read where beta != 0, of c_dtype's size
    float alpha, beta;
    float diag;              // RG_SYM: added on the diagonal
    float* resid;            // RG_SYM: see RgParams
    int64_t stride_resid;
    int resid_in;
    const float* bias;
    int64_t stride_bias;
    int act;
    bool pdl;          // the kernel enqueued just before prepares an operand
    bool a8;           // the lane operand is int8, K-major, ld and stride in bytes
};
// The kernel variant a problem takes (CTAs per tile, columns), its parameters, and
// a bound on its tiles.
void rg_variant(const RgProblem& q, const DeviceInfo& d, int* cg, int* bt);
gemm_status_t rg_fill(const RgProblem& q, const DeviceInfo& d, int cg, int bt, RgParams* p,
                      int64_t* tiles);
gemm_status_t rg_run(const RgProblem& q, const DeviceInfo& d, cudaStream_t stream);

// ---- few rows: 4-bit weights, and 16-bit ones for decoding steps (w4.cu)
struct W4Params {
    CUtensorMap tmap_q;      // [groups][N][K / 2] bytes, boxes of 128 bytes x rows (x blocks);
                             // 16-bit weights: 64 x rows x 2 blocks, or 64 columns x 128 k
    CUtensorMap tmap_x;      // [T][K], boxes of 64 x the tokens of a tile (x blocks)
    const void* scales;
    const uint8_t* zeros;
    const int32_t* offsets;  // or null
    int32_t groups, T, N, K;
    int32_t group;           // weights per scale; 0: 16-bit weights
    int32_t w_mn;            // 16-bit weights: 1: stored with N contiguous
    int32_t w_z;             // 16-bit weights: 1: the map's z coordinate is the group
    int32_t vec;             // 1: scales and zeros of a stage load as vectors
    int32_t q4, x4;          // 1: the map has blocks as a dimension, a stage is one load
    int32_t n_tiles, splits; // row tiles; CTAs (K slices) of a cluster
    int32_t grid;            // clusters
    void* C;
    int64_t ldc;
    int32_t c_dtype;
    float alpha, beta;
    const float* bias;
    int64_t stride_bias;
    int32_t act;
    int32_t test_stall;      // test only: leave one stage unfilled
    int* status;
    uint64_t timeout_ns;
#if DG_DEBUG
    int64_t dbg_c_elems;
#endif
};
// Shape of the kernel for `tokens` token columns and a scale per `group` weights (0: 16-bit
// weights): weight rows of a unit, and weights of a row per stage.
struct W4Shape {
    int rows, step;
};
W4Shape w4_shape(int tokens, int group);
cudaError_t w4_launch(int dt, int tokens, const W4Params& p, cudaStream_t stream);
cudaError_t w4_prepare();
// Dense [groups][N][K] weights of type dt: (q - z) * s, rounded once.
cudaError_t w4_dequantise(int dt, const uint8_t* q, const void* scales, const uint8_t* zeros,
                          int64_t rows, int64_t K, int group, void* out, cudaStream_t stream);

// ---- element-wise passes of the orthogonalised update (newton_schulz.cu)
struct NsParams {
    const void* G;
    int64_t ldg, stride_g;
    int32_t g_dtype, g_vec;
    int64_t batch;
    int32_t M, N;
    int32_t parts;           // blocks per matrix
    float* partials;         // [batch][parts][3]
    void* X;                 // fp16, [batch][M][ldx]
    int64_t ldx;
    float eps, scale;
    unsigned int* arrived;   // [batch], zeroed for the sequence that follows
};
cudaError_t ns_norm_launch(const NsParams& p, cudaStream_t stream);
cudaError_t ns_scale_launch(const NsParams& p, cudaStream_t stream);

}  // namespace dg
