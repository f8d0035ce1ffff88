// Declarations of the 8-bit product's kernel and of the passes that prepare its operands
// (not part of the ABI).
#pragma once

#include "ragged.h"

namespace dg {

// Tiles, maps and the output are those of a row product (RgParams); its lane operand is
// the int8 weights, its column operand the tokens' integers as fp16.
struct I8Params {
    RgParams g;
    const float* x_scales;   // [T]
    const float* w_scales;   // [groups][n_lane], stride_ws apart
    int64_t stride_ws;
    int32_t splits;          // CTAs of a cluster that share a tile's contraction
};
constexpr int kI8PairCols = 192;  // columns of a pair's tile at most
// CTAs per tile (1, or 2 with cta_group::2 MMAs) and columns of a tile at most.
cudaError_t i8_launch(int cg, int bt, const I8Params& p, int grid, cudaStream_t stream);
cudaError_t i8_prepare();  // kernel attributes (once per device)

// Tokens as fp16 integers in rows of `pad` (a multiple of 64, zeros past K): quantised row
// by row, or from int8.  sms: CTAs of a wave.
cudaError_t i8_widen_quantized(int dt, const void* x, int64_t ld, int64_t T, int64_t K, int64_t pad,
                               void* out, float* scales, int sms, cudaStream_t stream);
cudaError_t i8_widen(const void* x, int64_t ld, int64_t T, int64_t K, int64_t pad, void* out, int sms,
                     cudaStream_t stream);
// A copy of int8 matrices with rows of ld_dst bytes, one after another.
cudaError_t i8_pack(const void* src, int64_t ld, int64_t stride, int64_t rows, int64_t cols,
                    int64_t depth, void* dst, int64_t ld_dst, int sms, cudaStream_t stream);

}  // namespace dg
