// Host helpers that the expert-layer entry points share: checks of extents, pointers and
// epilogues, and operands that are copied into the workspace (not part of the ABI).
#pragma once

#include <stdint.h>

#include "gemm.h"
#include "internal.h"
#include "ragged.h"
#include "span_check.h"

namespace dg {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int dt_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }
constexpr int64_t kLim = 0x7FFFFFFF;

// The kernels walk extents in 32 bits, by up to 2048 at a time, and round them up to
// whole tiles: an extent this close to 2^31 would wrap.
constexpr int64_t kMaxExtent = kLim - 4095;

inline bool size_ok(int64_t v) { return v >= 0 && v <= kLim; }
inline gemm_status_t extents(int64_t a, int64_t b, int64_t c, int64_t d) {
    if (!size_ok(a) || !size_ok(b) || !size_ok(c) || !size_ok(d)) return GEMM_ERR_INVALID_ARG;
    return a > kMaxExtent || b > kMaxExtent || c > kMaxExtent || d > kMaxExtent
               ? GEMM_ERR_UNSUPPORTED
               : GEMM_OK;
}
// Tiles are dealt in 32 bits, with the grid's size to spare.  The bounds below count the
// smallest tiles there are, so that a call is refused before an operand's copy is
// enqueued, whichever tile the device's size then chooses.
constexpr int64_t kMaxTiles = kLim - 65535;

// Row products, with a last tile for every group that has rows: 128 lanes by 32 columns,
// or 64 lanes by 8 rows in the kernel for few rows (`few`).
inline bool row_tiles_ok(int64_t groups, int64_t T, int64_t N, bool few) {
    const int64_t active = groups < T ? groups : T;
    return cdiv(N, few ? 64 : 128) <= kMaxTiles / (cdiv(T, few ? 8 : 32) + active);
}

inline bool wgrad_tiles_ok(int64_t groups, int64_t M, int64_t N) {
    return cdiv(N, 128) * cdiv(M, 128) <= kMaxTiles / groups;
}

inline bool is16(int dt) { return dt == DT_BF16 || dt == DT_F16; }
inline bool is_dt(int dt) { return is16(dt) || dt == DT_F32; }

// Activation and bias of a gemm_epilogue_t; the row-bias forms have no meaning
// for rows that belong to groups.
inline gemm_status_t epilogue_of(int epi, const float* bias, int64_t stride_bias, int64_t N,
                          int64_t groups, int* act) {
    if (epi < 0 || epi > 15 || ((epi & 8) && !(epi & 1))) return GEMM_ERR_INVALID_ARG;
    if (epi & 8) return GEMM_ERR_UNSUPPORTED;
    if (epi & 1) {
        if (!bias || !aligned(bias, 4) || stride_bias < 0) return GEMM_ERR_INVALID_ARG;
        if (!strided_span_ok(groups, N, stride_bias, 1, 1, 0)) return GEMM_ERR_INVALID_ARG;
    }
    switch ((epi >> 1) & 3) {
        case 1: *act = ACT_GELU_TANH; break;
        case 2: *act = ACT_RELU; break;
        case 3: *act = ACT_GELU_ERF; break;
        default: *act = ACT_NONE;
    }
    return GEMM_OK;
}

// Can TMA address this 16-bit matrix (`depth` of them, `stride` apart)?  Matrices side by
// side, whose stride is less than a row's, are copied: a map's strides ascend.
inline bool in_place(const void* ptr, int64_t ld, int64_t depth, int64_t stride) {
    return aligned(ptr, 16) && ld % 8 == 0 &&
           (depth <= 1 || stride == 0 || (stride % 8 == 0 && stride >= ld));
}

// Workspace bytes of the dense copy of an outer x inner matrix, `depth` times.
inline size_t copy_bytes(int64_t outer, int64_t inner, int64_t depth) {
    return static_cast<size_t>(round_up(depth * outer * round_up(inner, 8) * 2, 256));
}

// Uses the operand in place or copies it into the workspace at *off.
struct Stored {
    const void* ptr;
    int64_t ld, stride;
};
inline gemm_status_t place(Stored* m, int64_t outer, int64_t inner, int64_t depth, char* ws,
                    size_t ws_bytes, size_t* off, bool launch, cudaStream_t stream) {
    if (in_place(m->ptr, m->ld, depth, m->stride)) return GEMM_OK;
    const int64_t n = depth > 1 && m->stride != 0 ? depth : 1;
    const size_t need = copy_bytes(outer, inner, n);
    if (!ws || *off + need > ws_bytes) return GEMM_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return GEMM_ERR_INVALID_ARG;
    const int64_t ld = round_up(inner, 8);
    if (launch && pack16_launch(m->ptr, m->ld, n > 1 ? m->stride : 0, outer, inner, n, ws + *off,
                                ld, stream) != cudaSuccess)
        return GEMM_ERR_CUDA;
    m->ptr = ws + *off;
    m->ld = ld;
    m->stride = n > 1 ? outer * ld : 0;
    *off += need;
    return GEMM_OK;
}

// Do the matrices of a batch stay clear of each other: one after another, or side by side
// (the rows of one between those of the others, as column blocks of one wide matrix)?
inline bool apart(int64_t outer, int64_t inner, int64_t ld, int64_t depth, int64_t stride) {
    return depth <= 1 || stride >= (outer - 1) * ld + inner ||
           (stride >= inner && (ld - inner) / stride >= depth - 1);
}

inline bool c_ok(const void* C, int64_t rows, int64_t cols, int64_t ld, int64_t depth, int64_t stride,
          int dt) {
    return C && aligned(C, dt_bytes(dt)) && ld >= cols &&
           strided_span_ok(rows, cols, ld, 1, depth, stride) && count_ok(depth, rows, cols);
}

}  // namespace dg
