/*
 * gemm_experts.h -- operators of an expert layer, next to the dense products
 * of gemm.h and in the same library (libdgemm_gb300.so): products grouped by
 * expert with ragged row counts, their weight gradient, the orthogonalised
 * update of the weights (Newton-Schulz products), and products with 4-bit
 * weights.  The conventions of gemm.h hold: device pointers, caller-owned
 * buffers and workspaces, work enqueued on `stream`, argument errors by return
 * code before anything is enqueued, no allocation.  An extent above 2^31 - 4096
 * is GEMM_ERR_UNSUPPORTED: the kernels walk extents in 32 bits, tile by tile.
 *
 * Group offsets.  `offsets` is a device array of groups + 1 ascending int32
 * values: group e owns the rows offsets[e] .. offsets[e+1] - 1 of the row
 * operands (none when they are equal).  Rows that belong to no group are
 * neither read as results nor written.  The offsets are read by the kernels,
 * never by the host, so a call needs no synchronisation with whatever computes
 * them.  Offsets that descend or leave [0, T] are reported:
 * gemm_check_device_status then returns GEMM_ERR_INVALID_ARG, and the groups
 * from the first such one on (gemm_grouped_wgrad: that group) count as empty.
 */
#ifndef DGEMM_GB300_GEMM_EXPERTS_H
#define DGEMM_GB300_GEMM_EXPERTS_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gemm_grouped -- for every group e and every row t of it,
 *
 *     C[t, :] <- act( alpha * A[t, :] @ B[e] + beta * C[t, :] + bias[e, :] )
 *
 *   ab_dtype     GEMM_DT_BF16 or GEMM_DT_F16 (GEMM_DT_F32: GEMM_ERR_UNSUPPORTED).
 *   groups, T    number of groups; rows of A and C.
 *   A, lda       T x K, row-major.
 *   B, ldb, lb, stride_b   one K x N matrix per group, stride_b elements apart
 *                (0: the same matrix for all), row- or column-major: one after
 *                another, or side by side (column blocks of one wide matrix:
 *                ldb >= (groups - 1) * stride_b + a row), which are copied.  The
 *                gradient of A is the same call with the other layout of B.
 *   C, ldc       T x N, row-major, c_dtype ab_dtype or GEMM_DT_F32.
 *   bias, stride_bias  fp32, N values per group, stride_bias elements apart
 *                (0: the same for all); required iff epi uses a bias.  The
 *                row-bias epilogues are GEMM_ERR_UNSUPPORTED.
 *   workspace    256-byte aligned; needed only for an A or B that TMA cannot
 *                address (a base, leading dimension or group stride that is not
 *                a multiple of 16 bytes, or matrices side by side), which is
 *                copied first.
 *                gemm_grouped_workspace_size() always suffices.
 *
 * Products accumulate in fp32 (an fp32 C: at most 768 in the tensor core's
 * accumulator, which cuts off towards zero, then added to nearest) and are rounded
 * once.  Calls repeat bit for bit.
 * T, groups, N and the operands' layout choose the kernel and its tiles, and with
 * them the order of a row's sum; where they are equal, a group's results do not
 * depend on the other groups' rows, weights or sizes, bit for bit.  (One more row,
 * of any group, may change the last bits of all.)
 */
gemm_status_t gemm_grouped(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t N, int64_t K,
                           const void* A, int64_t lda,
                           const void* B, int64_t ldb, gemm_layout_t lb, int64_t stride_b,
                           void* C, int64_t ldc, gemm_dtype_t c_dtype, const int32_t* offsets,
                           float alpha, float beta, const float* bias, int64_t stride_bias,
                           gemm_epilogue_t epi, void* workspace, size_t workspace_bytes,
                           gemm_stream_t stream);

/* Bytes of workspace that suffice for gemm_grouped with these arguments (0 when
 * both operands are used in place, or for invalid arguments). */
size_t gemm_grouped_workspace_size(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t N,
                                   int64_t K, const void* A, int64_t lda, const void* B,
                                   int64_t ldb, gemm_layout_t lb, int64_t stride_b);

/*
 * gemm_grouped_wgrad -- the weights' gradient of gemm_grouped: for every group e
 *
 *     C[e] <- alpha * A_e^T @ D_e + beta * C[e]
 *
 * with A_e (D_e) the rows of group e of A (D).  A group without rows gives
 * beta * C[e] (zeros when beta == 0).  Rows of other groups never enter a sum,
 * whatever they hold (NaN and infinities included).
 *
 *   A, lda       T x M, row-major.     D, ldd   T x N, row-major.
 *   C, ldc, stride_c   one M x N row-major matrix per group, c_dtype ab_dtype
 *                or GEMM_DT_F32; stride_c must keep them apart (one after
 *                another, or side by side as B of gemm_grouped).
 *   Other arguments as gemm_grouped.
 */
gemm_status_t gemm_grouped_wgrad(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t M,
                                 int64_t N, const void* A, int64_t lda, const void* D, int64_t ldd,
                                 void* C, int64_t ldc, int64_t stride_c, gemm_dtype_t c_dtype,
                                 const int32_t* offsets, float alpha, float beta, void* workspace,
                                 size_t workspace_bytes, gemm_stream_t stream);

size_t gemm_grouped_wgrad_workspace_size(gemm_dtype_t ab_dtype, int64_t groups, int64_t T,
                                         int64_t M, int64_t N, const void* A, int64_t lda,
                                         const void* D, int64_t ldd);

/*
 * gemm_newton_schulz -- the orthogonalised form of every matrix of a batch, by
 * `steps` odd quintic steps:
 *
 *     X <- G / (||G||_F + eps)
 *     steps times:  S = X X^T;  X <- a X + (b S + c S S) X
 *     O <- X
 *
 * (with X^T X in place of X X^T, on the right, when M > N: the same values).
 * a = 3.4445, b = -4.7750, c = 2.0315 and 5 steps bring singular values of
 * 1e-2 and more into about [0.7, 1.2].
 *
 *   batch, M, N  matrices M x N, row-major with leading dimensions ldg, ldo
 *                and batch strides stride_g, stride_o (elements).
 *   g_dtype      GEMM_DT_F32, GEMM_DT_BF16 or GEMM_DT_F16.
 *   o_dtype      GEMM_DT_BF16 or GEMM_DT_F16 (GEMM_DT_F32: GEMM_ERR_UNSUPPORTED,
 *                the products round their operands to 16 bits).  O may be G.
 *   steps        1 to 64.     eps   >= 0 (0 gives NaN for a zero matrix).
 *   workspace    gemm_newton_schulz_workspace_size() bytes, 256-byte aligned.
 *
 * The norm and every product accumulate in fp32.  Between products X and the
 * symmetric matrices S + b / (2 c) and a + b S + c S S are held in fp16 times a
 * power of two (eight times finer than bf16), with what the first one's diagonal
 * loses carried on in fp32; coefficients must keep singular
 * values below 4 and both matrices below 8 in norm, which the values above do.
 * Both symmetric products compute the tiles on and below the diagonal only.
 */
gemm_status_t gemm_newton_schulz(gemm_dtype_t g_dtype, int64_t batch, int64_t M, int64_t N,
                                 const void* G, int64_t ldg, int64_t stride_g,
                                 void* O, int64_t ldo, int64_t stride_o, gemm_dtype_t o_dtype,
                                 int steps, float a, float b, float c, float eps,
                                 void* workspace, size_t workspace_bytes, gemm_stream_t stream);

size_t gemm_newton_schulz_workspace_size(int64_t batch, int64_t M, int64_t N);

/*
 * gemm_w4 -- products with 4-bit weights that carry one scale (and optionally
 * one zero point) per `group` neighbours along K:
 *
 *     C[t, n] <- act( sum_k A[t, k] * (q[e, n, k] - z[e, n, k/group]) * s[e, n, k/group]
 *                     + bias[e, n] )
 *
 *   ab_dtype     GEMM_DT_BF16 or GEMM_DT_F16: type of A and of the scales.
 *   A, lda       T x K, row-major.
 *   Q            [groups][N][K / 2] bytes, dense, 16-byte aligned: byte k/2 of a
 *                row holds q[k] in its low half for even k, in its high half
 *                for odd k.
 *   scales       [groups][N][K / group], dense, type ab_dtype.
 *   zeros        [groups][N][K / group] bytes with values 0..15, or NULL: 8.
 *   group        32, 64 or 128; K must be a multiple of it.
 *   C, ldc       T x N, row-major, c_dtype ab_dtype or GEMM_DT_F32.
 *   offsets      device group offsets as above, or NULL with groups == 1: one
 *                matrix for all rows.
 *   bias, epi    as gemm_grouped.
 *   workspace    gemm_w4_workspace_size() bytes, 256-byte aligned.
 *
 * Few rows (a 16-bit C with T <= 64, or T <= 40 * groups for several groups, or
 * any fp32 C) multiply the 4-bit integers themselves and scale fp32 sums once
 * per group, so nothing is rounded before the output.  More rows with a 16-bit
 * C multiply weights that were rounded to ab_dtype in the workspace, unless
 * GEMM_OPT_W4_EXACT is set.  A row's last bits may so depend on how many rows the
 * call has.
 */
gemm_status_t gemm_w4(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t N, int64_t K,
                      const void* A, int64_t lda, const uint8_t* Q, const void* scales,
                      const uint8_t* zeros, int group, void* C, int64_t ldc, gemm_dtype_t c_dtype,
                      const int32_t* offsets, const float* bias, int64_t stride_bias,
                      gemm_epilogue_t epi, void* workspace, size_t workspace_bytes,
                      gemm_stream_t stream);

size_t gemm_w4_workspace_size(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t N,
                              int64_t K, const void* A, int64_t lda, gemm_dtype_t c_dtype);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_GB300_GEMM_EXPERTS_H */
