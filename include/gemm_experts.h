/*
 * gemm_experts.h -- operators of an expert layer, next to the dense products
 * of gemm.h and in the same library (libdgemm_gb300.so): tokens sorted by
 * expert and their results added up again, products grouped by
 * expert with ragged row counts, their weight gradient, the orthogonalised
 * update of the weights (Newton-Schulz products), products with 4-bit
 * weights, and products of 8-bit integers.  The conventions of gemm.h hold: device pointers, caller-owned
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
 * gemm_expert_dispatch -- tokens to the rows of their experts.  Token t chose the
 * experts ids[t, 0 .. top-1]; the pairs (t, j) that have an expert get the rows
 * 0, 1, ... in the order of (expert, t, j), so that expert e owns the rows
 * offsets[e] .. offsets[e+1] - 1, as the products below take them:
 *
 *     rows[slots[t, j], :] <- X[t, :]      row_scales[slots[t, j]] <- scales[t]
 *
 *   elem_bytes   1, 2 or 4: size of an element; rows are copied as they are.
 *   T, K         tokens; elements of a row.        X, ldx   T x K, row-major.
 *   scales       T fp32 values that go along, or NULL (row_scales is then not
 *                written).
 *   id_bytes     4 (int32_t) or 8 (int64_t).   ids, ld_ids   T x top, row-major.
 *                A negative id is no expert: the pair gets no row.  An id of
 *                `groups` or more gets none either and is reported:
 *                gemm_check_device_status then returns GEMM_ERR_INVALID_ARG.  An
 *                expert may be chosen twice by a token, which gives two rows.
 *   groups       experts, at most 4096 (more: GEMM_ERR_UNSUPPORTED).
 *   rows, ld_rows, row_scales   room for T * top rows.  Rows past the last
 *                expert's are not written.
 *   offsets      groups + 1 values.      slots   T x top values, dense; -1: no row.
 *   workspace    gemm_expert_dispatch_workspace_size() bytes, 256-byte aligned.
 *
 * No output may overlap an input.  The gradient of X is gemm_expert_combine of the
 * rows' gradient, without weights.
 */
gemm_status_t gemm_expert_dispatch(int elem_bytes, int64_t T, int64_t K, const void* X, int64_t ldx,
                                   const float* scales, int id_bytes, const void* ids,
                                   int64_t ld_ids, int64_t top, int64_t groups, void* rows,
                                   int64_t ld_rows, float* row_scales, int32_t* offsets,
                                   int32_t* slots, void* workspace, size_t workspace_bytes,
                                   gemm_stream_t stream);

size_t gemm_expert_dispatch_workspace_size(int64_t T, int64_t top, int64_t groups);

/*
 * gemm_expert_combine -- the experts' rows added up per token:
 *
 *     Y[t, :] <- sum_j weights[t, j] * rows[slots[t, j], :]
 *
 * in fp32, j ascending, rounded once.  Pairs without a row (a negative slot) add
 * nothing; a token without any gets zeros.  A slot of R or more is reported
 * (GEMM_ERR_INVALID_ARG of gemm_check_device_status) and adds nothing.
 *
 *   dtype        GEMM_DT_BF16, GEMM_DT_F16 or GEMM_DT_F32.
 *   rows, R, ld_rows   R x K, row-major.      slots   T x top, dense; top at most 512
 *                (more: GEMM_ERR_UNSUPPORTED).
 *   weights, w_dtype, ld_weights   T x top, of any of the three types, or NULL: ones.
 *   Y, ldy       T x K, row-major, y_dtype dtype or GEMM_DT_F32; not over an input.
 */
gemm_status_t gemm_expert_combine(gemm_dtype_t dtype, int64_t T, int64_t K, int64_t top,
                                  const void* rows, int64_t R, int64_t ld_rows,
                                  const int32_t* slots, const void* weights,
                                  gemm_dtype_t w_dtype, int64_t ld_weights, void* Y, int64_t ldy,
                                  gemm_dtype_t y_dtype, gemm_stream_t stream);

/*
 * gemm_expert_combine_grad -- the gradient of gemm_expert_combine, in one pass:
 *
 *     d_rows[slots[t, j], :] <- weights[t, j] * DY[t, :]
 *     d_weights[t, j]        <- sum_k DY[t, k] * rows[slots[t, j], k]
 *
 * Rows that no pair names are not written; pairs without a row get a d_weights of
 * zero.  No two pairs may name one row (those of gemm_expert_dispatch do not).
 *
 *   DY, lddy, d_rows, ld_drows   of type dtype; d_rows holds R rows.
 *   rows         of the forward call; read only if d_weights is wanted.
 *   d_weights, dw_dtype, ld_dweights   T x top of any of the three types, summed in
 *                fp32, or NULL: not wanted.
 *   Other arguments as gemm_expert_combine; no output may overlap an input.  Without
 *   weights and d_weights this copies tokens to rows that exist already (a second
 *   tensor's dispatch).
 */
gemm_status_t gemm_expert_combine_grad(gemm_dtype_t dtype, int64_t T, int64_t K, int64_t top,
                                       const void* DY, int64_t lddy, const int32_t* slots,
                                       const void* weights, gemm_dtype_t w_dtype,
                                       int64_t ld_weights, const void* rows, int64_t R,
                                       int64_t ld_rows, void* d_rows, int64_t ld_drows,
                                       void* d_weights, gemm_dtype_t dw_dtype, int64_t ld_dweights,
                                       gemm_stream_t stream);

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

/*
 * gemm_i8_quantize -- rows to 8-bit integers with a scale each:
 *
 *     scales[t] <- max_k |X[t, k]| / 127
 *     Q[t, k]   <- 127 X[t, k] / max_k |X[t, k]|, to the nearest integer, ties to even
 *
 * (-127 .. 127; decided as in exact arithmetic).  A row of zeros gives zeros and the
 * scale 0; a row with an infinity or a NaN gives zeros and a NaN scale, so that what is
 * computed from it is NaN.  Tokens are quantised over their features, weights stored as
 * [N][K] over the inputs of each output channel.
 *
 *   dtype        GEMM_DT_BF16, GEMM_DT_F16 or GEMM_DT_F32.   X, ldx   T x K, row-major.
 *   Q, ldq       T x K, row-major, not over X.      scales   T values.
 */
gemm_status_t gemm_i8_quantize(gemm_dtype_t dtype, int64_t T, int64_t K, const void* X, int64_t ldx,
                               int8_t* Q, int64_t ldq, float* scales, gemm_stream_t stream);

/*
 * gemm_i8 -- products of 8-bit integers with a scale for each token and each output
 * channel:
 *
 *     C[t, n] <- act( (sum_k x[t, k] * Q[e, n, k]) * x_scales[t] * w_scales[e, n]
 *                     + bias[e, n] )
 *
 * The sum is the integer sum, exactly; it is scaled in fp32 (token first) and the result
 * rounded once, so a row's bits do not depend on the other rows, their number or the
 * kernel's form.
 *
 *   x_dtype      GEMM_DT_I8: X holds the integers, x_scales their T scales.
 *                GEMM_DT_BF16, GEMM_DT_F16 or GEMM_DT_F32: X is quantised row by row on
 *                the way, as by gemm_i8_quantize, and x_scales is NULL.
 *   X, ldx       T x K, row-major.      K at most 131071 (more: GEMM_ERR_UNSUPPORTED; an
 *                int32 would not hold every sum).
 *   Q, ldq, stride_q   one N x K row-major matrix per group, stride_q bytes apart (0: the
 *                same for all).  Matrices whose base, ldq and stride_q are multiples of 16
 *                bytes (stride_q at least ldq) are used in place, others copied first.
 *   w_scales, stride_ws   fp32, N values per group, stride_ws elements apart (0: the same).
 *   C, ldc       T x N, row-major, GEMM_DT_BF16, GEMM_DT_F16 or GEMM_DT_F32; not over an
 *                input.
 *   offsets      device group offsets as above, or NULL with groups == 1: one matrix for
 *                all rows.
 *   bias, stride_bias, epi   as gemm_grouped, but ReLU keeps a NaN, so that a token or a
 *                channel with a NaN scale gives NaN through every epilogue.
 *   workspace    gemm_i8_workspace_size() bytes, 256-byte aligned: the tokens' integers as
 *                16-bit operands, and copies of weights that are not used in place.
 */
gemm_status_t gemm_i8(gemm_dtype_t x_dtype, int64_t groups, int64_t T, int64_t N, int64_t K,
                      const void* X, int64_t ldx, const float* x_scales, const int8_t* Q,
                      int64_t ldq, int64_t stride_q, const float* w_scales, int64_t stride_ws,
                      void* C, int64_t ldc, gemm_dtype_t c_dtype, const int32_t* offsets,
                      const float* bias, int64_t stride_bias, gemm_epilogue_t epi, void* workspace,
                      size_t workspace_bytes, gemm_stream_t stream);

size_t gemm_i8_workspace_size(gemm_dtype_t x_dtype, int64_t groups, int64_t T, int64_t N, int64_t K,
                              const int8_t* Q, int64_t ldq, int64_t stride_q);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_GB300_GEMM_EXPERTS_H */
