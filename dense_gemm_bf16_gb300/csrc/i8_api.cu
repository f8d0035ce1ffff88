// Host side of gemm_i8: checks, the operands' preparation, the choice of the kernel's form.
#include <cstring>

#include "experts_host.h"
#include "gemm_experts.h"
#include "i8.h"

namespace dg {
namespace {

// Products of at most 2^14 whose sum an int32 holds.
constexpr int64_t kI8MaxK = (int64_t(1) << 17) - 1;

struct I8Layout {
    int64_t pad;        // row of the tokens' fp16 integers, elements
    int64_t ldq;        // row of a weights' copy, bytes
    size_t x_bytes, s_bytes, q_bytes;
};

bool i8_in_place(const void* Q, int64_t ldq, int64_t groups, int64_t stride_q) {
    return aligned(Q, 16) && ldq % 16 == 0 &&
           (groups <= 1 || stride_q == 0 || (stride_q % 16 == 0 && stride_q >= ldq));
}

I8Layout i8_layout(int x_dtype, int64_t groups, int64_t T, int64_t N, int64_t K, const void* Q,
                   int64_t ldq, int64_t stride_q) {
    I8Layout l{};
    l.pad = round_up(K, 64);
    l.ldq = round_up(K, 16);
    l.x_bytes = static_cast<size_t>(round_up(T * l.pad * 2, 256));
    if (x_dtype != GEMM_DT_I8) l.s_bytes = static_cast<size_t>(round_up(T * 4, 256));
    if (K > 0 && !i8_in_place(Q, ldq, groups, stride_q))
        l.q_bytes = static_cast<size_t>(
            round_up((groups > 1 && stride_q != 0 ? groups : 1) * N * l.ldq, 256));
    return l;
}

gemm_status_t check_i8(int x_dtype, int64_t groups, int64_t T, int64_t N, int64_t K, const void* Q,
                       int64_t ldq, int64_t stride_q) {
    if (x_dtype != GEMM_DT_I8 && !is_dt(x_dtype)) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = extents(groups, T, N, K);
    if (st != GEMM_OK) return st;
    if (K > kI8MaxK) return GEMM_ERR_UNSUPPORTED;
    if (groups == 0 || T == 0 || N == 0 || K == 0) return GEMM_OK;
    if (!Q || ldq < K || stride_q < 0 || !strided_span_ok(N, K, ldq, 1, groups, stride_q) ||
        !count_ok(groups, N, K + 16) || !count_ok(1, T, K + 64))
        return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

// CTAs per tile and columns of a tile: the widest tile whose tiles fill the GPU, pairs
// where theirs fill at least half of it.
void i8_variant(const RgProblem& q, const DeviceInfo& d, int* cg, int* bt) {
    const int64_t cols = q.offsets ? cdiv(q.T, q.groups) : q.T;
    auto tiles = [&](int64_t lanes, int64_t w) {
        return cdiv(q.n_lane, lanes) * (q.offsets ? q.groups : 1) * cdiv(cols, w);
    };
    *cg = 1;
    if (cols > 128 && q.n_lane > 128 && d.max_pairs > 0 && tiles(256, kI8PairCols) >= d.max_pairs / 2) {
        *cg = 2, *bt = kI8PairCols;
        return;
    }
    *bt = cols <= 32 ? 32 : (cols <= 64 ? 64 : 128);
    while (*bt > 32 && tiles(128, *bt) * 2 <= d.sm_count) *bt /= 2;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

size_t gemm_i8_workspace_size(gemm_dtype_t x_dtype, int64_t groups, int64_t T, int64_t N, int64_t K,
                              const int8_t* Q, int64_t ldq, int64_t stride_q) {
    if (check_i8(x_dtype, groups, T, N, K, Q, ldq, stride_q) != GEMM_OK) return 0;
    if (groups == 0 || T == 0 || N == 0) return 0;
    const I8Layout l = i8_layout(x_dtype, groups, T, N, K, Q, ldq, stride_q);
    return l.x_bytes + l.s_bytes + l.q_bytes;
}

gemm_status_t gemm_i8(gemm_dtype_t x_dtype, int64_t groups, int64_t T, int64_t N, int64_t K,
                      const void* X, int64_t ldx, const float* x_scales, const int8_t* Q,
                      int64_t ldq, int64_t stride_q, const float* w_scales, int64_t stride_ws,
                      void* C, int64_t ldc, gemm_dtype_t c_dtype, const int32_t* offsets,
                      const float* bias, int64_t stride_bias, gemm_epilogue_t epi, void* workspace,
                      size_t workspace_bytes, gemm_stream_t stream) {
    gemm_status_t st = check_i8(x_dtype, groups, T, N, K, Q, ldq, stride_q);
    if (st != GEMM_OK) return st;
    if (!is_dt(c_dtype)) return GEMM_ERR_INVALID_ARG;
    int act = ACT_NONE;
    st = epilogue_of(epi, bias, stride_bias, N, groups, &act);
    if (st != GEMM_OK) return st;
    if (groups == 0 || T == 0 || N == 0) return GEMM_OK;
    if (offsets ? !aligned(offsets, 4) : groups != 1) return GEMM_ERR_INVALID_ARG;
    const bool given = x_dtype == GEMM_DT_I8;
    if (given != (x_scales != nullptr) || !aligned(x_scales, 4)) return GEMM_ERR_INVALID_ARG;
    if (!w_scales || !aligned(w_scales, 4) || stride_ws < 0 ||
        !strided_span_ok(groups, N, stride_ws, 1, 1, 0))
        return GEMM_ERR_INVALID_ARG;
    if (!c_ok(C, T, N, ldc, 1, 0, c_dtype)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!X || !aligned(X, given ? 1 : dt_bytes(x_dtype)) || ldx < K ||
                  !strided_span_ok(T, K, ldx, 1, 1, 0)))
        return GEMM_ERR_INVALID_ARG;
    if (!row_tiles_ok(groups, T, N, false)) return GEMM_ERR_UNSUPPORTED;
    if (groups == 1) stride_q = 0;
    const I8Layout l = i8_layout(x_dtype, groups, T, N, K, Q, ldq, stride_q);
    const size_t need = l.x_bytes + l.s_bytes + l.q_bytes;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo d;
    st = device_info(&d);
    if (st != GEMM_OK) return st;
    if (!d.i8) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    float* made = reinterpret_cast<float*>(ws + l.x_bytes);

    RgProblem q{};
    q.form = RG_ROWS;
    q.dt = DT_F16;
    q.groups = groups;
    q.T = T;
    q.n_lane = N;
    q.n_col = T;
    q.K = K;
    q.offsets = offsets;
    q.a8 = true;
    q.a = RgOperand{Q, ldq, groups > 1 ? stride_q : 0, false, N, K};
    if (l.q_bytes > 0) {
        q.a.ptr = ws + l.x_bytes + l.s_bytes;
        q.a.ld = l.ldq;
        q.a.stride = q.a.stride != 0 ? N * l.ldq : 0;
    }
    q.b = RgOperand{ws, l.pad, 0, false, T, l.pad};
    q.C = C;
    q.ldc = ldc;
    q.c_dtype = q.cin_dtype = c_dtype;
    q.alpha = 1.0f;
    q.bias = (epi & 1) ? bias : nullptr;
    q.stride_bias = stride_bias;
    q.act = act;
    // (the product starts where the tokens' pass leaves an SM free, a CTA of it fits beside no
    // block of the pass, and reads offsets and weights before it waits for the pass: weights must
    // not be copied in front of it, and there must be a pass)
    q.pdl = l.q_bytes == 0 && K > 0;
    int cg, bt;
    i8_variant(q, d, &cg, &bt);
    I8Params p;
    std::memset(&p, 0, sizeof(p));
    int64_t tiles = 0;
    st = rg_fill(q, d, cg, bt, &p.g, &tiles);
    if (st != GEMM_OK) return st;
    p.x_scales = given ? x_scales : made;
    p.w_scales = w_scales;
    p.stride_ws = groups > 1 ? stride_ws : 0;
    // CTAs of a cluster share a tile where all tiles there may be leave half of the SMs
    // idle, each with two 256-deep stages at least
    p.splits = 1;
    if (cg == 1 && bt == 32)
        while (p.splits < 4 && tiles * p.splits * 2 <= d.sm_count && cdiv(K, 256) >= p.splits * 4)
            p.splits *= 2;
    int64_t grid = cg == 2 ? d.max_pairs : d.sm_count;
    if (tiles < grid) grid = tiles;
    cudaError_t e = cudaSuccess;
    if (l.q_bytes > 0)
        e = i8_pack(Q, ldq, groups > 1 ? stride_q : 0, N, K, q.a.stride != 0 ? groups : 1,
                    ws + l.x_bytes + l.s_bytes, l.ldq, d.sm_count, s);
    if (e == cudaSuccess && !given)
        e = i8_widen_quantized(x_dtype, X, ldx, T, K, l.pad, ws, made, d.sm_count, s);
    if (e == cudaSuccess && given && K > 0) e = i8_widen(X, ldx, T, K, l.pad, ws, d.sm_count, s);
    if (e == cudaSuccess)
        e = i8_launch(cg, bt, p, static_cast<int>(grid * (cg == 2 ? 2 : p.splits)), s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

}  // extern "C"
