// Host side of include/gemm_experts.h: argument validation, planning, operand
// copies, tensor maps and launches.  No device memory is allocated here.
#include <stdint.h>

#include <cmath>
#include <cstring>
#include <new>

#include "experts_host.h"
#include "gemm_experts.h"
#include "internal.h"
#include "ptx.cuh"
#include "ragged.h"

namespace dg {

// ---------------------------------------------------------------- the ragged kernel's launches

// With l = ceil(log2 d) and m = floor(2^(31 + l) / d) + 1, n m / 2^(31 + l) exceeds
// n / d by less than n / 2^(31 + l) < 1 / d, so its integer part is n / d.
static RgDiv make_div(int64_t d) {
    if (d < 1) d = 1;
    uint32_t l = 0;
    while ((int64_t(1) << l) < d) ++l;
    if (l == 0) return RgDiv{0u, 0u};  // (division by 1)
    const uint64_t m = (uint64_t(1) << (31 + l)) / static_cast<uint64_t>(d) + 1;
    return RgDiv{static_cast<uint32_t>(m), l - 1};
}

// Lanes (128 per CTA) and columns of a tile: CTA pairs with 256 x 256 tiles where
// they fill at least half of the GPU, narrower single-CTA tiles for few rows.
void rg_variant(const RgProblem& q, const DeviceInfo& d, int* cg, int* bt) {
    const int64_t cols = q.form == RG_ROWS && q.offsets ? cdiv(q.T, q.groups) : q.n_col;
    *cg = 2;
    *bt = 256;
    if (q.form == RG_ROWS && cols <= 32) {
        *cg = 1, *bt = 32;
    } else if (cols <= 128 || q.n_lane <= 128) {
        *cg = 1, *bt = 128;
    } else {
        const int64_t tiles = q.groups * cdiv(q.n_lane, 256) *
                              (q.form == RG_SYM ? (cdiv(cols, 256) + 1) / 2 : cdiv(cols, 256));
        if (d.max_pairs == 0 || tiles < d.max_pairs / 2) *cg = 1, *bt = 128;
    }
}

gemm_status_t rg_fill(const RgProblem& q, const DeviceInfo& d, int cg, int bt, RgParams* out,
                      int64_t* tiles) {
    RgParams& p = *out;
    std::memset(&p, 0, sizeof(p));
    const int64_t lanes = 128 * cg;
    const int64_t lane_tiles = cdiv(q.n_lane, lanes);
    p.col_tile = bt;
    int64_t total = 0, bound = 0;
    if (q.form == RG_ROWS && q.offsets) {
        bound = lane_tiles * (cdiv(q.T, bt) + (q.groups < q.T ? q.groups : q.T));
    } else if (q.form == RG_SYM) {
        const int64_t cols = cdiv(q.n_col, bt), whole = lanes / bt * lane_tiles;
        total = bound = q.groups * (lanes / bt * (lane_tiles * (lane_tiles - 1) / 2) +
                                    (cols < whole ? cols : whole));
    } else {
        if (q.form == RG_ROWS) {
            // equal groups: the tile width (a multiple of 32) whose waves over the
            // GPU take the fewest columns, a tile's own cost counted as 24 more
            const int64_t P = cg == 2 ? d.max_pairs : d.sm_count;
            const int64_t n0 = cdiv(q.n_col, bt);
            int64_t best = INT64_MAX;
            for (int64_t n = n0; n <= 2 * n0; ++n) {
                const int64_t w = round_up(cdiv(q.n_col, n), 32);
                const int64_t cost = cdiv(q.groups * lane_tiles * cdiv(q.n_col, w), P) * (w + 24);
                if (cost < best) {
                    best = cost;
                    p.col_tile = static_cast<int32_t>(w);
                }
            }
        }
        total = bound = q.groups * lane_tiles * cdiv(q.n_col, p.col_tile);
    }
    // (the triangle's index arithmetic takes up to 32767 tile rows; the sequence of
    // products fills its parameters before it enqueues anything)
    if (bound > kMaxTiles || (q.form == RG_SYM && lane_tiles > 32767)) return GEMM_ERR_UNSUPPORTED;
    *tiles = bound;
    p.total_tiles = static_cast<int32_t>(total);
    p.per_group = static_cast<int32_t>(q.groups > 0 ? total / q.groups : 0);
    p.chunks = static_cast<int32_t>(lane_tiles > 0 ? p.per_group / lane_tiles : 0);
    p.div_group = make_div(p.per_group);
    p.div_band = make_div(RG_BAND * lane_tiles);
    p.offsets = q.offsets;
    p.groups = static_cast<int32_t>(q.groups);
    p.rows = static_cast<int32_t>(q.T);
    p.n_lane = static_cast<int32_t>(q.n_lane);
    p.n_col = static_cast<int32_t>(q.n_col);
    p.K = static_cast<int32_t>(q.K);
    p.lane_tiles = static_cast<int32_t>(lane_tiles);
    p.a_mn = q.a.mn;
    p.b_mn = q.b.mn;
    const int64_t az = q.a.stride != 0 ? q.groups : 1, bz = q.b.stride != 0 ? q.groups : 1;
    p.a_z = az > 1;
    p.b_z = bz > 1;
    p.maps = q.form == RG_WGRAD ? q.T > 0 : q.K > 0;
    if (p.maps) {
        // MN-major boxes bring two 64-deep K blocks; K-major ones too where K is a
        // whole number of blocks, else one block each
        p.a_k4 = !q.a.mn && q.a.k % 64 == 0;
        p.b_k4 = !q.b.mn && q.b.k % 64 == 0;
        auto k_major = [&](CUtensorMap* map, const RgOperand& o, int64_t z, bool k4, int rows) {
            return k4 ? encode_map16_k4(map, q.dt, o.ptr, o.k, o.rows, z, o.ld * 2, o.stride * 2, rows)
                      : encode_map16(map, q.dt, o.ptr, o.k, o.rows, z, o.ld * 2, o.stride * 2, 64,
                                     rows);
        };
        auto mn_major = [&](CUtensorMap* map, const RgOperand& o, int64_t z) {
            return encode_map16(map, q.dt, o.ptr, o.rows, o.k, z, o.ld * 2, o.stride * 2, 64, 128);
        };
        auto tails = [&](CUtensorMap* map, const RgOperand& o) {
            return encode_map16(map, q.dt, o.ptr, o.rows, o.k, 1, o.ld * 2, 0, 64, 16);
        };
        const bool ok =
            (q.form != RG_WGRAD || (tails(&p.tmap_a16, q.a) && tails(&p.tmap_b32, q.b))) &&
            (q.a8     ? encode_map8_rows(&p.tmap_a, q.a.ptr, q.a.k, q.a.rows, az, q.a.ld, q.a.stride, 128)
             : q.a.mn ? mn_major(&p.tmap_a, q.a, az)
                      : k_major(&p.tmap_a, q.a, az, p.a_k4, 128)) &&
            (q.b.mn ? mn_major(&p.tmap_b, q.b, bz)
                    : k_major(&p.tmap_b, q.b, bz, p.b_k4, bt / cg) &&
                          k_major(&p.tmap_b32, q.b, bz, false, q.a8 && bt == 32 ? 16 : 32));
        if (!ok) return GEMM_ERR_CUDA;
    }
    p.idesc = make_idesc_f16(q.dt == DT_BF16, q.a.mn, q.b.mn, 128 * cg, 0);
    p.C = q.C;
    p.Cin = q.Cin;
    p.ldc = q.ldc;
    p.stride_c = q.stride_c;
    p.ldcin = q.ldcin;
    p.stride_cin = q.stride_cin;
    p.c_dtype = q.c_dtype;
    p.cin_dtype = q.cin_dtype;
    const int es = dt_bytes(q.c_dtype);
    p.c_vec = aligned(q.C, 16) && q.ldc * es % 16 == 0 && q.stride_c * es % 16 == 0 &&
              (q.beta == 0.0f || (aligned(q.Cin, 16) && q.ldcin * es % 16 == 0 &&
                                  q.stride_cin * es % 16 == 0));
    p.c_tma = q.form == RG_WGRAD && p.c_vec && (q.groups <= 1 || q.stride_c >= q.ldc) &&
              encode_map_out(&p.tmap_c, q.c_dtype, q.C, q.n_lane, q.n_col, q.groups, q.ldc * es,
                             q.stride_c * es);
    p.alpha = q.alpha;
    p.beta = q.beta;
    p.diag = q.diag;
    p.resid = q.resid;
    p.stride_resid = q.stride_resid;
    p.resid_in = q.resid_in;
    p.bias = q.bias;
    p.stride_bias = q.stride_bias;
    p.act = q.act;
    p.status = d.status;
    p.timeout_ns = option_timeout_ns();
    p.test_stall = take_test_stall();
    p.pdl = q.pdl && option_overlap_copy();
#if DG_DEBUG
    const int64_t out_rows = q.form == RG_ROWS && q.offsets ? q.T : q.n_col;
    p.dbg_c_elems = (q.offsets && q.form == RG_ROWS ? 0 : (q.groups - 1) * q.stride_c) +
                    (out_rows - 1) * q.ldc + (q.form == RG_SYM ? q.ldc : q.n_lane);
#endif
    return GEMM_OK;
}

// Few rows (RG_ROWS with offsets): the kernel of w4.cu, with 16-bit weights.  Against
// the ragged kernel, K = 2048 (us): 8 rows, 8 experts of N = 1024 10.5 : 15.3, of
// N = 4096 28.0 : 43.5; 32 rows, 32 experts of N = 1024 28.4 : 28.8, of N = 4096
// 88.1 : 85.6; 64 rows, 64 experts of N = 1024 46.4 : 51.1; one expert with 64 rows
// 9.8 : 13.5; but 192 rows over 64 experts of N = 2048 90.3 : 83.6.
constexpr int64_t kFewRows = 64;

static bool few_rows(const RgProblem& q) {
    return q.form == RG_ROWS && q.offsets && q.K > 0 && q.T <= kFewRows;
}

static gemm_status_t few_run(const RgProblem& q, const DeviceInfo& d, cudaStream_t stream) {
    const int64_t avg = cdiv(q.T, q.groups);
    const int tokens = (q.T < 2 * avg ? q.T : 2 * avg) <= 8 ? 8 : 16;
    const W4Shape shape = w4_shape(tokens, 0);
    W4Params p;
    std::memset(&p, 0, sizeof(p));
    const int64_t z = q.a.stride != 0 ? q.groups : 1;
    p.w_mn = q.a.mn;
    p.w_z = z > 1;
    p.q4 = !q.a.mn && q.K % 64 == 0;
    p.x4 = q.K % 64 == 0;
    const bool ok =
        (q.a.mn ? encode_map16(&p.tmap_q, q.dt, q.a.ptr, q.n_lane, q.K, z, q.a.ld * 2, q.a.stride * 2,
                               static_cast<uint32_t>(shape.rows), static_cast<uint32_t>(shape.step))
         : p.q4 ? encode_map16_k4(&p.tmap_q, q.dt, q.a.ptr, q.K, q.n_lane, z, q.a.ld * 2,
                                  q.a.stride * 2, static_cast<uint32_t>(shape.rows))
                : encode_map16(&p.tmap_q, q.dt, q.a.ptr, q.K, q.n_lane, z, q.a.ld * 2,
                               q.a.stride * 2, 64, static_cast<uint32_t>(shape.rows))) &&
        (p.x4 ? encode_map16_blocks(&p.tmap_x, q.dt, q.b.ptr, q.K, q.T, q.b.ld * 2,
                                    static_cast<uint32_t>(tokens),
                                    static_cast<uint32_t>(shape.step / 64))
              : encode_map16(&p.tmap_x, q.dt, q.b.ptr, q.K, q.T, 1, q.b.ld * 2, 0, 64,
                             static_cast<uint32_t>(tokens)));
    if (!ok) return GEMM_ERR_CUDA;
    p.offsets = q.offsets;
    p.groups = static_cast<int32_t>(q.groups);
    p.T = static_cast<int32_t>(q.T);
    p.N = static_cast<int32_t>(q.n_lane);
    p.K = static_cast<int32_t>(q.K);
    const int64_t n_tiles = cdiv(q.n_lane, shape.rows), steps = cdiv(q.K, shape.step);
    const int64_t units = n_tiles * (q.T / tokens + (q.groups < q.T ? q.groups : q.T));
    int splits = 1;
    while (splits < 4 && units * splits * 2 <= d.sm_count && steps >= splits * 8) splits *= 2;
    p.n_tiles = static_cast<int32_t>(n_tiles);
    p.splits = splits;
    p.grid = static_cast<int32_t>(units < d.sm_count ? units : d.sm_count);
    p.C = q.C;
    p.ldc = q.ldc;
    p.c_dtype = q.c_dtype;
    p.alpha = q.alpha;
    p.beta = q.beta;
    p.bias = q.bias;
    p.stride_bias = q.stride_bias;
    p.act = q.act;
    p.test_stall = take_test_stall();
    p.status = d.status;
    p.timeout_ns = option_timeout_ns();
#if DG_DEBUG
    p.dbg_c_elems = (q.T - 1) * q.ldc + q.n_lane;
#endif
    if (w4_launch(q.dt, tokens, p, stream) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

gemm_status_t rg_run(const RgProblem& q, const DeviceInfo& d, cudaStream_t stream) {
    if (few_rows(q)) return few_run(q, d, stream);
    int cg, bt;
    rg_variant(q, d, &cg, &bt);
    RgParams p;
    int64_t tiles = 0;
    const gemm_status_t st = rg_fill(q, d, cg, bt, &p, &tiles);
    if (st != GEMM_OK) return st;
    int64_t grid = cg == 2 ? d.max_pairs : d.sm_count;
    if (tiles < grid) grid = tiles;
    const int ctas = static_cast<int>(grid * cg);
    const cudaError_t e = q.form == RG_ROWS ? rg_launch_rows(cg, bt, p, ctas, stream)
                                            : rg_launch_wgrad(cg, bt, p, ctas, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

namespace {

gemm_status_t check_grouped(int ab, int64_t groups, int64_t T, int64_t N, int64_t K, const void* A,
                            int64_t lda, const void* B, int64_t ldb, int lb, int64_t stride_b) {
    if (!is_dt(ab)) return GEMM_ERR_INVALID_ARG;
    if (lb != GEMM_ROW_MAJOR && lb != GEMM_COL_MAJOR) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = extents(groups, T, N, K);
    if (st != GEMM_OK) return st;
    if (ab == DT_F32) return GEMM_ERR_UNSUPPORTED;
    if (groups == 0 || T == 0 || N == 0 || K == 0) return GEMM_OK;
    if (!A || !B || !aligned(A, 2) || !aligned(B, 2)) return GEMM_ERR_INVALID_ARG;
    const int64_t inner = lb == GEMM_ROW_MAJOR ? N : K, outer = lb == GEMM_ROW_MAJOR ? K : N;
    if (lda < K || ldb < inner || stride_b < 0) return GEMM_ERR_INVALID_ARG;
    if (!strided_span_ok(T, K, lda, 1, 1, 0) || !count_ok(1, T, K) ||
        !strided_span_ok(outer, inner, ldb, 1, groups, stride_b) || !count_ok(groups, K, N))
        return GEMM_ERR_INVALID_ARG;
    if (stride_b != 0 && !apart(outer, inner, ldb, groups, stride_b)) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

gemm_status_t gemm_grouped(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t N, int64_t K,
                           const void* A, int64_t lda, const void* B, int64_t ldb,
                           gemm_layout_t lb, int64_t stride_b, void* C, int64_t ldc,
                           gemm_dtype_t c_dtype, const int32_t* offsets, float alpha, float beta,
                           const float* bias, int64_t stride_bias, gemm_epilogue_t epi,
                           void* workspace, size_t workspace_bytes, gemm_stream_t stream) {
    // alpha == 0: A and B are not read
    const int64_t Kc = alpha == 0.0f ? 0 : K;
    if (!size_ok(K)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_grouped(ab_dtype, groups, T, N, Kc, A, lda, B, ldb, lb, stride_b);
    if (st != GEMM_OK) return st;
    if (!is_dt(c_dtype)) return GEMM_ERR_INVALID_ARG;
    if (c_dtype != ab_dtype && c_dtype != GEMM_DT_F32) return GEMM_ERR_UNSUPPORTED;
    int act = ACT_NONE;
    st = epilogue_of(epi, bias, stride_bias, N, groups, &act);
    if (st != GEMM_OK) return st;
    if (groups == 0 || T == 0 || N == 0) return GEMM_OK;
    if (!offsets || !aligned(offsets, 4)) return GEMM_ERR_INVALID_ARG;
    if (!c_ok(C, T, N, ldc, 1, 0, c_dtype)) return GEMM_ERR_INVALID_ARG;
    if (!row_tiles_ok(groups, T, N, T <= kFewRows)) return GEMM_ERR_UNSUPPORTED;
    const bool b_mn = lb == GEMM_ROW_MAJOR;
    Stored a{A, lda, 0}, b{B, ldb, groups > 1 ? stride_b : 0};
    DeviceInfo d;
    st = device_info(&d);
    if (st != GEMM_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (Kc > 0) {
        // first without launching, so that an error enqueues nothing
        for (const bool launch : {false, true}) {
            size_t off = 0;
            Stored ta{A, lda, 0}, tb{B, ldb, groups > 1 ? stride_b : 0};
            st = place(&ta, T, K, 1, static_cast<char*>(workspace), workspace_bytes, &off, launch, s);
            if (st == GEMM_OK)
                st = place(&tb, b_mn ? K : N, b_mn ? N : K, groups, static_cast<char*>(workspace),
                           workspace_bytes, &off, launch, s);
            if (st != GEMM_OK) return st;
            a = ta;
            b = tb;
        }
    }
    RgProblem q{};
    q.form = RG_ROWS;
    q.dt = ab_dtype;
    q.groups = groups;
    q.T = T;
    q.n_lane = N;
    q.n_col = T;
    q.K = Kc;
    q.offsets = offsets;
    q.a = RgOperand{b.ptr, b.ld, b.stride, b_mn, N, Kc};
    q.b = RgOperand{a.ptr, a.ld, 0, false, T, Kc};
    q.C = C;
    q.Cin = C;
    q.ldc = q.ldcin = ldc;
    q.c_dtype = q.cin_dtype = c_dtype;
    q.alpha = alpha;
    q.beta = beta;
    q.bias = (epi & 1) ? bias : nullptr;
    q.stride_bias = stride_bias;
    q.act = act;
    q.pdl = a.ptr != A || b.ptr != B;
    return rg_run(q, d, s);
}

size_t gemm_grouped_workspace_size(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t N,
                                   int64_t K, const void* A, int64_t lda, const void* B,
                                   int64_t ldb, gemm_layout_t lb, int64_t stride_b) {
    if (check_grouped(ab_dtype, groups, T, N, K, A, lda, B, ldb, lb, stride_b) != GEMM_OK) return 0;
    if (groups == 0 || T == 0 || N == 0 || K == 0) return 0;
    size_t need = 0;
    const bool b_mn = lb == GEMM_ROW_MAJOR;
    if (groups == 1) stride_b = 0;
    if (!in_place(A, lda, 1, 0)) need += copy_bytes(T, K, 1);
    if (!in_place(B, ldb, groups, stride_b))
        need += copy_bytes(b_mn ? K : N, b_mn ? N : K, stride_b != 0 ? groups : 1);
    return need;
}

static gemm_status_t check_wgrad(int ab, int64_t groups, int64_t T, int64_t M, int64_t N,
                                 const void* A, int64_t lda, const void* D, int64_t ldd) {
    if (!is_dt(ab)) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = extents(groups, T, N, M);
    if (st != GEMM_OK) return st;
    if (ab == DT_F32) return GEMM_ERR_UNSUPPORTED;
    if (groups == 0 || T == 0 || N == 0 || M == 0) return GEMM_OK;
    if (!A || !D || !aligned(A, 2) || !aligned(D, 2)) return GEMM_ERR_INVALID_ARG;
    if (lda < M || ldd < N) return GEMM_ERR_INVALID_ARG;
    if (!strided_span_ok(T, M, lda, 1, 1, 0) || !count_ok(1, T, M) ||
        !strided_span_ok(T, N, ldd, 1, 1, 0) || !count_ok(1, T, N))
        return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

gemm_status_t gemm_grouped_wgrad(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t M,
                                 int64_t N, const void* A, int64_t lda, const void* D, int64_t ldd,
                                 void* C, int64_t ldc, int64_t stride_c, gemm_dtype_t c_dtype,
                                 const int32_t* offsets, float alpha, float beta, void* workspace,
                                 size_t workspace_bytes, gemm_stream_t stream) {
    if (!size_ok(T)) return GEMM_ERR_INVALID_ARG;
    const int64_t Tc = alpha == 0.0f ? 0 : T;  // alpha == 0: A and D are not read
    gemm_status_t st = check_wgrad(ab_dtype, groups, Tc, M, N, A, lda, D, ldd);
    if (st != GEMM_OK) return st;
    if (!is_dt(c_dtype)) return GEMM_ERR_INVALID_ARG;
    if (c_dtype != ab_dtype && c_dtype != GEMM_DT_F32) return GEMM_ERR_UNSUPPORTED;
    if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
    if (!c_ok(C, M, N, ldc, groups, groups > 1 ? stride_c : 0, c_dtype)) return GEMM_ERR_INVALID_ARG;
    if (!apart(M, N, ldc, groups, stride_c)) return GEMM_ERR_INVALID_ARG;
    if (Tc > 0 && (!offsets || !aligned(offsets, 4))) return GEMM_ERR_INVALID_ARG;
    if (!wgrad_tiles_ok(groups, M, N)) return GEMM_ERR_UNSUPPORTED;
    DeviceInfo d;
    st = device_info(&d);
    if (st != GEMM_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Stored a{A, lda, 0}, b{D, ldd, 0};
    if (Tc > 0) {
        for (const bool launch : {false, true}) {
            size_t off = 0;
            Stored ta{A, lda, 0}, tb{D, ldd, 0};
            st = place(&ta, T, M, 1, static_cast<char*>(workspace), workspace_bytes, &off, launch, s);
            if (st == GEMM_OK)
                st = place(&tb, T, N, 1, static_cast<char*>(workspace), workspace_bytes, &off,
                           launch, s);
            if (st != GEMM_OK) return st;
            a = ta;
            b = tb;
        }
    }
    RgProblem q{};
    q.form = RG_WGRAD;
    q.dt = ab_dtype;
    q.groups = groups;
    q.T = Tc;
    q.n_lane = N;
    q.n_col = M;
    q.K = 0;
    q.offsets = Tc > 0 ? offsets : nullptr;
    q.a = RgOperand{b.ptr, b.ld, 0, true, N, Tc};
    q.b = RgOperand{a.ptr, a.ld, 0, true, M, Tc};
    q.C = C;
    q.Cin = C;
    q.ldc = q.ldcin = ldc;
    q.stride_c = q.stride_cin = groups > 1 ? stride_c : 0;
    q.c_dtype = q.cin_dtype = c_dtype;
    q.alpha = alpha;
    q.beta = beta;
    q.pdl = a.ptr != A || b.ptr != D;
    return rg_run(q, d, s);
}

size_t gemm_grouped_wgrad_workspace_size(gemm_dtype_t ab_dtype, int64_t groups, int64_t T,
                                         int64_t M, int64_t N, const void* A, int64_t lda,
                                         const void* D, int64_t ldd) {
    if (check_wgrad(ab_dtype, groups, T, M, N, A, lda, D, ldd) != GEMM_OK) return 0;
    if (groups == 0 || T == 0 || N == 0 || M == 0) return 0;
    size_t need = 0;
    if (!in_place(A, lda, 1, 0)) need += copy_bytes(T, M, 1);
    if (!in_place(D, ldd, 1, 0)) need += copy_bytes(T, N, 1);
    return need;
}

// ---------------------------------------------------------------- orthogonalised update

namespace {

// fp16 scales of the stored states: X times 2^13, S and b S + c S S times 2^12.
// With singular values of X below 4 and the polynomial below 8 in norm no
// stored value passes 32768, and an entry 2^-10 of a typical one (1 / sqrt(n) of
// an orthogonalised 8192-wide matrix is 90 when stored) is still a normal number.
constexpr float kNsX = 8192.0f, kNsS = 4096.0f;

struct NsLayout {
    int64_t side, ldx, lds, parts;
    size_t x_bytes, s_bytes, part_bytes, total;
};

bool ns_layout(int64_t batch, int64_t M, int64_t N, NsLayout* l) {
    if (!size_ok(batch) || !size_ok(M) || !size_ok(N)) return false;
    l->side = M < N ? M : N;
    l->ldx = round_up(N, 8);
    l->lds = round_up(l->side, 8);
    if (!count_ok(batch, M, l->ldx) || !count_ok(batch, l->side, l->lds)) return false;
    int64_t parts = cdiv(1216, batch > 0 ? batch : 1);  // 8 blocks for each of 152 SMs
    if (parts > M) parts = M;
    if (parts < 1) parts = 1;
    l->parts = parts;
    if (batch * parts > kLim) return false;
    l->x_bytes = static_cast<size_t>(round_up(batch * M * l->ldx * 2, 256));
    l->s_bytes = static_cast<size_t>(round_up(batch * l->side * l->lds * 2, 256));
    l->part_bytes = static_cast<size_t>(round_up(batch * parts * 12, 256));
    l->total = 2 * l->x_bytes + 2 * l->s_bytes + l->part_bytes +
               static_cast<size_t>(round_up(batch * 4, 256));
    return true;
}

}  // namespace

size_t gemm_newton_schulz_workspace_size(int64_t batch, int64_t M, int64_t N) {
    NsLayout l;
    if (batch <= 0 || M <= 0 || N <= 0 || !ns_layout(batch, M, N, &l)) return 0;
    return l.total;
}

gemm_status_t gemm_newton_schulz(gemm_dtype_t g_dtype, int64_t batch, int64_t M, int64_t N,
                                 const void* G, int64_t ldg, int64_t stride_g, void* O,
                                 int64_t ldo, int64_t stride_o, gemm_dtype_t o_dtype, int steps,
                                 float a, float b, float c, float eps, void* workspace,
                                 size_t workspace_bytes, gemm_stream_t stream) {
    if (!is_dt(g_dtype) || !is_dt(o_dtype)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = extents(batch, M, N, 0);
    if (st != GEMM_OK) return st;
    if (steps < 1 || steps > 64 || !(eps >= 0.0f)) return GEMM_ERR_INVALID_ARG;
    if (o_dtype == GEMM_DT_F32) return GEMM_ERR_UNSUPPORTED;
    if (batch == 0 || M == 0 || N == 0) return GEMM_OK;
    if (!G || !aligned(G, dt_bytes(g_dtype)) || ldg < N || (batch > 1 && stride_g < 0))
        return GEMM_ERR_INVALID_ARG;
    if (!strided_span_ok(M, N, ldg, 1, batch, batch > 1 ? stride_g : 0)) return GEMM_ERR_INVALID_ARG;
    if (!c_ok(O, M, N, ldo, batch, batch > 1 ? stride_o : 0, o_dtype)) return GEMM_ERR_INVALID_ARG;
    if (!apart(M, N, ldo, batch, stride_o)) return GEMM_ERR_INVALID_ARG;
    NsLayout l;
    if (!ns_layout(batch, M, N, &l)) return GEMM_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < l.total) return GEMM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo d;
    st = device_info(&d);
    if (st != GEMM_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    char* x[2] = {ws, ws + l.x_bytes};
    char* S = ws + 2 * l.x_bytes;
    char* P = S + l.s_bytes;

    NsParams n{};
    n.G = G;
    n.ldg = ldg;
    n.stride_g = batch > 1 ? stride_g : 0;
    n.g_dtype = g_dtype;
    n.g_vec = aligned(G, 16) && ldg * dt_bytes(g_dtype) % 16 == 0 &&
              n.stride_g * dt_bytes(g_dtype) % 16 == 0;
    n.batch = batch;
    n.M = static_cast<int32_t>(M);
    n.N = static_cast<int32_t>(N);
    n.parts = static_cast<int32_t>(l.parts);
    n.partials = reinterpret_cast<float*>(P + l.s_bytes);
    n.X = x[0];
    n.ldx = l.ldx;
    n.eps = eps;
    n.scale = kNsX;
    n.arrived = reinterpret_cast<unsigned int*>(P + l.s_bytes + l.part_bytes);
    // a X + b S X + c S S X = P X, with P from a square completed, so that no product
    // reads its own kind of matrix back: with Y = S + b / (2 c),
    //   P = a + b S + c S S = c Y Y + (a - b b / (4 c)).
    // Where b / (2 c) would cost Y its bits (or c is zero), Y is S and P adds b S.
    // The shift would cost Y's diagonal bits of S too (fp16 steps of 2^-11 near 1.2): what
    // an entry Y_ii loses, r_i, comes back as the 2 c r_i Y_ii that P_ii lacks for it.  The
    // products lie in the buffer of the next X, which is not in use between the two.  (The
    // result's error before its own rounding: 128 x 2048 1.6e-3 -> 8.5e-4, 64 x 64 1.9e-3
    // -> 1.5e-3; rounding the products c (r_i + r_j) Y_ij beside the diagonal is left.)
    const bool squared = std::fabs(b) <= 4.0f * std::fabs(c) && c != 0.0f;
    const float shift = squared ? b / (2.0f * c) : 0.0f;
    const bool wide = M <= N;
    const int64_t xs = batch > 1 ? M * l.ldx : 0, ss = batch > 1 ? l.side * l.lds : 0;
    int cg = 0, bt = 0;
    int64_t most = 0;
    auto add = [&](const RgProblem& q, RgParams* out) {
        if (cg == 0) {
            // (the sequence's shapes: pairs, or 128 lanes by 128 columns, or by 64
            // where those would leave more than half of the SMs idle, which shortens
            // each product of the chain: 256 x 256 80 us with 128 columns, 73 with 64)
            rg_variant(q, d, &cg, &bt);
            if (cg == 1)
                bt = batch * cdiv(M, 128) * cdiv(N, 128) * 2 <= d.sm_count ? 64 : 128;
        }
        int64_t tiles = 0;
        const gemm_status_t e = rg_fill(q, d, cg, bt, out, &tiles);
        if (tiles > most) most = tiles;
        return e;
    };
    RgSeq* seq = new (std::nothrow) RgSeq;
    if (!seq) return GEMM_ERR_CUDA;
    std::memset(seq, 0, sizeof(*seq));
    seq->steps = steps;
    seq->arrived = n.arrived;
    for (int odd = 0; odd < 2 && st == GEMM_OK; ++odd) {
        const void* X = x[odd];
        // Y = X X^T (K-major) or X^T X (MN-major), shifted, times kNsS
        RgProblem q{};
        q.form = RG_SYM;
        q.dt = DT_F16;
        q.groups = batch;
        q.n_lane = q.n_col = l.side;
        q.K = wide ? N : M;
        q.a = q.b = RgOperand{X, l.ldx, xs, !wide, l.side, q.K};
        q.C = S;
        q.ldc = q.ldcin = l.lds;
        q.stride_c = q.stride_cin = ss;
        q.c_dtype = q.cin_dtype = DT_F16;
        q.alpha = kNsS / (kNsX * kNsX);
        q.diag = shift * kNsS;
        if (squared) {
            q.resid = reinterpret_cast<float*>(x[1 - odd]);
            q.stride_resid = xs / 2;
        }
        st = add(q, &seq->ph[3 * odd]);
        // P = c Y Y + beta Y + constant, times kNsS
        q.K = l.side;
        q.a = q.b = RgOperand{S, l.lds, ss, false, l.side, l.side};
        q.resid_in = 1;
        q.C = P;
        q.Cin = S;
        q.alpha = c / kNsS;
        q.beta = squared ? 0.0f : b;
        q.diag = (squared ? static_cast<float>(a - 0.25 * b * (static_cast<double>(b) / c)) : a) * kNsS;
        if (st == GEMM_OK) st = add(q, &seq->ph[3 * odd + 1]);
        // X <- P X, or X P
        RgProblem u{};
        u.form = RG_ROWS;
        u.dt = DT_F16;
        u.groups = batch;
        u.n_lane = N;
        u.n_col = M;
        u.K = l.side;
        const RgOperand sym{P, l.lds, ss, false, l.side, l.side};
        u.a = wide ? RgOperand{X, l.ldx, xs, true, N, M} : sym;
        u.b = wide ? sym : RgOperand{X, l.ldx, xs, false, M, N};
        u.alpha = 1.0f / kNsS;
        u.c_dtype = u.cin_dtype = DT_F16;
        u.C = x[1 - odd];
        u.ldc = l.ldx;
        u.stride_c = xs;
        if (st == GEMM_OK) st = add(u, &seq->ph[3 * odd + 2]);
        if (((steps - 1) & 1) == odd) {
            u.alpha /= kNsX;
            u.C = O;
            u.ldc = ldo;
            u.stride_c = batch > 1 ? stride_o : 0;
            u.c_dtype = o_dtype;
            if (st == GEMM_OK) st = add(u, &seq->ph[6]);
        }
    }
    if (st == GEMM_OK) {
        int64_t grid = cg == 2 ? d.max_pairs : d.sm_count;
        if (most < grid) grid = most;
        if (ns_norm_launch(n, s) != cudaSuccess || ns_scale_launch(n, s) != cudaSuccess ||
            rg_launch_seq(cg, bt, *seq, static_cast<int>(grid * cg), s) != cudaSuccess) {
            cudaGetLastError();
            st = GEMM_ERR_CUDA;
        }
    }
    delete seq;
    return st;
}

// ---------------------------------------------------------------- 4-bit weights

namespace {

// Rows (of a group, on average) up to which the 4-bit integers are multiplied directly;
// more rows multiply 16-bit weights in the workspace, rounded once more (bf16 output: 2.2e-3
// of the result against 1.7e-3).  Direct : 16-bit (us), K x N = 4096 x 4096, one matrix:
// 64 rows 19.7 : 29, 96 rows 32 : 29.  Experts of 2048 x 4096, where the host knows the
// average alone: 32 of them with 16 rows each 133 : 215, 25 rows 207 : 221, 37 rows
// 223 : 214 unevenly and 192 : 215 evenly spread, 50 rows 261 : 221 and 203 : 215;
// 8 of them with 37 rows 62.1 : 62.6, 50 rows 85 : 63.  So past 40 rows, evenly spread
// rows over many experts lose up to a tenth of their time, and uneven ones or few experts
// win more.
constexpr int64_t kW4DirectRows = 64, kW4DirectGroupRows = 40;

bool w4_direct(int64_t groups, int64_t T, int c_dtype) {
    return c_dtype == DT_F32 || option_w4_exact() || T <= (groups > 1 ? kW4DirectGroupRows * groups : kW4DirectRows);
}

size_t w4_need(bool direct, int64_t groups, int64_t T, int64_t N, int64_t K, const void* A,
               int64_t lda) {
    size_t need = 0;
    if (!in_place(A, lda, 1, 0)) need += copy_bytes(T, K, 1);
    if (!direct) need += copy_bytes(N, K, groups);
    return need;
}

}  // namespace

size_t gemm_w4_workspace_size(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t N,
                              int64_t K, const void* A, int64_t lda, gemm_dtype_t c_dtype) {
    if (!is16(ab_dtype) || !is_dt(c_dtype) || !size_ok(groups) || !size_ok(T) || !size_ok(N) ||
        !size_ok(K) || groups == 0 || T == 0 || N == 0 || K == 0 || !count_ok(groups, N, K) ||
        !count_ok(1, T, K + 8))
        return 0;
    return w4_need(w4_direct(groups, T, c_dtype), groups, T, N, K, A, lda);
}

gemm_status_t gemm_w4(gemm_dtype_t ab_dtype, int64_t groups, int64_t T, int64_t N, int64_t K,
                      const void* A, int64_t lda, const uint8_t* Q, const void* scales,
                      const uint8_t* zeros, int group, void* C, int64_t ldc, gemm_dtype_t c_dtype,
                      const int32_t* offsets, const float* bias, int64_t stride_bias,
                      gemm_epilogue_t epi, void* workspace, size_t workspace_bytes,
                      gemm_stream_t stream) {
    if (!is_dt(ab_dtype) || !is_dt(c_dtype)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = extents(groups, T, N, K);
    if (st != GEMM_OK) return st;
    if (group != 32 && group != 64 && group != 128) return GEMM_ERR_INVALID_ARG;
    if (K % group != 0) return GEMM_ERR_INVALID_ARG;
    if (ab_dtype == GEMM_DT_F32 || (c_dtype != ab_dtype && c_dtype != GEMM_DT_F32))
        return GEMM_ERR_UNSUPPORTED;
    int act = ACT_NONE;
    st = epilogue_of(epi, bias, stride_bias, N, groups, &act);
    if (st != GEMM_OK) return st;
    if (groups == 0 || T == 0 || N == 0) return GEMM_OK;
    if (offsets ? !aligned(offsets, 4) : groups != 1) return GEMM_ERR_INVALID_ARG;
    if (!c_ok(C, T, N, ldc, 1, 0, c_dtype)) return GEMM_ERR_INVALID_ARG;
    if (K == 0)  // act(bias), rows outside the groups untouched
        return offsets ? gemm_grouped(ab_dtype, groups, T, N, 0, nullptr, 0, nullptr, 0,
                                      GEMM_COL_MAJOR, 0, C, ldc, c_dtype, offsets, 1.0f, 0.0f, bias,
                                      stride_bias, epi, nullptr, 0, stream)
                       : gemm_batched(ab_dtype, 1, T, N, 0, nullptr, 0, GEMM_ROW_MAJOR, 0, nullptr,
                                      N, GEMM_ROW_MAJOR, 0, C, ldc, GEMM_ROW_MAJOR, 0, c_dtype, 1.0f,
                                      0.0f, bias, epi, 0, nullptr, 0, stream);
    if (!A || !aligned(A, 2) || lda < K || !Q || !aligned(Q, 16) || !scales || !aligned(scales, 2))
        return GEMM_ERR_INVALID_ARG;
    if (!strided_span_ok(T, K, lda, 1, 1, 0) || !count_ok(groups, N, K)) return GEMM_ERR_INVALID_ARG;
    // (once: the option may change meanwhile)
    const bool direct = w4_direct(groups, T, c_dtype);
    if (!row_tiles_ok(groups, T, N, direct)) return GEMM_ERR_UNSUPPORTED;
    const size_t need = w4_need(direct, groups, T, N, K, A, lda);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo d;
    st = device_info(&d);
    if (st != GEMM_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    size_t off = 0;
    Stored a{A, lda, 0};
    st = place(&a, T, K, 1, ws, workspace_bytes, &off, true, s);
    if (st != GEMM_OK) return st;
    if (!direct) {
        if (w4_dequantise(ab_dtype, Q, scales, zeros, groups * N, K, group, ws + off, s) !=
            cudaSuccess)
            return GEMM_ERR_CUDA;
        RgProblem q{};
        q.form = RG_ROWS;
        q.dt = ab_dtype;
        q.groups = groups;
        q.T = T;
        q.n_lane = N;
        q.n_col = T;
        q.K = K;
        q.offsets = offsets;
        q.a = RgOperand{ws + off, K, groups > 1 ? N * K : 0, false, N, K};
        q.b = RgOperand{a.ptr, a.ld, 0, false, T, K};
        q.C = C;
        q.Cin = C;
        q.ldc = q.ldcin = ldc;
        q.c_dtype = q.cin_dtype = c_dtype;
        q.alpha = 1.0f;
        q.bias = (epi & 1) ? bias : nullptr;
        q.stride_bias = stride_bias;
        q.act = act;
        q.pdl = true;
        return rg_run(q, d, s);
    }
    // tokens of a tile: the rows a group is expected to have
    const int64_t avg = cdiv(T, groups);
    const int64_t want = offsets ? (T < 2 * avg ? T : 2 * avg) : T;
    const int tokens = want <= 8 ? 8 : (want <= 16 ? 16 : (want <= 32 ? 32 : 64));
    const W4Shape shape = w4_shape(tokens, group);
    W4Params p;
    std::memset(&p, 0, sizeof(p));
    p.q4 = K % 256 == 0;
    p.x4 = K % 64 == 0;
    if (!encode_map8(&p.tmap_q, Q, K / 2, N, groups, static_cast<uint32_t>(shape.rows),
                     p.q4 ? static_cast<uint32_t>(shape.step / 256) : 0u) ||
        !(p.x4 ? encode_map16_blocks(&p.tmap_x, ab_dtype, a.ptr, K, T, a.ld * 2,
                                     static_cast<uint32_t>(tokens),
                                     static_cast<uint32_t>(shape.step / 64))
               : encode_map16(&p.tmap_x, ab_dtype, a.ptr, K, T, 1, a.ld * 2, 0, 64,
                              static_cast<uint32_t>(tokens))))
        return GEMM_ERR_CUDA;
    p.scales = scales;
    p.zeros = zeros;
    p.offsets = offsets;
    p.groups = static_cast<int32_t>(groups);
    p.T = static_cast<int32_t>(T);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.group = group;
    const int stage_k = shape.step;
    p.vec = K % stage_k == 0 && aligned(scales, 16) && (!zeros || aligned(zeros, 8));
    const int64_t n_tiles = cdiv(N, shape.rows), steps = cdiv(K, stage_k);
    // units there may be: full token tiles and one more for each non-empty group
    const int64_t units = n_tiles * (T / tokens + (groups < T ? groups : T));
    // K slices (a cluster per unit) where the units would leave SMs idle, each of
    // at least one stage for every set of consumer warps.  (Clusters of 8 do not all
    // fit at once: N = 1024, K = 8192 took 11.9 us in 8 slices.)
    int splits = 1;
    if (!offsets)
        while (splits < 4 && n_tiles * cdiv(T, tokens) * splits * 2 <= d.sm_count &&
               steps >= splits * 8)
            splits *= 2;
    p.n_tiles = static_cast<int32_t>(n_tiles);
    p.splits = splits;
    p.grid = static_cast<int32_t>(splits > 1 ? n_tiles * cdiv(T, tokens)
                                             : (units < d.sm_count ? units : d.sm_count));
    p.C = C;
    p.ldc = ldc;
    p.c_dtype = c_dtype;
    p.alpha = 1.0f;
    p.bias = (epi & 1) ? bias : nullptr;
    p.stride_bias = stride_bias;
    p.act = act;
    p.test_stall = take_test_stall();
    p.status = d.status;
    p.timeout_ns = option_timeout_ns();
#if DG_DEBUG
    p.dbg_c_elems = (T - 1) * ldc + N;
#endif
    if (w4_launch(ab_dtype, tokens, p, s) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

}  // extern "C"
