// The ragged-product kernel: persistent, warp-specialised tcgen05 products
// whose tiles come from groups of unequal size.
//
// Every form computes tiles of  D[col][lane] = sum_k B[col][k] * A[lane][k]
// with the LANE operand A on the MMA's M side (128 rows per CTA, 256 per CTA
// pair) and the COLUMN operand B on its N side:
//
//   RG_ROWS   y[t, n] = sum_k x[t, k] w_e[k, n] for the rows t of group e.
//             Lanes are the weights' output features n, columns the tokens t.
//             Groups end anywhere, so the ragged dimension is the MMA's N,
//             which the instruction descriptor sets per tile in steps of 16
//             (32 for a pair): a group of R rows becomes ceil(R / BT) tiles of
//             equal width and wastes at most 31 columns per tile, where tokens
//             on the M side would round every group up to 256 rows.  A few
//             tokens still fill the 128 lanes with weights, which is what a
//             decoding batch has to read (192 rows over 64 experts of 2048 x 2048:
//             83.5 us, 6.4 TB/s; below 65 rows the kernel of w4.cu is faster).
//   RG_WGRAD  dw_e[m, n] = sum_{t in group e} x[t, m] d[t, n].  Lanes are n,
//             columns m; the contraction is ragged.  Both operands are
//             MN-major.  A group's last K = 16 step may end inside the next
//             group: its 16 rows are loaded apart, at the start of the tile, the
//             rows past the group's end (finite or not) are overwritten with
//             zeros in shared memory, and the tile's last MMA takes them.
//   RG_SYM    X X^T (or X^T X), plus beta Cin and a multiple of the unit matrix:
//             only tiles on or below the diagonal are computed, and each is
//             written to both places.
//
// Warps: 0 TMA producer, 1 MMA issuer, 10 (RG_WGRAD) ragged tails, 2-9 epilogue,
// two per tensor-memory lane quarter taking 32-column chunks in
// turn (fp32 outputs: 2 tails, 4-11 epilogue).  Two accumulators let a tile's epilogue
// overlap the next main loop.
// The output's contiguous dimension runs along the lanes.  A 16-bit chunk is
// read from tensor memory in the MMA-fragment layout, turned by transposing
// 8 x 8 matrix stores into a shared-memory tile of 32 columns by 32 lanes (rows
// of 64 bytes, 16-byte parts swizzled by the row: conflict-free both ways) and
// leaves as 16-byte stores along the lanes; beta * Cin takes the same way in.
// An fp32 chunk is read one lane per thread and stored directly: 32 lanes are
// 128 contiguous bytes.  Rows of another group are masked per column.  (A
// first form that turned fp32 values through padded rows with 4-byte stores
// took 10.6 thousand cycles for a CTA's 128 x 256 tile, more than the main
// loop of K = 1024.)  RG_WGRAD's tiles end with their matrix, so its staged tiles
// leave as TMA boxes that end there too (16 groups, 16384 rows, 2048 x 4096, fp32:
// 209 -> 196 us).  For the other forms, whose whole boxes could do the same, it gave
// nothing (187 -> 191 us for the forward product of that size).
//
// Work: tiles are dealt round robin to CTAs (pairs).  Where group sizes are on
// the device, each warp finds its tile by a 32-group window of prefix sums held
// one group per lane: no table, no extra launch, no limit on the groups.
//
// Every mbarrier wait is bounded; on expiry the kernel sets the status word,
// drains its copies and MMAs, frees tensor memory and returns.
#pragma once
#include <stdint.h>

#include <type_traits>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "ragged.h"

namespace dg {
namespace {

constexpr uint32_t kRgMaxSmem = 232448;  // 227 KB opt-in limit per CTA

template <int CG, int BT>
struct RgCfg {
    static constexpr int B_ROWS = BT / CG;  // column-operand rows a CTA holds
    // a stage holds two 64-deep K blocks: half as many waits, loads and commits
    // for the single threads that issue them
    static constexpr uint32_t A_BYTES = 2 * 128 * 128;
    static constexpr uint32_t B_BYTES = 2 * B_ROWS * 128;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARPS = 8;
    // (RG_WGRAD has one warp more, for the ragged tails; fp32 outputs take four warps
    // before the epilogue's, so that registers move between whole warpgroups)
    static constexpr int threads(int form, bool sum = false) {
        return sum ? 128 + 32 * EPI_WARPS : 64 + 32 * EPI_WARPS + (form == RG_WGRAD ? 32 : 0);
    }
    static constexpr uint32_t EPI_WARP = 2 * 2048;  // two tiles of 32 x 32 16-bit elements
    static constexpr uint32_t EPI_SMEM = EPI_WARPS * EPI_WARP;
    static constexpr uint32_t BAR_BYTES = 512;
    static constexpr int FIT = (kRgMaxSmem - 1024 - BAR_BYTES - EPI_SMEM) / STAGE_BYTES;
    static constexpr int STAGES = FIT > 12 ? 12 : FIT;
    static constexpr uint32_t TMEM_COLS = 2 * BT < 32 ? 32 : 2 * BT;
    static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE_BYTES + EPI_SMEM + BAR_BYTES;
    static_assert(BT % 32 == 0 && BT <= 256 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "tile width");
    static_assert(CG == 1 || BT == 256, "pairs take 256-column tiles (two 64-wide atoms per CTA)");
    // RG_WGRAD: half of the staging (one tile a warp), and two buffers of 16 rows of
    // both operands for the ragged ends of groups
    static constexpr uint32_t TAIL_A = 2 * 16 * 128, TAIL_B = (B_ROWS / 64) * 16 * 128;
    static constexpr uint32_t TAIL_AT = EPI_SMEM / 2, TAIL_BYTES = 8192;
    static_assert(B_ROWS < 64 || 2 * TAIL_BYTES <= EPI_SMEM / 2, "tail buffers");
    static_assert(TAIL_A + TAIL_B <= TAIL_BYTES, "tail buffer");
    static_assert((2 * STAGES + 11) * 8 + 8 <= BAR_BYTES, "barrier area too small");
};

struct RgTile {
    int group;
    int lane0;   // first lane of this CTA
    int col0;    // first column, in the group
    int ncols;   // valid columns
    int n_mma;   // MMA N
    int b_row;   // row (or feature) coordinate of column 0 of the tile
    int out_row; // output row of column 0 of the tile
    int k0;      // first contraction coordinate
    int klen;    // contraction length
    bool diag;   // RG_SYM: on the diagonal
};

// A 32-group window of tile counts, one group per lane.
struct RgWalk {
    int base;    // first group of the window
    int before;  // tiles of the groups before it
    int incl;    // this lane's inclusive tile count inside the window
    int row0, rows;
    bool last;   // no group follows the window
};

// Offsets that do not ascend inside [0, rows] are reported.  RG_ROWS then takes
// the groups from the first such one on as empty (so that rows, and tiles, stay
// within the host's bounds), RG_WGRAD that group alone.
__device__ __forceinline__ void rg_window(const RgParams& p, RgWalk& w, int lane) {
    const int g = w.base + lane;
    int lo = 0, hi = 0;
    if (g < p.groups) {
        lo = __ldg(p.offsets + g);
        hi = __ldg(p.offsets + g + 1);
    }
    const uint32_t bad = __ballot_sync(0xffffffffu, lo < 0 || hi < lo || hi > p.rows);
    w.last = bad != 0 || w.base + 32 >= p.groups;
    if (bad) {
        if (lane == 0 && p.status) atomicOr(p.status, STATUS_BAD_OFFSETS);
        if (lane >= __ffs(bad) - 1) lo = hi = 0;
    }
    w.row0 = lo;
    w.rows = hi - lo;
    int tiles = ((w.rows + p.col_tile - 1) / p.col_tile) * p.lane_tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, tiles, d);
        if (lane >= d) tiles += o;
    }
    w.incl = tiles;
}

// Tile r of a group's chunks x lane_tiles: bands of RG_BAND chunks, in a band
// the chunks of one lane tile after another, so that the tiles in flight at
// once (76 pairs) share few operand panels (16384 x 4096 x 8192 in one group:
// 643 us against 759 us with all 64 chunks in one band).
__device__ __forceinline__ int rg_div(int n, RgDiv d) {
    return d.m == 0u ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), d.m) >> d.s);
}
__device__ __forceinline__ void rg_band(const RgParams& p, int r, int chunks, int& lt, int& c) {
    const int c0 = rg_div(r, p.div_band) * RG_BAND;
    const int in = r - c0 * p.lane_tiles;
    if (chunks - c0 >= RG_BAND) {
        lt = in / RG_BAND;
        c = c0 + in % RG_BAND;
    } else {
        lt = in / (chunks - c0);
        c = c0 + in - lt * (chunks - c0);
    }
}

template <int FORM>
__device__ __forceinline__ RgWalk rg_begin(const RgParams& p, int lane) {
    RgWalk w{0, 0, 0, 0, 0, false};
    if (FORM == RG_ROWS && p.offsets) rg_window(p, w, lane);
    return w;
}

// Tile t of the problem, by a whole (converged) warp; false past the last one.
template <int CG, int BT, int FORM>
__device__ __forceinline__ bool rg_tile(const RgParams& p, RgWalk& w, int t, int lane,
                                        uint32_t rank, RgTile& o) {
    constexpr int LANES = 128 * CG;
    constexpr int GRAN = 16 * CG;  // granularity of the MMA's N
    o.k0 = 0;
    o.klen = p.K;
    o.diag = false;
    if (FORM == RG_ROWS && p.offsets) {
        int total = __shfl_sync(0xffffffffu, w.incl, 31);
        while (t - w.before >= total) {
            if (w.last) return false;
            w.before += total;
            w.base += 32;
            rg_window(p, w, lane);
            total = __shfl_sync(0xffffffffu, w.incl, 31);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, w.incl > t - w.before);
        const int l = __ffs(m) - 1;
        const int rows = __shfl_sync(0xffffffffu, w.rows, l);
        const int row0 = __shfl_sync(0xffffffffu, w.row0, l);
        const int incl = __shfl_sync(0xffffffffu, w.incl, l);
        const int chunks = (rows + BT - 1) / BT;  // (col_tile is BT here)
        const int r = t - w.before - (incl - chunks * p.lane_tiles);
        int lt, c;
        rg_band(p, r, chunks, lt, c);
        const int width = ((rows + chunks - 1) / chunks + GRAN - 1) / GRAN * GRAN;
        o.group = w.base + l;
        o.lane0 = lt * LANES + static_cast<int>(rank) * 128;
        o.col0 = c * width;
        o.ncols = rows - o.col0 < width ? rows - o.col0 : width;
        o.b_row = o.out_row = row0 + o.col0;
    } else {
        if (t >= p.total_tiles) return false;
        o.group = rg_div(t, p.div_group);
        const int r = t - o.group * p.per_group;
        if (FORM == RG_SYM) {
            // F column tiles to a lane tile; those on the diagonal are computed whole
            constexpr int F = LANES / BT;
            const int q = r / F;
            int i = static_cast<int>((sqrtf(8.0f * static_cast<float>(q) + 1.0f) - 1.0f) * 0.5f);
            while (i * (i + 1) / 2 > q) --i;
            while ((i + 1) * (i + 2) / 2 <= q) ++i;
            const int j = r - F * (i * (i + 1) / 2);
            o.diag = j >= F * i;
            o.lane0 = i * LANES + static_cast<int>(rank) * 128;
            o.col0 = j * p.col_tile;
        } else {
            int lt, c;
            rg_band(p, r, p.chunks, lt, c);
            o.lane0 = lt * LANES + static_cast<int>(rank) * 128;
            o.col0 = c * p.col_tile;
        }
        o.ncols = p.n_col - o.col0 < p.col_tile ? p.n_col - o.col0 : p.col_tile;
        o.b_row = o.out_row = o.col0;
        if (FORM == RG_WGRAD) {
            int lo = 0, hi = 0;
            if (p.offsets) {  // (none: alpha == 0 or no rows)
                lo = __ldg(p.offsets + o.group);
                hi = __ldg(p.offsets + o.group + 1);
                if (lo < 0 || hi < lo || hi > p.rows) {
                    if (lane == 0 && p.status) atomicOr(p.status, STATUS_BAD_OFFSETS);
                    lo = hi = 0;
                }
            }
            o.k0 = lo;
            o.klen = hi - lo;
        }
    }
    // MN-major columns come in 64-wide swizzle atoms per CTA
    const int gran = p.b_mn ? 64 * CG : GRAN;
    o.n_mma = (o.ncols + gran - 1) / gran * gran;
    return true;
}

// A value that all lanes hold, in a register that the compiler knows to be uniform:
// the tensor-core and TMA instructions take their operands from uniform registers.
__device__ __forceinline__ int rg_uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Bounded wait of a whole warp (all lanes poll, and agree on the result).
__device__ __forceinline__ bool rg_all_wait(uint32_t bar, uint32_t parity, const RgParams& p,
                                            volatile int* abort_flag) {
    const bool ok = mbar_wait_short(bar, parity, abort_flag, p.status, p.timeout_ns);
    return __all_sync(0xffffffffu, ok) != 0;
}

// Bounded wait of a whole warp (one lane polls).
__device__ __forceinline__ bool rg_warp_wait(uint32_t bar, uint32_t parity, int lane,
                                             volatile int* abort_flag, const RgParams& p) {
    int ok = 1;
    if (lane == 0) ok = mbar_wait_short(bar, parity, abort_flag, p.status, p.timeout_ns) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

__device__ __forceinline__ bool rg_drain(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > timeout_ns) return false;
    return true;
}

__device__ __forceinline__ uint32_t rg_pack(int dt, float lo, float hi) {
    if (dt == DT_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 rg_unpack(int dt, uint32_t u) {
    if (dt == DT_BF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ bool rg_span_ok(const RgParams& p, int64_t off, int n) {
#if DG_DEBUG
    return DG_CHECK(off >= 0 && off + n <= p.dbg_c_elems, p.status, STATUS_CHECK_BOUNDS);
#else
    (void)p, (void)off, (void)n;
    return true;
#endif
}

// Byte offset of 16-byte part `part` of row `row` in a staged 32 x 32 tile.
__device__ __forceinline__ uint32_t rg_at(int row, int part) {
    return static_cast<uint32_t>(row * 64 + ((part ^ ((row >> 1) & 3)) << 4));
}

// Eight 16-bit elements of which `n` exist, one at a time (out of line, so that
// the epilogue's common path stays short in the instruction cache).
__device__ __noinline__ uint4 rg_load8_slow(const char* src, int n) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n)
            w[i >> 1] |= static_cast<uint32_t>(__ldcg(reinterpret_cast<const uint16_t*>(src + 2 * i)))
                         << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __noinline__ void rg_store8_slow(char* dst, int n, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n)
            *reinterpret_cast<uint16_t*>(dst + 2 * i) =
                static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

// A staged tile's first `rows` rows and `cols` columns to a C whose rows start anywhere:
// row by row, one element per lane (64 contiguous bytes; as eight stores of two bytes
// for each 16-byte piece, 64 groups of 521 x 1001 took 160 us, now 76).
__device__ __noinline__ void rg_put_rows(const RgParams& p, const uint8_t* tile, int64_t off,
                                         int rows, int cols, int lane) {
    if (lane >= cols) return;
    uint16_t* dst = static_cast<uint16_t*>(p.C) + off + lane;
#pragma unroll 8
    for (int c = 0; c < rows; ++c)
        if (rg_span_ok(p, off + c * p.ldc + lane, 1))
            dst[c * p.ldc] = *reinterpret_cast<const uint16_t*>(tile + rg_at(c, lane >> 3) +
                                                                (lane & 7) * 2);
}

__device__ __noinline__ float rg_gelu_erf(float x) { return gelu_erf(x); }

// The activation over 32 values.
__device__ __forceinline__ void rg_act(float (&v)[32], int act) {
    if (act == ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = gelu_tanh(v[i]);
    } else if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = relu(v[i]);
    } else if (act == ACT_GELU_ERF) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = rg_gelu_erf(v[i]);
    }
}

// Elements off .. off + 7 of Cin, of which `n` exist (16-bit types); through L2: in
// a sequence of products other SMs wrote Cin in the same launch.
// PAD: rows are padded to whole 16 bytes on 16-byte boundaries (RG_SYM's buffers).
template <bool PAD>
__device__ __forceinline__ uint4 rg_load8(const RgParams& p, int64_t off, int n) {
    const char* src = static_cast<const char*>(p.Cin) + off * 2;
    if (PAD || (p.c_vec && n >= 8)) return __ldcg(reinterpret_cast<const uint4*>(src));
    return rg_load8_slow(src, n);
}

template <bool PAD>
__device__ __forceinline__ void rg_store8(const RgParams& p, int64_t off, int n, uint4 v) {
    if (!rg_span_ok(p, off, n < 8 ? n : 8)) return;
    char* dst = static_cast<char*>(p.C) + off * 2;
    if (PAD || (p.c_vec && n >= 8))
        *reinterpret_cast<uint4*>(dst) = v;
    else
        rg_store8_slow(dst, n, v);
}

// A chunk's accumulators (two 16-lane loads of 32 columns) to values:
// [16-lane half][8-column block][2 lanes x 2 columns], bias by lane.
__device__ __forceinline__ void rg_values(const RgParams& p, const uint32_t (&r)[32],
                                          const float (&bias)[4], float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = fmaf(p.alpha, __uint_as_float(r[i]), bias[(i >> 4) * 2 + ((i >> 1) & 1)]);
}

// Values to packed 16-bit pairs, pk[column block][8-lane part].
__device__ __forceinline__ void rg_pack16(int dt, const float (&v)[32], uint32_t (&pk)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float* x = v + 16 * (m >> 1) + 4 * i + 2 * (m & 1);
            pk[i][m] = rg_pack(dt, x[0], x[1]);
        }
}

// Epilogue of a warp's 32 lanes (output columns nl0 ..) of tile w for a 16-bit
// C: the 32-column chunks half, half + 2, ...  `ready` waits for the accumulator
// (false: gave up); `release` runs once it has been read.
template <int FORM, bool ACT, typename Ready, typename Release>
__device__ __forceinline__ void rg_out16(const RgParams& p, const RgTile& w, uint32_t tmem_row,
                                         int nl0, int half, int lane, uint8_t* buf, bool empty,
                                         Ready ready, Release release) {
    const int64_t c_base = w.group * p.stride_c + nl0;
    const int64_t in_base = w.group * p.stride_cin + nl0;
    const bool beta = p.beta != 0.0f;
    const int pcol = lane >> 2, part = lane & 3;  // this lane's 16 bytes of a staged tile
    const int nn = p.n_lane - nl0 - 8 * part;     // of which this many columns exist
    // (RG_WGRAD has one staged tile, which Cin and the output share)
    constexpr uint32_t IN = FORM == RG_WGRAD ? 0u : 2048u;
    const uint32_t s_out = smem_u32(buf), s_in = s_out + IN;
    const uint32_t mat = rg_at(lane & 7, lane >> 3);  // this lane's row of a transposed store
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = nl0 + 8 * i + pcol;
        bias[i] = p.bias && n < p.n_lane ? __ldg(p.bias + w.group * p.stride_bias + n) : 0.0f;
    }
    uint4 cin[4];
    auto load_in = [&](int c0) {
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int c = c0 + 8 * it + pcol;
            cin[it] = c < w.ncols && nn > 0
                          ? rg_load8<FORM == RG_SYM>(p, in_base + (w.out_row + c) * p.ldcin + 8 * part, nn)
                          : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_acc = [&](int c0, uint32_t (&r)[32]) {
        if (empty) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
        } else {
            tmem_ld_16x256_x4(tmem_row + static_cast<uint32_t>(c0), r, 0);
            tmem_ld_16x256_x4(tmem_row + (16u << 16) + static_cast<uint32_t>(c0), r, 1);
        }
    };
    // a staged tile's four 16-byte parts of this lane, to rows c0 .. of C
    auto store_tile = [&](int c0, uint32_t tile) {
        if (FORM != RG_SYM && !p.c_vec) {
            rg_put_rows(p, buf + tile, c_base + (w.out_row + c0) * p.ldc,
                        w.ncols - c0 < 32 ? w.ncols - c0 : 32, p.n_lane - nl0, lane);
            return;
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int c = c0 + 8 * it + pcol;
            if (c < w.ncols && nn > 0)
                rg_store8<FORM == RG_SYM>(p, c_base + (w.out_row + c) * p.ldc + 8 * part, nn,
                          *reinterpret_cast<const uint4*>(buf + tile + rg_at(8 * it + pcol, part)));
        }
    };
    const bool tma = FORM == RG_WGRAD && p.c_tma;
    const int first = half * 32;
    if (first >= w.ncols || nl0 >= p.n_lane) {
        if (ready()) release();
        return;
    }
    if (FORM == RG_ROWS && !beta) {
        // two chunks at a time, one in each staged tile
        if (!ready()) return;
#pragma unroll 1
        for (int c0 = first; c0 < w.ncols; c0 += 128) {
            const bool two = c0 + 64 < w.ncols;
            uint32_t r0[32], r1[32], pk[4][4];
            float v[32];
            load_acc(c0, r0);
            if (two) load_acc(c0 + 64, r1);
            if (!empty) tmem_ld_wait2(r0, r1);
            if (c0 + 128 >= w.ncols) release();
            __syncwarp();  // the previous chunks have left the staged tiles
            rg_values(p, r0, bias, v);
            if (ACT) rg_act(v, p.act);
            rg_pack16(p.c_dtype, v, pk);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                stmatrix_x4_trans(s_out + mat + 512u * i, pk[i][0], pk[i][1], pk[i][2], pk[i][3]);
            if (two) {
                rg_values(p, r1, bias, v);
                if (ACT) rg_act(v, p.act);
                rg_pack16(p.c_dtype, v, pk);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    stmatrix_x4_trans(s_in + mat + 512u * i, pk[i][0], pk[i][1], pk[i][2],
                                      pk[i][3]);
            }
            __syncwarp();
            store_tile(c0, 0u);
            if (two) store_tile(c0 + 64, 2048u);
        }
        return;
    }
    // (RG_SYM: Cin comes from the product before, which is known to be complete only here)
    if (FORM == RG_SYM && !ready()) return;
    // RG_SYM: the chunk of this warp on the diagonal, if any, and what its rounding lost
    const int c_diag = FORM == RG_SYM && w.diag ? nl0 - w.col0 : -1;
    float* resid = FORM == RG_SYM && p.resid ? p.resid + w.group * p.stride_resid + nl0 + pcol : nullptr;
    float lost[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (FORM == RG_SYM && p.resid_in && resid && w.diag) {
#pragma unroll
        for (int hg = 0; hg < 4; ++hg)
            if (nl0 + 8 * hg + pcol < p.n_lane) lost[hg] = __ldcg(resid + 8 * hg);
    }
    if (beta) load_in(first);
    if (FORM != RG_SYM && !ready()) return;
#pragma unroll 1
    for (int c0 = first; c0 < w.ncols; c0 += 64) {
        uint32_t r[32], pk[4][4];
        float v[32];
        load_acc(c0, r);
        if (!empty) tmem_ld_wait(r);
        const bool more = c0 + 64 < w.ncols;
        if (!more) release();
        rg_values(p, r, bias, v);
        // the previous chunk has left the staged tiles
        if (tma && lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        if (beta) {
#pragma unroll
            for (int it = 0; it < 4; ++it)
                *reinterpret_cast<uint4*>(buf + IN + rg_at(8 * it + pcol, part)) = cin[it];
            if (more) load_in(c0 + 64);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t u[4];
                ldmatrix_x4_trans(s_in + mat + 512u * i, u[0], u[1], u[2], u[3]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 f = rg_unpack(p.cin_dtype, u[m]);
                    float* x = v + 16 * (m >> 1) + 4 * i + 2 * (m & 1);
                    x[0] = fmaf(p.beta, f.x, x[0]);
                    x[1] = fmaf(p.beta, f.y, x[1]);
                }
            }
            if (FORM != RG_ROWS) __syncwarp();  // (Cin's place is written again)
        }
        if (FORM == RG_SYM && c0 == c_diag && pcol >> 1 == part) {
            // a 32 x 32 block on the diagonal: lane 16 h + 8 g + pcol, column 8 b + 2 part + k
#pragma unroll
            for (int hg = 0; hg < 4; ++hg) {
                const int i = 16 * (hg >> 1) + 4 * hg + 2 * (hg & 1);
                float y = (pcol & 1 ? v[i + 1] : v[i]) + p.diag;
                if (p.resid_in) y = fmaf(p.alpha, lost[hg], y);
                v[i] = pcol & 1 ? v[i] : y;
                v[i + 1] = pcol & 1 ? y : v[i + 1];
                if (resid && !p.resid_in && nl0 + 8 * hg + pcol < p.n_lane) {
                    const float h = __half2float(__float2half_rn(y));
                    resid[8 * hg] = 2.0f * h * (y - h);
                }
            }
        }
        if (ACT) rg_act(v, p.act);
        rg_pack16(p.c_dtype, v, pk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            stmatrix_x4_trans(s_out + mat + 512u * i, pk[i][0], pk[i][1], pk[i][2], pk[i][3]);
            // the mirrored tile: lanes as rows (an off-diagonal tile's columns all exist)
            if (FORM == RG_SYM && !w.diag)
                stmatrix_x4(s_in + rg_at(lane, i), pk[i][0], pk[i][1], pk[i][2], pk[i][3]);
        }
        if (tma) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(&p.tmap_c, s_out, nl0, w.out_row + c0, w.group, l2_policy_evict_normal());
                bulk_commit_group();
            }
            continue;
        }
        __syncwarp();
        store_tile(c0, 0u);
        if (FORM == RG_SYM && !w.diag) {
#pragma unroll
            for (int it = 0; it < 4; ++it)
                if (nl0 + 8 * it + pcol < p.n_lane)
                    rg_store8<FORM == RG_SYM>(p, w.group * p.stride_c + (nl0 + 8 * it + pcol) * p.ldc + w.col0 +
                                     c0 + 8 * part,
                              8, *reinterpret_cast<const uint4*>(buf + 2048 +
                                                                 rg_at(8 * it + pcol, part)));
        }
    }
}

// Columns c0 .. c0 + 31 of an fp32 C from their sums v: one lane (output column) per
// thread, stores of 32 neighbouring columns of one row (RG_WGRAD: TMA boxes of 16 rows by
// 32 columns).  MORE: with beta * C or an activation.
template <int FORM, bool MORE>
__device__ __forceinline__ void rg_out32(const RgParams& p, const RgTile& w, int nl0, int c0,
                                         float bias, int lane, uint8_t* buf,
                                         const uint32_t (&v)[32]) {
    const int n = nl0 + lane;
    const bool in = n < p.n_lane;
    float o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = fmaf(p.alpha, __uint_as_float(v[i]), bias);
    const int64_t row = w.out_row + c0;
    if (MORE && p.beta != 0.0f && in) {
        const float* src = static_cast<const float*>(p.Cin) + w.group * p.stride_cin +
                           row * p.ldcin + n;
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = c0 + i < w.ncols ? src[i * p.ldcin] : 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = fmaf(p.beta, f[i], o[i]);
    }
    if (MORE && FORM == RG_ROWS) rg_act(o, p.act);
    if (FORM == RG_WGRAD && p.c_tma) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (c0 + 16 * h >= w.ncols) break;
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                *reinterpret_cast<float*>(buf + i * 128 + lane * 4) = o[16 * h + i];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(&p.tmap_c, smem_u32(buf), nl0, w.out_row + c0 + 16 * h, w.group,
                             l2_policy_evict_normal());
                bulk_commit_group();
            }
        }
        return;
    }
    if (!in) return;
    const int64_t off = w.group * p.stride_c + row * p.ldc + n;
    float* dst = static_cast<float*>(p.C) + off;
    const int left = w.ncols - c0;
    if (left >= 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (rg_span_ok(p, off + i * p.ldc, 1)) dst[i * p.ldc] = o[i];
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < left && rg_span_ok(p, off + i * p.ldc, 1)) dst[i * p.ldc] = o[i];
    }
}

// Stages of 128 of a tile's contraction (RG_WGRAD: of its whole K = 16 steps), and for an
// fp32 output the sums that it is cut into: RG_SUM stages each, the last one the rest
// and the ragged tail.
constexpr int RG_SUM = 6;

template <int FORM>
__device__ __forceinline__ int rg_stages(int klen) {
    return ((FORM == RG_WGRAD ? klen & ~15 : klen) + 127) / 128;
}

template <int FORM>
__device__ __forceinline__ int rg_sums(int klen) {
    const int stages = rg_stages<FORM>(klen);
    return klen == 0 ? 0 : stages <= RG_SUM ? 1 : (stages + RG_SUM - 1) / RG_SUM;
}

// Products that stand alone wait for nothing and tell no one.
struct RgAlone {
    __device__ bool operator()(int) const { return true; }
};

// What the roles of a CTA share.
struct RgCta {
    uint8_t* smem;
    uint32_t sA0, sB0;
    uint32_t full0, empty0, tail0, tfull0, tempty0, drain_bar;
    uint32_t tmem_base;
    volatile int* abort_flag;
    uint32_t rank;   // CTA of the pair
    bool leader;
    int cl, ncl;     // this cluster, clusters of the grid
    int lane;
};

// Where a role stands in the ring and the accumulators.
struct RgRole {
    int stage = 0;
    uint32_t phase = 0;
    uint32_t armed = 0;                    // producer: stages filled
    uint32_t tails = 0;                    // ragged ends so far
    int abuf = 0;
    uint32_t aphase = 0;
    bool issued = false, ok = true;
};

// ------------------------------------------------ TMA producer (a warp)
// Tiles first, first + clusters, ...  gate(group) runs in lane 0 before a tile's loads
// (false: gave up).
template <int CG, int BT, int FORM, typename Gate>
__device__ __forceinline__ void rg_produce(const RgParams& p, const RgCta& x, RgRole& r, int first,
                                           Gate gate) {
    using C = RgCfg<CG, BT>;
    const uint64_t pol = l2_policy_evict_normal();
    RgWalk walk = rg_begin<FORM>(p, x.lane);
    RgTile w;
    if (p.pdl) griddep_wait();
    for (int t = first; r.ok && rg_tile<CG, BT, FORM>(p, walk, t, x.lane, x.rank, w); t += x.ncl) {
        // As in the MMA warp, the whole warp walks the stages and one lane issues.
        w.group = rg_uniform(w.group);
        w.lane0 = rg_uniform(w.lane0);
        w.n_mma = rg_uniform(w.n_mma);
        w.b_row = rg_uniform(w.b_row);
        w.k0 = rg_uniform(w.k0);
        w.klen = rg_uniform(w.klen);
        const int rows_b = w.n_mma / CG;  // column rows of this CTA
        const int b_row = w.b_row + static_cast<int>(x.rank) * rows_b;
        const int za = p.a_z ? w.group : 0, zb = p.b_z ? w.group : 0;
        const bool a_mn = p.a_mn, b_mn = p.b_mn, a_k4 = p.a_k4, b_k4 = p.b_k4;
        // K-major columns: whole-tile boxes, or 32-row boxes where those are fewer bytes
        // (one load a block costs as much issue time as bytes: half a tile suffices there)
        const bool big = !b_mn && 4 * rows_b > 3 * C::B_ROWS;
        const int nb = b_mn ? rows_b / 64 : (big ? 1 : (rows_b + 31) / 32);
        const uint32_t b_bytes = b_mn ? nb * 16384u : (big ? C::B_BYTES : nb * 8192u);
        const CUtensorMap* map_b = big || b_mn ? &p.tmap_b : &p.tmap_b32;
        const uint32_t bytes = C::A_BYTES + b_bytes;
        // (RG_WGRAD: whole K = 16 steps; the tail warp loads the rest)
        const int ksteps = rg_stages<FORM>(w.klen);
        if constexpr (!std::is_same<Gate, RgAlone>::value) {
            int open = 1;
            if (x.lane == 0) open = gate(w.group) ? 1 : 0;
            r.ok = __all_sync(0xffffffffu, open) != 0;
        }
        for (int ks = 0; r.ok && ks < ksteps; ++ks) {
            r.ok = rg_all_wait(x.empty0 + 8u * r.stage, r.phase ^ 1u, p, x.abort_flag);
            if (p.test_stall == 1 && r.armed == 0)
                r.ok = false;  // test only: the MMA warp's bounded wait must expire
            if (!r.ok) break;
            const uint32_t fb = x.full0 + 8u * r.stage;
            const uint32_t bar = CG == 1 || x.leader ? fb : mapa_shared(fb, 0u);
            const uint32_t a_dst = x.sA0 + r.stage * C::A_BYTES;
            const uint32_t b_dst = x.sB0 + r.stage * C::B_BYTES;
            const int k = w.k0 + ks * 128;
            if (x.lane == 0) {
                if (x.leader) mbar_arrive_expect_tx(fb, CG * bytes);
                auto load = [&](uint32_t dst, const CUtensorMap* map, int cx, int cy, int cz) {
                    if constexpr (CG == 2)
                        tma_load_3d_pair(dst, map, bar, cx, cy, cz, pol);
                    else
                        tma_load_3d(dst, map, bar, cx, cy, cz, pol);
                };
                // K-major: the second block's rows follow the first's; MN-major:
                // 64-wide atom columns of 128 K rows (16 KB)
                if (a_k4) {
                    tma_load_4d_cg<CG>(a_dst, &p.tmap_a, bar, 0, w.lane0, 2 * ks, za, pol);
                } else if (a_mn) {
                    load(a_dst, &p.tmap_a, w.lane0, k, za);
                    load(a_dst + 16384u, &p.tmap_a, w.lane0 + 64, k, za);
                } else {
                    load(a_dst, &p.tmap_a, k, w.lane0, za);
                    load(a_dst + 16384u, &p.tmap_a, k + 64, w.lane0, za);
                }
                if (b_mn) {
                    for (int h = 0; h < nb; ++h)
                        load(b_dst + 16384u * h, map_b, b_row + 64 * h, k, zb);
                } else if (big) {
                    if (b_k4) {
                        tma_load_4d_cg<CG>(b_dst, map_b, bar, 0, b_row, 2 * ks, zb, pol);
                    } else {
                        load(b_dst, map_b, k, b_row, zb);
                        load(b_dst + C::B_BYTES / 2, map_b, k + 64, b_row, zb);
                    }
                } else {
                    // (32-row boxes one block at a time: the blocks lie B_BYTES / 2 apart)
                    for (int h = 0; h < nb; ++h) {
                        load(b_dst + 4096u * h, map_b, k, b_row + 32 * h, zb);
                        load(b_dst + C::B_BYTES / 2 + 4096u * h, map_b, k + 64, b_row + 32 * h, zb);
                    }
                }
            }
            ++r.armed;
            if (++r.stage == C::STAGES) {
                r.stage = 0;
                r.phase ^= 1u;
            }
        }
        r.ok = __all_sync(0xffffffffu, r.ok) != 0;
    }
}

// Every issued copy lands before the CTA exits.  A pair's peer completes its
// copies on the leader's barriers: after a normal run the leader has consumed
// them before the final cluster barrier; after an abort the peer gives them a
// fixed time.
template <int CG, int BT>
__device__ __forceinline__ void rg_produce_end(const RgParams& p, const RgCta& x, const RgRole& r) {
    using C = RgCfg<CG, BT>;
    if (x.lane != 0) return;
    if (CG == 2 && !x.leader) {
        if (!r.ok) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000ull) {
            }
        }
    } else {
        for (int s = 0; s < C::STAGES && static_cast<uint32_t>(s) < r.armed; ++s) {
            const uint32_t fills = (r.armed - 1u - s) / C::STAGES + 1u;
            rg_drain(x.full0 + 8u * s, (fills - 1u) & 1u, p.timeout_ns);
        }
    }
}

// ------------------------------------------------ MMA issuer (a warp)
// (nothing to do in the pair's peer)
template <int CG, int BT, int FORM, bool SUM = false>
__device__ __forceinline__ void rg_issue(const RgParams& p, const RgCta& x, RgRole& r, int first) {
    using C = RgCfg<CG, BT>;
    constexpr uint16_t kPair = 3u;
    const bool a_mn = p.a_mn != 0, b_mn = p.b_mn != 0;
    // descriptors of stage 0; a stage or K = 16 step adds to their address fields
    // (in 16 bytes; K-major: 32 bytes a step inside a block, MN-major: 16 rows)
    const uint64_t a_desc0 = smem_desc_sw128(x.sA0, a_mn ? 16384u : 16u, 1024u);
    const uint64_t b_desc0 = smem_desc_sw128(x.sB0, b_mn ? 16384u : 16u, 1024u);
    const uint32_t a_step = a_mn ? 128u : 2u, b_step = b_mn ? 128u : 2u;
    const uint32_t a_block = a_mn ? 512u : C::A_BYTES >> 5, b_block = b_mn ? 512u : C::B_BYTES >> 5;
    if (CG == 2 && !x.leader) return;
    RgWalk walk = rg_begin<FORM>(p, x.lane);
    RgTile w;
    for (int t = first; r.ok && rg_tile<CG, BT, FORM>(p, walk, t, x.lane, x.rank, w); t += x.ncl) {
        if (w.klen == 0) continue;  // no rows: the epilogue writes zeros
        w.klen = rg_uniform(w.klen);
        w.n_mma = rg_uniform(w.n_mma);
        const bool tail = FORM == RG_WGRAD && (w.klen & 15) != 0;
        const int klen = FORM == RG_WGRAD ? w.klen & ~15 : w.klen;
        const int ksteps = rg_stages<FORM>(w.klen);
        const uint32_t tmem0 = static_cast<uint32_t>(rg_uniform(static_cast<int>(x.tmem_base)));
        uint32_t d_tmem = 0;
        const uint32_t idesc = p.idesc | (static_cast<uint32_t>(w.n_mma >> 3) << 17);
        // `fresh`: the first stage of a sum; `last`: the accumulator goes to the epilogue
        auto issue = [&](bool fresh, bool last, int steps) {
            const uint64_t ad = a_desc0 + static_cast<uint32_t>(r.stage) * (C::A_BYTES >> 4);
            const uint64_t bd = b_desc0 + static_cast<uint32_t>(r.stage) * (C::B_BYTES >> 4);
            const uint32_t empty = x.empty0 + 8u * r.stage;
            if (x.lane == 0) {
                if (steps == 8) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        umma_f16_cg<CG>(d_tmem, ad + (k >> 2) * a_block + (k & 3) * a_step,
                                        bd + (k >> 2) * b_block + (k & 3) * b_step, idesc,
                                        (!fresh || k > 0) ? 1u : 0u);
                } else {
                    for (int k = 0; k < steps; ++k)
                        umma_f16_cg<CG>(d_tmem, ad + (k >> 2) * a_block + (k & 3) * a_step,
                                        bd + (k >> 2) * b_block + (k & 3) * b_step, idesc,
                                        (!fresh || k > 0) ? 1u : 0u);
                }
                if constexpr (CG > 1)
                    umma_commit_mc_cg<CG>(empty, kPair);
                else
                    umma_commit_cg<CG>(empty);
                if (last) {
                    if constexpr (CG > 1)
                        umma_commit_mc_cg<CG>(x.tfull0 + 8u * r.abuf, kPair);
                    else
                        umma_commit_cg<CG>(x.tfull0 + 8u * r.abuf);
                }
            }
        };
        // The whole warp walks the stages and one lane issues, so that the stage's
        // addresses stay in uniform registers (16384 x 4096 x 2048: 174 -> 154 us; one
        // lane alone took as long to issue eight MMAs as they take to run).
        auto open = [&]() {
            d_tmem = tmem0 + static_cast<uint32_t>(r.abuf * BT);
            r.ok = rg_all_wait(x.tempty0 + 8u * r.abuf, r.aphase ^ 1u, p, x.abort_flag);
            if (r.ok) tc_fence_after_sync();
        };
        auto close = [&]() {
            if (++r.abuf == 2) {
                r.abuf = 0;
                r.aphase ^= 1u;
            }
        };
        open();
        for (int ks = 0; r.ok && ks < ksteps; ++ks) {
            const bool fresh = SUM ? ks % RG_SUM == 0 : ks == 0;
            if (SUM && fresh && ks > 0) {
                close();
                open();
                if (!r.ok) break;
            }
            r.ok = rg_all_wait(x.full0 + 8u * r.stage, r.phase, p, x.abort_flag);
            if (!r.ok) break;
            tc_fence_after_sync();
            const int left = klen - ks * 128;
            issue(fresh, ks == ksteps - 1 ? !tail : SUM && ks % RG_SUM == RG_SUM - 1,
                  left >= 128 ? 8 : (left + 15) / 16);
            r.issued = true;
            if (++r.stage == C::STAGES) {
                r.stage = 0;
                r.phase ^= 1u;
            }
        }
        if (FORM == RG_WGRAD && tail && r.ok) {
            const uint32_t b = r.tails & 1u;
            r.ok = rg_all_wait(x.tail0 + 16u + 8u * b, r.tails >> 1 & 1u, p, x.abort_flag);
            ++r.tails;
            if (r.ok) {
                fence_proxy_async_smem();
                tc_fence_after_sync();
                // 64-wide atom columns of 16 rows (2 KB)
                const uint32_t at = x.sA0 + C::STAGES * C::STAGE_BYTES + C::TAIL_AT + b * C::TAIL_BYTES;
                const uint64_t ad = smem_desc_sw128(at, 2048u, 1024u);
                const uint64_t bd = smem_desc_sw128(at + C::TAIL_A, 2048u, 1024u);
                if (x.lane == 0) {
                    umma_f16_cg<CG>(d_tmem, ad, bd, idesc, ksteps > 0 ? 1u : 0u);
                    if constexpr (CG > 1) {
                        umma_commit_mc_cg<CG>(x.tail0 + 32u + 8u * b, kPair);
                        umma_commit_mc_cg<CG>(x.tfull0 + 8u * r.abuf, kPair);
                    } else {
                        umma_commit_cg<CG>(x.tail0 + 32u + 8u * b);
                        umma_commit_cg<CG>(x.tfull0 + 8u * r.abuf);
                    }
                }
                r.issued = true;
            }
        }
        close();
        r.ok = __all_sync(0xffffffffu, r.ok) != 0;
    }
}

// ------------------------------------------------ ragged tails (a warp, RG_WGRAD)
// Loads the 16 rows that a group's last, partial K = 16 step reads into one of two
// buffers, overwrites the rows past the group's end with zeros, and hands them to
// the MMA warp of the leader, up to two tiles ahead.  (Zeroing inside the ring's
// last stage made every ragged tile wait for its own loads: 247 us against 197 for
// 16 groups of 1021 and of 1024 rows.)
template <int CG, int BT>
__device__ __forceinline__ void rg_tails(const RgParams& p, const RgCta& x, RgRole& r) {
    using C = RgCfg<CG, BT>;
    const uint64_t pol = l2_policy_evict_normal();
    RgWalk walk = rg_begin<RG_WGRAD>(p, x.lane);
    RgTile w;
    if (p.pdl) griddep_wait();
    for (int t = x.cl; rg_tile<CG, BT, RG_WGRAD>(p, walk, t, x.lane, x.rank, w); t += x.ncl) {
        const int v = w.klen & 15;  // valid rows
        if (v == 0) continue;
        const uint32_t b = r.tails & 1u, turn = r.tails >> 1 & 1u;
        ++r.tails;
        const uint32_t loaded = x.tail0 + 8u * b, ready = x.tail0 + 16u + 8u * b;
        if (!rg_warp_wait(x.tail0 + 32u + 8u * b, turn ^ 1u, x.lane, x.abort_flag, p)) return;
        uint8_t* buf = x.smem + C::STAGES * C::STAGE_BYTES + C::TAIL_AT + b * C::TAIL_BYTES;
        const uint32_t dst = smem_u32(buf);
        const int rows_b = w.n_mma / CG, nb = rows_b / 64;
        const int b_row = w.b_row + static_cast<int>(x.rank) * rows_b;
        if (x.lane == 0) {
            const int k = w.k0 + (w.klen & ~15);
            mbar_arrive_expect_tx(loaded, (2 + nb) * 2048u);
            tma_load_3d(dst, &p.tmap_a16, loaded, w.lane0, k, 0, pol);
            tma_load_3d(dst + 2048u, &p.tmap_a16, loaded, w.lane0 + 64, k, 0, pol);
            for (int h = 0; h < nb; ++h)
                tma_load_3d(dst + C::TAIL_A + 2048u * h, &p.tmap_b32, loaded, b_row + 64 * h, k, 0,
                            pol);
        }
        __syncwarp();
        // (gives up only after its copies have had their time to land)
        if (!rg_warp_wait(loaded, turn, x.lane, x.abort_flag, p)) {
            if (x.lane == 0) rg_drain(loaded, turn, p.timeout_ns);
            return;
        }
        __syncwarp();
        // rows v .. 15: one row is 128 bytes of every 64-wide atom column (whole
        // rows, so the swizzle inside them does not matter)
        for (int i = x.lane; i < (2 + nb) * 128; i += 32) {
            const int row = i >> 3 & 15;
            if (row >= v)
                *reinterpret_cast<uint4*>(buf + (i >> 7) * 2048 + row * 128 + (i & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (x.lane == 0) {
            if (CG == 2 && !x.leader)
                mbar_arrive_remote(mapa_shared(ready, 0u));
            else
                mbar_arrive(ready);
        }
    }
}

// All MMAs complete before tensor memory is released.
template <int CG>
__device__ __forceinline__ void rg_issue_end(const RgParams& p, const RgCta& x, const RgRole& r) {
    if (r.issued && x.lane == 0) {
        umma_commit_cg<CG>(x.drain_bar);
        rg_drain(x.drain_bar, 0u, p.timeout_ns);
    }
    __syncwarp();
}

// ------------------------------------------------ epilogue (a warp of eight)
// told(group) runs in the whole warp after its part of a tile has been stored; r.ok goes
// false when a wait gave up.
template <int CG, int BT, int FORM, bool ACT, typename Told>
__device__ __forceinline__ void rg_epilogue(const RgParams& p, const RgCta& x, RgRole& r, int first,
                                            int warp, uint8_t* buf, Told told) {
    const int q = warp & 3;            // tensor-memory lane quarter of this warp
    const int half = (warp - 2) >> 2;  // which 32-column chunks it takes
    const uint32_t lane_field = static_cast<uint32_t>(q * 32) << 16;
    RgWalk walk = rg_begin<FORM>(p, x.lane);
    RgTile w;
    for (int t = first; rg_tile<CG, BT, FORM>(p, walk, t, x.lane, x.rank, w); t += x.ncl) {
        const bool empty = w.klen == 0;
        const int nl0 = w.lane0 + q * 32;  // first output column of this warp
        auto ready = [&]() {
            if (empty) return true;
            r.ok = rg_warp_wait(x.tfull0 + 8u * r.abuf, r.aphase, x.lane, x.abort_flag, p);
            tc_fence_after_sync();
            return r.ok;
        };
        const uint32_t tmem_row = x.tmem_base + lane_field + static_cast<uint32_t>(r.abuf * BT);
        // the accumulator goes back to the MMA warp as soon as it is in registers
        auto release = [&]() {
            if (empty) return;
            tc_fence_before_sync();
            __syncwarp();
            if (x.lane == 0)
                mbar_arrive_relaxed(mapa_shared(x.tempty0 + 8u * r.abuf, 0u));
        };
        rg_out16<FORM, ACT>(p, w, tmem_row, nl0, half, x.lane, buf, empty, ready, release);
        if (!r.ok) break;
        told(w.group);
        if (!empty && ++r.abuf == 2) {
            r.abuf = 0;
            r.aphase ^= 1u;
        }
    }
    if (FORM == RG_WGRAD && x.lane == 0) bulk_wait_group_all();  // the staged tiles have been read
    __syncwarp();
}

// The same for an fp32 output (warps 4 to 11).  The tensor core cuts off what an addition
// leaves below its accumulator's 24 bits, always towards zero, so that the error grows
// with the length of the sum (2.1e-6 of the result for 2048 products, 1.9e-5 for 16384).
// Here an accumulator takes RG_SUM stages (768 products) and the epilogue adds it to sums
// in its registers, rounding to nearest, while the MMAs go on in the other one: 7e-7 at
// any length.  It costs 192 -> 197 us for the weight gradient of 16384 rows over 16
// groups, 2048 x 4096, and nothing measurable for row products; stages of 4 (4.7e-7) and
// 8 (1.0e-6) took 199 and 195 us.
template <int CG, int BT, int FORM>
__device__ __forceinline__ void rg_epilogue_sum(const RgParams& p, const RgCta& x, RgRole& r,
                                                int first, int warp, uint8_t* buf) {
    constexpr int NC = BT < 64 ? 1 : BT / 64;  // 32-column chunks of a warp
    const int q = warp & 3;                    // tensor-memory lane quarter of this warp
    const int c_first = ((warp - 4) >> 2) * 32;
    const uint32_t tmem_row = x.tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                              static_cast<uint32_t>(c_first);
    RgWalk walk = rg_begin<FORM>(p, x.lane);
    RgTile w;
    for (int t = first; rg_tile<CG, BT, FORM>(p, walk, t, x.lane, x.rank, w); t += x.ncl) {
        const int nl0 = w.lane0 + q * 32;  // first output column of this warp
        const bool mine = c_first < w.ncols && nl0 < p.n_lane;
        const int sums = rg_sums<FORM>(w.klen);
        uint32_t v[NC][32];                // (bits of the fp32 sums)
        if (sums == 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[c][i] = 0u;
        }
#pragma unroll 1
        for (int s = 0; s < sums; ++s) {
            r.ok = rg_warp_wait(x.tfull0 + 8u * r.abuf, r.aphase, x.lane, x.abort_flag, p);
            if (!r.ok) break;
            tc_fence_after_sync();
            const uint32_t from = tmem_row + static_cast<uint32_t>(r.abuf * BT);
            if (mine && s == 0) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (c_first + 64 * c < w.ncols) tmem_ld_x32(from + 64u * c, v[c]);
#pragma unroll
                for (int c = 0; c < NC; ++c) tmem_ld_wait(v[c]);
            } else if (mine) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (c_first + 64 * c < w.ncols) {
                        uint32_t u[32];
                        tmem_ld_x32(from + 64u * c, u);
                        tmem_ld_wait(u);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[c][i] = __float_as_uint(__uint_as_float(v[c][i]) + __uint_as_float(u[i]));
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (x.lane == 0) mbar_arrive_relaxed(mapa_shared(x.tempty0 + 8u * r.abuf, 0u));
            if (++r.abuf == 2) {
                r.abuf = 0;
                r.aphase ^= 1u;
            }
        }
        if (!r.ok) break;
        if (mine) {
            const int n = nl0 + x.lane;
            const float bias =
                p.bias && n < p.n_lane ? __ldg(p.bias + w.group * p.stride_bias + n) : 0.0f;
            if (p.beta != 0.0f || p.act != ACT_NONE) {
                // (one copy of this code, which takes registers of its own: the next chunk
                // moves to the front)
#pragma unroll 1
                for (int c0 = c_first; c0 < w.ncols; c0 += 64) {
                    rg_out32<FORM, true>(p, w, nl0, c0, bias, x.lane, buf, v[0]);
#pragma unroll
                    for (int c = 0; c + 1 < NC; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[c][i] = v[c + 1][i];
                }
            } else {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (c_first + 64 * c < w.ncols)
                        rg_out32<FORM, false>(p, w, nl0, c_first + 64 * c, bias, x.lane, buf, v[c]);
            }
        }
        __syncwarp();
    }
    if (FORM == RG_WGRAD && x.lane == 0) bulk_wait_group_all();  // the staged tiles have been read
    __syncwarp();
}

// Barriers, tensor memory and the CTA's view of them (all threads).
template <int CG, int BT>
__device__ __forceinline__ RgCta rg_setup(const RgParams& p, uint8_t* smem_raw) {
    using C = RgCfg<CG, BT>;
    RgCta x;
    x.rank = CG > 1 ? cluster_ctarank() : 0u;
    x.leader = x.rank == 0;
    x.cl = static_cast<int>(blockIdx.x) / CG;
    x.ncl = static_cast<int>(gridDim.x) / CG;
    x.lane = threadIdx.x & 31;
    x.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                        ~static_cast<uintptr_t>(1023));
    x.sA0 = smem_u32(x.smem);
    x.sB0 = x.sA0 + C::STAGES * C::A_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(x.smem + C::STAGES * C::STAGE_BYTES + C::EPI_SMEM);
    // full[STAGES], empty[STAGES], tail_full[2], tail_ready[2], tail_empty[2],
    // tmem_full[2], tmem_empty[2], drain
    x.full0 = smem_u32(bars);
    x.empty0 = x.full0 + 8u * C::STAGES;
    x.tail0 = x.full0 + 16u * C::STAGES;
    x.tfull0 = x.tail0 + 48u;
    x.tempty0 = x.tfull0 + 16u;
    x.drain_bar = x.tempty0 + 16u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 11);
    x.abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(x.full0 + 8u * s, 1);
            mbar_init(x.empty0 + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(x.tail0 + 8u * b, 1);        // loaded (own bytes)
            mbar_init(x.tail0 + 16u + 8u * b, CG);  // zeroed, by every CTA of the pair
            mbar_init(x.tail0 + 32u + 8u * b, 1);  // read by the MMA
            mbar_init(x.tfull0 + 8u * b, 1);
            mbar_init(x.tempty0 + 8u * b, CG * C::EPI_WARPS);
        }
        mbar_init(x.drain_bar, 1);
        *x.abort_flag = 0;
        fence_mbar_init();
        if (p.maps) {
            prefetch_tmap(&p.tmap_a);
            prefetch_tmap(&p.tmap_b);
            if (p.c_tma) prefetch_tmap(&p.tmap_c);
            if (!p.b_mn) prefetch_tmap(&p.tmap_b32);
        }
    }
    if (warp == 1) {
        tmem_alloc_cg<CG>(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish_cg<CG>();
    }
    tc_fence_before_sync();
    if constexpr (CG > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after_sync();
    x.tmem_base = *tmem_slot;
    return x;
}

template <int CG, int BT>
__device__ __forceinline__ void rg_teardown(const RgCta& x) {
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG > 1) cluster_sync();
    if ((threadIdx.x >> 5) == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<CG>(x.tmem_base, RgCfg<CG, BT>::TMEM_COLS);
    }
}

// Registers of an fp32 kernel: 128 sums a thread of the epilogue's two warpgroups, for
// which the first one (producer, MMA issuer, tails) gives some of its own up.  384 threads
// are launched with at least 160 (rg_prepare checks it): 128 x 80 + 256 x 200 fit.
constexpr int RG_LAUNCH_REGS = 160, RG_FEW_REGS = 80, RG_SUM_REGS = 200;
static_assert(128 * RG_FEW_REGS + 256 * RG_SUM_REGS <= 384 * RG_LAUNCH_REGS, "register split");

// SUM: an fp32 output, with its sums cut (see rg_epilogue_sum).
template <int CG, int BT, int FORM, bool SUM>
__global__ void __launch_bounds__(RgCfg<CG, BT>::threads(FORM, SUM), 1)
    ragged_kernel(const __grid_constant__ RgParams p) {
    using C = RgCfg<CG, BT>;
    extern __shared__ uint8_t smem_raw[];
    const RgCta x = rg_setup<CG, BT>(p, smem_raw);
    const int warp = threadIdx.x >> 5;
    constexpr int EPI0 = SUM ? 4 : 2;                           // the epilogue's first warp
    constexpr int TAILS = SUM ? 2 : 2 + C::EPI_WARPS;           // RG_WGRAD
    uint8_t* buf = x.smem + C::STAGES * C::STAGE_BYTES +
                   (warp - EPI0) * (FORM == RG_WGRAD ? C::EPI_WARP / 2 : C::EPI_WARP);
    RgRole r;
    if (SUM && warp >= EPI0) {
        if (BT == 256) reg_inc<RG_SUM_REGS>();
        rg_epilogue_sum<CG, BT, FORM>(p, x, r, x.cl, warp, buf);
        rg_teardown<CG, BT>(x);
        return;
    }
    if (SUM && BT == 256) reg_dec<RG_FEW_REGS>();
    if (warp == 0) {
        rg_produce<CG, BT, FORM>(p, x, r, x.cl, RgAlone());
        rg_produce_end<CG, BT>(p, x, r);
    } else if (warp == 1) {
        rg_issue<CG, BT, FORM, SUM>(p, x, r, x.cl);
        rg_issue_end<CG>(p, x, r);
    } else if (FORM == RG_WGRAD && warp == TAILS) {
        rg_tails<CG, BT>(p, x, r);
    } else if (!SUM) {
        rg_epilogue<CG, BT, FORM, FORM == RG_ROWS>(p, x, r, x.cl, warp, buf, RgAlone());
    }
    rg_teardown<CG, BT>(x);
}

template <int CG, int BT, int FORM, bool SUM>
cudaError_t rg_launch_as(const RgParams& p, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(RgCfg<CG, BT>::threads(FORM, SUM));
    cfg.dynamicSmemBytes = RgCfg<CG, BT>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (p.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    if (CG > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = CG;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, ragged_kernel<CG, BT, FORM, SUM>, p);
}

template <int CG, int BT, int FORM>
cudaError_t rg_launch(const RgParams& p, int grid, cudaStream_t stream) {
    return p.c_dtype == DT_F32 ? rg_launch_as<CG, BT, FORM, true>(p, grid, stream)
                               : rg_launch_as<CG, BT, FORM, false>(p, grid, stream);
}

template <int CG, int BT, int FORM>
cudaError_t rg_prepare() {
    const int smem = static_cast<int>(RgCfg<CG, BT>::SMEM);
    cudaError_t e = cudaFuncSetAttribute(ragged_kernel<CG, BT, FORM, false>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ragged_kernel<CG, BT, FORM, true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    // (a wait for registers that the launch does not have would never end)
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, ragged_kernel<CG, BT, FORM, true>);
    if (e == cudaSuccess && BT == 256 && a.numRegs < RG_LAUNCH_REGS) e = cudaErrorInvalidConfiguration;
    return e;
}

}  // namespace
}  // namespace dg
