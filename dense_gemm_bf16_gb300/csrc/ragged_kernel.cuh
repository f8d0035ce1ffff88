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
//             decoding step has to read.
//   RG_WGRAD  dw_e[m, n] = sum_{t in group e} x[t, m] d[t, n].  Lanes are n,
//             columns m; the contraction is ragged.  Both operands are
//             MN-major; a group's last K = 16 step may end inside the next
//             group, whose rows (finite or not) are overwritten with zeros in
//             shared memory before the MMA reads them.
//   RG_SYM    S = X X^T (or X^T X), and b S + c S S: only tiles on or below
//             the diagonal are computed, and each is written to both places.
//
// Warps: 0 TMA producer, 1 MMA issuer (and the zeroing of ragged tails),
// 2-9 epilogue, two per tensor-memory lane quarter taking 32-column chunks in
// turn.  Two accumulators let a tile's epilogue overlap the next main loop.
// The output's contiguous dimension runs along the lanes, so a chunk goes
// through a shared-memory tile of 16 columns by 32 lanes (rows of 36 words:
// conflict-free both ways) and leaves as 16-byte stores along the lanes; rows
// of another group are masked per column.
//
// Work: tiles are dealt round robin to CTAs (pairs).  Where group sizes are on
// the device, each warp finds its tile by a 32-group window of prefix sums held
// one group per lane: no table, no extra launch, no limit on the groups.
//
// Every mbarrier wait is bounded; on expiry the kernel sets the status word,
// drains its copies and MMAs, frees tensor memory and returns.
#pragma once
#include <stdint.h>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "ragged.h"

namespace dg {
namespace {

constexpr uint32_t kRgMaxSmem = 232448;  // 227 KB opt-in limit per CTA
constexpr int RG_LD = 36;                // words per staged column

template <int CG, int BT>
struct RgCfg {
    static constexpr int B_ROWS = BT / CG;  // column-operand rows a CTA holds
    static constexpr uint32_t A_BYTES = 128 * 128;
    static constexpr uint32_t B_BYTES = B_ROWS * 128;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr uint32_t EPI_WARP = 16 * RG_LD * 4;
    static constexpr uint32_t EPI_SMEM = EPI_WARPS * EPI_WARP;
    static constexpr uint32_t BAR_BYTES = 512;
    static constexpr int FIT = (kRgMaxSmem - 1024 - BAR_BYTES - EPI_SMEM) / STAGE_BYTES;
    static constexpr int STAGES = FIT > 12 ? 12 : FIT;
    static constexpr uint32_t TMEM_COLS = 2 * BT < 32 ? 32 : 2 * BT;
    static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE_BYTES + EPI_SMEM + BAR_BYTES;
    static_assert(BT % 32 == 0 && BT <= 256 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "tile width");
    static_assert(CG == 1 || BT == 256, "pairs take 256-column tiles (two 64-wide atoms per CTA)");
    static_assert((4 * STAGES + 5) * 8 + 8 <= BAR_BYTES, "barrier area too small");
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
};

__device__ __forceinline__ void rg_bounds(const RgParams& p, int g, int& lo, int& hi) {
    lo = __ldg(p.offsets + g);
    hi = __ldg(p.offsets + g + 1);
    if (lo < 0 || hi < lo || hi > p.rows) {
        // offsets that are not ascending inside [0, rows]: reported, and
        // clamped so that no access leaves the operands
        if (p.status) atomicOr(p.status, STATUS_BAD_OFFSETS);
        lo = lo < 0 ? 0 : (lo > p.rows ? p.rows : lo);
        hi = hi < lo ? lo : (hi > p.rows ? p.rows : hi);
    }
}

__device__ __forceinline__ void rg_window(const RgParams& p, RgWalk& w, int lane) {
    const int g = w.base + lane;
    int tiles = 0;
    w.row0 = w.rows = 0;
    if (g < p.groups) {
        int lo, hi;
        rg_bounds(p, g, lo, hi);
        w.row0 = lo;
        w.rows = hi - lo;
        tiles = ((w.rows + p.col_tile - 1) / p.col_tile) * p.lane_tiles;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, tiles, d);
        if (lane >= d) tiles += o;
    }
    w.incl = tiles;
}

// Tile t of the problem, by a whole (converged) warp; false past the last one.
template <int CG, int FORM>
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
            w.before += total;
            w.base += 32;
            if (w.base >= p.groups) return false;
            rg_window(p, w, lane);
            total = __shfl_sync(0xffffffffu, w.incl, 31);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, w.incl > t - w.before);
        const int l = __ffs(m) - 1;
        const int rows = __shfl_sync(0xffffffffu, w.rows, l);
        const int row0 = __shfl_sync(0xffffffffu, w.row0, l);
        const int incl = __shfl_sync(0xffffffffu, w.incl, l);
        const int chunks = (rows + p.col_tile - 1) / p.col_tile;
        const int r = t - w.before - (incl - chunks * p.lane_tiles);
        const int lt = r / chunks;
        const int c = r - lt * chunks;
        const int width = ((rows + chunks - 1) / chunks + GRAN - 1) / GRAN * GRAN;
        o.group = w.base + l;
        o.lane0 = lt * LANES + static_cast<int>(rank) * 128;
        o.col0 = c * width;
        o.ncols = rows - o.col0 < width ? rows - o.col0 : width;
        o.b_row = o.out_row = row0 + o.col0;
    } else {
        if (t >= p.total_tiles) return false;
        const int per_group = p.total_tiles / p.groups;
        o.group = t / per_group;
        const int r = t - o.group * per_group;
        if (FORM == RG_SYM) {
            int i = static_cast<int>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
            while (i * (i + 1) / 2 > r) --i;
            while ((i + 1) * (i + 2) / 2 <= r) ++i;
            const int j = r - i * (i + 1) / 2;
            o.diag = i == j;
            o.lane0 = i * LANES + static_cast<int>(rank) * 128;
            o.col0 = j * p.col_tile;
        } else {
            const int chunks = per_group / p.lane_tiles;
            const int lt = r / chunks;
            o.lane0 = lt * LANES + static_cast<int>(rank) * 128;
            o.col0 = (r - lt * chunks) * p.col_tile;
        }
        o.ncols = p.n_col - o.col0 < p.col_tile ? p.n_col - o.col0 : p.col_tile;
        o.b_row = o.out_row = o.col0;
        if (FORM == RG_WGRAD) {
            int lo = 0, hi = 0;
            if (p.offsets) rg_bounds(p, o.group, lo, hi);  // (none: alpha == 0 or no rows)
            o.k0 = lo;
            o.klen = hi - lo;
        }
    }
    // MN-major columns come in 64-wide swizzle atoms per CTA
    const int gran = p.b_mn ? 64 * CG : GRAN;
    o.n_mma = (o.ncols + gran - 1) / gran * gran;
    return true;
}

// Bounded wait of a whole warp (one lane polls).
__device__ __forceinline__ bool rg_warp_wait(uint32_t bar, uint32_t parity, int lane,
                                             volatile int* abort_flag, const RgParams& p) {
    int ok = 1;
    if (lane == 0) ok = mbar_wait(bar, parity, abort_flag, p.status, p.timeout_ns) ? 1 : 0;
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

// NV (8 for 16-bit outputs, 4 for fp32: 16 bytes) neighbouring outputs of one
// output row, columns n .. n + NV - 1 of which those below n_lane exist.
// beta * Cin is added here unless MIRROR (RG_SYM adds it before).
template <int NV, bool MIRROR>
__device__ __forceinline__ void rg_store(const RgParams& p, int64_t off, int64_t off_in, int n,
                                         float (&v)[NV]) {
    const bool whole = p.c_vec && n + NV <= p.n_lane;
    const bool beta = !MIRROR && p.beta != 0.0f;
    constexpr int ES = NV == 8 ? 2 : 4;
    if (!rg_span_ok(p, off, n + NV <= p.n_lane ? NV : p.n_lane - n)) return;
    if (whole) {
        char* dst = static_cast<char*>(p.C) + off * ES;
        if (beta) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.Cin) + off_in * ES);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            if constexpr (NV == 8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = rg_unpack(p.cin_dtype, w[i]);
                    v[2 * i] = fmaf(p.beta, f.x, v[2 * i]);
                    v[2 * i + 1] = fmaf(p.beta, f.y, v[2 * i + 1]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = fmaf(p.beta, __uint_as_float(w[i]), v[i]);
            }
            act_inplace<NV>(v, p.act);
        }
        uint4 o;
        if constexpr (NV == 8)
            o = make_uint4(rg_pack(p.c_dtype, v[0], v[1]), rg_pack(p.c_dtype, v[2], v[3]),
                           rg_pack(p.c_dtype, v[4], v[5]), rg_pack(p.c_dtype, v[6], v[7]));
        else
            o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                           __float_as_uint(v[3]));
        *reinterpret_cast<uint4*>(dst) = o;
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (n + i >= p.n_lane) break;
        float x = v[i];
        if (beta) {
            x = fmaf(p.beta, load_elem(static_cast<const char*>(p.Cin) + (off_in + i) * ES, p.cin_dtype), x);
            x = apply_act(x, p.act);
        }
        store_elem(static_cast<char*>(p.C) + (off + i) * ES, p.c_dtype, x);
    }
}

template <int CG, int BT, int FORM>
__global__ void __launch_bounds__(RgCfg<CG, BT>::THREADS, 1)
    ragged_kernel(const __grid_constant__ RgParams p) {
    using C = RgCfg<CG, BT>;
    constexpr uint16_t kPair = 3u;
    const uint32_t rank = CG > 1 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int cl = static_cast<int>(blockIdx.x) / CG;
    const int ncl = static_cast<int>(gridDim.x) / CG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sA0 = smem_u32(smem);
    const uint32_t sB0 = sA0 + C::STAGES * C::A_BYTES;
    uint8_t* epi_smem = smem + C::STAGES * C::STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(epi_smem + C::EPI_SMEM);
    // full[STAGES], empty[STAGES], tail[STAGES], peer_tail[STAGES], tmem_full[2],
    // tmem_empty[2], drain
    const uint32_t full0 = smem_u32(bars);
    const uint32_t empty0 = full0 + 8u * C::STAGES;
    const uint32_t tail0 = full0 + 16u * C::STAGES;
    const uint32_t peer_tail0 = full0 + 24u * C::STAGES;
    const uint32_t tfull0 = full0 + 32u * C::STAGES;
    const uint32_t tempty0 = tfull0 + 16u;
    const uint32_t drain_bar = tempty0 + 16u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * C::STAGES + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8u * s, 1);
            mbar_init(empty0 + 8u * s, 1);
            mbar_init(tail0 + 8u * s, 1);
            mbar_init(peer_tail0 + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8u * b, 1);
            mbar_init(tempty0 + 8u * b, CG * C::EPI_WARPS);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (p.maps) {
            prefetch_tmap(&p.tmap_a);
            prefetch_tmap(&p.tmap_b);
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
    const uint32_t tmem_base = *tmem_slot;
    if (p.pdl) {
        griddep_launch_dependents();
        griddep_wait();
        fence_proxy_async_global();  // the previous grid's plain stores, read by TMA below
    }

    RgWalk walk{0, 0, 0, 0, 0};
    if (FORM == RG_ROWS && p.offsets) rg_window(p, walk, lane);
    RgTile w;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        const uint64_t pol = l2_policy_evict_normal();
        int stage = 0;
        uint32_t phase = 0, armed = 0;
        uint32_t tail_used = 0, tail_odd = 0;  // per stage: tails armed; an odd number of them
        bool ok = true;
        for (int t = cl; ok && rg_tile<CG, FORM>(p, walk, t, lane, rank, w); t += ncl) {
            if (lane == 0) {
                const int rows_b = w.n_mma / CG;  // column rows of this CTA
                const int b_row = w.b_row + static_cast<int>(rank) * rows_b;
                const int za = p.a_z ? w.group : 0, zb = p.b_z ? w.group : 0;
                // K-major columns: one whole-tile box, or 32-row boxes where those are fewer bytes
                const bool big = p.b_mn == 0 && 4 * rows_b > 3 * C::B_ROWS;
                const int nb = p.b_mn ? rows_b / 64 : (big ? 1 : (rows_b + 31) / 32);
                const uint32_t b_bytes = p.b_mn ? nb * 8192u : (big ? C::B_BYTES : nb * 4096u);
                const uint32_t bytes = C::A_BYTES + b_bytes;
                const int kblocks = (w.klen + 63) / 64;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait(empty0 + 8u * stage, phase ^ 1u, abort_flag, p.status, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (p.test_stall == 1 && armed == 0) {
                        ok = false;  // test only: the MMA warp's bounded wait must expire
                        break;
                    }
                    const uint32_t fb = full0 + 8u * stage;
                    // a ragged tail lands on each CTA's own barrier, for the zeroing
                    const bool tail = FORM == RG_WGRAD && kb == kblocks - 1 && (w.klen & 15) != 0;
                    uint32_t bar;
                    if (tail) {
                        mbar_arrive_expect_tx(tail0 + 8u * stage, bytes);
                        if (leader) mbar_arrive(fb);
                        bar = tail0 + 8u * stage;
                        tail_used |= 1u << stage;
                        tail_odd ^= 1u << stage;
                    } else {
                        if (leader) mbar_arrive_expect_tx(fb, CG * bytes);
                        bar = CG == 1 || leader ? fb : mapa_shared(fb, 0u);
                    }
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                        if constexpr (CG == 2)
                            tma_load_3d_pair(dst, map, bar, x, y, z, pol);
                        else
                            tma_load_3d(dst, map, bar, x, y, z, pol);
                    };
                    const uint32_t a_dst = sA0 + stage * C::A_BYTES;
                    const uint32_t b_dst = sB0 + stage * C::B_BYTES;
                    const int k = w.k0 + kb * 64;
                    if (p.a_mn) {
                        load(a_dst, &p.tmap_a, w.lane0, k, za);
                        load(a_dst + 8192u, &p.tmap_a, w.lane0 + 64, k, za);
                    } else {
                        load(a_dst, &p.tmap_a, k, w.lane0, za);
                    }
                    if (p.b_mn) {
                        for (int h = 0; h < nb; ++h)
                            load(b_dst + 8192u * h, &p.tmap_b, b_row + 64 * h, k, zb);
                    } else if (big) {
                        load(b_dst, &p.tmap_b, k, b_row, zb);
                    } else {
                        for (int h = 0; h < nb; ++h)
                            load(b_dst + 4096u * h, &p.tmap_b32, k, b_row + 32 * h, zb);
                    }
                    ++armed;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        // Every issued copy lands before the CTA exits.  A pair's peer completes
        // its copies on the leader's barriers: after a normal run the leader has
        // consumed them before the final cluster barrier; after an abort the
        // peer gives them a fixed time.
        if (lane == 0) {
            for (int s = 0; s < C::STAGES; ++s)
                if (tail_used >> s & 1u)  // an odd count: its last phase has parity 0
                    rg_drain(tail0 + 8u * s, (tail_odd >> s & 1u) ^ 1u, p.timeout_ns);
            if (CG == 2 && !leader) {
                if (!ok) {
                    const uint64_t t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < 200000ull) {
                    }
                }
            } else {
                for (int s = 0; s < C::STAGES && static_cast<uint32_t>(s) < armed; ++s) {
                    const uint32_t fills = (armed - 1u - s) / C::STAGES + 1u;
                    rg_drain(full0 + 8u * s, (fills - 1u) & 1u, p.timeout_ns);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        // (the pair's peer walks the same tiles for the tails only)
        int stage = 0;
        uint32_t phase = 0, tail_phase = 0;  // tail_phase: one bit per stage
        int abuf = 0;
        uint32_t aphase = 0;
        bool issued = false, ok = true;
        const bool a_mn = p.a_mn != 0, b_mn = p.b_mn != 0;
        const uint32_t a_lbo = a_mn ? 8192u : 16u, b_lbo = b_mn ? 8192u : 16u;
        const uint32_t a_step = a_mn ? 2048u : 32u, b_step = b_mn ? 2048u : 32u;
        for (int t = cl; ok && rg_tile<CG, FORM>(p, walk, t, lane, rank, w); t += ncl) {
            const int kblocks = (w.klen + 63) / 64;
            if (kblocks == 0) continue;  // no rows: the epilogue writes zeros
            const bool issuer = CG == 1 || leader;
            if (issuer) {
                if (!rg_warp_wait(tempty0 + 8u * abuf, aphase ^ 1u, lane, abort_flag, p)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
            }
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(abuf * BT);
            const uint32_t idesc = p.idesc | (static_cast<uint32_t>(w.n_mma >> 3) << 17);
            if (!issuer && FORM != RG_WGRAD) continue;
            for (int kb = 0; kb < kblocks; ++kb) {
                const bool tail = FORM == RG_WGRAD && kb == kblocks - 1 && (w.klen & 15) != 0;
                if (issuer) {
                    if (!rg_warp_wait(full0 + 8u * stage, phase, lane, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                }
                if (tail) {
                    if (!rg_warp_wait(tail0 + 8u * stage, tail_phase >> stage & 1u, lane,
                                      abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    __syncwarp();
                    // rows klen % 64 .. up to the end of the last K = 16 step: one
                    // row is 128 bytes of every 64-wide atom column (whole rows,
                    // so the swizzle inside them does not matter)
                    const int v = w.klen - kb * 64;
                    const int nz = ((v + 15) & ~15) - v;
                    const int acols = 2 + w.n_mma / CG / 64;
                    for (int i = lane; i < acols * nz * 8; i += 32) {
                        const int chunk = i & 7, r = v + (i >> 3) % nz, col = (i >> 3) / nz;
                        const uint32_t base =
                            col < 2 ? stage * C::A_BYTES + col * 8192u
                                    : C::STAGES * C::A_BYTES + stage * C::B_BYTES + (col - 2) * 8192u;
                        *reinterpret_cast<uint4*>(smem + base + r * 128 + chunk * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (CG == 2 && !leader) {
                        if (lane == 0) mbar_arrive_remote(mapa_shared(peer_tail0 + 8u * stage, 0u));
                    } else if (CG == 2) {
                        if (!rg_warp_wait(peer_tail0 + 8u * stage, tail_phase >> stage & 1u, lane,
                                          abort_flag, p)) {
                            ok = false;
                            break;
                        }
                        fence_proxy_async_smem();
                    }
                    tail_phase ^= 1u << stage;
                }
                if (issuer) {
                    tc_fence_after_sync();
                    if (lane == 0) {
                        const uint32_t a_base = sA0 + stage * C::A_BYTES;
                        const uint32_t b_base = sB0 + stage * C::B_BYTES;
                        const int left = w.klen - kb * 64;
                        const int steps = left >= 64 ? 4 : (left + 15) / 16;
                        for (int k = 0; k < steps; ++k)
                            umma_f16_cg<CG>(d_tmem,
                                            smem_desc_sw128(a_base + k * a_step, a_lbo, 1024u),
                                            smem_desc_sw128(b_base + k * b_step, b_lbo, 1024u),
                                            idesc, (kb > 0 || k > 0) ? 1u : 0u);
                        if constexpr (CG > 1)
                            umma_commit_mc_cg<CG>(empty0 + 8u * stage, kPair);
                        else
                            umma_commit_cg<CG>(empty0 + 8u * stage);
                        if (kb == kblocks - 1) {
                            if constexpr (CG > 1)
                                umma_commit_mc_cg<CG>(tfull0 + 8u * abuf, kPair);
                            else
                                umma_commit_cg<CG>(tfull0 + 8u * abuf);
                        }
                    }
                    issued = true;
                }
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (++abuf == 2) {
                abuf = 0;
                aphase ^= 1u;
            }
        }
        if (issued && lane == 0) {
            umma_commit_cg<CG>(drain_bar);
            rg_drain(drain_bar, 0u, p.timeout_ns);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ epilogue
        const int q = warp & 3;           // tensor-memory lane quarter of this warp
        const int half = (warp - 2) >> 2; // which 32-column chunks it takes
        const uint32_t lane_field = static_cast<uint32_t>(q * 32) << 16;
        float* stg = reinterpret_cast<float*>(epi_smem + (warp - 2) * C::EPI_WARP);
        int abuf = 0;
        uint32_t aphase = 0;
        const bool late = p.beta != 0.0f && FORM != RG_SYM;  // beta * Cin read at the stores
        for (int t = cl; rg_tile<CG, FORM>(p, walk, t, lane, rank, w); t += ncl) {
            const bool empty = w.klen == 0;
            const int nl0 = w.lane0 + q * 32;   // first output column of this warp
            const int n = nl0 + lane;
            const float bias = p.bias && n < p.n_lane ? p.bias[w.group * p.stride_bias + n] : 0.0f;
            if (!empty) {
                if (!rg_warp_wait(tfull0 + 8u * abuf, aphase, lane, abort_flag, p)) break;
                tc_fence_after_sync();
            }
            const uint32_t tmem_row = tmem_base + lane_field + static_cast<uint32_t>(abuf * BT);
            if (nl0 < p.n_lane) {
#pragma unroll 1
                for (int c0 = half * 32; c0 < w.ncols; c0 += 64) {
                    uint32_t r[32];
                    if (!empty) {
                        tmem_ld_x32(tmem_row + static_cast<uint32_t>(c0), r);
                        tmem_ld_wait(r);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = 0u;
                    }
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = fmaf(p.alpha, __uint_as_float(r[i]), bias);
                    if constexpr (FORM == RG_SYM) {
                        // Cin is symmetric: its row n, columns of this chunk
                        if (p.beta != 0.0f && n < p.n_lane) {
                            const char* src = static_cast<const char*>(p.Cin) +
                                              (w.group * p.stride_cin + n * p.ldcin + w.col0 + c0) * 2;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (w.col0 + c0 + 8 * i >= p.n_lane) break;
                                const uint4 u = *reinterpret_cast<const uint4*>(src + 16 * i);
                                const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float2 f = rg_unpack(p.cin_dtype, uw[j]);
                                    v[8 * i + 2 * j] = fmaf(p.beta, f.x, v[8 * i + 2 * j]);
                                    v[8 * i + 2 * j + 1] = fmaf(p.beta, f.y, v[8 * i + 2 * j + 1]);
                                }
                            }
                        }
                        // the mirrored tile: this lane's row, 64 bytes (an
                        // off-diagonal tile's columns all exist)
                        if (!w.diag && n < p.n_lane) {
                            const int64_t off = w.group * p.stride_c + n * p.ldc + w.col0 + c0;
                            if (rg_span_ok(p, off, 32)) {
                                char* dst = static_cast<char*>(p.C) + off * 2;
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    *reinterpret_cast<uint4*>(dst + 16 * i) = make_uint4(
                                        rg_pack(p.c_dtype, v[8 * i], v[8 * i + 1]),
                                        rg_pack(p.c_dtype, v[8 * i + 2], v[8 * i + 3]),
                                        rg_pack(p.c_dtype, v[8 * i + 4], v[8 * i + 5]),
                                        rg_pack(p.c_dtype, v[8 * i + 6], v[8 * i + 7]));
                            }
                        }
                    }
                    if (!late) act_inplace<32>(v, p.act);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 16; ++i) stg[i * RG_LD + lane] = v[16 * h + i];
                        __syncwarp();
                        const int cbase = c0 + 16 * h;
                        if (p.c_dtype == DT_F32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int c = 4 * i + (lane >> 3), n4 = (lane & 7) * 4;
                                if (cbase + c < w.ncols && nl0 + n4 < p.n_lane) {
                                    const float4 f = *reinterpret_cast<const float4*>(stg + c * RG_LD + n4);
                                    float o[4] = {f.x, f.y, f.z, f.w};
                                    const int64_t row = w.out_row + cbase + c;
                                    const int64_t nn = nl0 + n4;
                                    rg_store<4, FORM == RG_SYM>(p, w.group * p.stride_c + row * p.ldc + nn,
                                                w.group * p.stride_cin + row * p.ldcin + nn,
                                                nl0 + n4, o);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int c = 8 * i + (lane >> 2), n8 = (lane & 3) * 8;
                                if (cbase + c < w.ncols && nl0 + n8 < p.n_lane) {
                                    const float4 f = *reinterpret_cast<const float4*>(stg + c * RG_LD + n8);
                                    const float4 g =
                                        *reinterpret_cast<const float4*>(stg + c * RG_LD + n8 + 4);
                                    float o[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
                                    const int64_t row = w.out_row + cbase + c;
                                    const int64_t nn = nl0 + n8;
                                    rg_store<8, FORM == RG_SYM>(p, w.group * p.stride_c + row * p.ldc + nn,
                                                w.group * p.stride_cin + row * p.ldcin + nn,
                                                nl0 + n8, o);
                                }
                            }
                        }
                    }
                }
            }
            if (empty) continue;
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2 && !leader)
                    mbar_arrive_remote(mapa_shared(tempty0 + 8u * abuf, 0u));
                else
                    mbar_arrive(tempty0 + 8u * abuf);
            }
            if (++abuf == 2) {
                abuf = 0;
                aphase ^= 1u;
            }
        }
        __syncwarp();
    }
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG > 1) cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<CG>(tmem_base, C::TMEM_COLS);
    }
}

template <int CG, int BT, int FORM>
cudaError_t rg_launch(const RgParams& p, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(RgCfg<CG, BT>::THREADS);
    cfg.dynamicSmemBytes = RgCfg<CG, BT>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (CG > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = CG;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (p.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, ragged_kernel<CG, BT, FORM>, p);
}

template <int CG, int BT, int FORM>
cudaError_t rg_prepare() {
    return cudaFuncSetAttribute(ragged_kernel<CG, BT, FORM>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(RgCfg<CG, BT>::SMEM));
}

}  // namespace
}  // namespace dg
