// Products of 8-bit integers with a scale for each token and each output channel:
//
//   y[t, n] = act( (sum_k x[t, k] q_e[n, k]) * sx[t] * sw_e[n] + bias_e[n] )
//
// for the rows t of group e.  The tensor cores of sm_103a multiply no 8-bit integers at a
// useful rate, but an int8 is an exact fp16 number, a product of two at most 2^14, and 1024
// of them sum to at most 2^24, which the fp32 accumulator holds exactly.  So the kernel
// multiplies fp16 (at the 16-bit rate), takes at most 1024 products into an accumulator and
// adds that to 32-bit integers in registers (or two of them in fp32, which rounds their sum as
// the integer would be): the sum is the integer sum, whatever the tiles, splits and order, and
// a row's result does not depend on the call's other rows.
//
// What it saves against 16-bit weights is bytes, so the weights stay bytes up to the SM:
//
//   warp 2       loads 128 weight rows x 128 bytes by TMA (128-byte swizzle);
//   warps 4-11   read half of their lane's row, make fp16 pairs by byte permutes (b ^ 128 under the
//                exponent of 1024 is 1152 + b; one packed subtraction) and store them to
//                tensor memory, 64 columns for 128 of them;
//   warp 0       loads the tokens' fp16 rows by TMA (made once per call in the workspace);
//   warp 1       issues tcgen05.mma with its A operand in tensor memory;
//   warps 12-19  add accumulators up and write the result.
//
// Weights in tensor memory rather than back in shared memory: a pair's stage then moves 16 KB
// in and out of shared memory for the weights and 24 KB in and out for the tokens in 768
// clocks of MMAs, 107 of the 128 bytes a clock; with fp16 weights stored to shared memory
// and read from there it would be 192.  Tiles have the weights on the MMA's M side (128 rows
// a CTA, 256 a pair) and the tokens on its N side, which is ragged in steps of 16: as in
// ragged_kernel.cuh, whose tiles, walk and bounded waits this kernel shares.  A pair's tile
// has 192 columns, so that two accumulators (384 columns) and two stages of weights (128)
// fill tensor memory: with 256 columns and one accumulator the MMAs would wait for every
// one of its hand-overs.
//
// Few tokens leave one tile per 128 weight rows; where those do not fill half of the SMs,
// the CTAs of a cluster share a tile's contraction and send their integer sums to the first
// one's shared memory.
//
// Bounds and times (graph replay, with the tokens' pass, inputs in turn).  One token of 8192 x
// 8192: 19 us (weights in L2: 16), the bytes take 10: start-up, the pass in front, and 128 of the
// 152 SMs have a tile.  192 rows over 64 experts of 2048 x 2048: 47 us, the bytes 40.  1500 tokens
// of 4096 x 4096: 40 us, the products 26: two rounds of 128 tiles on 76 pairs, and the pass (5).
// 16384 rows over 16 experts, 2048 to 4096, GELU: 190 us (1024 rows each: 197), the products 143:
// issue slots, most of them taken by the sums, scales, GELU and the conversion of the weights, and
// the pass (17).
#include "i8.h"
#include "ragged_kernel.cuh"

namespace dg {
namespace {

constexpr int kI8Convert = 8;    // warps that make fp16 weights
constexpr int kI8Epilogue = 4 + kI8Convert;  // the epilogue's first warp
constexpr int kI8Threads = 32 * (kI8Epilogue + 8);
constexpr int kI8Sum = 8;        // 128-deep blocks that an accumulator takes
constexpr int kI8MaxSplits = 4;

template <int CG, int BT, bool SPLIT>
struct I8Cfg {
    static constexpr int B_ROWS = BT / CG;                       // token rows a CTA holds
    // 128-deep blocks of a stage: a stage costs its roles 500 clocks beside its work, which
    // narrow tiles, bound by the weights' bytes, do not hide (192 rows over 64 experts, 2048 x
    // 2048: 59 us with one block, 47 with two)
    static constexpr int KS = BT <= 64 ? 2 : 1;
    static constexpr uint32_t A_BLOCK = 128 * 128;               // int8
    static constexpr uint32_t A_BYTES = KS * A_BLOCK;
    static constexpr uint32_t B_BLOCK = B_ROWS * 128;            // 64 deep, fp16
    static constexpr uint32_t B_BYTES = 2 * KS * B_BLOCK;
    static constexpr int A_COLS = 64 * KS;                       // of a stage in tensor memory
    static constexpr int SUM = kI8Sum / KS;                      // stages that an accumulator takes
    static constexpr int SMALL = BT == 32 ? 16 : 32;             // rows of the smaller token boxes
    static constexpr int NC = (BT + 63) / 64;        // 32-column chunks of an epilogue warp
    static constexpr uint32_t D_COLS = 2 * BT;              // two accumulators
    static constexpr int TA = (512 - D_COLS) / A_COLS < 4 ? (512 - D_COLS) / A_COLS : 4;
    static constexpr uint32_t RED_BYTES = SPLIT ? (kI8MaxSplits - 1) * BT * 128 * 4 : 0;
    static constexpr uint32_t BAR_BYTES = 512;
    static constexpr uint32_t EPI_WARP = 2048;  // a staged tile of 32 x 32 16-bit elements
    // stages of tokens, and of weights with what is left
    static constexpr int SB = CG == 2 ? 4 : 3;
    static constexpr int FIT = (kRgMaxSmem - 1024 - BAR_BYTES - RED_BYTES - 8 * EPI_WARP - SB * B_BYTES) / A_BYTES;
    static constexpr int SA = FIT > 10 ? 10 : FIT;
    static constexpr size_t SMEM = 1024 + size_t(SA) * A_BYTES + SB * B_BYTES + RED_BYTES + 8 * EPI_WARP + BAR_BYTES;
    static_assert(TA >= 2 && SA >= 3, "rings");
    static_assert(B_BLOCK % 1024 == 0, "blocks start on swizzle atoms");
    static_assert((2 * (SA + SB + TA) + 6) * 8 + 8 <= BAR_BYTES, "barrier area too small");
    static_assert(!SPLIT || CG == 1, "a tile is shared by single CTAs");
};

// What the roles of a CTA share.
struct I8Cta {
    uint32_t sA0, sB0;
    int* red;
    uint32_t afull, aempty;    // weights in shared memory
    uint32_t wfull, wempty;    // weights in tensor memory
    uint32_t bfull, bempty;    // tokens
    uint32_t tfull, tempty;    // accumulators
    uint32_t drain_bar, red_bar;
    uint32_t tmem;
    volatile int* abort_flag;
    uint32_t rank;             // CTA of the pair, or of the split
    bool leader;
    int cl, ncl;               // this cluster, clusters of the grid
    int lane;
};

// D += A B with A in tensor memory (a row per lane, two fp16 of it per column).
template <int CG>
__device__ __forceinline__ void umma_f16_tmem_a(uint32_t d, uint32_t a, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
            ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
            ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Four int8 as two pairs of fp16.
__device__ __forceinline__ void i8_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const uint32_t bias = 0x64806480u;  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&bias));
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&bias));
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

// One lane of a converged warp.  (elect.sync, not a comparison of the lane: the compiler then
// keeps the operands of tensor-core and copy instructions in uniform registers.)
__device__ __forceinline__ bool i8_elect() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ uint4 i8_ld_shared(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// 16 lanes x 32 columns of tensor memory in the layout of tmem_ld_16x256_x4, complete on
// return.
__device__ __forceinline__ void i8_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void i8_st_cluster(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Bounded wait of a whole warp.  All lanes ask and vote, which costs least where the phase has
// completed, and the compiler knows a vote to be the same in all lanes (see i8_issue).  A wait
// that runs out is voted on too: a lane that gave up by its own clock would leave the others at
// their next shuffle for ever.  A warp that has to wait is suspended: polling, it took issue
// slots from the epilogue, which shares its scheduler.  CLUSTER: acquires what the CTAs of the
// cluster wrote before they arrived.
constexpr uint32_t kI8Suspend = 20000;  // ns

template <bool CLUSTER = false>
__device__ __forceinline__ bool i8_wait(uint32_t bar, uint32_t parity, const I8Params& p, const I8Cta& x) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        const bool done = CLUSTER ? mbar_try_wait_cluster_ns(bar, parity, kI8Suspend)
                                  : mbar_try_wait_ns(bar, parity, kI8Suspend);
        if (__all_sync(0xffffffffu, done)) return true;
        if ((it & 7u) == 0) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            const bool late = now - t0 > p.g.timeout_ns;
            if (late) {
                *x.abort_flag = 1;
                if (p.g.status) DG_SET_TIMEOUT(p.g.status);
            }
            if (__any_sync(0xffffffffu, late || *x.abort_flag != 0)) return false;
        }
    }
}

// Stages of a tile's contraction that this CTA takes.
template <bool SPLIT, int KS>
__device__ __forceinline__ void i8_range(const I8Params& p, const I8Cta& x, int& s0, int& s1) {
    const int steps = (p.g.K + 128 * KS - 1) / (128 * KS);
    s0 = SPLIT ? static_cast<int>(static_cast<int64_t>(steps) * x.rank / p.splits) : 0;
    s1 = SPLIT ? static_cast<int>(static_cast<int64_t>(steps) * (x.rank + 1) / p.splits) : steps;
}

// Where a role stands in a ring.
template <int N>
struct I8Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            phase ^= 1u;
        }
    }
};

// Every copy armed on a ring's barriers lands before the CTA exits.
template <int N>
__device__ __forceinline__ void i8_drain(uint32_t full, uint32_t armed, uint64_t timeout_ns) {
    for (int s = 0; s < N && static_cast<uint32_t>(s) < armed; ++s) {
        const uint32_t fills = (armed - 1u - s) / N + 1u;
        rg_drain(full + 8u * s, (fills - 1u) & 1u, timeout_ns);
    }
}

// ------------------------------------------------ weights, by TMA (a warp)
template <int CG, int BT, bool SPLIT>
__device__ __forceinline__ void i8_load_weights(const I8Params& p, const I8Cta& x) {
    using C = I8Cfg<CG, BT, SPLIT>;
    // (few tokens read a weight once; many read it for every tile of tokens)
    const uint64_t pol = BT <= 32 ? l2_policy_evict_first() : l2_policy_evict_normal();
    RgWalk walk = rg_begin<RG_ROWS>(p.g, x.lane);
    RgTile w;
    I8Ring<C::SA> ring;
    uint32_t armed = 0;
    bool ok = true;
    for (int t = x.cl; ok && rg_tile<CG, BT, RG_ROWS>(p.g, walk, t, x.lane, SPLIT ? 0u : x.rank, w); t += x.ncl) {
        int s0, s1;
        i8_range<SPLIT, C::KS>(p, x, s0, s1);
        for (int s = s0; s < s1; ++s) {
            // (from here on it waits for the MMAs, which wait for the tokens' pass: that pass's
            // time is not the bounded wait's)
            if (p.g.pdl && armed == C::SA) griddep_wait();
            ok = i8_wait(x.aempty + 8u * ring.at, ring.phase ^ 1u, p, x);
            if (p.g.test_stall == 1 && armed == 0) ok = false;  // test only: the others' bounded waits must expire
            if (!ok) break;
            if (i8_elect()) {
                const uint32_t bar = x.afull + 8u * ring.at;
                mbar_arrive_expect_tx(bar, C::A_BYTES);
#pragma unroll
                for (int j = 0; j < C::KS; ++j)
                    tma_load_3d(x.sA0 + ring.at * C::A_BYTES + j * C::A_BLOCK, &p.g.tmap_a, bar,
                                (s * C::KS + j) * 128, w.lane0, p.g.a_z ? w.group : 0, pol);
            }
            ++armed;
            ring.next();
        }
    }
    if (x.lane == 0) i8_drain<C::SA>(x.afull, armed, p.g.timeout_ns);
    __syncwarp();
}

// ------------------------------------------------ tokens, by TMA (a warp)
template <int CG, int BT, bool SPLIT>
__device__ __forceinline__ void i8_load_tokens(const I8Params& p, const I8Cta& x) {
    using C = I8Cfg<CG, BT, SPLIT>;
    const uint64_t pol = l2_policy_evict_last();
    RgWalk walk = rg_begin<RG_ROWS>(p.g, x.lane);
    RgTile w;
    I8Ring<C::SB> ring;
    uint32_t armed = 0;
    bool ok = true;
    if (p.g.pdl) griddep_wait();
    for (int t = x.cl; ok && rg_tile<CG, BT, RG_ROWS>(p.g, walk, t, x.lane, SPLIT ? 0u : x.rank, w); t += x.ncl) {
        const int n_mma = rg_uniform(w.n_mma);
        const int rows_b = n_mma / CG;
        const int b_row = rg_uniform(w.b_row) + (CG == 2 ? static_cast<int>(x.rank) * rows_b : 0);
        // whole-tile boxes, or smaller ones where those are fewer bytes
        const bool big = 4 * rows_b > 3 * C::B_ROWS;
        const int nb = big ? 1 : (rows_b + C::SMALL - 1) / C::SMALL;
        const uint32_t bytes = big ? C::B_BYTES : nb * (C::SMALL * 256u * C::KS);
        int s0, s1;
        i8_range<SPLIT, C::KS>(p, x, s0, s1);
        for (int s = s0; s < s1; ++s) {
            ok = i8_wait(x.bempty + 8u * ring.at, ring.phase ^ 1u, p, x);
            if (!ok) break;
            if (i8_elect()) {
                const uint32_t fb = x.bfull + 8u * ring.at;
                const uint32_t bar = CG == 1 || x.leader ? fb : mapa_shared(fb, 0u);
                const uint32_t dst = x.sB0 + ring.at * C::B_BYTES;
                if (CG == 1 || x.leader) mbar_arrive_expect_tx(fb, CG * bytes);
                if (big) {
#pragma unroll
                    for (int j = 0; j < C::KS; ++j)
                        tma_load_4d_cg<CG>(dst + 2 * j * C::B_BLOCK, &p.g.tmap_b, bar, 0, b_row,
                                           2 * (s * C::KS + j), 0, pol);
                } else {
                    for (int h = 0; h < nb; ++h)
#pragma unroll
                        for (int blk = 0; blk < 2 * C::KS; ++blk) {
                            const uint32_t to = dst + blk * C::B_BLOCK + C::SMALL * 128u * h;
                            const int k = (2 * C::KS * s + blk) * 64, row = b_row + C::SMALL * h;
                            if constexpr (CG == 2)
                                tma_load_3d_pair(to, &p.g.tmap_b32, bar, k, row, 0, pol);
                            else
                                tma_load_3d(to, &p.g.tmap_b32, bar, k, row, 0, pol);
                        }
                }
            }
            ++armed;
            ring.next();
        }
    }
    if (x.lane == 0) {
        if (CG == 2 && !x.leader) {
            // (its copies complete on the leader's barriers: after an abort they get a
            // fixed time, otherwise the leader has consumed them before the last barrier)
            if (!ok) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 200000ull) {
                }
            }
        } else {
            i8_drain<C::SB>(x.bfull, armed, p.g.timeout_ns);
        }
    }
    __syncwarp();
}

// ------------------------------------------------ weights to tensor memory (eight warps)
// Two warps per tensor-memory lane quarter, each for 64 of a stage's 128 weights a row.  They
// are converted before the wait for their place in tensor memory: a pair's two stages there
// leave 768 clocks from one MMA's end to the next one's start, of which the hand-over takes
// 600 (the commit's arrival 300, the weights' 250).
template <int CG, int BT, bool SPLIT>
__device__ __forceinline__ void i8_convert(const I8Params& p, const I8Cta& x, int warp) {
    using C = I8Cfg<CG, BT, SPLIT>;
    const int q = warp & 3, row = q * 32 + x.lane, half = (warp - 4) >> 2;
    // (16-byte part 4 half + c of the row, swizzled by the row)
    const uint32_t a_row = x.sA0 + row * 128 + ((half << 6) ^ ((row & 4) << 4)), swz = (row & 3) << 4;
    const uint32_t to = x.tmem + (static_cast<uint32_t>(q * 32) << 16) + C::D_COLS + half * 32;
    RgWalk walk = rg_begin<RG_ROWS>(p.g, x.lane);
    RgTile w;
    I8Ring<C::SA> in;
    I8Ring<C::TA> out;
    bool ok = true;
    uint32_t done = 0;  // stages, while the tokens' pass may still run
    int s0, s1;
    i8_range<SPLIT, C::KS>(p, x, s0, s1);
    for (int t = x.cl; ok; t += x.ncl) {
        const bool more = rg_tile<CG, BT, RG_ROWS>(p.g, walk, t, x.lane, SPLIT ? 0u : x.rank, w);
        if (!__all_sync(0xffffffffu, more)) break;
        for (int s = s0; s < s1; ++s) {
            // (the tokens' pass's time is not the bounded waits': it is waited for in front of the
            // first of them that depends on it, which is for a stage that the loader fills behind
            // the pass or, where shared memory has more stages than tensor memory, for a place
            // there that an MMA gives back)
            if (C::SA <= C::TA && p.g.pdl && done == C::SA) griddep_wait();
            ok = i8_wait(x.afull + 8u * in.at, in.phase, p, x);
            if (!ok) break;
            const uint32_t src = a_row + in.at * C::A_BYTES;
#pragma unroll
            for (int j = 0; j < C::KS; ++j) {
                uint32_t r[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 v = i8_ld_shared(src + j * C::A_BLOCK + ((c << 4) ^ swz));
                    i8_halves(v.x, r[8 * c], r[8 * c + 1]);
                    i8_halves(v.y, r[8 * c + 2], r[8 * c + 3]);
                    i8_halves(v.z, r[8 * c + 4], r[8 * c + 5]);
                    i8_halves(v.w, r[8 * c + 6], r[8 * c + 7]);
                }
                if (j == 0) {
                    if (C::SA > C::TA && p.g.pdl && done == C::TA) griddep_wait();
                    ++done;
                    ok = i8_wait(x.wempty + 8u * out.at, out.phase ^ 1u, p, x);
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                tmem_st_x32(to + out.at * C::A_COLS + j * 64, r);
            }
            if (!ok) break;
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (x.lane == 0) {
                // (nothing but tensor memory is handed over, which the fence above orders: a
                // release at cluster scope took 500 to 1500 clocks here)
                const uint32_t bar = x.wfull + 8u * out.at;
                if (CG == 2 && !x.leader)
                    mbar_arrive_relaxed(mapa_shared(bar, 0u));
                else
                    mbar_arrive(bar);
                // (the stage goes back only now that its values have been used: an arrival
                // right behind the loads overtook them where the epilogue's stores held them
                // up, and the next copy overwrote what single lanes had still to read)
                mbar_arrive(x.aempty + 8u * in.at);
            }
            in.next();
            out.next();
        }
    }
}

// ------------------------------------------------ MMA issuer (a warp; of the pair's leader)
// The whole warp walks tiles and stages, every branch decided by a vote, and an elected lane
// issues.  (Chosen by its number, that lane took 67 clocks to issue an MMA of any size and 100
// for a commit, 1200 a stage in all: 4096 tokens, 4096 x 4096, 166 us against 129.)
template <int CG, int BT, bool SPLIT>
__device__ __forceinline__ void i8_issue(const I8Params& p, const I8Cta& x) {
    using C = I8Cfg<CG, BT, SPLIT>;
    constexpr uint16_t kPair = 3u;
    if (CG == 2 && !x.leader) return;
    if (p.g.pdl) griddep_wait();
    const uint64_t b_desc0 = smem_desc_sw128(x.sB0, 16u, 1024u);
    const uint32_t tmem = static_cast<uint32_t>(rg_uniform(static_cast<int>(x.tmem)));
    RgWalk walk = rg_begin<RG_ROWS>(p.g, x.lane);
    RgTile w;
    I8Ring<C::TA> wr;
    I8Ring<C::SB> br;
    I8Ring<2> acc;
    bool ok = true, issued = false;
    auto commit = [&](uint32_t bar) {
        if constexpr (CG == 2)
            umma_commit_mc_cg<CG>(bar, kPair);
        else
            umma_commit_cg<CG>(bar);
    };
    int s0, s1;
    i8_range<SPLIT, C::KS>(p, x, s0, s1);
    const int steps = rg_uniform(s1 - s0);
    for (int t = x.cl; ok; t += x.ncl) {
        const bool more = rg_tile<CG, BT, RG_ROWS>(p.g, walk, t, x.lane, SPLIT ? 0u : x.rank, w);
        if (!__all_sync(0xffffffffu, more)) break;
        const uint32_t idesc = p.g.idesc | (static_cast<uint32_t>(rg_uniform(w.n_mma) >> 3) << 17);
        for (int s = 0; s < steps; ++s) {
            const bool fresh = s % C::SUM == 0;
            const bool last = s + 1 == steps || s % C::SUM == C::SUM - 1;
            if (fresh) {
                ok = i8_wait(x.tempty + 8u * acc.at, acc.phase ^ 1u, p, x);
                if (!ok) break;
            }
            const uint32_t bbar = x.bfull + 8u * br.at, wbar = x.wfull + 8u * wr.at;
            ok = i8_wait(bbar, br.phase, p, x) && i8_wait(wbar, wr.phase, p, x);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d = tmem + static_cast<uint32_t>(acc.at * BT);
            const uint32_t a = tmem + C::D_COLS + static_cast<uint32_t>(wr.at * C::A_COLS);
            const uint64_t b = b_desc0 + static_cast<uint32_t>(br.at) * (C::B_BYTES >> 4);
            const uint32_t wdone = x.wempty + 8u * wr.at, bdone = x.bempty + 8u * br.at;
            const uint32_t tdone = x.tfull + 8u * acc.at;
            if (i8_elect()) {
                // (past K both operands are zeros)
#pragma unroll
                for (int k = 0; k < 8 * C::KS; ++k)
                    umma_f16_tmem_a<CG>(d, a + 8 * k, b + (k >> 2) * (C::B_BLOCK >> 4) + (k & 3) * 2,
                                        idesc, (!fresh || k > 0) ? 1u : 0u);
                commit(wdone);
                commit(bdone);
                if (last) commit(tdone);
            }
            issued = true;
            wr.next();
            br.next();
            if (last) acc.next();
        }
    }
    // all MMAs complete before tensor memory is released
    if (issued && x.lane == 0) {
        umma_commit_cg<CG>(x.drain_bar);
        rg_drain(x.drain_bar, 0u, p.g.timeout_ns);
    }
    __syncwarp();
}

// A chunk's results (`cols` of its tokens and `lanes` of its output columns exist) from
// element `base` of C on: 16-bit ones through a staged tile, 16 bytes at a time.
__device__ __forceinline__ void i8_store16(const RgParams& p, int64_t base, int cols, int lanes,
                                           int lane, uint8_t* buf, const float (&o)[32]) {
    const int row = lane >> 2, part = lane & 3;
    uint32_t pk[4][4];
    rg_pack16(p.c_dtype, o, pk);
    __syncwarp();  // (the chunk before has left the staged tile)
#pragma unroll
    for (int i = 0; i < 4; ++i)
        stmatrix_x4_trans(smem_u32(buf) + rg_at(lane & 7, lane >> 3) + 512u * i, pk[i][0], pk[i][1],
                          pk[i][2], pk[i][3]);
    __syncwarp();
    if (!p.c_vec) {
        rg_put_rows(p, buf, base, cols < 32 ? cols : 32, lanes, lane);
        return;
    }
    uint16_t* dst = static_cast<uint16_t*>(p.C) + base + row * p.ldc + 8 * part;
    if (cols >= 32 && lanes >= 32) {
        const int64_t step = 8 * p.ldc;
#pragma unroll
        for (int it = 0; it < 4; ++it)
            if (rg_span_ok(p, base + (8 * it + row) * p.ldc + 8 * part, 8))
                *reinterpret_cast<uint4*>(dst + it * step) =
                    *reinterpret_cast<const uint4*>(buf + rg_at(8 * it + row, part));
        return;
    }
    const int n = lanes - 8 * part;
#pragma unroll 1
    for (int it = 0; it < 4; ++it)
        if (8 * it + row < cols && n > 0)
            rg_store8<false>(p, base + (8 * it + row) * p.ldc + 8 * part, n,
                             *reinterpret_cast<const uint4*>(buf + rg_at(8 * it + row, part)));
}

// fp32 ones: whole chunks through the staged tile, 16 tokens of 128 bytes at a time (16-byte
// parts swizzled by the token, conflict-free both ways), others directly: a store of 32 lanes is
// then 32 bytes in each of four rows.
__device__ __forceinline__ void i8_store32(const RgParams& p, int64_t base, int cols, int lanes,
                                           int lane, uint8_t* buf, const float (&o)[32]) {
    const int pcol = lane >> 2, part = lane & 3;
    if (p.c_vec && cols >= 32 && lanes >= 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            __syncwarp();  // (the tokens before have left the staged tile)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (((i >> 3) & 1) != h) continue;
                const int tok = 8 * ((i >> 2) & 1) + 2 * part + (i & 1);
                const int n = 8 * (2 * (i >> 4) + ((i >> 1) & 1)) + pcol;
                *reinterpret_cast<float*>(buf + tok * 128 + (((n >> 2) ^ (2 * part)) << 4) + (n & 3) * 4) = o[i];
            }
            __syncwarp();
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int tok = 4 * it + (lane >> 3), unit = lane & 7;
                const int64_t off = base + (16 * h + tok) * p.ldc + 4 * unit;
                if (rg_span_ok(p, off, 4))
                    *reinterpret_cast<uint4*>(static_cast<float*>(p.C) + off) =
                        *reinterpret_cast<const uint4*>(buf + tok * 128 + ((unit ^ (((tok >> 1) & 3) * 2)) << 4));
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int n = 8 * (2 * (i >> 4) + ((i >> 1) & 1)) + pcol;
        const int col = 8 * ((i >> 2) & 3) + 2 * part + (i & 1);
        const int64_t off = base + col * p.ldc + n;
        if (n < lanes && col < cols && rg_span_ok(p, off, 1)) static_cast<float*>(p.C)[off] = o[i];
    }
}

// GELU's tanh form as x / (1 + exp(-2 y)), y = sqrt(2 / pi) (x + 0.044715 x^3): half the
// instructions of 0.5 x (1 + tanh y), as the other kernels have it: their issue slots are free, this
// one's are not (16384 rows over 16 experts, 2048 to 4096: 190 us against 204).  The exponent is taken to base 2.
__device__ __forceinline__ float i8_gelu_tanh(float x) {
    constexpr float k = -2.0f * 0.7978845608028654f * 1.4426950408889634f;
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * fmaf(0.044715f * k, x * x, k)));
    return __fdividef(x, 1.0f + e);
}

// max(x, 0) that keeps a NaN: a token with an infinity or a NaN has a NaN scale, which has to show
// in its results (the other kernels' relu makes it 0).
__device__ __forceinline__ float i8_relu(float x) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void i8_act(float (&v)[32], int act) {
    if (act == ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i8_gelu_tanh(v[i]);
    } else if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i8_relu(v[i]);
    } else {
        rg_act(v, act);
    }
}

// ------------------------------------------------ epilogue (a warp of eight)
// Sums stay in the registers in the layout of the matrix loads: of a chunk of 32 tokens, value
// i is output column 8 (2 (i / 16) + (i / 2) % 2) + lane / 4 and token 8 ((i / 4) % 4) +
// 2 (lane % 4) + i % 2 of the warp's.  16-bit results go through a staged tile, as
// in rg_out16, and leave 16 bytes at a time.  (One output column per thread, a shuffle for
// each token's scale and a two-byte store for each result took 4.5 us a tile: 1500 tokens of
// 4096 x 4096 46 us, then 42.)
template <int CG, int BT, bool SPLIT>
__device__ __forceinline__ void i8_epilogue(const I8Params& p, const I8Cta& x, int warp, uint8_t* buf) {
    using C = I8Cfg<CG, BT, SPLIT>;
    const int q = warp & 3;  // tensor-memory lane quarter of this warp
    const int c_first = ((warp - kI8Epilogue) >> 2) * 32;
    const int pcol = x.lane >> 2, part = x.lane & 3;
    const uint32_t row = x.tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c_first);
    RgWalk walk = rg_begin<RG_ROWS>(p.g, x.lane);
    RgTile w;
    I8Ring<2> acc;
    if (p.g.pdl) griddep_wait();  // (the tokens' scales)
    for (int t = x.cl; rg_tile<CG, BT, RG_ROWS>(p.g, walk, t, x.lane, SPLIT ? 0u : x.rank, w); t += x.ncl) {
        int s0, s1;
        i8_range<SPLIT, C::KS>(p, x, s0, s1);
        const int nl0 = w.lane0 + q * 32;  // first output column of this warp
        const bool mine = c_first < w.ncols && nl0 < p.g.n_lane;
        // the scale and bias of one output column and, of each chunk, one token's scale (on
        // their way before the sums: they took 1000 clocks in front of every tile's output)
        const bool in = mine && nl0 + x.lane < p.g.n_lane;
        const float sw_lane = in ? __ldg(p.w_scales + w.group * p.stride_ws + nl0 + x.lane) : 0.0f;
        const float bias_lane =
            in && p.g.bias ? __ldg(p.g.bias + w.group * p.g.stride_bias + nl0 + x.lane) : 0.0f;
        float sx[C::NC];
#pragma unroll
        for (int c = 0; c < C::NC; ++c) {
            const int at = c_first + 64 * c + x.lane;
            sx[c] = at < w.ncols ? __ldcg(p.x_scales + w.out_row + at) : 0.0f;
        }
        int v[C::NC][32];
        bool ok = true;
        // Two accumulators' sum in fp32 is rounded as its integer would be for the scaling: with no
        // more than two the sums stay fp32 numbers and save the conversions, whose rate
        // is a fraction of an addition's (16384 rows over 16 experts, 2048 to 4096, GELU: 196 us with
        // them, 190 without).
        const bool two = !SPLIT && s1 - s0 <= 2 * C::SUM;
        // an accumulator to the sums (the first one replaces them)
        auto add = [&](auto first, auto exact) {
            const uint32_t from = row + static_cast<uint32_t>(acc.at * BT);
#pragma unroll
            for (int c = 0; c < C::NC; ++c) {
                if (c_first + 64 * c < w.ncols) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t u[16];
                        i8_ld16(from + 64u * c + (static_cast<uint32_t>(h) << 20), u);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            int& sum = v[c][16 * h + i];
                            const float f = __uint_as_float(u[i]);
                            if (decltype(exact)::value)
                                sum = decltype(first)::value ? __float_as_int(f)
                                                             : __float_as_int(__int_as_float(sum) + f);
                            else
                                sum = decltype(first)::value ? __float2int_rn(f) : sum + __float2int_rn(f);
                        }
                    }
                }
            }
        };
        if (s0 == s1) {
#pragma unroll
            for (int c = 0; c < C::NC; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[c][i] = 0;
        }
#pragma unroll 1
        for (int s = s0; s < s1; s += C::SUM) {
            ok = i8_wait(x.tfull + 8u * acc.at, acc.phase, p, x);
            if (!ok) break;
            tc_fence_after_sync();
            if (mine && two) {
                if (s == s0)
                    add(std::true_type(), std::true_type());
                else
                    add(std::false_type(), std::true_type());
            } else if (mine) {
                if (s == s0)
                    add(std::true_type(), std::false_type());
                else
                    add(std::false_type(), std::false_type());
            }
            tc_fence_before_sync();
            __syncwarp();
            if (x.lane == 0)
                mbar_arrive_relaxed(mapa_shared(x.tempty + 8u * acc.at, CG == 2 ? 0u : x.rank));
            acc.next();
        }
        if (!ok) return;
        if (SPLIT) {
            // (one tile a cluster) the other CTAs' sums go to the first one
            if (x.rank != 0) {
                if (mine) {
                    // (value by value, 32 lanes side by side)
                    const uint32_t at = mapa_shared(smem_u32(x.red), 0u) +
                                        ((x.rank - 1) * BT * 128 + q * 32 + x.lane) * 4u;
#pragma unroll
                    for (int c = 0; c < C::NC; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            i8_st_cluster(at + (c_first + 64 * c + i) * 512u, v[c][i]);
                }
                __syncwarp();
                // (test only: with test_stall 2 they never arrive, so the first CTA's wait expires)
                if (x.lane == 0 && p.g.test_stall != 2) mbar_arrive_remote(mapa_shared(x.red_bar, 0u));
                return;
            }
            if (!i8_wait<true>(x.red_bar, 0u, p, x)) return;
            if (mine)
                for (int r = 1; r < p.splits; ++r) {
                    const int* from = x.red + (r - 1) * BT * 128 + q * 32 + x.lane;
#pragma unroll
                    for (int c = 0; c < C::NC; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[c][i] += from[(c_first + 64 * c + i) * 128];
                }
        }
        if (!mine) continue;
        if (!two) {
#pragma unroll
            for (int c = 0; c < C::NC; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[c][i] = __float_as_int(__int2float_rn(v[c][i]));
        }
        float sw[4], bias[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sw[i] = __shfl_sync(0xffffffffu, sw_lane, 8 * i + pcol);
            bias[i] = __shfl_sync(0xffffffffu, bias_lane, 8 * i + pcol);
        }
        // (one copy of the code, the next chunk's sums move to the front: unrolled, it did not
        // stay in the instruction cache beside the other roles')
#pragma unroll 1
        for (int c0 = c_first; c0 < w.ncols; c0 += 64) {
            float o[32];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float s = __shfl_sync(0xffffffffu, sx[0], 8 * (k >> 1) + 2 * part + (k & 1));
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int i = 16 * (h >> 1) + 4 * (k >> 1) + 2 * (h & 1) + (k & 1);
                    o[i] = fmaf(__int_as_float(v[0][i]) * s, sw[h], bias[h]);
                }
            }
#pragma unroll
            for (int c = 0; c + 1 < C::NC; ++c) {
                sx[c] = sx[c + 1];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[c][i] = v[c + 1][i];
            }
            i8_act(o, p.g.act);
            const int left = w.ncols - c0;
            const int64_t base = (w.out_row + c0) * p.g.ldc + nl0;
            if (p.g.c_dtype == DT_F32)
                i8_store32(p.g, base, left, p.g.n_lane - nl0, x.lane, buf, o);
            else
                i8_store16(p.g, base, left, p.g.n_lane - nl0, x.lane, buf, o);
        }
    }
}

// Registers: up to 96 sums a thread of the epilogue's two warpgroups.  640 threads are
// launched with 96 (i8_prepare checks it): 48 + 2 x 56 + 2 x 160 fit 5 x 96.
constexpr int I8_LAUNCH_REGS = 96, I8_ISSUE_REGS = 48, I8_CONVERT_REGS = 56, I8_SUM_REGS = 160;
static_assert(I8_ISSUE_REGS + 2 * I8_CONVERT_REGS + 2 * I8_SUM_REGS <= 5 * I8_LAUNCH_REGS, "register split");

template <int CG, int BT, bool SPLIT>
__global__ void __launch_bounds__(kI8Threads, 1) i8_kernel(const __grid_constant__ I8Params p) {
    using C = I8Cfg<CG, BT, SPLIT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int per_tile = SPLIT ? p.splits : CG;
    I8Cta x;
    x.rank = CG > 1 || SPLIT ? cluster_ctarank() : 0u;
    x.leader = x.rank == 0;
    x.cl = static_cast<int>(blockIdx.x) / per_tile;
    x.ncl = static_cast<int>(gridDim.x) / per_tile;
    x.lane = threadIdx.x & 31;
    x.sA0 = smem_u32(smem);
    x.sB0 = x.sA0 + C::SA * C::A_BYTES;
    x.red = reinterpret_cast<int*>(smem + C::SA * C::A_BYTES + C::SB * C::B_BYTES);
    uint8_t* staged = reinterpret_cast<uint8_t*>(x.red) + C::RED_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staged + 8 * C::EPI_WARP);
    x.afull = smem_u32(bars);
    x.aempty = x.afull + 8u * C::SA;
    x.bfull = x.aempty + 8u * C::SA;
    x.bempty = x.bfull + 8u * C::SB;
    x.wfull = x.bempty + 8u * C::SB;
    x.wempty = x.wfull + 8u * C::TA;
    x.tfull = x.wempty + 8u * C::TA;
    x.tempty = x.tfull + 16u;
    x.drain_bar = x.tempty + 16u;
    x.red_bar = x.drain_bar + 8u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * (C::SA + C::SB + C::TA) + 6);
    x.abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::SA; ++s) {
            mbar_init(x.afull + 8u * s, 1);
            mbar_init(x.aempty + 8u * s, kI8Convert);
        }
        for (int s = 0; s < C::SB; ++s) {
            mbar_init(x.bfull + 8u * s, 1);
            mbar_init(x.bempty + 8u * s, 1);
        }
        for (int s = 0; s < C::TA; ++s) {
            mbar_init(x.wfull + 8u * s, kI8Convert * CG);
            mbar_init(x.wempty + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(x.tfull + 8u * b, 1);
            mbar_init(x.tempty + 8u * b, 8 * CG);
        }
        mbar_init(x.drain_bar, 1);
        mbar_init(x.red_bar, SPLIT ? 8 * (p.splits - 1) : 1);
        *x.abort_flag = 0;
        fence_mbar_init();
        if (p.g.maps) {
            prefetch_tmap(&p.g.tmap_a);
            prefetch_tmap(&p.g.tmap_b);
            prefetch_tmap(&p.g.tmap_b32);
        }
    }
    if (warp == 1) {
        tmem_alloc_cg<CG>(smem_u32(tmem_slot), 512u);
        tmem_relinquish_cg<CG>();
    }
    tc_fence_before_sync();
    if constexpr (CG > 1 || SPLIT)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after_sync();
    x.tmem = *tmem_slot;

    if (warp >= kI8Epilogue) {
        reg_inc<I8_SUM_REGS>();
        i8_epilogue<CG, BT, SPLIT>(p, x, warp, staged + (warp - kI8Epilogue) * C::EPI_WARP);
    } else if (warp >= 4) {
        reg_dec<I8_CONVERT_REGS>();
        i8_convert<CG, BT, SPLIT>(p, x, warp);
    } else {
        reg_dec<I8_ISSUE_REGS>();
        if (warp == 0)
            i8_load_tokens<CG, BT, SPLIT>(p, x);
        else if (warp == 1)
            i8_issue<CG, BT, SPLIT>(p, x);
        else if (warp == 2)
            i8_load_weights<CG, BT, SPLIT>(p, x);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG > 1 || SPLIT) cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<CG>(x.tmem, 512u);
    }
}

template <int CG, int BT, bool SPLIT>
cudaError_t launch_form(const I8Params& p, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kI8Threads);
    cfg.dynamicSmemBytes = I8Cfg<CG, BT, SPLIT>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (p.g.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    if (CG > 1 || SPLIT) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = SPLIT ? static_cast<unsigned>(p.splits) : CG;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, i8_kernel<CG, BT, SPLIT>, p);
}

template <int CG, int BT, bool SPLIT>
cudaError_t prepare_form() {
    cudaError_t e = cudaFuncSetAttribute(i8_kernel<CG, BT, SPLIT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(I8Cfg<CG, BT, SPLIT>::SMEM));
    // (a wait for registers that the launch does not have would never end)
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, i8_kernel<CG, BT, SPLIT>);
    if (e == cudaSuccess && a.numRegs < I8_LAUNCH_REGS) e = cudaErrorInvalidConfiguration;
    return e;
}

}  // namespace

cudaError_t i8_launch(int cg, int bt, const I8Params& p, int grid, cudaStream_t stream) {
    if (p.splits > 1) return launch_form<1, 32, true>(p, grid, stream);
    if (cg == 2) return launch_form<2, kI8PairCols, false>(p, grid, stream);
    if (bt == 128) return launch_form<1, 128, false>(p, grid, stream);
    if (bt == 64) return launch_form<1, 64, false>(p, grid, stream);
    return launch_form<1, 32, false>(p, grid, stream);
}

cudaError_t i8_prepare() {
    cudaError_t e = prepare_form<1, 32, true>();
    if (e == cudaSuccess) e = prepare_form<1, 32, false>();
    if (e == cudaSuccess) e = prepare_form<1, 64, false>();
    if (e == cudaSuccess) e = prepare_form<1, 128, false>();
    if (e == cudaSuccess) e = prepare_form<2, kI8PairCols, false>();
    return e;
}

}  // namespace dg
