// Products of few rows, which are bound by reading the weights: 4-bit weights with group
// scales (gemm_w4's direct form, and the dequantising pass of its other form),
//
//   y[t, n] = sum_G s[n, G] * sum_{k in G} x[t, k] (q[n, k] - z[n, G])
//
// and 16-bit weights (gemm_grouped with up to 64 rows).
//
// One CTA per SM streams units of 64 (128 for more than 16 tokens) weight rows through a
// ring of 128-byte-swizzled TMA boxes, with the tokens' values of the same columns,
// filled by one producer warp that runs ahead over the CTA's units.  Of its sixteen
// (eight) consumer warps, each set of RT / 16 takes a range of the stages of its own, a
// warp 16 rows by a whole stage.  The arithmetic stays near the loads by going through
// mma.sync m16n8k16 with the weights on its M side and 8 tokens as its columns.
// (tcgen05.mma would need the 4-bit weights written back to shared memory as 16 bits; and
// for 16-bit ones its tiles of 128 weight rows leave most SMs idle in a decoding step:
// 8 experts with a row each, 2048 x 1024, were 64 tiles of half a megabyte, loaded at the
// 55 bytes a clock that an SM takes and multiplied at 115 clocks an instruction, 15.3 us;
// here 128 units take 10.5 us, of which 4.5 are what any one unit takes, against 5.0 us
// for reading the 34 MB.)
//
// 4-bit integers are exact bf16 (fp16) numbers, made by a byte permute, one masking and
// one packed subtraction for every two weights.  The products x (q - z) are summed in
// fp32 and scaled by s once per group, so nothing is rounded but the output.  The sum
// over k may be taken in any order, so lane t of a quad takes the 8 weights of 32-bit
// word t of a 16-byte chunk (32 weights) and 8 values of its token; the swizzle makes the
// word reads of 8 rows x 4 words conflict-free.  What bounds it: instructions and their
// latencies, 34 for 16 rows x 32 weights and 78 with groups of 32, where the schedulers
// issue in 53 % of the cycles, no pipe is busy for more than 47 %, and warps wait in
// about equal parts for fixed latencies, the integer pipe, loads and the unit's barriers;
// and where there is less than one unit a CTA, start-up.  Measured: one token, 8192 x 8192, groups of 128, 13.6 us
// (2.5 TB/s); 32 rows over 32 experts of 2048 x 4096, groups of 32 and zero points,
// 48.1 us (2.3 TB/s).
//
// Units (group, 64 rows, tokens of a tile) are dealt round robin; where they are fewer
// than half of the SMs, K is cut over the CTAs of a cluster (at most 4), whose fp32 sums
// meet in distributed shared memory and are added in rank order, so results repeat.  All
// waits are bounded, as in the other kernels.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "ragged.h"

namespace dg {
namespace {

template <int MT, int GROUP>
struct W4Cfg {
    static constexpr int WARPS = MT <= 16 ? 16 : 8;  // consumer warps
    static constexpr int THREADS = 32 * (WARPS + 1); // and the producer, warp 0
    // (registers come to four warps at once: 9 warps have 168 each, 17 have 96; 64 tokens
    // spill 28 to 64 bytes a thread there, 16 and 32 with groups of 64 spill 4)
    static constexpr int RT = MT <= 16 ? 64 : 128;   // weight rows (outputs) of a unit
    static constexpr int RG = RT / 16;               // row groups of a stage
    static constexpr int SG = WARPS / RG;            // stages in work at once
    // 256-weight blocks of a stage (one where many tokens' or groups' values take
    // the registers)
    static constexpr int BLK = MT <= 16 && GROUP > 32 ? 2 : 1;
    static constexpr int STEP = GROUP == 0 ? 128 : 256 * BLK;  // weights of a row per stage
    static constexpr uint32_t Q_BYTES = RT * 128;    // of a block of 4-bit weights
    static constexpr uint32_t W_BYTES = GROUP == 0 ? RT * STEP * 2 : BLK * Q_BYTES;
    static constexpr uint32_t X_BOX = MT * 128;      // 64 values of MT tokens
    static constexpr int X_BOXES = STEP / 64;
    static constexpr uint32_t STAGE = W_BYTES + X_BOXES * X_BOX;
    static constexpr int R_LD = RT + 4;
    static constexpr uint32_t R_BYTES = SG * MT * R_LD * 4;
    static constexpr int FIT = (232448 - 1024 - 512 - R_BYTES) / STAGE;
    static constexpr int STAGES = FIT > 16 ? 16 : FIT;
    static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE + R_BYTES + 512;
    static_assert(STAGES >= 3 && (2 * STAGES + 1) * 8 <= 512, "ring");
    static_assert(W_BYTES % 1024 == 0 && X_BOX % 1024 == 0, "swizzle atoms");
};

template <int DT>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (DT == DT_BF16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same onto zero.
template <int DT>
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    if constexpr (DT == DT_BF16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Weights 2 j and 2 j + 1 of word w (w4 = w >> 4) as 16-bit floats minus the pair
// `sub`: or-ing q into the mantissa of 128 (bf16) or 1024 (fp16), where one unit is
// the last bit, gives 128 + q (1024 + q) exactly, and sub holds 128 + z (1024 + z).
struct W4Bits {
    uint32_t mask, magic;
};

template <int DT>
__device__ __forceinline__ W4Bits w4_bits() {
    W4Bits k;
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(k.mask));
    asm volatile("mov.b32 %0, %1;" : "=r"(k.magic) : "n"(DT == DT_BF16 ? 0x43004300 : 0x64006400));
    return k;
}

template <int DT, int J>
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t w4, uint32_t sub, W4Bits k) {
    // (one three-input operation: mask and magic stay in registers)
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(v)
        : "r"(__byte_perm(w, w4, 0x4400 + 0x1111 * J)), "r"(k.mask), "r"(k.magic));
    if constexpr (DT == DT_BF16) {
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                         *reinterpret_cast<const __nv_bfloat162*>(&sub));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v),
                                  *reinterpret_cast<const __half2*>(&sub));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}

// 128 + z (1024 + z) twice, for the default and for byte `i` of four zero points
// (0 .. 15 each).
template <int DT>
__device__ __forceinline__ uint32_t w4_sub(int z) {
    return (DT == DT_BF16 ? 0x43004300u : 0x64006400u) + static_cast<uint32_t>(z) * 0x00010001u;
}

template <int DT>
__device__ __forceinline__ uint32_t w4_sub(uint32_t z, int i) {
    return (__byte_perm(z, 0u, 0x4040 + 0x0101 * i) & 0x000F000Fu) |
           (DT == DT_BF16 ? 0x43004300u : 0x64006400u);
}

template <int DT>
__device__ __forceinline__ float w4_float(uint16_t u) {
    if constexpr (DT == DT_BF16) return __uint_as_float(static_cast<uint32_t>(u) << 16);
    return __half2float(__ushort_as_half(u));
}

// (volatile: in order with the waits around them)
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint4 ld_shared_u128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// The units in order: group by group, its row tiles, the token tiles of one row
// tile after another.  One group per lane, a window of 32 groups at a time.
struct W4Walk {
    int base, before, incl, row0, rows;
    bool last;  // no group follows the window
};

template <int MT>
__device__ __forceinline__ void w4_window(const W4Params& p, W4Walk& w, int lane) {
    const int g = w.base + lane;
    int lo = 0, hi = 0;
    if (g < p.groups) {
        if (p.offsets) {
            lo = __ldg(p.offsets + g);
            hi = __ldg(p.offsets + g + 1);
        } else {
            hi = p.T;
        }
    }
    // offsets that do not ascend inside [0, T]: reported, and the groups from
    // there on have no rows
    const uint32_t bad = __ballot_sync(0xffffffffu, lo < 0 || hi < lo || hi > p.T);
    w.last = bad != 0 || w.base + 32 >= p.groups;
    if (bad) {
        if (lane == 0 && p.status) atomicOr(p.status, STATUS_BAD_OFFSETS);
        if (lane >= __ffs(bad) - 1) lo = hi = 0;
    }
    w.row0 = lo;
    w.rows = hi - lo;
    int units = (w.rows + MT - 1) / MT * p.n_tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, units, d);
        if (lane >= d) units += o;
    }
    w.incl = units;
}

struct W4Unit {
    int group, n0, row0, tokens;  // first output row; first token row, tokens
};

template <int MT>
__device__ __forceinline__ bool w4_unit(const W4Params& p, W4Walk& w, int u, int lane, W4Unit& o) {
    int total = __shfl_sync(0xffffffffu, w.incl, 31);
    while (u - w.before >= total) {
        if (w.last) return false;
        w.before += total;
        w.base += 32;
        w4_window<MT>(p, w, lane);
        total = __shfl_sync(0xffffffffu, w.incl, 31);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, w.incl > u - w.before);
    const int l = __ffs(m) - 1;
    const int rows = __shfl_sync(0xffffffffu, w.rows, l);
    const int row0 = __shfl_sync(0xffffffffu, w.row0, l);
    const int incl = __shfl_sync(0xffffffffu, w.incl, l);
    const int chunks = (rows + MT - 1) / MT;
    const int r = u - w.before - (incl - chunks * p.n_tiles);
    const int tile = r / chunks;
    const int t0 = (r - tile * chunks) * MT;
    o.group = w.base + l;
    o.n0 = tile * W4Cfg<MT, 128>::RT;
    o.row0 = row0 + t0;
    o.tokens = rows - t0 < MT ? rows - t0 : MT;
    return true;
}

// Scales and zero points of a warp's rows r, r + 8 for one stage, as loaded:
// NG neighbouring 16-bit scales and bytes of each row.
template <int NG>
struct W4Scales {
    uint32_t s[2][NG / 2];
    uint32_t z[2][(NG + 3) / 4];
};

// (vec: every stage's groups of a row start on a 16-byte boundary, or on their size)
template <int NG>
__device__ __forceinline__ void w4_fetch(const W4Params& p, int64_t row, int gi, int kg, int i,
                                         W4Scales<NG>& v) {
    const uint16_t* s = static_cast<const uint16_t*>(p.scales) + row * kg;
    const uint8_t* z = p.zeros + row * kg;
    if (p.vec && gi + NG <= kg) {
        if constexpr (NG >= 8) {
#pragma unroll
            for (int k = 0; k < NG / 8; ++k) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(s + gi) + k);
                v.s[i][4 * k] = u.x; v.s[i][4 * k + 1] = u.y;
                v.s[i][4 * k + 2] = u.z; v.s[i][4 * k + 3] = u.w;
            }
        } else if constexpr (NG == 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(s + gi));
            v.s[i][0] = u.x; v.s[i][1] = u.y;
        } else {
            v.s[i][0] = __ldg(reinterpret_cast<const uint32_t*>(s + gi));
        }
        if (p.zeros) {
            if constexpr (NG >= 8) {
#pragma unroll
                for (int k = 0; k < NG / 8; ++k) {
                    const uint2 u = __ldg(reinterpret_cast<const uint2*>(z + gi) + k);
                    v.z[i][2 * k] = u.x; v.z[i][2 * k + 1] = u.y;
                }
            } else if constexpr (NG == 4) {
                v.z[i][0] = __ldg(reinterpret_cast<const uint32_t*>(z + gi));
            } else {
                v.z[i][0] = __ldg(reinterpret_cast<const uint16_t*>(z + gi));
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < NG / 2; ++k) v.s[i][k] = 0u;
#pragma unroll
    for (int k = 0; k < (NG + 3) / 4; ++k) v.z[i][k] = 0u;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        // (groups past K: zero times zero)
        if (gi + k < kg) {
            v.s[i][k / 2] |= static_cast<uint32_t>(__ldg(s + gi + k)) << (16 * (k & 1));
            if (p.zeros) v.z[i][k / 4] |= static_cast<uint32_t>(__ldg(z + gi + k)) << (8 * (k & 3));
        }
    }
}

// A warp's 16 rows of a stage of 16-bit weights (128 of each row): K-major as two
// 64-wide blocks of 64 rows, or with the rows contiguous as 128 k of 64 rows.
template <int DT, int NT, uint32_t X_BOX>
__device__ __forceinline__ void w16_stage(uint32_t w0, uint32_t x0, int rg, int lane,
                                          bool mn, float (&total)[NT][4]) {
    // ldmatrix: lane l gives a row of matrix l >> 3; the matrices are (rows 0-7, k 0-7),
    // (rows 8-15, k 0-7), (rows 0-7, k 8-15), (rows 8-15, k 8-15) of 16 rows x 16 k
    const int l = lane & 7, m = lane >> 3;
    const int row = rg * 16 + (m & 1) * 8 + l;       // K-major: a row's 8 k
    const int col = rg * 2 + (m & 1);                // rows contiguous: 8 rows of one k
    // (two chains of a stage's sums, added to the total to nearest: a matrix instruction
    // cuts its sum off towards zero, which over a long row would add up)
    float acc[2][NT][4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // 32 k
        uint32_t a[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int kk = 2 * h + s;                // 16 k
            if (mn) {
                const int k = kk * 16 + (m >> 1) * 8 + l;
                ldmatrix_x4_trans(w0 + k * 128 + ((col ^ (k & 7)) << 4), a[s][0], a[s][1], a[s][2],
                                  a[s][3]);
            } else {
                const int part = (kk & 3) * 2 + (m >> 1);
                ldmatrix_x4(w0 + (kk >> 2) * 8192 + row * 128 + ((part ^ (row & 7)) << 4), a[s][0],
                            a[s][1], a[s][2], a[s][3]);
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint32_t b[4];                           // k 0-7, 8-15, 16-23, 24-31 of 8 tokens
            const int part = (h & 1) * 4 + m;
            ldmatrix_x4(x0 + (h >> 1) * X_BOX + (8 * j + l) * 128 + ((part ^ l) << 4), b[0], b[1],
                        b[2], b[3]);
            if (h == 0) {
                mma16816_first<DT>(acc[0][j], a[0], b[0], b[1]);
                mma16816_first<DT>(acc[1][j], a[1], b[2], b[3]);
            } else {
                mma16816<DT>(acc[0][j], a[0], b[0], b[1]);
                mma16816<DT>(acc[1][j], a[1], b[2], b[3]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) total[j][i] += acc[0][j][i] + acc[1][j][i];
}

template <int DT, int MT, int GROUP>
__global__ void __launch_bounds__(W4Cfg<MT, GROUP>::THREADS, 1) w4_kernel(const __grid_constant__ W4Params p) {
    using C = W4Cfg<MT, GROUP>;
    constexpr int NT = MT / 8;
    constexpr int GR = GROUP == 0 ? 128 : GROUP;  // (16-bit weights have no scales)
    constexpr int CPG = GR / 32;           // 16-byte chunks per group
    constexpr int NG = GROUP == 0 ? 2 : C::STEP / GR;  // groups of a row per stage
    constexpr int NGB = 256 / GR;          // ... per block
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* red = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red) + C::R_BYTES);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * C::STAGES;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * C::STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int u0 = static_cast<int>(blockIdx.x) / p.splits;
    const int nu = static_cast<int>(gridDim.x) / p.splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8u * s, 1);
            mbar_init(empty0 + 8u * s, C::RG);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        prefetch_tmap(&p.tmap_q);
        prefetch_tmap(&p.tmap_x);
    }
    W4Walk walk{0, 0, 0, 0, 0, false};
    w4_window<MT>(p, walk, lane);
    __syncthreads();

    // Stages of this CTA's K slice.  Each set of consumer warps walks a range of its
    // own, so that its scales come as neighbours; the ring holds the sets' first
    // stages, their second ones, and so on (the ranges' lengths differ by one at most).
    const int steps = (p.K + C::STEP - 1) / C::STEP;
    const int st0 = static_cast<int>(static_cast<int64_t>(steps) * rank / p.splits);
    const int st1 = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / p.splits);
    W4Unit w;

    if (warp == 0) {
        // ------------------------------------------------ producer
        int stage = 0;
        uint32_t phase = 0, armed = 0;
        bool ok = true;
        // (after a failed wait the units' cluster barriers still run)
        for (int u = u0; (ok || p.splits > 1) && w4_unit<MT>(p, walk, u, lane, w); u += nu) {
            if (ok && lane == 0) {
                const uint64_t pol_q = l2_policy_evict_first();
                const uint64_t pol_x = l2_policy_evict_last();
                const int n = st1 - st0;
                for (int i = 0, round = 0; ok && i < n; ++round)
                    for (int k = 0; k < C::SG; ++k) {
                        const int st = st0 + n * k / C::SG + round;
                        if (st >= st0 + n * (k + 1) / C::SG) continue;
                        if (!mbar_wait_short(empty0 + 8u * stage, phase ^ 1u, abort_flag, p.status,
                                       p.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb = full0 + 8u * stage;
                        if (p.test_stall == 1 && armed == 0) {
                            ok = false;  // test only: the consumers' bounded waits must expire
                            break;
                        }
                        mbar_arrive_expect_tx(fb, C::STAGE);
                        const uint32_t dst = smem_u32(smem) + stage * C::STAGE;
                        const uint32_t xdst = dst + C::W_BYTES;
                        if constexpr (GROUP == 0) {
                            const int k0 = st * C::STEP, wz = p.w_z ? w.group : 0;
                            if (p.w_mn) {
                                tma_load_3d(dst, &p.tmap_q, fb, w.n0, k0, wz, pol_q);
                            } else if (p.q4) {
                                tma_load_4d_cg<1>(dst, &p.tmap_q, fb, 0, w.n0, k0 / 64, wz,
                                                  pol_q);
                            } else {
                                tma_load_3d(dst, &p.tmap_q, fb, k0, w.n0, wz, pol_q);
                                tma_load_3d(dst + C::W_BYTES / 2, &p.tmap_q, fb, k0 + 64, w.n0,
                                            wz, pol_q);
                            }
                        } else if (p.q4) {
                            tma_load_4d_cg<1>(dst, &p.tmap_q, fb, 0, w.n0, st * C::BLK, w.group, pol_q);
                        } else {
#pragma unroll
                            for (int j = 0; j < C::BLK; ++j)
                                tma_load_3d(dst + j * C::Q_BYTES, &p.tmap_q, fb,
                                            (st * C::BLK + j) * 128, w.n0, w.group, pol_q);
                        }
                        if (p.x4) {
                            tma_load_3d(xdst, &p.tmap_x, fb, 0, w.row0, st * C::X_BOXES, pol_x);
                        } else {
#pragma unroll
                            for (int j = 0; j < C::X_BOXES; ++j)
                                tma_load_3d(xdst + j * C::X_BOX, &p.tmap_x, fb,
                                            st * C::STEP + 64 * j, w.row0, 0, pol_x);
                        }
                        ++armed;
                        ++i;
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (p.splits > 1) {
                // the consumers' two cluster barriers of the unit
                cluster_sync();
                cluster_sync();
            }
        }
        // every issued copy lands before the CTA exits
        if (lane == 0)
            for (int s = 0; s < C::STAGES && static_cast<uint32_t>(s) < armed; ++s) {
                const uint32_t fills = (armed - 1u - s) / C::STAGES + 1u;
                const uint64_t begin = globaltimer_ns();
                while (!mbar_try_wait(full0 + 8u * s, (fills - 1u) & 1u))
                    if (globaltimer_ns() - begin > p.timeout_ns) break;
            }
        __syncwarp();
    } else {
        // ------------------------------------------------ consumers
        const int cw = warp - 1, gr = lane >> 2, t = lane & 3;
        const int rg = cw % C::RG, sg = cw / C::RG;
        const int r = rg * 16 + gr;  // rows r and r + 8 of the unit
        const int kg = p.K / GR;
        // word t of chunk c of row r of a stage: the chunk is swizzled by the row
        const uint32_t q_at = static_cast<uint32_t>(r * 128 + t * 4) | static_cast<uint32_t>(gr << 4);
        const W4Bits bits = w4_bits<DT>();
        bool ok = true;
        uint32_t it0 = 0;  // stages of the units before
        const int n = st1 - st0;
        const int a0 = st0 + n * sg / C::SG, a1 = st0 + n * (sg + 1) / C::SG;
        const int shortest = n / C::SG;  // stages of the shorter ranges
        int longer_before = 0;           // sets before this one that have one more
#pragma unroll
        for (int k = 0; k < C::SG; ++k)
            if (k < sg && n * (k + 1) / C::SG - n * k / C::SG > shortest) ++longer_before;
        W4Scales<NG> cur, nxt;
        int64_t row_lo, row_hi;
        // the unit's rows of scales, and its first stage's ones
        auto open_unit = [&](const W4Unit& v) {
            // (rows past N read the last one: their sums are not stored)
            const int n_lo = v.n0 + r < p.N ? v.n0 + r : p.N - 1;
            const int n_hi = v.n0 + r + 8 < p.N ? v.n0 + r + 8 : p.N - 1;
            row_lo = static_cast<int64_t>(v.group) * p.N + n_lo;
            row_hi = static_cast<int64_t>(v.group) * p.N + n_hi;
        };
        auto fetch = [&](int st) {
            if (GROUP == 0) return;
            w4_fetch<NG>(p, row_lo, st * NG, kg, 0, nxt);
            w4_fetch<NG>(p, row_hi, st * NG, kg, 1, nxt);
        };
        bool have = w4_unit<MT>(p, walk, u0, lane, w);
        if (have) {
            open_unit(w);
            if (a0 < a1) fetch(a0);
        }
        for (int u = u0; have; u += nu, it0 += st1 - st0) {
            float total[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) total[j][i] = 0.0f;
            // (one tile of tokens: the lanes of those that do not exist read the first
            // one's values along with its lane; a column of the product has only its
            // own token)
            const int xr = NT > 1 || gr < w.tokens ? gr : 0;
            const uint32_t x_at = static_cast<uint32_t>(xr * 128 + ((t ^ xr) << 4));
            for (int st = a0; ok && st < a1; ++st) {
                const int round = st - a0;
                const uint32_t it = it0 + static_cast<uint32_t>(
                                              round * C::SG + (round < shortest ? sg : longer_before));
                const uint32_t turn = it / C::STAGES;
                const uint32_t stage = it - turn * C::STAGES;
                cur = nxt;
                if (st + 1 < a1) fetch(st + 1);
                ok = mbar_wait_short(full0 + 8u * stage, turn & 1u, abort_flag, p.status, p.timeout_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t ws = smem_u32(smem) + stage * C::STAGE;
                if constexpr (GROUP == 0)
                    w16_stage<DT, NT, C::X_BOX>(ws, ws + C::W_BYTES, rg, lane, p.w_mn != 0, total);
                // (stages are aligned, so that the swizzle is an exclusive or of addresses)
                uint32_t qs = ws + q_at, xs = ws + C::W_BYTES + x_at;
#pragma unroll 1
                for (int blk = 0; GROUP != 0 && blk < C::BLK; ++blk, qs += C::Q_BYTES, xs += 4 * C::X_BOX) {
                const uint32_t xs2 = xs ^ 64u;
#pragma unroll
                for (int gg = 0; gg < NGB; ++gg) {
                    // (two chains of sums where neither tokens nor a short group give
                    // independent ones)
                    constexpr bool two = NT == 1 && CPG > 1;
                    float acc[NT][4], acc2[4];
                    uint32_t sub_lo = w4_sub<DT>(8), sub_hi = sub_lo;
                    if (p.zeros) {
                        sub_lo = w4_sub<DT>(cur.z[0][gg / 4], gg & 3);
                        sub_hi = w4_sub<DT>(cur.z[1][gg / 4], gg & 3);
                    }
#pragma unroll
                    for (int cc = 0; cc < CPG; ++cc) {
                        const int c = gg * CPG + cc;
                        const uint32_t src = qs ^ static_cast<uint32_t>(c << 4);
                        const uint32_t lo = ld_shared_u32(src), hi = ld_shared_u32(src + 1024u);
                        const uint32_t lo4 = lo >> 4, hi4 = hi >> 4;
                        const uint32_t a1[4] = {w4_pair<DT, 0>(lo, lo4, sub_lo, bits),
                                                w4_pair<DT, 0>(hi, hi4, sub_hi, bits),
                                                w4_pair<DT, 1>(lo, lo4, sub_lo, bits),
                                                w4_pair<DT, 1>(hi, hi4, sub_hi, bits)};
                        const uint32_t a2[4] = {w4_pair<DT, 2>(lo, lo4, sub_lo, bits),
                                                w4_pair<DT, 2>(hi, hi4, sub_hi, bits),
                                                w4_pair<DT, 3>(lo, lo4, sub_lo, bits),
                                                w4_pair<DT, 3>(hi, hi4, sub_hi, bits)};
                        const uint32_t xsrc = ((c & 1) ? xs2 : xs) + (c >> 1) * C::X_BOX;
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const uint4 x = ld_shared_u128(xsrc + 1024u * j);
                            if (cc == 0)
                                mma16816_first<DT>(acc[j], a1, x.x, x.y);
                            else
                                mma16816<DT>(acc[j], a1, x.x, x.y);
                            if (two && cc == 0)
                                mma16816_first<DT>(acc2, a2, x.z, x.w);
                            else
                                mma16816<DT>(two ? acc2 : acc[j], a2, x.z, x.w);
                        }
                    }
                    const float s_lo = w4_float<DT>(
                        static_cast<uint16_t>(cur.s[0][gg / 2] >> (16 * (gg & 1))));
                    const float s_hi = w4_float<DT>(
                        static_cast<uint16_t>(cur.s[1][gg / 2] >> (16 * (gg & 1))));
                    if (two) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[0][i] += acc2[i];
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        total[j][0] = fmaf(s_lo, acc[j][0], total[j][0]);
                        total[j][1] = fmaf(s_lo, acc[j][1], total[j][1]);
                        total[j][2] = fmaf(s_hi, acc[j][2], total[j][2]);
                        total[j][3] = fmaf(s_hi, acc[j][3], total[j][3]);
                    }
                }
                    // the next block's scales move to the front
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int k = 0; C::BLK > 1 && k < NGB / 2; ++k)
                            cur.s[i][k] = cur.s[i][k + NGB / 2];
                        if constexpr (C::BLK > 1 && NGB >= 4) {
#pragma unroll
                            for (int k = 0; k < NGB / 4; ++k) cur.z[i][k] = cur.z[i][k + NGB / 4];
                        } else if constexpr (C::BLK > 1) {
                            cur.z[i][0] >>= 16;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8u * stage);
            }
            // the next unit's first scales are on their way while this one's sums meet
            const W4Unit done = w;
            have = w4_unit<MT>(p, walk, u + nu, lane, w);
            if (have) {
                open_unit(w);
                if (a0 < a1) fetch(a0);
            }
            // [stage set][token][row] sums of this CTA
            float* part = red + sg * MT * C::R_LD;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                part[(8 * j + 2 * t) * C::R_LD + r] = total[j][0];
                part[(8 * j + 2 * t + 1) * C::R_LD + r] = total[j][1];
                part[(8 * j + 2 * t) * C::R_LD + r + 8] = total[j][2];
                part[(8 * j + 2 * t + 1) * C::R_LD + r + 8] = total[j][3];
            }
            auto sync = [&]() {
                if (p.splits > 1)
                    cluster_sync();
                else
                    asm volatile("bar.sync 1, %0;" ::"n"(32 * C::WARPS) : "memory");
            };
            sync();
            // each CTA of the cluster adds and writes its share of the rows
            const int share = C::RT / p.splits;
            if (!*abort_flag) {
                for (int i = threadIdx.x - 32; i < done.tokens * share; i += 32 * C::WARPS) {
                    const int tok = i / share, rr = rank * share + i % share;
                    const int n = done.n0 + rr;
                    if (n >= p.N) continue;
                    const float* src = red + tok * C::R_LD + rr;
                    float v = 0.0f;
                    if (p.splits > 1) {
                        for (int k = 0; k < p.splits; ++k) {
                            const uint32_t at = mapa_shared(smem_u32(src), static_cast<uint32_t>(k));
#pragma unroll
                            for (int m = 0; m < C::SG; ++m)
                                v += ld_cluster_f32(at + 4u * m * MT * C::R_LD);
                        }
                    } else {
#pragma unroll
                        for (int m = 0; m < C::SG; ++m) v += src[m * MT * C::R_LD];
                    }
                    const int64_t off = static_cast<int64_t>(done.row0 + tok) * p.ldc + n;
#if DG_DEBUG
                    if (!DG_CHECK(off >= 0 && off < p.dbg_c_elems, p.status, STATUS_CHECK_BOUNDS))
                        continue;
#endif
                    char* dst = static_cast<char*>(p.C) + off * dt_size(p.c_dtype);
                    if (GROUP == 0) {
                        v *= p.alpha;
                        if (p.beta != 0.0f) v = fmaf(p.beta, load_elem(dst, p.c_dtype), v);
                    }
                    if (p.bias) v += __ldg(p.bias + done.group * p.stride_bias + n);
                    store_elem(dst, p.c_dtype, apply_act(v, p.act));
                }
            }
            // the sums are read before the next unit's (or the exit) replace them;
            // after a failed wait (ok stays false) the units' barriers still run
            sync();
        }
    }
}

template <int DT, int MT, int GROUP>
cudaError_t launch_one(const W4Params& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.grid) * p.splits);
    cfg.blockDim = dim3(W4Cfg<MT, GROUP>::THREADS);
    cfg.dynamicSmemBytes = W4Cfg<MT, GROUP>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, w4_kernel<DT, MT, GROUP>, p);
}

template <int DT, int MT>
cudaError_t launch_group(const W4Params& p, cudaStream_t stream) {
    if constexpr (MT <= 16)
        if (p.group == 0) return launch_one<DT, MT, 0>(p, stream);
    if (p.group == 32) return launch_one<DT, MT, 32>(p, stream);
    if (p.group == 64) return launch_one<DT, MT, 64>(p, stream);
    return launch_one<DT, MT, 128>(p, stream);
}

template <int DT>
cudaError_t launch_tokens(int tokens, const W4Params& p, cudaStream_t stream) {
    if (tokens == 8) return launch_group<DT, 8>(p, stream);
    if (tokens == 16) return launch_group<DT, 16>(p, stream);
    if (tokens == 32) return launch_group<DT, 32>(p, stream);
    return launch_group<DT, 64>(p, stream);
}

template <int DT, int MT, int GROUP>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(w4_kernel<DT, MT, GROUP>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(W4Cfg<MT, GROUP>::SMEM));
}

template <int DT, int MT>
cudaError_t prepare_group() {
    cudaError_t e = prepare_one<DT, MT, 32>();
    if constexpr (MT <= 16)
        if (e == cudaSuccess) e = prepare_one<DT, MT, 0>();
    if (e == cudaSuccess) e = prepare_one<DT, MT, 64>();
    if (e == cudaSuccess) e = prepare_one<DT, MT, 128>();
    return e;
}

template <int DT>
cudaError_t prepare_tokens() {
    cudaError_t e = prepare_group<DT, 8>();
    if (e == cudaSuccess) e = prepare_group<DT, 16>();
    if (e == cudaSuccess) e = prepare_group<DT, 32>();
    if (e == cudaSuccess) e = prepare_group<DT, 64>();
    return e;
}

// Dense weights: one thread turns 4 bytes (8 weights of one group) into 16.
template <int DT>
__global__ void __launch_bounds__(256) w4_dequantise_kernel(const uint32_t* q, const uint16_t* scales,
                                                            const uint8_t* zeros, int64_t words,
                                                            int shift, uint4* out) {
    griddep_launch_dependents();  // the product sets itself up meanwhile
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
#pragma unroll 4
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < words;
         i += stride) {
        const uint32_t w = __ldg(q + i);
        const int64_t gi = i >> shift;  // K is a multiple of the group, so rows need no division
        const float s = w4_float<DT>(__ldg(scales + gi));
        const float z = zeros ? static_cast<float>(__ldg(zeros + gi) & 15) : 8.0f;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = (static_cast<float>((w >> (8 * j)) & 15u) - z) * s;
            const float hi = (static_cast<float>((w >> (8 * j + 4)) & 15u) - z) * s;
            if constexpr (DT == DT_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                o[j] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(lo, hi);
                o[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        out[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

W4Shape w4_shape(int tokens, int group) {
    if (tokens > 16) return W4Shape{W4Cfg<64, 128>::RT, W4Cfg<64, 128>::STEP};
    return W4Shape{W4Cfg<16, 128>::RT, group == 0 ? W4Cfg<16, 0>::STEP
                                                  : (group > 32 ? W4Cfg<16, 128>::STEP : W4Cfg<16, 32>::STEP)};
}

cudaError_t w4_launch(int dt, int tokens, const W4Params& p, cudaStream_t stream) {
    return dt == DT_BF16 ? launch_tokens<DT_BF16>(tokens, p, stream)
                         : launch_tokens<DT_F16>(tokens, p, stream);
}

cudaError_t w4_prepare() {
    const cudaError_t e = prepare_tokens<DT_BF16>();
    return e != cudaSuccess ? e : prepare_tokens<DT_F16>();
}

cudaError_t w4_dequantise(int dt, const uint8_t* q, const void* scales, const uint8_t* zeros,
                          int64_t rows, int64_t K, int group, void* out, cudaStream_t stream) {
    const int64_t words = rows * K / 8;
    const int shift = group == 32 ? 2 : (group == 64 ? 3 : 4);  // words per group, as a power of 2
    int64_t blocks = (words + 1023) / 1024;
    if (blocks > 152 * 8) blocks = 152 * 8;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(q);
    const uint16_t* sc = static_cast<const uint16_t*>(scales);
    uint4* dst = static_cast<uint4*>(out);
    if (dt == DT_BF16)
        w4_dequantise_kernel<DT_BF16><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
            src, sc, zeros, words, shift, dst);
    else
        w4_dequantise_kernel<DT_F16><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
            src, sc, zeros, words, shift, dst);
    return cudaGetLastError();
}

}  // namespace dg
