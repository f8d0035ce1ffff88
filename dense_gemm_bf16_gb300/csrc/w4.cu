// Products with 4-bit weights and group scales (gemm_w4's direct form) and the
// dequantising pass of its other form.
//
//   y[t, n] = sum_G s[n, G] * sum_{k in G} x[t, k] (q[n, k] - z[n, G])
//
// With few tokens the call is bound by the N K / 2 bytes of weights.  So a CTA
// streams 64 rows of them through a ring of TMA boxes (128 bytes = 256 weights
// of 64 rows, 8 KB a stage, filled by one producer warp), and four consumer
// warps keep 16 rows each.  The arithmetic stays ahead of the loads by going
// through mma.sync m16n8k16 with the weights on its M side: a 4-bit integer is
// an exact bf16 (fp16) number, made from two bits operations and one packed
// subtraction for every two weights, and the tokens are the 8 columns.  The
// products x (q - z) are summed in fp32 and scaled by s once per group, so the
// direct form rounds nothing but its output.
//
// The sum over k may be taken in any order, so lane t of a quad takes the 8
// weights of 32-bit word t of a 16-byte chunk (32 weights) in the order that
// masking leaves them, (0,4) (1,5) (2,6) (3,7), and the same 8 tokens' values,
// paired by byte permutes.  The boxes are 128-byte swizzled, which makes the
// word reads of 8 rows x 4 words conflict-free.
//
// K is cut over the CTAs of a cluster (at most 8); their fp32 sums meet in
// distributed shared memory and are added in rank order, so results repeat.
// Scales (and zero points) of up to 4096 weights' columns are staged in shared
// memory at a time.
//
// All waits are bounded, as in the other kernels.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "ragged.h"

namespace dg {
namespace {

constexpr int W4_ROWS = 64;      // weight rows (outputs) of a CTA
constexpr int W4_STEP = 256;     // weights of a row per stage
constexpr int W4_PANEL = 4096;   // weights of a row whose scales are staged at once
constexpr int W4_THREADS = 160;  // warp 0 producer, warps 1-4 consumers

template <int MT, int GROUP>
struct W4Cfg {
    static constexpr uint32_t Q_BYTES = W4_ROWS * 128;
    static constexpr uint32_t X_BOX = MT * 128;  // 64 values of MT tokens
    static constexpr uint32_t STAGE = Q_BYTES + 4 * X_BOX;
    static constexpr int STAGES = MT == 8 ? 5 : 4;
    static constexpr int GROUPS = W4_PANEL / GROUP;
    static constexpr int S_LD = GROUPS + 2;  // (one word more than a multiple of 32 banks)
    static constexpr int Z_LD = GROUPS + 4;
    static constexpr uint32_t S_BYTES = W4_ROWS * S_LD * 2;
    static constexpr uint32_t Z_BYTES = W4_ROWS * Z_LD;
    static constexpr int R_LD = W4_ROWS + 4;
    static constexpr uint32_t R_BYTES = MT * R_LD * 4;
    static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE + S_BYTES + Z_BYTES + R_BYTES + 256;
    static_assert(S_BYTES % 16 == 0 && Z_BYTES % 16 == 0 && R_BYTES % 16 == 0, "alignment");
};

template <int DT>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (DT == DT_BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The pair of 4-bit values at bits 0-3 and 16-19 of w as 16-bit floats minus
// the pair `sub`: or-ing q into the mantissa of 128 (bf16) or 1024 (fp16), where
// one unit is the last bit, gives 128 + q (1024 + q) exactly, and sub holds
// 128 + z (1024 + z).
template <int DT>
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t sub) {
    constexpr uint32_t magic = DT == DT_BF16 ? 0x43004300u : 0x64006400u;
    const uint32_t v = (w & 0x000F000Fu) | magic;
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

template <int DT>
__device__ __forceinline__ uint32_t w4_sub(int z) {
    return (DT == DT_BF16 ? 0x43004300u : 0x64006400u) + static_cast<uint32_t>(z) * 0x00010001u;
}

template <int DT>
__device__ __forceinline__ float w4_float(uint16_t u) {
    if constexpr (DT == DT_BF16) return __uint_as_float(static_cast<uint32_t>(u) << 16);
    return __half2float(__ushort_as_half(u));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// The slot-th non-empty group (whole warp), or -1; with its rows.
__device__ __forceinline__ int w4_group(const W4Params& p, int slot, int lane, int& row0, int& rows) {
    if (!p.offsets) {
        row0 = 0;
        rows = p.T;
        return 0;
    }
    int seen = 0;
    for (int base = 0; base < p.groups; base += 32) {
        const int g = base + lane;
        int lo = 0, hi = 0;
        if (g < p.groups) {
            lo = __ldg(p.offsets + g);
            hi = __ldg(p.offsets + g + 1);
            if (lo < 0 || hi < lo || hi > p.T) {
                if (p.status) atomicOr(p.status, STATUS_BAD_OFFSETS);
                lo = lo < 0 ? 0 : (lo > p.T ? p.T : lo);
                hi = hi < lo ? lo : (hi > p.T ? p.T : hi);
            }
        }
        const uint32_t m = __ballot_sync(0xffffffffu, hi > lo);
        const int n = __popc(m);
        if (slot < seen + n) {
            const int l = __fns(m, 0, slot - seen + 1);
            row0 = __shfl_sync(0xffffffffu, lo, l);
            rows = __shfl_sync(0xffffffffu, hi - lo, l);
            return base + l;
        }
        seen += n;
    }
    return -1;
}

template <int DT, int MT, int GROUP>
__global__ void __launch_bounds__(W4_THREADS) w4_kernel(const __grid_constant__ W4Params p) {
    using C = W4Cfg<MT, GROUP>;
    constexpr int NT = MT / 8;
    constexpr int CPG = GROUP / 32;  // 16-byte chunks per group
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint16_t* s_sm = reinterpret_cast<uint16_t*>(smem + C::STAGES * C::STAGE);
    uint8_t* z_sm = reinterpret_cast<uint8_t*>(s_sm) + C::S_BYTES;
    float* red = reinterpret_cast<float*>(z_sm + C::Z_BYTES);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red) + C::R_BYTES);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * C::STAGES;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * C::STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int unit = static_cast<int>(blockIdx.x) / p.splits;
    const int rank = static_cast<int>(blockIdx.x) - unit * p.splits;
    const int slot = unit / p.n_tiles;
    const int n0 = (unit - slot * p.n_tiles) * W4_ROWS;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8u * s, 1);
            mbar_init(empty0 + 8u * s, 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&p.tmap_q);
        prefetch_tmap(&p.tmap_x);
    }
    int row0 = 0, rows = 0;
    const int g = w4_group(p, slot, lane, row0, rows);
    __syncthreads();
    if (g < 0) return;  // (every CTA of the cluster alike)

    const int steps = (p.K + W4_STEP - 1) / W4_STEP;
    const int st0 = static_cast<int>(static_cast<int64_t>(steps) * rank / p.splits);
    const int st1 = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / p.splits);
    int stage = 0;
    uint32_t phase = 0;
    uint32_t armed = 0;

    for (int t0 = 0; t0 < rows; t0 += MT) {
        if (warp == 0) {
            if (lane == 0) {
                const uint64_t pol_q = rows <= MT ? l2_policy_evict_first() : l2_policy_evict_normal();
                const uint64_t pol_x = l2_policy_evict_last();
                for (int st = st0; st < st1; ++st) {
                    if (!mbar_wait(empty0 + 8u * stage, phase ^ 1u, abort_flag, p.status, p.timeout_ns))
                        break;
                    const uint32_t fb = full0 + 8u * stage;
                    mbar_arrive_expect_tx(fb, C::STAGE);
                    const uint32_t dst = smem_u32(smem) + stage * C::STAGE;
                    tma_load_3d(dst, &p.tmap_q, fb, st * 128, n0, g, pol_q);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tma_load_3d(dst + C::Q_BYTES + i * C::X_BOX, &p.tmap_x, fb,
                                    st * W4_STEP + 64 * i, row0 + t0, 0, pol_x);
                    ++armed;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            __syncwarp();
        } else {
            const int cw = warp - 1, gr = lane >> 2, t = lane & 3;
            const int r = cw * 16 + gr;  // rows r and r + 8 of the CTA's 64
            float total[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) total[j][i] = 0.0f;
            const int kg = p.K / GROUP;
            int panel = -1;
            bool ok = true;
            for (int st = st0; ok && st < st1; ++st) {
                const int in_panel = st - st0;
                if (in_panel / (W4_PANEL / W4_STEP) != panel) {
                    // stage the scales of the next panel (each warp its own 16 rows)
                    panel = in_panel / (W4_PANEL / W4_STEP);
                    const int gp0 = (st0 + panel * (W4_PANEL / W4_STEP)) * (W4_STEP / GROUP);
                    int n_g = (st1 - st) * (W4_STEP / GROUP);
                    if (n_g > C::GROUPS) n_g = C::GROUPS;
                    const int64_t base = (static_cast<int64_t>(g) * p.N + n0) * kg;
                    __syncwarp();
                    const uint16_t* src = static_cast<const uint16_t*>(p.scales);
#pragma unroll 4
                    for (int i = lane; i < 16 * n_g; i += 32) {
                        const int rr = cw * 16 + i / n_g, gg = i % n_g;
                        const bool in = n0 + rr < p.N && gp0 + gg < kg;
                        const int64_t at = base + static_cast<int64_t>(rr) * kg + gp0 + gg;
                        s_sm[rr * C::S_LD + gg] = in ? __ldg(src + at) : static_cast<uint16_t>(0);
                        if (p.zeros) z_sm[rr * C::Z_LD + gg] = in ? __ldg(p.zeros + at) : static_cast<uint8_t>(8);
                    }
                    __syncwarp();
                }
                int got = 1;
                if (lane == 0)
                    got = mbar_wait(full0 + 8u * stage, phase, abort_flag, p.status, p.timeout_ns) ? 1 : 0;
                ok = __shfl_sync(0xffffffffu, got, 0) != 0;
                if (!ok) break;
                // (every lane's reads below follow the barrier's completion)
                mbar_try_wait(full0 + 8u * stage, phase);
                const uint8_t* qs = smem + stage * C::STAGE;
                const uint8_t* xs = qs + C::Q_BYTES;
                const int gl0 = (in_panel % (W4_PANEL / W4_STEP)) * (W4_STEP / GROUP);
#pragma unroll
                for (int gg = 0; gg < W4_STEP / GROUP; ++gg) {
                    float acc[NT][4];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
                    const int gl = gl0 + gg;
                    uint32_t sub_lo = w4_sub<DT>(8), sub_hi = sub_lo;
                    if (p.zeros) {
                        sub_lo = w4_sub<DT>(z_sm[r * C::Z_LD + gl] & 15);
                        sub_hi = w4_sub<DT>(z_sm[(r + 8) * C::Z_LD + gl] & 15);
                    }
                    const float s_lo = w4_float<DT>(s_sm[r * C::S_LD + gl]);
                    const float s_hi = w4_float<DT>(s_sm[(r + 8) * C::S_LD + gl]);
#pragma unroll
                    for (int cc = 0; cc < CPG; ++cc) {
                        const int c = gg * CPG + cc;
                        const uint32_t at = static_cast<uint32_t>((c ^ gr) << 4) + t * 4;
                        const uint32_t lo = *reinterpret_cast<const uint32_t*>(qs + r * 128 + at);
                        const uint32_t hi = *reinterpret_cast<const uint32_t*>(qs + (r + 8) * 128 + at);
                        const uint32_t a1[4] = {w4_pair<DT>(lo, sub_lo), w4_pair<DT>(hi, sub_hi),
                                                w4_pair<DT>(lo >> 4, sub_lo),
                                                w4_pair<DT>(hi >> 4, sub_hi)};
                        const uint32_t a2[4] = {
                            w4_pair<DT>(lo >> 8, sub_lo), w4_pair<DT>(hi >> 8, sub_hi),
                            w4_pair<DT>(lo >> 12, sub_lo), w4_pair<DT>(hi >> 12, sub_hi)};
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const uint4 x = *reinterpret_cast<const uint4*>(
                                xs + (c >> 1) * C::X_BOX + (8 * j + gr) * 128 +
                                ((((c & 1) * 4 + t) ^ gr) << 4));
                            mma16816<DT>(acc[j], a1, __byte_perm(x.x, x.z, 0x5410),
                                         __byte_perm(x.x, x.z, 0x7632));
                            mma16816<DT>(acc[j], a2, __byte_perm(x.y, x.w, 0x5410),
                                         __byte_perm(x.y, x.w, 0x7632));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        total[j][0] = fmaf(s_lo, acc[j][0], total[j][0]);
                        total[j][1] = fmaf(s_lo, acc[j][1], total[j][1]);
                        total[j][2] = fmaf(s_hi, acc[j][2], total[j][2]);
                        total[j][3] = fmaf(s_hi, acc[j][3], total[j][3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8u * stage);
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            // [token][row] sums of this CTA
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                red[(8 * j + 2 * t) * C::R_LD + r] = total[j][0];
                red[(8 * j + 2 * t + 1) * C::R_LD + r] = total[j][1];
                red[(8 * j + 2 * t) * C::R_LD + r + 8] = total[j][2];
                red[(8 * j + 2 * t + 1) * C::R_LD + r + 8] = total[j][3];
            }
        }
        if (p.splits > 1)
            cluster_sync();
        else
            __syncthreads();
        // each CTA of the cluster adds and writes its share of the 64 rows
        const int share = W4_ROWS / p.splits;
        const int nt = rows - t0 < MT ? rows - t0 : MT;
        if (!*abort_flag) {
            for (int i = threadIdx.x; i < nt * share; i += W4_THREADS) {
                const int tok = i / share, rr = rank * share + i % share;
                const int n = n0 + rr;
                if (n >= p.N) continue;
                float v = 0.0f;
                if (p.splits > 1) {
                    const uint32_t at = smem_u32(red + tok * C::R_LD + rr);
                    for (int k = 0; k < p.splits; ++k)
                        v += ld_cluster_f32(mapa_shared(at, static_cast<uint32_t>(k)));
                } else {
                    v = red[tok * C::R_LD + rr];
                }
                if (p.bias) v += p.bias[g * p.stride_bias + n];
                v = apply_act(v, p.act);
                const int64_t off = static_cast<int64_t>(row0 + t0 + tok) * p.ldc + n;
#if DG_DEBUG
                if (!DG_CHECK(off >= 0 && off < p.dbg_c_elems, p.status, STATUS_CHECK_BOUNDS)) continue;
#endif
                store_elem(static_cast<char*>(p.C) + off * dt_size(p.c_dtype), p.c_dtype, v);
            }
        }
        // the sums are read before the next tokens' (or the exit) replace them
        if (p.splits > 1)
            cluster_sync();
        else
            __syncthreads();
    }
    // every issued copy lands before the CTA exits
    if (warp == 0 && lane == 0)
        for (int s = 0; s < C::STAGES && static_cast<uint32_t>(s) < armed; ++s) {
            const uint32_t fills = (armed - 1u - s) / C::STAGES + 1u;
            const uint64_t begin = globaltimer_ns();
            while (!mbar_try_wait(full0 + 8u * s, (fills - 1u) & 1u))
                if (globaltimer_ns() - begin > p.timeout_ns) break;
        }
}

template <int DT, int MT, int GROUP>
cudaError_t launch_one(const W4Params& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.n_tiles) * p.slots * p.splits);
    cfg.blockDim = dim3(W4_THREADS);
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
