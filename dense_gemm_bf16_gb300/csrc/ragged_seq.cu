// The products of the orthogonalised update in one launch: per step
//   S = X X^T,  P = b S + c S S  (both symmetric: tiles on and below the diagonal),
//   X <- a X + P X,
// every one needing all of the one before.  As fifteen launches the chain spent
// 6 to 8 us a product on launch, set-up and the first loads, whatever its size
// (a 256 x 256 matrix took 122 us); here the CTAs stay, and between products
// meet at one counter: each CTA's epilogue warps finish their stores, one thread
// adds to the counter (release), and the producers' next loads wait for all CTAs
// (acquire).  The launch is cooperative, so every CTA the counter waits for is
// resident; the wait is bounded like all others.
#include "ragged_kernel.cuh"

namespace dg {
namespace {

// Waits (bounded) until `target` CTA arrivals have been counted.
__device__ __forceinline__ bool seq_wait(const unsigned int* arrived, unsigned int target,
                                         const RgParams& p, volatile int* abort_flag) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        unsigned int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(arrived) : "memory");
        if (v >= target) return true;
        if ((it & 15u) == 0) {
            if (*abort_flag) return false;
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > p.timeout_ns) {
                *abort_flag = 1;
                if (p.status) DG_SET_TIMEOUT(p.status);
                return false;
            }
        }
    }
}

__device__ __forceinline__ int seq_phase(const RgSeq& q, int step, int k) {
    return k == 2 && step == q.steps - 1 ? 6 : (step & 1) * 3 + k;
}

template <int CG, int BT>
__global__ void __launch_bounds__(RgCfg<CG, BT>::threads(RG_SYM), 1)
    ragged_seq_kernel(const __grid_constant__ RgSeq q) {
    using C = RgCfg<CG, BT>;
    extern __shared__ uint8_t smem_raw[];
    const RgCta x = rg_setup<CG, BT>(q.ph[0], smem_raw);
    const int warp = threadIdx.x >> 5;
    RgRole r;
    if (warp == 0) {
        for (int step = 0; r.ok && step < q.steps; ++step)
#pragma unroll 1
            for (int k = 0; r.ok && k < 3; ++k) {
                const RgParams& p = q.ph[seq_phase(q, step, k)];
                const unsigned int done = static_cast<unsigned int>(3 * step + k);
                // (lane 0, with the first tile of the product already known)
                auto gate = [&]() {
                    if (done == 0) return true;
                    if (!seq_wait(q.arrived, done * gridDim.x, p, x.abort_flag)) return false;
                    fence_proxy_async_global();  // plain stores before, TMA reads after
                    mbar_arrive(x.gate_bar);
                    return true;
                };
                if (x.lane == 0) {
                    prefetch_tmap(&p.tmap_a);
                    prefetch_tmap(&p.tmap_b);
                }
                if (k == 2)
                    rg_produce<CG, BT, RG_ROWS>(p, x, r, gate);
                else
                    rg_produce<CG, BT, RG_SYM>(p, x, r, gate);
            }
        rg_produce_end<CG, BT>(q.ph[0], x, r);
    } else if (warp == 1) {
        for (int step = 0; r.ok && step < q.steps; ++step)
#pragma unroll 1
            for (int k = 0; r.ok && k < 3; ++k) {
                const RgParams& p = q.ph[seq_phase(q, step, k)];
                if (k == 2)
                    rg_issue<CG, BT, RG_ROWS>(p, x, r);
                else
                    rg_issue<CG, BT, RG_SYM>(p, x, r);
            }
        rg_issue_end<CG>(q.ph[0], x, r);
    } else {
        uint8_t* buf = x.smem + C::STAGES * C::STAGE_BYTES + (warp - 2) * C::EPI_WARP;
        uint32_t gate_phase = 0;
        for (int step = 0; step < q.steps; ++step)
#pragma unroll 1
            for (int k = 0; k < 3; ++k) {
                const RgParams& p = q.ph[seq_phase(q, step, k)];
                const unsigned int done = static_cast<unsigned int>(3 * step + k);
                const bool tile = x.cl < p.total_tiles;  // this CTA has a tile of the product
                auto gate = [&]() {
                    if (done == 0) return true;
                    const bool ok = rg_warp_wait(x.gate_bar, gate_phase, x.lane, x.abort_flag, p);
                    gate_phase ^= 1u;
                    return ok;
                };
                // (after a failed wait the barriers below still run, so that no
                // warp is left at them)
                if (r.ok) {
                    if (k == 2)
                        rg_epilogue<CG, BT, RG_ROWS, false>(p, x, r, warp, buf, gate);
                    else
                        rg_epilogue<CG, BT, RG_SYM, false>(p, x, r, warp, buf, gate);
                }
                fence_proxy_async_global();  // this thread's stores before TMA reads of others
                asm volatile("bar.sync 2, %0;" ::"n"(32 * C::EPI_WARPS) : "memory");
                if (threadIdx.x == 64) {
                    // (a CTA without a tile must not count for this product before
                    // every CTA has finished the one before)
                    if (!tile) seq_wait(q.arrived, done * gridDim.x, p, x.abort_flag);
                    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(q.arrived)
                                 : "memory");
                }
            }
    }
    rg_teardown<CG, BT>(x);
}

template <int CG, int BT>
cudaError_t launch_seq(const RgSeq& q, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(RgCfg<CG, BT>::threads(RG_SYM));
    cfg.dynamicSmemBytes = RgCfg<CG, BT>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ragged_seq_kernel<CG, BT>, q);
}

template <int CG, int BT>
cudaError_t prepare_seq() {
    return cudaFuncSetAttribute(ragged_seq_kernel<CG, BT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(RgCfg<CG, BT>::SMEM));
}

}  // namespace

cudaError_t rg_launch_seq(int cg, int bt, const RgSeq& q, int grid, cudaStream_t stream) {
    if (cg == 2 && bt == 256) return launch_seq<2, 256>(q, grid, stream);
    if (cg == 1 && bt == 128) return launch_seq<1, 128>(q, grid, stream);
    return cudaErrorInvalidValue;
}

cudaError_t rg_prepare_seq() {
    const cudaError_t e = prepare_seq<2, 256>();
    return e != cudaSuccess ? e : prepare_seq<1, 128>();
}

}  // namespace dg
