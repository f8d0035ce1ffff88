// The products of the orthogonalised update in one launch: per step
//   Y = X X^T + shift,  P = c Y Y + constant  (both symmetric: tiles on and below
//   the diagonal),  X <- P X,
// each needing the one before, but matrix by matrix only.  As fifteen launches the
// chain spent 6 to 8 us a product on launch, set-up and the first loads, whatever
// its size (a 256 x 256 matrix took 122 us); here the CTAs stay.  The tiles of all
// products are dealt to them in one order, and a matrix has one counter: each
// epilogue warp adds to it (release) after storing its part of a tile, and before
// a tile's loads the producer waits (acquire) for all tiles of the matrix's
// products before.  With several matrices the products overlap and their last,
// partly filled rounds of tiles with them (16 matrices of 1024 x 2048: 510 us,
// against 663 with a barrier over the grid after every product and with a X and b S
// read back in the epilogues instead of the constants on the diagonals).  The launch is
// cooperative, so every CTA is resident, and a tile waits only for tiles that come
// before it in that order; the wait is bounded like all others.
#include "ragged_kernel.cuh"

namespace dg {
namespace {

// Waits (bounded) until `target` arrivals have been counted.
__device__ __forceinline__ bool seq_wait(const unsigned int* arrived, unsigned int target,
                                         const RgParams& p, volatile int* abort_flag) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        unsigned int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(arrived) : "memory");
        if (static_cast<int>(v - target) >= 0) return true;
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

// One role's walk over the products: body(parameters, product of the step, first
// tile, arrivals of a matrix before the product).
template <int CG, int BT, typename Body>
__device__ __forceinline__ void seq_walk(const RgSeq& q, const RgCta& x, const RgRole& r, Body body) {
    int base = 0;               // tiles of the products before, modulo the clusters
    unsigned int before = 0;
    for (int step = 0; r.ok && step < q.steps; ++step)
#pragma unroll 1
        for (int k = 0; r.ok && k < 3; ++k) {
            const RgParams& p = q.ph[seq_phase(q, step, k)];
            body(p, k, x.cl >= base ? x.cl - base : x.cl - base + x.ncl, before);
            base = (base + p.total_tiles) % x.ncl;
            before += static_cast<unsigned int>(p.per_group) * (RgCfg<CG, BT>::EPI_WARPS * CG);
        }
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
        seq_walk<CG, BT>(q, x, r, [&](const RgParams& p, int k, int first, unsigned int before) {
            auto gate = [&](int group) {
                if (before == 0) return true;
                if (!seq_wait(q.arrived + group, before, p, x.abort_flag)) return false;
                fence_proxy_async_global();  // plain stores before, TMA reads after
                return true;
            };
            if (x.lane == 0) {
                prefetch_tmap(&p.tmap_a);
                prefetch_tmap(&p.tmap_b);
            }
            if (k == 2)
                rg_produce<CG, BT, RG_ROWS>(p, x, r, first, gate);
            else
                rg_produce<CG, BT, RG_SYM>(p, x, r, first, gate);
        });
        rg_produce_end<CG, BT>(q.ph[0], x, r);
    } else if (warp == 1) {
        seq_walk<CG, BT>(q, x, r, [&](const RgParams& p, int k, int first, unsigned int) {
            if (k == 2)
                rg_issue<CG, BT, RG_ROWS>(p, x, r, first);
            else
                rg_issue<CG, BT, RG_SYM>(p, x, r, first);
        });
        rg_issue_end<CG>(q.ph[0], x, r);
    } else {
        uint8_t* buf = x.smem + C::STAGES * C::STAGE_BYTES + (warp - 2) * C::EPI_WARP;
        auto told = [&](int group) {
            fence_proxy_async_global();  // this thread's stores before TMA reads of others
            __syncwarp();
            if (x.lane == 0)
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(q.arrived + group)
                             : "memory");
        };
        seq_walk<CG, BT>(q, x, r, [&](const RgParams& p, int k, int first, unsigned int) {
            if (k == 2)
                rg_epilogue<CG, BT, RG_ROWS, false>(p, x, r, first, warp, buf, told);
            else
                rg_epilogue<CG, BT, RG_SYM, false>(p, x, r, first, warp, buf, told);
        });
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
    if (cg == 1 && bt == 64) return launch_seq<1, 64>(q, grid, stream);
    return cudaErrorInvalidValue;
}

cudaError_t rg_prepare_seq() {
    cudaError_t e = prepare_seq<2, 256>();
    if (e == cudaSuccess) e = prepare_seq<1, 128>();
    if (e == cudaSuccess) e = prepare_seq<1, 64>();
    return e;
}

}  // namespace dg
