// Instantiations of the ragged kernel for products grouped by expert.
#include "ragged_kernel.cuh"

namespace dg {

cudaError_t rg_launch_rows(int cg, int bt, const RgParams& p, int grid, cudaStream_t stream) {
    if (cg == 2 && bt == 256) return rg_launch<2, 256, RG_ROWS>(p, grid, stream);
    if (cg == 1 && bt == 128) return rg_launch<1, 128, RG_ROWS>(p, grid, stream);
    if (cg == 1 && bt == 32) return rg_launch<1, 32, RG_ROWS>(p, grid, stream);
    return cudaErrorInvalidValue;
}

cudaError_t rg_prepare_rows() {
    cudaError_t e = rg_prepare<2, 256, RG_ROWS>();
    if (e == cudaSuccess) e = rg_prepare<1, 128, RG_ROWS>();
    if (e == cudaSuccess) e = rg_prepare<1, 32, RG_ROWS>();
    return e;
}

}  // namespace dg
