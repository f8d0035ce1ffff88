// Instantiations of the ragged kernel: symmetric products.
#include "ragged_kernel.cuh"

namespace dg {

cudaError_t rg_launch_sym(int cg, int bt, const RgParams& p, int grid, cudaStream_t stream) {
    if (cg == 2 && bt == 256) return rg_launch<2, 256, RG_SYM>(p, grid, stream);
    if (cg == 1 && bt == 128) return rg_launch<1, 128, RG_SYM>(p, grid, stream);
    return cudaErrorInvalidValue;
}

cudaError_t rg_prepare_sym() {
    cudaError_t e = rg_prepare<2, 256, RG_SYM>();
    if (e == cudaSuccess) e = rg_prepare<1, 128, RG_SYM>();
    return e;
}

}  // namespace dg
