// Grouped fp32 products and their weight gradients on the tiles of
// gemm_grouped_tile.hpp.
#include "gemm_grouped_tile.hpp"

namespace gemm {
namespace {

// One kernel by name, so that this source shows which template it makes (and counts among those whose
// kernels the resource table has to list); the launchers below make the others.
template __global__ void grouped_tile_kernel<TileConfig<GEMM_DTYPE_F32, 2, 2, 2, 2, false, false, true>>(GroupedParams, int, int);

}  // namespace

hipError_t launch_grouped_f32(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream) {
    return launch_typed<GEMM_DTYPE_F32>(op_b, dma, p, stream);
}

hipError_t launch_wgrad_f32(bool dma, const GroupedParams &p, hipStream_t stream) {
    return launch_wgrad<GEMM_DTYPE_F32>(dma, p, stream);
}

}  // namespace gemm
