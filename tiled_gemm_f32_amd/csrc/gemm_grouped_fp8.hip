// fp8 products with block scales on the tiles of gemm_grouped_tile.hpp.
#include "gemm_grouped_tile.hpp"

namespace gemm {

hipError_t launch_grouped_fp8(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream) {
    return launch_typed<GEMM_DTYPE_FP8F32>(op_b, dma, p, stream);
}

}  // namespace gemm
