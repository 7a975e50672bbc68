// Grouped bf16 products and their weight gradients on the tiles of
// gemm_grouped_tile.hpp.
#include "gemm_grouped_tile.hpp"

namespace gemm {

hipError_t launch_grouped_bf16(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream) {
    return launch_typed<GEMM_DTYPE_BF16F32>(op_b, dma, p, stream);
}

// Weight gradients: both operands are walked down their rows.
hipError_t launch_wgrad_bf16(bool dma, const GroupedParams &p, hipStream_t s) {
    auto tiles = [&](int64_t b) { return ((p.N + b - 1) / b) * ((p.K + b - 1) / b) * p.groups; };
    constexpr int DT = GEMM_DTYPE_BF16F32;
    if (tiles(128) < 256)
        return dma ? launch_grouped_tile<TileConfig<DT, 1, 2, 2, 2, true, true, true>>(p, s)
                   : launch_grouped_tile<TileConfig<DT, 1, 2, 2, 2, true, true, false>>(p, s);
    if (!dma) return launch_grouped_tile<TileConfig<DT, 2, 2, 2, 2, true, true, false>>(p, s);
    return tiles(256) >= 256 ? launch_grouped_tile<TileConfig<DT, 4, 2, 2, 4, true, true, true>>(p, s)
                             : launch_grouped_tile<TileConfig<DT, 2, 2, 2, 2, true, true, true>>(p, s);
}

}  // namespace gemm
