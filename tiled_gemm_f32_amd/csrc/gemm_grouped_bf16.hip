// Grouped bf16 products and their weight gradients on the tiles of
// gemm_grouped_tile.hpp.
#include "gemm_grouped_tile.hpp"

namespace gemm {

hipError_t launch_grouped_bf16(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream) {
    return launch_typed<GEMM_DTYPE_BF16F32>(op_b, dma, p, stream);
}

// Weight gradients: both operands are walked down their rows.  Results are
// fp32, so a tile's store takes twice the time.
hipError_t launch_wgrad_bf16(bool dma, const GroupedParams &p, hipStream_t s) {
    constexpr int DT = GEMM_DTYPE_BF16F32;
    // The outputs of all groups together, each as deep as a group has rows.
    const double slabs = std::ceil((double)p.M / p.groups / 64);
    switch (tile_size((double)p.N * p.groups, p.K, slabs, p.groups, dma ? kTile256 : kTile128, 2.0)) {
        case kTile256:
        case kTileWide:
            if (dma) return launch_grouped_tile<TileConfig<DT, 4, 2, 2, 4, true, true, true>>(p, s);
        case kTile128:
            return dma ? launch_grouped_tile<TileConfig<DT, 2, 2, 2, 2, true, true, true>>(p, s)
                       : launch_grouped_tile<TileConfig<DT, 2, 2, 2, 2, true, true, false>>(p, s);
        default:
            return dma ? launch_grouped_tile<TileConfig<DT, 1, 2, 2, 2, true, true, true>>(p, s)
                       : launch_grouped_tile<TileConfig<DT, 1, 2, 2, 2, true, true, false>>(p, s);
    }
}

}  // namespace gemm
