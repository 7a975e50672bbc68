// Products of 8-bit integers with a scale for each token and channel: the tiles of gemm_grouped_tile.hpp with
// 32-bit accumulators, and a general kernel for the calls that those do not take, where a row of an operand is
// shorter than one 16-byte load, or rows lie so far apart that a tile's panel passes the 2 GiB a buffer load can
// address.  Every layout, stride and alignment is right here.  An output tile of 64 x 64, 64 k of both operands
// staged a byte at a time through registers into LDS as [row][k], four waves each keeping a quarter of the tile
// in 32-bit accumulators, two v_mfma_i32_32x32x32_i8 a slab.  Such calls are bound by their results' stores, or
// by one memory transaction a row.
#include "gemm_grouped_tile.hpp"

namespace gemm {
namespace {

constexpr int BT = 64, kBK = 64, kThreads = 256;
constexpr int kStride = kBK + 16;            // bytes a panel row takes in LDS

// 16 values of a panel's slab into LDS.  KCONT: element (r, k) at base[r * ld + k], else at base[k * ld + r].
template <bool KCONT>
__device__ __forceinline__ void stage_panel(const int8_t *base, int64_t ld, int rows, int len, int k0, char *lds) {
#pragma unroll
    for (int i = 0; i < BT * kBK / kThreads; ++i) {
        const int at = threadIdx.x + i * kThreads;
        const int r = KCONT ? at / kBK : at % BT, k = KCONT ? at % kBK : at / BT;
        char v = 0;
        if (r < rows && k < len - k0) v = base[KCONT ? (int64_t)r * ld + k0 + k : ((int64_t)k0 + k) * ld + r];
        lds[r * kStride + k] = v;
    }
}

template <bool BN>
__global__ void __launch_bounds__(kThreads)
int8_general_kernel(GroupedParams p, int tiles_n) {
    __shared__ __attribute__((aligned(16))) char lds_a[BT * kStride], lds_b[BT * kStride];
    const GroupTile t = find_tile(p, blockIdx.x, BT, tiles_n, 8);
    if (t.rows <= 0) return;
    const int group = max(t.group, 0), row0 = t.row0, n0 = t.tn * BT, cols = min(BT, p.N - n0);
    const int len = t.group < 0 ? 0 : p.K;
    const int8_t *a = static_cast<const int8_t *>(p.A) + (int64_t)row0 * p.lda;
    const int8_t *b = static_cast<const int8_t *>(p.B) + (int64_t)group * p.stride_b +
                      (BN ? (int64_t)n0 : (int64_t)n0 * p.ldb);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, l32 = lane & 31;
    i32x16 acc = {};
    for (int k0 = 0; k0 < len; k0 += kBK) {
        stage_panel<true>(a, p.lda, t.rows, len, k0, lds_a);
        stage_panel<!BN>(b, p.ldb, cols, len, k0, lds_b);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kBK / 32; ++q) {
            const i32x4 fa = *reinterpret_cast<const i32x4 *>(&lds_a[(wm * 32 + l32) * kStride + 32 * q + 16 * h]);
            const i32x4 fb = *reinterpret_cast<const i32x4 *>(&lds_b[(wn * 32 + l32) * kStride + 32 * q + 16 * h]);
            acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa, fb, acc, 0, 0, 0);
        }
        __syncthreads();
    }
    // Register r of lane (h, l32) is row 8*(r/4) + 4*h + r%4, column l32 of its block.
    const int col = wn * 32 + l32;
    if (col >= cols) return;
    const bool owned = t.group >= 0, scaled = len > 0;
    const float sb = scaled ? p.ts.b[(int64_t)group * p.ts.b_group + (int64_t)(n0 + col) * p.ts.b_col] : 0.0f;
    const float bias = owned && p.ts.bias != nullptr ? p.ts.bias[(int64_t)group * p.ts.bias_group + n0 + col] : 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = wm * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row >= t.rows) continue;
        const int64_t at = (int64_t)(row0 + row) * p.ldo + n0 + col;
        const float v = scaled ? int8_value((float)acc[r], p.ts.a[(int64_t)(row0 + row) * p.ts.a_row], sb, bias) : bias;
        if (p.out_type == GEMM_OUT_BF16) static_cast<uint16_t *>(p.out)[at] = to_bf16(v);
        else static_cast<float *>(p.out)[at] = v;
    }
}

template <bool BN> hipError_t launch_general(const GroupedParams &p, hipStream_t stream) {
    GroupedParams args = p;
    int tiles_n = (p.N + BT - 1) / BT;
    const int64_t tiles = most_row_tiles(p.M, p.groups, BT, p.ends != nullptr) * tiles_n;
    void *argv[] = {&args, &tiles_n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&int8_general_kernel<BN>), dim3((unsigned)tiles),
                           dim3(kThreads), argv, 0, stream);
}

}  // namespace

hipError_t launch_grouped_int8(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream) {
    return launch_typed<kInt8>(op_b, dma, p, stream);
}

hipError_t launch_int8_general(int32_t op_b, const GroupedParams &p, hipStream_t stream) {
    return op_b == GEMM_OP_N ? launch_general<true>(p, stream) : launch_general<false>(p, stream);
}

}  // namespace gemm
