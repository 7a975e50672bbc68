// Grouped and block-scaled products with few output tiles: the waves of a
// workgroup share out k instead of the tile.
//
// A workgroup makes 32 rows by one 32-column fragment of one group, or by the
// columns that 128 bytes of a k row hold where B is walked down k.  Its waves
// take the slabs of 128 bytes of k in turn, each through an LDS stage of its
// own, so that the loop has no barrier; a slab's fragments are read into
// registers at once, and the next one lands under their products.  The waves'
// partial tiles are added through LDS in a fixed order.  A larger tile moves
// fewer bytes a product, but its slabs follow one another: with no more tiles
// than compute units a call takes as long as one tile's chain of slabs, which
// is an eighth here.  (Two stages a wave, and so one workgroup a compute unit
// instead of two, were no faster at 256 tiles and slower at more: 1000 x 512 x
// 4096 bf16, 512 tiles, 17.4 us, 15.2 so.)
//
// On inputs that change from call to call: 128 x 2000 x 8000 fp8 12.0 us (16 MB
// of weights: 1.3 TB/s, bound by the latency of eight slabs a wave; 11 where
// the caches hold the weights); 16 x 4096 x 4096 fp8 against K x N weights 13.5
// us (9.9), 16 x 8192 x 8192 24 us: a workgroup for each 128 columns, which is
// none for most compute units; 64 rows over 32 experts of 4096 x 4096 fp8, K x
// N, 21 of them with rows, 72 us (4.9 TB/s); 64 x 1000 x 1024 fp32 7.8 us, 3.5 of
// them matrix instructions.
//
// Loads, layouts and fragments are those of gemm_grouped_tile.hpp with one
// wave.  fp8: the products of the two block scales are made once a workgroup,
// in LDS, under the first loads.
#include "gemm_grouped_tile.hpp"

namespace gemm {
namespace {

// Waves, and (fp8) floats of LDS beside the stages for 32 rows' scales: two workgroups of
// one-fragment tiles share a compute unit's 160 KB.
template <class C> struct Deep {
    static constexpr int kWaves = C::FN == 4 ? 7 : 8;
    static constexpr int kScales = C::DT != GEMM_DTYPE_FP8F32 ? 1 : C::FN == 4 ? 4864 : 4000;
};
template <class C>
__global__ void __launch_bounds__(64 * Deep<C>::kWaves, C::FN == 1 ? 4 : 2)
grouped_deep_kernel(GroupedParams p, int tiles_n) {
    constexpr bool FP8 = C::DT == GEMM_DTYPE_FP8F32;
    constexpr int FN = C::FN, BN = C::BN, WAVES = Deep<C>::kWaves;
    constexpr int NA = Loader<C, false, 32>::kLoads, NB = Loader<C, C::BKN, BN>::kLoads;
    static_assert(C::BM == 32 && C::NW == 1, "");
    static_assert(!C::BKN || BN * C::esz == kSlab, "a k row of the tile is a slab's 128 bytes");
    __shared__ __attribute__((aligned(1024))) char stages[WAVES * C::kStage];
    __shared__ float scales[Deep<C>::kScales];

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    GroupTile t = find_tile(p, blockIdx.x, 32, tiles_n, 4);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (t.rows <= 0) return;
    const int owner = __builtin_amdgcn_readfirstlane(t.group), group = max(owner, 0);
    const int row0 = __builtin_amdgcn_readfirstlane(t.row0), n0 = BN * __builtin_amdgcn_readfirstlane(t.tn);
    const int out_cols = min(BN, p.N - n0);

    Loader<C, false, 32> a;
    Loader<C, C::BKN, BN> b;
    a.base = static_cast<const char *>(p.A) + (int64_t)row0 * p.lda * C::esz;
    b.base = static_cast<const char *>(p.B) +
             ((int64_t)group * p.stride_b + (C::BKN ? (int64_t)n0 : (int64_t)n0 * p.ldb)) * C::esz;
    a.rows = t.rows;
    b.rows = out_cols;
    const int len = owner < 0 ? 0 : p.K;
    a.len = b.len = len;
    a.ld = p.lda * C::esz;
    b.ld = p.ldb * C::esz;
    a.init(0, lane);
    b.init(0, lane);

    char *const st = stages + wave * C::kStage;
    auto fetch = [&](int slab) __attribute__((always_inline)) {
        if constexpr (C::DMA) {
            const rsrc_t ra = a.source(slab), rb = b.source(slab);
#pragma unroll
            for (int j = 0; j < NB; ++j) b.load(rb, st + C::kA, 0, j);
#pragma unroll
            for (int j = 0; j < NA; ++j) a.load(ra, st, 0, j);
        } else {
            a.hold(slab, 0);
            b.hold(slab, 0);
        }
    };

    const int slabs = slabs_of(len, C::BK);
    f32x16 acc[FN] = {};
    // This wave's slabs: wave, wave + WAVES, ...
    const int mine = (slabs - wave + WAVES - 1) / WAVES;
    if (mine > 0) fetch(wave);
    if constexpr (FP8) {
        const float *sa = p.sc.a + (int64_t)row0 * p.sc.a_row;
        const float *sb = p.sc.b + (int64_t)group * p.sc.b_group + (int64_t)(n0 / GEMM_SCALE_BLOCK) * p.sc.b_n;
        for (int i = tid; i < 32 * slabs; i += 64 * WAVES) {
            const int k = i / 32, r = min(i % 32, t.rows - 1);
            scales[i] = sa[(int64_t)r * p.sc.a_row + k * p.sc.a_block] * sb[k * p.sc.b_k];
        }
        __syncthreads();
    }
    const uint32_t a_base = frag_base<C, false>(0, lane), b_base = frag_base<C, C::BKN>(0, lane);
    // Slab i of the wave's; `last`: it may end K.
    auto step = [&](int i, bool last) __attribute__((always_inline)) {
        const int slab = wave + i * WAVES;
        if constexpr (C::DMA) {
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
        } else {
            a.stash(st, 0, 0, lane);
            b.stash(st + C::kA, 0, 0, lane);
        }
        if (last && (!C::DMA || len % C::BK != 0) && slab == slabs - 1) {
            a.cut(slab, st, lane);
            b.cut(slab, st + C::kA, lane);
        }
        const FragOf<C::esz> fa = read_frag<C, false>(st, a_base, 0);
        FragOf<C::esz> fb[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = read_frag<C, C::BKN>(st + C::kA, b_base, j);
        const float s = FP8 ? scales[32 * slab + l32] : 0.0f;
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));          // read before the next slab lands on them
        __builtin_amdgcn_sched_barrier(0);
        if (!last) fetch(slab + WAVES);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if constexpr (FP8) {
                const f32x16 part = product<1>(fa, fb[j], 1, product<1>(fa, fb[j], 0, f32x16{}));
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[j][e] = fmaf(part[e], s, acc[j][e]);
            } else {
                acc[j] = product<C::esz>(fa, fb[j], 1, product<C::esz>(fa, fb[j], 0, acc[j]));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int i = 0; i + 1 < mine; ++i) step(i, false);
    if (mine > 0) step(mine - 1, true);

    // Partial tiles: row l32 of 8 * FN chunks of 4 columns, chunk c at c ^ (row & 7).
    float *const tile = reinterpret_cast<float *>(st);
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f32x4 *>(tile + BN * l32 + 4 * ((8 * j + 2 * g + h) ^ (l32 & 7))) =
                f32x4{acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
    __syncthreads();
    for (int e = tid; e < 32 * BN / 2; e += 64 * WAVES) {
        const int row = e / (BN / 2), col = 2 * (e % (BN / 2));
        if (row >= t.rows || col >= out_cols) continue;
        const char *from = stages + 4 * (BN * row + 4 * ((col >> 2) ^ (row & 7)) + (col & 3));
        float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float *at = reinterpret_cast<const float *>(from + w * C::kStage);
            v0 += at[0];
            v1 += at[1];
        }
        v0 *= p.alpha;
        v1 *= p.alpha;
        const int64_t at = (int64_t)(row0 + row) * p.ldo + n0 + col;
        const bool both = col + 1 < out_cols;
        if (p.out_type == GEMM_OUT_BF16) {
            uint16_t *o = static_cast<uint16_t *>(p.out) + at;
            o[0] = to_bf16(v0);
            if (both) o[1] = to_bf16(v1);
        } else {
            float *o = static_cast<float *>(p.out) + at;
            o[0] = v0;
            if (both) o[1] = v1;
        }
    }
}

template <int DT, bool BKN, bool DMA> hipError_t launch(const GroupedParams &p, hipStream_t stream) {
    constexpr int FN = deep_columns(DT, BKN) / 32;
    typedef TileConfig<DT, 1, FN, 1, 1, false, BKN, DMA> C;
    GroupedParams args = p;
    int tiles_n = (p.N + C::BN - 1) / C::BN;
    const int64_t tiles = most_row_tiles(p.M, p.groups, 32, p.ends != nullptr) * tiles_n;
    void *argv[] = {&args, &tiles_n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&grouped_deep_kernel<C>), dim3((unsigned)tiles),
                           dim3(64 * Deep<C>::kWaves), argv, 0, stream);
}
template <int DT> hipError_t launch_op(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t s) {
    if (op_b == GEMM_OP_T) return dma ? launch<DT, false, true>(p, s) : launch<DT, false, false>(p, s);
    if constexpr (DT != GEMM_DTYPE_FP8F32)
        if (!dma) return launch<DT, true, false>(p, s);
    return launch<DT, true, true>(p, s);
}

}  // namespace

bool deep_takes(int32_t dtype, int32_t op_b, bool dma, const GroupedParams &p) {
    if (dtype == GEMM_DTYPE_FP8F32) {
        // (128 columns of a slab, their fragments and the partial tile leave no registers to stage through.)
        if (op_b == GEMM_OP_N && !dma) return false;
        const int64_t most = op_b == GEMM_OP_N ? 4864 : 4000;       // Deep::kScales
        if (((int64_t)p.K + GEMM_SCALE_BLOCK - 1) / GEMM_SCALE_BLOCK * 32 > most) return false;
    }
    // (A launch counts its threads in 32 bits.)
    return most_row_tiles(p.M, p.groups, 32, p.ends != nullptr) * ((p.N + 31) / 32) < 1 << 20;
}

hipError_t launch_grouped_deep(int32_t dtype, int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream) {
    if (dtype == GEMM_DTYPE_F32) return launch_op<GEMM_DTYPE_F32>(op_b, dma, p, stream);
    if (dtype == GEMM_DTYPE_BF16F32) return launch_op<GEMM_DTYPE_BF16F32>(op_b, dma, p, stream);
    return launch_op<GEMM_DTYPE_FP8F32>(op_b, dma, p, stream);
}

}  // namespace gemm
