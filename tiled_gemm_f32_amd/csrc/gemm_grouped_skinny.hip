// Products of few rows (of a decoding step, or of a group that few tokens
// went to) with weights stored N x K: bound by reading the weights once.
//
// out[i][j] = sum over k of A[i][k] * B[j][k], in blocks of 128 bytes of k.
// A lane of the 16-row matrix instructions (fp8: v_mfma_f32_16x16x128_f8f6f4,
// bf16: two v_mfma_f32_16x16x32_bf16) holds 32 bytes of one weight row and 32
// of one row of A, so both go from memory straight into its operands, with no
// trip through LDS.  A workgroup makes 16*MT rows by 16*CG columns; its waves
// take the blocks in turn, each keeping two batches of them in flight.  Eight
// partial sums of every result are added through LDS in a fixed order: one a
// wave of eight, or two a wave of four.  Four waves leave room for two
// workgroups a compute unit, whose starts and ends hide behind each other's
// loads; eight cover the memory's latency where a call has no more workgroups
// than compute units.  Workgroups start at blocks spread over K and wrap
// around, so that rows a power of two apart do not press on the same memory
// channels at once; where a column starts depends on the column only, so a
// row's results do not depend on the other rows and groups of a call.
//
// 16 x 8192 x 8192 fp8: 17.5 to 19 us (3.5 to 3.8 TB/s of weights; a third is
// the launch and the first loads' latency).  64 rows over 32 experts of 4096 x
// 4096 fp8, 26 of them with rows: 88 to 95 us (4.6 to 5 TB/s, a copy's rate).
//
// fp8 with block scales: a block is one scale block.  Its partial sums are
// multiplied by a(row) * b(column block) as they are added; the products of
// the two scales are made once a workgroup, in LDS, under the first loads.
#include "gemm_grouped.hpp"

namespace gemm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kSums = 8;                  // partial sums of a result: blocks b with equal b % 8
constexpr int kBlock = 128;               // bytes of k a block
constexpr int kScaleFloats = 16384;       // of LDS: 16*MT rows by ceil(K / 128) blocks

template <int DT> struct Skinny;
template <> struct Skinny<GEMM_DTYPE_FP8F32> {
    static constexpr int esz = 1;
    static __device__ __forceinline__ f32x4 mma(const u32x4 (&w)[2], const u32x4 (&a)[2], f32x4 acc) {
        i32x8 wv, av;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            wv[e] = (int)w[e >> 2][e & 3];
            av[e] = (int)a[e >> 2][e & 3];
        }
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, acc, 0, 0, 0, 0, 0, 0);
    }
};
template <> struct Skinny<GEMM_DTYPE_BF16F32> {
    static constexpr int esz = 2;
    static __device__ __forceinline__ f32x4 mma(const u32x4 (&w)[2], const u32x4 (&a)[2], f32x4 acc) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[h]),
                                                          __builtin_bit_cast(bf16x8, a[h]), acc, 0, 0, 0);
        return acc;
    }
};

template <int DT, int MT, int CG, int UNROLL, int WAVES>
__global__ void __launch_bounds__(64 * WAVES)
grouped_skinny_kernel(GroupedParams p, int tiles_n) {
    typedef Skinny<DT> E;
    constexpr bool FP8 = DT == GEMM_DTYPE_FP8F32;
    constexpr int esz = E::esz, ROWS = 16 * MT, COLS = 16 * CG;
    constexpr int SUMS = kSums / WAVES;        // a wave's
    extern __shared__ __attribute__((aligned(16))) float lds[];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    GroupTile t = find_tile(p, blockIdx.x, ROWS, tiles_n, 8);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (t.rows <= 0) return;
    const int owner = __builtin_amdgcn_readfirstlane(t.group), group = max(owner, 0);
    const int row0 = __builtin_amdgcn_readfirstlane(t.row0);
    const int n0 = __builtin_amdgcn_readfirstlane(t.tn) * COLS;
    const int cols = min(COLS, p.N - n0);
    const int bytes = owner < 0 ? 0 : p.K * esz;                  // of k a row
    const int nb = (bytes + kBlock - 1) / kBlock;

    // Whole 16-byte chunks: the last one of a row holds at least one valid byte.
    const int wide = (bytes + 15) & ~15;
    const int lda = (int)p.lda * esz, ldb = (int)p.ldb * esz;
    const rsrc_t ra = make_rsrc(static_cast<const char *>(p.A) + (int64_t)row0 * p.lda * esz,
                                (uint32_t)((t.rows - 1) * lda + wide));
    const rsrc_t rw = make_rsrc(static_cast<const char *>(p.B) + ((int64_t)group * p.stride_b + (int64_t)n0 * p.ldb) * esz,
                                (uint32_t)((cols - 1) * ldb + wide));
    const int lc = lane & 15, g = lane >> 4;
    const uint32_t a_off = (uint32_t)(lc * lda + 32 * g), w_off = (uint32_t)(lc * ldb + 32 * g);
    const int rot = n0 / 32 % 32 * nb / 32;

    u32x4 av[2][UNROLL][MT][2], wv[2][UNROLL][CG][2];
    // Blocks first, first + WAVES, ... of this wave into register set `set`; past the end, zeros.
    auto issue = [&](int set, int first) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int b = first + u * WAVES;
            const int k = (b + rot < nb ? b + rot : b + rot - nb) * kBlock;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = b < nb && k + 32 * g + 16 * h < bytes;
                const uint32_t at = (uint32_t)(k + 16 * h);
#pragma unroll
                for (int i = 0; i < CG; ++i)
                    wv[set][u][i][h] = load_b128_nt(rw, in ? w_off + at + (uint32_t)(16 * i * ldb) : kOutOfRange);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    av[set][u][i][h] = load_b128(ra, in ? a_off + at + (uint32_t)(16 * i * lda) : kOutOfRange);
            }
        }
    };
    issue(0, wave);

    if constexpr (FP8) {
        const float *sa = p.sc.a + (int64_t)row0 * p.sc.a_row;
        const float *sb = p.sc.b + (int64_t)group * p.sc.b_group + (int64_t)(n0 / GEMM_SCALE_BLOCK) * p.sc.b_n;
        for (int i = tid; i < ROWS * nb; i += 64 * WAVES) {
            const int k = i / ROWS, r = min(i % ROWS, t.rows - 1);
            lds[i] = sa[(int64_t)r * p.sc.a_row + k * p.sc.a_block] * sb[k * p.sc.b_k];
        }
        __syncthreads();
    }

    f32x4 acc[SUMS][MT][CG] = {};
    // Weights as the first operand, A as the second: register r of lane (g,
    // lc) is column 4g + r of the 16, row lc.
    auto consume = [&](int set, int first) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int b = first + u * WAVES, q = (UNROLL > 1 ? u : set) % SUMS;
            const int kb = b + rot < nb ? b + rot : b + rot - nb;
            if (b < nb && kb == nb - 1 && bytes % 16 != 0) {
                // The chunk across the end of K: what follows a row in memory is not part of it.
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int n = bytes - (kb * kBlock + 32 * g + 16 * h + 4 * d);
                        const uint32_t keep = n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1;
#pragma unroll
                        for (int i = 0; i < CG; ++i) wv[set][u][i][h][d] &= keep;
#pragma unroll
                        for (int i = 0; i < MT; ++i) av[set][u][i][h][d] &= keep;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float s = FP8 && b < nb ? lds[kb * ROWS + 16 * i + lc] : 0.0f;
#pragma unroll
                for (int j = 0; j < CG; ++j) {
                    if constexpr (FP8) {
                        const f32x4 part = E::mma(wv[set][u][j], av[set][u][i], f32x4{});
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[q][i][j][r] = fmaf(part[r], s, acc[q][i][j][r]);
                    } else {
                        acc[q][i][j] = E::mma(wv[set][u][j], av[set][u][i], acc[q][i][j]);
                    }
                }
            }
        }
    };
    // The scheduling barriers keep each batch's loads ahead of the previous batch's products.
    constexpr int kStep = WAVES * UNROLL;
    for (int b = wave; b < nb; b += 2 * kStep) {
        issue(1, b + kStep);
        __builtin_amdgcn_sched_barrier(0);
        consume(0, b);
        __builtin_amdgcn_sched_barrier(0);
        issue(0, b + 2 * kStep);
        __builtin_amdgcn_sched_barrier(0);
        consume(1, b + kStep);
        __builtin_amdgcn_sched_barrier(0);
    }

    __syncthreads();                       // the scales are not needed any more
#pragma unroll
    for (int q = 0; q < SUMS; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < CG; ++j)
                *reinterpret_cast<f32x4 *>(lds + ((wave + q * WAVES) * ROWS + 16 * i + lc) * COLS + 16 * j + 4 * g) =
                    acc[q][i][j];
    __syncthreads();
    for (int i = tid; i < ROWS * COLS; i += 64 * WAVES) {
        const int row = i / COLS, col = i % COLS;
        if (row >= t.rows || col >= cols) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kSums; ++w) v += lds[w * ROWS * COLS + i];
        v *= p.alpha;
        const int64_t at = (int64_t)(row0 + row) * p.ldo + n0 + col;
        if (p.out_type == GEMM_OUT_BF16) static_cast<uint16_t *>(p.out)[at] = to_bf16(v);
        else static_cast<float *>(p.out)[at] = v;
    }
}

template <int DT, int MT, int CG, int UNROLL, int WAVES> hipError_t launch(const GroupedParams &p, hipStream_t stream) {
    GroupedParams args = p;
    int tiles_n = (p.N + 16 * CG - 1) / (16 * CG);
    const int64_t tiles = most_row_tiles(p.M, p.groups, 16 * MT, p.ends != nullptr) * tiles_n;
    const int blocks = DT == GEMM_DTYPE_FP8F32 ? (p.K + GEMM_SCALE_BLOCK - 1) / GEMM_SCALE_BLOCK : 0;
    const int floats = 16 * MT * (blocks > kSums * 16 * CG ? blocks : kSums * 16 * CG);
    void *argv[] = {&args, &tiles_n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&grouped_skinny_kernel<DT, MT, CG, UNROLL, WAVES>),
                           dim3((unsigned)tiles), dim3(64 * WAVES), argv, (size_t)floats * 4, stream);
}

// 32 columns a workgroup, which reads A half as often, where that leaves one
// for every compute unit, else 16; four waves where there are two or more.
template <int DT, int MT, int UNROLL> hipError_t launch_cols(const GroupedParams &p, hipStream_t s) {
    const int64_t groups = p.ends != nullptr ? (p.groups < p.M ? p.groups : p.M) : 1;
    const int64_t wide = groups * ((p.N + 31) / 32);
    if (wide >= 512) return launch<DT, MT, 2, UNROLL, 4>(p, s);
    if (wide >= 256) return launch<DT, MT, 2, UNROLL, 8>(p, s);
    return launch<DT, MT, 1, UNROLL, 8>(p, s);
}

template <int DT> hipError_t launch_rows(int rows, const GroupedParams &p, hipStream_t s) {
    if (rows <= 16) return launch_cols<DT, 1, 2>(p, s);
    if (rows <= 32) return launch_cols<DT, 2, 2>(p, s);
    return launch_cols<DT, 4, 1>(p, s);
}

}  // namespace

int skinny_rows(int32_t dtype, int32_t op_b, const GroupedParams &p) {
    if (op_b != GEMM_OP_T || p.K == 0) return 0;
    const int64_t groups = p.ends != nullptr ? (p.groups < p.M ? p.groups : p.M) : 1;
    const int64_t rows = (p.M + groups - 1) / groups;
    const int mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    // (A launch counts its threads in 32 bits.)
    if (rows > 64 || most_row_tiles(p.M, p.groups, 16 * mt, p.ends != nullptr) * ((p.N + 15) / 16) >= 1 << 23) return 0;
    if (dtype == GEMM_DTYPE_FP8F32 && 16 * mt * (int64_t)((p.K + GEMM_SCALE_BLOCK - 1) / GEMM_SCALE_BLOCK) > kScaleFloats)
        return 0;
    return 16 * mt;
}

hipError_t launch_grouped_skinny(int32_t dtype, int rows, const GroupedParams &p, hipStream_t stream) {
    return dtype == GEMM_DTYPE_FP8F32 ? launch_rows<GEMM_DTYPE_FP8F32>(rows, p, stream)
                                      : launch_rows<GEMM_DTYPE_BF16F32>(rows, p, stream);
}

}  // namespace gemm
