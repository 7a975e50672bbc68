// Grouped and block-scaled products for every operand type, layout, stride
// and alignment, and the fp32 ones' only kernel.
//
// The blocked method: an output tile of 128 x 128 (or 64 x 64, where there
// are too few large ones to fill the compute units), 32-deep slices of both
// operands staged through registers into double-buffered LDS, four waves
// each keeping a quarter of the tile in fp32 accumulators, products on
// v_mfma_f32_32x32x2_f32 (exact products for all three types).  Operands are
// read in units of 4 elements along the direction they are contiguous in,
// one 16-byte load a unit where fp32 alignment allows, four element loads
// otherwise, and widened to fp32 on the way to LDS; fp8 values take their
// block scale there (one fp32 rounding, 2^-24, a value).  Both panels sit in
// LDS as [row][k], so one consume loop serves every layout.
//
// fp32 is bound by the matrix cores (32 x 32 x 2 takes 64 cycles for 512 bytes
// of fragments, a fifth of what LDS delivers); 128 x 128 tiles ask L2 for 16
// bytes a cycle and compute unit.
#include "gemm_grouped.hpp"

namespace gemm {
namespace {

template <int DT> struct Elem;
template <> struct Elem<GEMM_DTYPE_F32> {
    typedef float T;
    static __device__ __forceinline__ float widen(T v) { return v; }
};
template <> struct Elem<GEMM_DTYPE_BF16F32> {
    typedef uint16_t T;
    static __device__ __forceinline__ float widen(T v) { return __uint_as_float((uint32_t)v << 16); }
};
template <> struct Elem<GEMM_DTYPE_FP8F32> {
    typedef uint8_t T;
    static __device__ __forceinline__ float widen(T v) { return __builtin_amdgcn_cvt_f32_fp8((int)v, 0); }
};

constexpr int kThreads = 256;
constexpr int kBK = 32;
constexpr int kStride = kBK + 4;       // floats a panel row takes in LDS

// One panel: `rows` of at most BT rows and `len` values of k at `base`.
// KCONT: element (r, k) at base[r * ld + k]; otherwise at base[k * ld + r].
template <int DT, int BT, bool KCONT, bool VEC>
struct Panel {
    typedef typename Elem<DT>::T T;
    static constexpr int kPer = BT * kBK / 4 / kThreads;     // units of 4 a thread
    const T *base;
    int64_t ld;
    int rows, len;
    f32x4 reg[kPer];

    static __device__ __forceinline__ void coord(int i, int &r, int &k) {
        const int c = threadIdx.x + i * kThreads;
        if (KCONT) {
            r = c / (kBK / 4);
            k = 4 * (c % (kBK / 4));
        } else {
            k = c / (BT / 4);
            r = 4 * (c % (BT / 4));
        }
    }
    // scale(r, k): what a unit's values are multiplied by (fp8; one block scale covers a unit).
    template <class S> __device__ __forceinline__ void fetch(int k0, S &&scale) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            int r, k;
            coord(i, r, k);
            k += k0;
            const int left = KCONT ? len - k : rows - r;     // valid elements from here on
            const bool in = KCONT ? r < rows : k < len;
            const T *src = base + (KCONT ? (int64_t)r * ld + k : (int64_t)k * ld + r);
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            if (VEC && in && left >= 4) {
                v = *reinterpret_cast<const f32x4 *>(src);
            } else if (in) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left) v[e] = Elem<DT>::widen(src[e]);
            }
            if (DT == GEMM_DTYPE_FP8F32 && in && left > 0) {
                const float s = scale(r, k);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left) v[e] *= s;
            }
            reg[i] = v;
        }
    }
    __device__ __forceinline__ void stash(float *lds) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            int r, k;
            coord(i, r, k);
            if (KCONT) {
                *reinterpret_cast<f32x4 *>(lds + r * kStride + k) = reg[i];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) lds[(r + e) * kStride + k] = reg[i][e];
            }
        }
    }
};

// WGRAD: rows of the result are columns of dY (A), its columns those of X
// (B), and k runs over the rows of one group.
template <int DT, int BT, bool WGRAD, bool BN, bool VEC>
__global__ void __launch_bounds__(kThreads)
grouped_general_kernel(GroupedParams p, int tiles_m, int tiles_n) {
    typedef typename Elem<DT>::T T;
    constexpr int F = BT / 64;            // 32 x 32 fragments a wave and direction
    __shared__ __attribute__((aligned(16))) float lds_a[2][BT * kStride];
    __shared__ __attribute__((aligned(16))) float lds_b[2][BT * kStride];

    Panel<DT, BT, !WGRAD, VEC> a;
    Panel<DT, BT, !WGRAD && !BN, VEC> b;
    int n0, group, row0;
    float *of = static_cast<float *>(p.out);
    uint16_t *oh = static_cast<uint16_t *>(p.out);
    if (WGRAD) {
        int tm, tn, lo, hi;
        tile_coords(blockIdx.x, tiles_m, tiles_n, 8, tm, tn);
        group = blockIdx.y;
        find_group(p, group, lo, hi);
        row0 = tm * BT;
        n0 = tn * BT;
        a.base = static_cast<const T *>(p.A) + (int64_t)lo * p.lda + row0;
        a.rows = min(BT, p.N - row0);
        b.base = static_cast<const T *>(p.B) + (int64_t)lo * p.ldb + n0;
        b.rows = min(BT, p.K - n0);
        a.len = b.len = hi - lo;
        of += (int64_t)group * p.stride_out + (int64_t)row0 * p.ldo + n0;
    } else {
        const GroupTile t = find_tile(p, blockIdx.x, BT, tiles_n, 8);
        if (t.rows <= 0) return;
        group = max(t.group, 0);
        row0 = t.row0;
        n0 = t.tn * BT;
        a.base = static_cast<const T *>(p.A) + (int64_t)row0 * p.lda;
        a.rows = t.rows;
        b.base = static_cast<const T *>(p.B) + (int64_t)group * p.stride_b + (BN ? (int64_t)n0 : (int64_t)n0 * p.ldb);
        b.rows = min(BT, p.N - n0);
        a.len = b.len = t.group < 0 ? 0 : p.K;
        of += (int64_t)row0 * p.ldo + n0;
        oh += (int64_t)row0 * p.ldo + n0;
    }
    a.ld = p.lda;
    b.ld = p.ldb;
    auto scale_a = [&](int r, int k) {
        return p.sc.a[(int64_t)(row0 + r) * p.sc.a_row + (int64_t)(k / GEMM_SCALE_BLOCK) * p.sc.a_block];
    };
    auto scale_b = [&](int r, int k) {
        return p.sc.b[(int64_t)group * p.sc.b_group + (int64_t)((n0 + r) / GEMM_SCALE_BLOCK) * p.sc.b_n +
                      (int64_t)(k / GEMM_SCALE_BLOCK) * p.sc.b_k];
    };

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int h = lane >> 5, l32 = lane & 31;
    f32x16 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = f32x16{};
    // Lane (l32, h) takes k = 16h .. 16h + 15 of its row; each matrix
    // instruction takes one k from each lane half.
    auto consume = [&](int buf) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f32x4 fa[F], fb[F];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int at = 32 * f + l32;
                fa[f] = *reinterpret_cast<const f32x4 *>(&lds_a[buf][(wm * 32 * F + at) * kStride + 16 * h + 4 * q]);
                fb[f] = *reinterpret_cast<const f32x4 *>(&lds_b[buf][(wn * 32 * F + at) * kStride + 16 * h + 4 * q]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < F; ++i)
#pragma unroll
                    for (int j = 0; j < F; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[i][e], fb[j][e], acc[i][j], 0, 0, 0);
        }
    };

    const int nk = (a.len + kBK - 1) / kBK;
    if (nk > 0) {
        a.fetch(0, scale_a);
        b.fetch(0, scale_b);
        a.stash(lds_a[0]);
        b.stash(lds_b[0]);
    }
    __syncthreads();
    for (int kt = 0; kt < nk; ++kt) {
        const int cur = kt & 1;
        const bool more = kt + 1 < nk;
        if (more) {
            a.fetch((kt + 1) * kBK, scale_a);
            b.fetch((kt + 1) * kBK, scale_b);
        }
        consume(cur);
        if (more) {
            a.stash(lds_a[cur ^ 1]);
            b.stash(lds_b[cur ^ 1]);
        }
        __syncthreads();
    }

    // Register r of lane (h, l32) is row 8*(r/4) + 4*h + r%4, column l32 of its block.
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int col = wn * 32 * F + 32 * j + l32;
            if (col >= b.rows) continue;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = wm * 32 * F + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
                if (row >= a.rows) continue;
                const int64_t at = (int64_t)row * p.ldo + col;
                float v = p.alpha * acc[i][j][r];
                if (WGRAD) {
                    if (p.beta != 0.0f) v = fmaf(p.beta, of[at], v);
                    of[at] = v;
                } else if (p.out_type == GEMM_OUT_BF16) {
                    oh[at] = to_bf16(v);
                } else {
                    of[at] = v;
                }
            }
        }
}

template <int DT, int BT, bool WGRAD, bool BN, bool VEC>
hipError_t launch(const GroupedParams &p, hipStream_t stream) {
    GroupedParams args = p;
    int tiles_m, tiles_n;
    dim3 grid;
    if (WGRAD) {
        tiles_m = (p.N + BT - 1) / BT;
        tiles_n = (p.K + BT - 1) / BT;
        grid = dim3((unsigned)(tiles_m * tiles_n), (unsigned)p.groups);
    } else {
        tiles_m = (int)most_row_tiles(p.M, p.groups, BT, p.ends != nullptr);
        tiles_n = (p.N + BT - 1) / BT;
        grid = dim3((unsigned)(tiles_m * tiles_n));
    }
    void *argv[] = {&args, &tiles_m, &tiles_n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&grouped_general_kernel<DT, BT, WGRAD, BN, VEC>), grid,
                           dim3(kThreads), argv, 0, stream);
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// fp32 rows that start on 16 bytes take 16-byte loads.
bool vectors(const GroupedParams &p) {
    return on16(p.A) && on16(p.B) && p.lda % 4 == 0 && p.ldb % 4 == 0 && p.stride_b % 4 == 0;
}

template <int DT, int BT, bool WGRAD, bool BN>
hipError_t launch_loads(const GroupedParams &p, hipStream_t s) {
    if constexpr (DT == GEMM_DTYPE_F32)
        if (vectors(p)) return launch<DT, BT, WGRAD, BN, true>(p, s);
    return launch<DT, BT, WGRAD, BN, false>(p, s);
}

template <int DT, int BT, bool WGRAD>
hipError_t launch_tile(int32_t op_b, const GroupedParams &p, hipStream_t s) {
    if constexpr (WGRAD) return launch_loads<DT, BT, true, true>(p, s);
    else return op_b == GEMM_OP_N ? launch_loads<DT, BT, false, true>(p, s) : launch_loads<DT, BT, false, false>(p, s);
}

// 128 x 128 where such tiles number at least the 256 compute units, else
// 64 x 64, whose four times as many tiles keep them busy.
template <int DT, bool WGRAD>
hipError_t launch_type(int32_t op_b, const GroupedParams &p, hipStream_t s) {
    const int64_t tiles = WGRAD ? (int64_t)((p.N + 127) / 128) * ((p.K + 127) / 128) * p.groups
                                : most_row_tiles(p.M, p.groups, 128, p.ends != nullptr) * ((p.N + 127) / 128);
    return tiles >= 256 ? launch_tile<DT, 128, WGRAD>(op_b, p, s) : launch_tile<DT, 64, WGRAD>(op_b, p, s);
}

}  // namespace

hipError_t launch_grouped_general(int32_t dtype, int32_t op_b, const GroupedParams &p, hipStream_t stream) {
    if (dtype == GEMM_DTYPE_F32) return launch_type<GEMM_DTYPE_F32, false>(op_b, p, stream);
    if (dtype == GEMM_DTYPE_BF16F32) return launch_type<GEMM_DTYPE_BF16F32, false>(op_b, p, stream);
    return launch_type<GEMM_DTYPE_FP8F32, false>(op_b, p, stream);
}

hipError_t launch_wgrad_general(int32_t dtype, const GroupedParams &p, hipStream_t stream) {
    if (dtype == GEMM_DTYPE_F32) return launch_type<GEMM_DTYPE_F32, true>(GEMM_OP_N, p, stream);
    return launch_type<GEMM_DTYPE_BF16F32, true>(GEMM_OP_N, p, stream);
}

}  // namespace gemm
