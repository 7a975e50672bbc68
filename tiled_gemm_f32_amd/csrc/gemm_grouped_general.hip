// Grouped and block-scaled products of the calls that the tiles do not take:
// a row of an operand is shorter than one 16-byte load, rows lie so far apart
// that a tile's panel passes the 2 GiB a buffer load can address, or the block
// scales do.  Every type, layout, stride and alignment is right here.
//
// The blocked method: an output tile of 64 x 64, 32-deep slices of both
// operands staged through registers into double-buffered LDS, four waves
// each keeping a quarter of the tile in fp32 accumulators, products on
// v_mfma_f32_32x32x2_f32 (exact products for all three types).  Operands are
// read element by element in units of 4 along the direction they are
// contiguous in and widened to fp32 on the way to LDS; fp8 values take their
// block scale there (one fp32 rounding, 2^-24, a value).  Both panels sit in
// LDS as [row][k], so one consume loop serves every layout.
//
// Products this short are bound by their results' stores, and rows this far
// apart by one memory transaction a row; larger tiles would change neither.
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
constexpr int BT = 64;                 // rows and columns of a tile
constexpr int kBK = 32;
constexpr int kStride = kBK + 4;       // floats a panel row takes in LDS

// One panel: `rows` of at most BT rows and `len` values of k at `base`.
// KCONT: element (r, k) at base[r * ld + k]; otherwise at base[k * ld + r].
template <int DT, bool KCONT>
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
            const int rest = len - k0 - k;                   // (k0 + k itself may pass 2^31)
            const int left = KCONT ? rest : rows - r;        // valid elements from here on
            const bool in = KCONT ? r < rows : rest > 0;
            const T *src = base + (KCONT ? (int64_t)r * ld + k0 + k : ((int64_t)k0 + k) * ld + r);
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            if (in) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left) v[e] = Elem<DT>::widen(src[e]);
            }
            if (DT == GEMM_DTYPE_FP8F32 && in && left > 0) {
                const float s = scale(r, k0 + k);
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
template <int DT, bool WGRAD, bool BN>
__global__ void __launch_bounds__(kThreads)
grouped_general_kernel(GroupedParams p, int tiles_m, int tiles_n) {
    typedef typename Elem<DT>::T T;
    __shared__ __attribute__((aligned(16))) float lds_a[2][BT * kStride];
    __shared__ __attribute__((aligned(16))) float lds_b[2][BT * kStride];

    Panel<DT, !WGRAD> a;
    Panel<DT, !WGRAD && !BN> b;
    int n0, group, row0;
    float *of = static_cast<float *>(p.out);
    uint16_t *oh = static_cast<uint16_t *>(p.out);
    if (WGRAD) {
        int tm, tn, lo, hi;
        tile_coords(blockIdx.x, tiles_m, tiles_n, 8, tm, tn);
        group = find_group(p, blockIdx.y, lo, hi);
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
    f32x16 acc = {};
    // Lane (l32, h) takes k = 16h .. 16h + 15 of its row; each matrix
    // instruction takes one k from each lane half.
    auto consume = [&](int buf) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4 fa = *reinterpret_cast<const f32x4 *>(&lds_a[buf][(wm * 32 + l32) * kStride + 16 * h + 4 * q]);
            const f32x4 fb = *reinterpret_cast<const f32x4 *>(&lds_b[buf][(wn * 32 + l32) * kStride + 16 * h + 4 * q]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[e], fb[e], acc, 0, 0, 0);
        }
    };

    const int nk = slabs_of(a.len, kBK);
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
    const int col = wn * 32 + l32;
    if (col >= b.rows) return;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = wm * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row >= a.rows) continue;
        const int64_t at = (int64_t)row * p.ldo + col;
        float v = p.alpha * acc[r];
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

template <int DT, bool WGRAD, bool BN>
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
    return hipLaunchKernel(reinterpret_cast<const void *>(&grouped_general_kernel<DT, WGRAD, BN>), grid,
                           dim3(kThreads), argv, 0, stream);
}

template <int DT> hipError_t launch_op(int32_t op_b, const GroupedParams &p, hipStream_t s) {
    return op_b == GEMM_OP_N ? launch<DT, false, true>(p, s) : launch<DT, false, false>(p, s);
}

}  // namespace

hipError_t launch_grouped_general(int32_t dtype, int32_t op_b, const GroupedParams &p, hipStream_t stream) {
    if (dtype == GEMM_DTYPE_F32) return launch_op<GEMM_DTYPE_F32>(op_b, p, stream);
    if (dtype == GEMM_DTYPE_BF16F32) return launch_op<GEMM_DTYPE_BF16F32>(op_b, p, stream);
    return launch_op<GEMM_DTYPE_FP8F32>(op_b, p, stream);
}

hipError_t launch_wgrad_general(int32_t dtype, const GroupedParams &p, hipStream_t stream) {
    if (dtype == GEMM_DTYPE_F32) return launch<GEMM_DTYPE_F32, true, true>(p, stream);
    return launch<GEMM_DTYPE_BF16F32, true, true>(p, stream);
}

}  // namespace gemm
