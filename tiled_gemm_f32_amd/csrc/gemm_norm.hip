// RMS norm with the residual's addition, its backward pass, and the block
// quantiser: passes over rows, bound by HBM.
//
// A row is read once and kept in registers, 8 consecutive values (a chunk) a
// lane at a time, while its sum of squares goes around: s = x + residual,
// r = (mean(s^2) + eps)^-1/2, y = s * r * weight.  Chunk c of a row belongs
// to lane c modulo the row's threads, so the 128 values of a scale block sit
// in 16 neighbouring lanes and their largest magnitude takes four
// lane-rotations, with no memory between the norm and its codes.  A row of
// up to 1024 values is one wave's, up to 4096 a team of four waves', up to
// 16384 of sixteen; longer rows are walked twice by sixteen waves, the second
// time from the caches.
//
// 8192 x 8192 bf16 with a residual to fp8: 470 MB in 85 us, 5.5 TB/s (a copy
// reaches 4.9 here).  8192 x 4096 bf16 in training, 268 MB each way: forward
// 48 us (5.6 TB/s), backward 45 us (6.0, some of it from the caches) and 4.5
// for the last sum over partial rows; in fp32 99 and 105 for all of the
// backward pass (5.4 and 5.1).  16 x 8192: 4.2 us, a launch and two trips to
// memory.  Codes of 8192 x 8192 bf16: 34 us with a scale for each 128 x 128
// (5.8 TB/s), 41 to 45 for each 128 columns of a row (4.5 to 5), where a lane
// has one 16-byte load under way.  Longer rows, 4096 x 20000 bf16: forward 150
// us (4.4 TB/s), backward 251 (2.6).
#include "gemm_device.hpp"
#include "gemm_norm.hpp"

namespace gemm {
namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));
constexpr int kChunk = 8;
constexpr float kMinAmax = 0x1p-100f;
constexpr float kE4m3Max = 448.0f;

template <int DT> struct Io;
template <> struct Io<GEMM_DTYPE_F32> {
    typedef float T;
    typedef f32x8 Raw;
    static __device__ __forceinline__ float widen(T v) { return v; }
    static __device__ __forceinline__ T narrow(float v) { return v; }
    static __device__ __forceinline__ f32x8 values(Raw r) { return r; }
};
template <> struct Io<GEMM_DTYPE_BF16F32> {
    typedef uint16_t T;
    typedef u32x4 Raw;
    static __device__ __forceinline__ float widen(T v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ T narrow(float v) { return to_bf16(v); }
    static __device__ __forceinline__ f32x8 values(Raw r) {
        f32x8 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
        return v;
    }
};

// A chunk at any alignment of its elements: the hardware takes unaligned
// 16-byte accesses, and rows of an odd length start anywhere.
template <class V> struct __attribute__((packed, aligned(1))) Anywhere {
    V v;
};
template <class V> __device__ __forceinline__ V get(const void *p) {
    return reinterpret_cast<const Anywhere<V> *>(p)->v;
}
template <class V> __device__ __forceinline__ void put(void *p, V v) { reinterpret_cast<Anywhere<V> *>(p)->v = v; }

// Up to 8 values, n of them valid (n <= 0: none; the rest read as zero).
template <int DT>
__device__ __forceinline__ typename Io<DT>::Raw load_raw(const void *base, int64_t at, int n) {
    typedef typename Io<DT>::T T;
    typedef typename Io<DT>::Raw Raw;
    const T *src = static_cast<const T *>(base) + at;
    Raw r = {};
    if (n >= kChunk) {
        r = get<Raw>(src);
    } else if constexpr (DT == GEMM_DTYPE_F32) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            if (e < n) r[e] = src[e];
    } else {
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            if (e < n) r[e / 2] |= (uint32_t)src[e] << (16 * (e & 1));
    }
    return r;
}
template <int DT>
__device__ __forceinline__ f32x8 load8(const void *base, int64_t at, int n) {
    return Io<DT>::values(load_raw<DT>(base, at, n));
}
template <int DT>
__device__ __forceinline__ void store8(void *base, int64_t at, f32x8 v, int n) {
    typedef typename Io<DT>::T T;
    T *dst = static_cast<T *>(base) + at;
    if (n >= kChunk) {
        if constexpr (DT == GEMM_DTYPE_F32) {
            put(dst, v);
        } else {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (uint32_t)to_bf16(v[2 * i]) | ((uint32_t)to_bf16(v[2 * i + 1]) << 16);
            put(dst, w);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            if (e < n) dst[e] = Io<DT>::narrow(v[e]);
    }
}

// Largest (or sum) over the 16 lanes of a row of lanes, in all of them:
// rotations by 8, 4, 2 and 1.
template <int N> __device__ __forceinline__ float ror16(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf,
                                                                 true));
}
__device__ __forceinline__ float max16(float v) {
    v = fmaxf(v, ror16<8>(v));
    v = fmaxf(v, ror16<4>(v));
    v = fmaxf(v, ror16<2>(v));
    return fmaxf(v, ror16<1>(v));
}
__device__ __forceinline__ float sum64(float v) {
    v += ror16<8>(v);
    v += ror16<4>(v);
    v += ror16<2>(v);
    v += ror16<1>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

__device__ __forceinline__ float finite_max(f32x8 v) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
        const float a = fabsf(v[e]);
        m = fmaxf(m, a < __builtin_inff() ? a : 0.0f);     // false for NaN too
    }
    return m;
}

// Codes of 8 values, inv = 448 / amax of their block: finite ones come out at
// most 448 * (1 + 2^-23), which rounds to 448.
__device__ __forceinline__ u32x2 codes8(f32x8 v, float inv) {
    float c[kChunk];
#pragma unroll
    for (int e = 0; e < kChunk; ++e) c[e] = fabsf(v[e]) < __builtin_inff() ? v[e] * inv : __builtin_nanf("");
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int q = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], q, true);
    }
    return w;
}
__device__ __forceinline__ void store_codes(uint8_t *dst, u32x2 w, int n) {
    if (n >= kChunk) {
        put(dst, w);
    } else {
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            if (e < n) dst[e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
    }
}

// Workgroup number of a launch folded into two grid dimensions (fold below).
__device__ __forceinline__ int64_t folded_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Sum over a team of THREADS threads (one or more whole waves) of a workgroup
// that is one team, or of one wave.  `red`: one float a wave, two sets used
// in turn so that one barrier a call suffices.
template <int THREADS> __device__ __forceinline__ float team_sum(float v, float *red, int set) {
    v = sum64(v);
    if (THREADS == 64) return v;
    constexpr int W = THREADS / 64;
    float *r = red + set * W;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += r[w];
    return t;
}

// One chunk's y out: fp32, bf16, or codes with their block's scale.  A chunk
// that is wholly past the row's end takes part in the lane rotations only.
__device__ __forceinline__ void put_norm(const NormParams &p, int64_t row, int64_t col, f32x8 y, int n) {
    if (p.out_type == GEMM_OUT_FP8) {
        const float amax = fmaxf(max16(finite_max(y)), kMinAmax);
        const u32x2 w = codes8(y, kE4m3Max / amax);
        if (n > 0) {
            store_codes(static_cast<uint8_t *>(p.out) + row * p.ldo + col, w, n);
            if ((col & (GEMM_SCALE_BLOCK - 1)) == 0)
                p.scales[row * p.ld_scales + col / GEMM_SCALE_BLOCK] = amax / kE4m3Max;
        }
    } else if (p.out_type == GEMM_OUT_BF16) {
        store8<GEMM_DTYPE_BF16F32>(p.out, row * p.ldo + col, y, n);
    } else {
        store8<GEMM_DTYPE_F32>(p.out, row * p.ldo + col, y, n);
    }
}

// s of one chunk, rounded to the operands' type as it is stored.
template <int DT>
__device__ __forceinline__ f32x8 norm_sum(const NormParams &p, int64_t row, int64_t col, int n) {
    f32x8 v = load8<DT>(p.x, row * p.ldx + col, n);
    if (p.residual != nullptr) {
        const f32x8 r = load8<DT>(p.residual, row * p.ldr + col, n);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[e] = Io<DT>::widen(Io<DT>::narrow(v[e] + r[e]));
    }
    return v;
}

template <int DT, int THREADS, int PER>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS)
rms_norm_kernel(NormParams p) {
    constexpr int TEAMS = THREADS < 256 ? 256 / THREADS : 1;
    __shared__ float red[THREADS / 64];
    const int64_t row = folded_block() * TEAMS + (TEAMS > 1 ? threadIdx.x / THREADS : 0);
    const int t = threadIdx.x % THREADS;
    if (row >= p.M) return;                    // the whole team together
    const int N = (int)p.N;
    f32x8 s[PER], w[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        s[i] = norm_sum<DT>(p, row, col, N - col);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        w[i] = load8<DT>(p.weight, col, N - col);
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) sq = fmaf(s[i][e], s[i][e], sq);
        const int col = kChunk * (t + i * THREADS);
        if (p.sum != nullptr) store8<DT>(p.sum, row * p.ld_sum + col, s[i], N - col);
    }
    const float r = 1.0f / sqrtf(team_sum<THREADS>(sq, red, 0) / (float)N + p.eps);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        f32x8 y;
#pragma unroll
        for (int e = 0; e < kChunk; ++e) y[e] = s[i][e] * r * w[i][e];
        put_norm(p, row, col, y, N - col);
    }
}

// Rows of any length: sixteen waves walk the row twice.
template <int DT>
__global__ void __launch_bounds__(1024)
rms_norm_long_kernel(NormParams p) {
    __shared__ float red[16];
    const int64_t row = folded_block();
    if (row >= p.M) return;
    float sq = 0.0f;
    for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024) {
        const int n = (int)min((int64_t)kChunk, p.N - col);
        const f32x8 s = norm_sum<DT>(p, row, col, n);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) sq = fmaf(s[e], s[e], sq);
    }
    const float r = 1.0f / sqrtf(team_sum<1024>(sq, red, 0) / (float)p.N + p.eps);
    // Every lane runs every round: the block maximum goes over 16 of them.
    for (int64_t c0 = 0; c0 < p.N; c0 += kChunk * 1024) {
        const int64_t col = c0 + kChunk * threadIdx.x;
        const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.N - col));
        f32x8 y = {};
        if (n > 0) {
            const f32x8 s = norm_sum<DT>(p, row, col, n);
            const f32x8 w = load8<DT>(p.weight, col, n);
            if (p.sum != nullptr) store8<DT>(p.sum, row * p.ld_sum + col, s, n);
#pragma unroll
            for (int e = 0; e < kChunk; ++e) y[e] = s[e] * r * w[e];
        }
        put_norm(p, row, col, y, n);
    }
}

// Backward pass: a team of threads takes rows team, team + teams, ... and
// keeps its columns' weights and weight-gradient sums in registers; the
// teams' sums go to `partials`, one row each, and dweight_kernel adds them.
template <int DT, int THREADS, int PER>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS)
rms_norm_backward_kernel(NormGradParams p) {
    constexpr int TEAMS = THREADS < 256 ? 256 / THREADS : 1;
    typedef typename Io<DT>::Raw Raw;
    __shared__ float red[4 * (THREADS / 64)];
    const int team = blockIdx.x * TEAMS + (TEAMS > 1 ? threadIdx.x / THREADS : 0), teams = gridDim.x * TEAMS;
    const int t = threadIdx.x % THREADS;
    const int N = (int)p.N;
    const float inv_n = 1.0f / (float)N;
    f32x8 w[PER], dw[PER];
    Raw dy[PER], s[PER], ds[PER];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int col = kChunk * (t + i * THREADS);
            dy[i] = load_raw<DT>(p.dy, row * p.lddy + col, N - col);
            s[i] = load_raw<DT>(p.s, row * p.lds + col, N - col);
            if (p.ds != nullptr) ds[i] = load_raw<DT>(p.ds, row * p.ldds + col, N - col);
        }
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        w[i] = load8<DT>(p.weight, col, N - col);
        dw[i] = f32x8{};
        ds[i] = Raw{};
    }
    int set = 0;
    for (int64_t row = team; row < p.M; row += teams, set ^= 2) {
        fetch(row);
        float sq = 0.0f, gs = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const f32x8 sv = Io<DT>::values(s[i]), yv = Io<DT>::values(dy[i]);
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                sq = fmaf(sv[e], sv[e], sq);
                gs = fmaf(yv[e] * w[i][e], sv[e], gs);
            }
        }
        sq = sum64(sq);
        gs = sum64(gs);
        if (THREADS > 64) {
            // Two sets of slots in turn: a wave that is a row ahead writes the other set, and it
            // cannot be two ahead past the next barrier.
            constexpr int W = THREADS / 64;
            if ((threadIdx.x & 63) == 0) {
                red[set * W + (threadIdx.x >> 6)] = sq;
                red[(set + 1) * W + (threadIdx.x >> 6)] = gs;
            }
            __syncthreads();
            sq = gs = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                sq += red[set * W + i];
                gs += red[(set + 1) * W + i];
            }
        }
        const float r = 1.0f / sqrtf(sq * inv_n + p.eps);
        const float along = r * (gs * inv_n);      // of the size of g: r^3 on its own could overflow
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int col = kChunk * (t + i * THREADS);
            const f32x8 sv = Io<DT>::values(s[i]), yv = Io<DT>::values(dy[i]), dv = Io<DT>::values(ds[i]);
            f32x8 dx;
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                dx[e] = fmaf(r, fmaf(-along, sv[e] * r, yv[e] * w[i][e]), dv[e]);
                dw[i][e] = fmaf(yv[e] * r, sv[e], dw[i][e]);
            }
            store8<DT>(p.dx, row * p.lddx + col, dx, N - col);
        }
    }
    if (p.dweight == nullptr) return;
    if constexpr (TEAMS > 1) {
        // One partial row a workgroup: its teams' sums are added through LDS, in order.
        __shared__ __attribute__((aligned(16))) float sums[TEAMS][PER * THREADS * kChunk];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            *reinterpret_cast<f32x8 *>(&sums[threadIdx.x / THREADS][kChunk * (t + i * THREADS)]) = dw[i];
        __syncthreads();
        for (int col = threadIdx.x; col < N; col += TEAMS * THREADS) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < TEAMS; ++i) v += sums[i][col];
            p.partials[(int64_t)blockIdx.x * N + col] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int col = kChunk * (t + i * THREADS);
            store8<GEMM_DTYPE_F32>(p.partials, (int64_t)team * N + col, dw[i], N - col);
        }
    }
}

// Rows past 16384 values (8192 in fp32): the row's sums first, then the row
// again from the caches.  The weight
// gradient's running sums live in `partials`.
template <int DT>
__global__ void __launch_bounds__(1024)
rms_norm_backward_long_kernel(NormGradParams p) {
    __shared__ float red[64];
    const int team = blockIdx.x, teams = gridDim.x;
    const float inv_n = 1.0f / (float)p.N;
    int set = 0;
    for (int64_t row = team; row < p.M; row += teams, set ^= 2) {
        float sq = 0.0f, gs = 0.0f;
        for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024) {
            const int n = (int)min((int64_t)kChunk, p.N - col);
            const f32x8 sv = load8<DT>(p.s, row * p.lds + col, n), yv = load8<DT>(p.dy, row * p.lddy + col, n);
            const f32x8 w = load8<DT>(p.weight, col, n);
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                sq = fmaf(sv[e], sv[e], sq);
                gs = fmaf(yv[e] * w[e], sv[e], gs);
            }
        }
        sq = sum64(sq);
        gs = sum64(gs);
        if ((threadIdx.x & 63) == 0) {
            red[set * 16 + (threadIdx.x >> 6)] = sq;
            red[(set + 1) * 16 + (threadIdx.x >> 6)] = gs;
        }
        __syncthreads();
        sq = gs = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            sq += red[set * 16 + i];
            gs += red[(set + 1) * 16 + i];
        }
        const float r = 1.0f / sqrtf(sq * inv_n + p.eps);
        const float along = r * (gs * inv_n);      // of the size of g: r^3 on its own could overflow
        for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024) {
            const int n = (int)min((int64_t)kChunk, p.N - col);
            const f32x8 sv = load8<DT>(p.s, row * p.lds + col, n), yv = load8<DT>(p.dy, row * p.lddy + col, n);
            const f32x8 w = load8<DT>(p.weight, col, n);
            f32x8 dv = {}, dx;
            if (p.ds != nullptr) dv = load8<DT>(p.ds, row * p.ldds + col, n);
            if (p.dweight != nullptr) {
                f32x8 dw = {};
                if (row != team) dw = load8<GEMM_DTYPE_F32>(p.partials, team * p.N + col, n);
#pragma unroll
                for (int e = 0; e < kChunk; ++e) dw[e] = fmaf(yv[e] * r, sv[e], dw[e]);
                store8<GEMM_DTYPE_F32>(p.partials, team * p.N + col, dw, n);
            }
#pragma unroll
            for (int e = 0; e < kChunk; ++e) dx[e] = fmaf(r, fmaf(-along, sv[e] * r, yv[e] * w[e]), dv[e]);
            store8<DT>(p.dx, row * p.lddx + col, dx, n);
        }
    }
}

// dweight[j] = sum of `parts` partial rows in a fixed order: 32 columns a
// workgroup, 32 threads a column each adding every 32nd row, eight rows in
// flight, then the threads' sums in turn.
__global__ void __launch_bounds__(1024)
dweight_kernel(const float *partials, float *dweight, int parts, int64_t N) {
    __shared__ float part[32][32];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t col = folded_block() * 32 + c;
    float s[8] = {};
    if (col < N)
        for (int i = g; i < parts; i += 256) {
#pragma unroll
            for (int u = 0; u < 8; ++u) s[u] += i + 32 * u < parts ? partials[(int64_t)(i + 32 * u) * N + col] : 0.0f;
        }
    part[g][c] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    if (g == 0 && col < N) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += part[i][c];
        dweight[col] = t;
    }
}

// A scale for each 128 columns of a row: 16 lanes a block.
template <int DT>
__global__ void __launch_bounds__(256)
quantize_rows_kernel(QuantParams p, int64_t blocks, int per_row) {
    const int64_t b = folded_block() * 16 + threadIdx.x / 16;
    if (b >= blocks) return;                   // sixteen lanes together
    // 32-bit division where it will do: the 64-bit one is some hundred instructions.
    const int64_t row = blocks >> 32 == 0 ? (int64_t)((uint32_t)b / (uint32_t)per_row) : b / per_row;
    const int j = (int)(b - row * per_row);
    const int64_t col = (int64_t)j * GEMM_SCALE_BLOCK + kChunk * (threadIdx.x & 15);
    const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.K - col));
    const f32x8 v = load8<DT>(p.x, row * p.ldx + col, n);
    const float amax = fmaxf(max16(finite_max(v)), kMinAmax);
    const u32x2 w = codes8(v, kE4m3Max / amax);
    if (n > 0) store_codes(p.q + row * p.ldq + col, w, n);
    if ((threadIdx.x & 15) == 0) p.scales[row * p.lds + j] = amax / kE4m3Max;
}

// A scale for each 128 x 128 tile: a workgroup each, the tile in registers.
template <int DT>
__global__ void __launch_bounds__(256)
quantize_tiles_kernel(QuantParams p, int64_t tiles, int per_row) {
    __shared__ float red[4];
    const int64_t b = folded_block();
    if (b >= tiles) return;                    // the whole workgroup
    const int64_t tile_row = b / per_row;
    const int tile_col = (int)(b - tile_row * per_row);
    const int64_t row0 = tile_row * GEMM_SCALE_BLOCK + threadIdx.x / 16;
    const int64_t col = (int64_t)tile_col * GEMM_SCALE_BLOCK + kChunk * (threadIdx.x & 15);
    const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.K - col));
    f32x8 v[8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 16 * i;
        v[i] = load8<DT>(p.x, row * p.ldx + col, row < p.M ? n : 0);
        amax = fmaxf(amax, finite_max(v[i]));
    }
    amax = max16(amax);
    amax = fmaxf(amax, __shfl_xor(amax, 16));
    amax = fmaxf(amax, __shfl_xor(amax, 32));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), kMinAmax);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 16 * i;
        if (row < p.M && n > 0) store_codes(p.q + row * p.ldq + col, codes8(v[i], kE4m3Max / amax), n);
    }
    if (threadIdx.x == 0) p.scales[tile_row * p.lds + tile_col] = amax / kE4m3Max;
}

template <typename... Args>
hipError_t go(void (*kernel)(Args...), dim3 grid, int threads, hipStream_t s, Args... args) {
    void *argv[] = {static_cast<void *>(&args)...};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, dim3((unsigned)threads), argv, 0, s);
}

// A launch counts its threads along x in 32 bits: workgroups past 2^20 go
// into further grid rows.
dim3 fold(int64_t workgroups) {
    const int64_t most = int64_t(1) << 20;
    return workgroups <= most ? dim3((unsigned)workgroups) : dim3((unsigned)most, (unsigned)((workgroups + most - 1) / most));
}

// How a row of N values is shared out: see the file's first comment.
enum Shape { kWave2, kFour2, kSixteen1, kSixteen2, kLong };
Shape shape_of(int64_t N) {
    return N <= 1024 ? kWave2 : N <= 4096 ? kFour2 : N <= 8192 ? kSixteen1 : N <= 16384 ? kSixteen2 : kLong;
}

template <int DT> hipError_t norm_type(const NormParams &p, hipStream_t s) {
    switch (shape_of(p.N)) {
        case kWave2: return go(&rms_norm_kernel<DT, 64, 2>, fold((p.M + 3) / 4), 256, s, p);
        case kFour2: return go(&rms_norm_kernel<DT, 256, 2>, fold(p.M), 256, s, p);
        case kSixteen1: return go(&rms_norm_kernel<DT, 1024, 1>, fold(p.M), 1024, s, p);
        case kSixteen2: return go(&rms_norm_kernel<DT, 1024, 2>, fold(p.M), 1024, s, p);
        default: return go(&rms_norm_long_kernel<DT>, fold(p.M), 1024, s, p);
    }
}

// Workgroups of the backward pass: enough to fill the compute units with
// teams that each still take several rows, so that the partial sums stay a
// small part of what is moved.
int grad_workgroups(int64_t M, int64_t N) {
    const Shape sh = shape_of(N);
    const int64_t rows = sh == kWave2 ? (M + 3) / 4 : M;     // rows a workgroup takes at once: 4, or 1
    const int64_t most = sh == kFour2 ? 768 : 512;
    return (int)(rows < most ? rows : most);
}

template <int DT> hipError_t grad_type(const NormGradParams &p, hipStream_t s) {
    const dim3 grid((unsigned)grad_workgroups(p.M, p.N));
    Shape sh = shape_of(p.N);
    // Two fp32 chunks a lane of everything the backward pass holds do not fit
    // the 128 registers that sixteen waves leave each.
    if (DT == GEMM_DTYPE_F32 && sh == kSixteen2) sh = kLong;
    switch (sh) {
        case kWave2: return go(&rms_norm_backward_kernel<DT, 64, 2>, grid, 256, s, p);
        case kFour2: return go(&rms_norm_backward_kernel<DT, 256, 2>, grid, 256, s, p);
        case kSixteen1: return go(&rms_norm_backward_kernel<DT, 1024, 1>, grid, 1024, s, p);
        case kSixteen2:
            if constexpr (DT != GEMM_DTYPE_F32) return go(&rms_norm_backward_kernel<DT, 1024, 2>, grid, 1024, s, p);
        default: return go(&rms_norm_backward_long_kernel<DT>, grid, 1024, s, p);
    }
}

}  // namespace

int norm_grad_partials(int64_t M, int64_t N) {
    if (M <= 0 || N <= 0) return 0;
    return grad_workgroups(M, N);
}

hipError_t launch_rms_norm(const NormParams &p, hipStream_t s) {
    return p.dtype == GEMM_DTYPE_F32 ? norm_type<GEMM_DTYPE_F32>(p, s) : norm_type<GEMM_DTYPE_BF16F32>(p, s);
}

hipError_t launch_rms_norm_backward(const NormGradParams &p, hipStream_t s) {
    hipError_t err = hipSuccess;
    if (p.M > 0)
        err = p.dtype == GEMM_DTYPE_F32 ? grad_type<GEMM_DTYPE_F32>(p, s) : grad_type<GEMM_DTYPE_BF16F32>(p, s);
    if (err != hipSuccess || p.dweight == nullptr) return err;
    return go(&dweight_kernel, fold((p.N + 31) / 32), 1024, s, (const float *)p.partials, p.dweight,
              norm_grad_partials(p.M, p.N), p.N);
}

hipError_t launch_quantize(const QuantParams &p, hipStream_t s) {
    const int64_t per_row = (p.K + GEMM_SCALE_BLOCK - 1) / GEMM_SCALE_BLOCK;
    if (p.block_rows == 1) {
        const int64_t blocks = p.M * per_row;
        const dim3 grid = fold((blocks + 15) / 16);
        return p.dtype == GEMM_DTYPE_F32
                   ? go(&quantize_rows_kernel<GEMM_DTYPE_F32>, grid, 256, s, p, blocks, (int)per_row)
                   : go(&quantize_rows_kernel<GEMM_DTYPE_BF16F32>, grid, 256, s, p, blocks, (int)per_row);
    }
    const int64_t tiles = (p.M + GEMM_SCALE_BLOCK - 1) / GEMM_SCALE_BLOCK * per_row;
    return p.dtype == GEMM_DTYPE_F32
               ? go(&quantize_tiles_kernel<GEMM_DTYPE_F32>, fold(tiles), 256, s, p, tiles, (int)per_row)
               : go(&quantize_tiles_kernel<GEMM_DTYPE_BF16F32>, fold(tiles), 256, s, p, tiles, (int)per_row);
}

}  // namespace gemm
