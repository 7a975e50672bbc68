// Shared by the kernels that pass over rows (gemm_norm.hip, gemm_layer_norm.hip, gemm_route.hip): chunks
// of 8 consecutive values a lane, sums over the lanes of a row, fp8 and 8-bit integer codes, launches.
#pragma once

#include "gemm_device.hpp"

#if defined(__HIPCC__)

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
// The same, non-temporal: a hint to the caches that the lines are not needed again soon.
template <class V> __device__ __forceinline__ V get_nt(const void *p) {
    typedef V Loose __attribute__((aligned(1)));
    return __builtin_nontemporal_load(static_cast<const Loose *>(p));
}
template <class V> __device__ __forceinline__ void put_nt(void *p, V v) {
    typedef V Loose __attribute__((aligned(1)));
    __builtin_nontemporal_store(v, static_cast<Loose *>(p));
}

// Up to 8 values, n of them valid (n <= 0: none; the rest read as zero).  In bf16 the values of a row's last,
// shorter chunk are loaded one after the other, each waited for before the next: 8192 rows bf16 of 4095 columns
// take 96 us forward and 146 backward in layer norm, of 4096 49 and 57.
template <int DT, bool NT = false>
__device__ __forceinline__ typename Io<DT>::Raw load_raw(const void *base, int64_t at, int n) {
    typedef typename Io<DT>::T T;
    typedef typename Io<DT>::Raw Raw;
    const T *src = static_cast<const T *>(base) + at;
    Raw r = {};
    if (n >= kChunk) {
        r = NT ? get_nt<Raw>(src) : get<Raw>(src);
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
template <int DT, bool NT = false>
__device__ __forceinline__ void store8(void *base, int64_t at, f32x8 v, int n) {
    typedef typename Io<DT>::T T;
    T *dst = static_cast<T *>(base) + at;
    if (n >= kChunk) {
        if constexpr (DT == GEMM_DTYPE_F32) {
            if constexpr (NT) put_nt(dst, v);
            else put(dst, v);
        } else {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (uint32_t)to_bf16(v[2 * i]) | ((uint32_t)to_bf16(v[2 * i + 1]) << 16);
            if constexpr (NT) put_nt(dst, w);
            else put(dst, w);
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
template <bool NT = false, class P>
__device__ __forceinline__ void put_norm(const P &p, int64_t row, int64_t col, f32x8 y, int n) {
    if (p.out_type == GEMM_OUT_FP8) {
        const float amax = fmaxf(max16(finite_max(y)), kMinAmax);
        const u32x2 w = codes8(y, kE4m3Max / amax);
        if (n > 0) {
            store_codes(static_cast<uint8_t *>(p.out) + row * p.ldo + col, w, n);
            if ((col & (GEMM_SCALE_BLOCK - 1)) == 0)
                p.scales[row * p.ld_scales + col / GEMM_SCALE_BLOCK] = amax / kE4m3Max;
        }
    } else if (p.out_type == GEMM_OUT_BF16) {
        store8<GEMM_DTYPE_BF16F32, NT>(p.out, row * p.ldo + col, y, n);
    } else {
        store8<GEMM_DTYPE_F32, NT>(p.out, row * p.ldo + col, y, n);
    }
}

// s of one chunk, rounded to the operands' type as it is stored.
template <int DT, class P>
__device__ __forceinline__ f32x8 norm_sum(const P &p, int64_t row, int64_t col, int n) {
    f32x8 v = load8<DT>(p.x, row * p.ldx + col, n);
    if (p.residual != nullptr) {
        const f32x8 r = load8<DT>(p.residual, row * p.ldr + col, n);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[e] = Io<DT>::widen(Io<DT>::narrow(v[e] + r[e]));
    }
    return v;
}

// 8-bit integer codes with a scale a row, 127 / amax being inv: finite values come out at most
// 127 * (1 + 2^-23), which rounds to 127.
constexpr float kInt8Max = 127.0f;
__device__ __forceinline__ u32x2 codes8_int(f32x8 v, float inv) {
    u32x2 w = {0, 0};
#pragma unroll
    for (int e = 0; e < kChunk; ++e) w[e / 4] |= ((uint32_t)(int)rintf(v[e] * inv) & 0xffu) << (8 * (e & 3));
    return w;
}
// Largest magnitude as bits, in the order of the magnitudes; infinities and NaN are above every finite one's.
constexpr uint32_t kInfBits = 0x7f800000u;
__device__ __forceinline__ uint32_t max_bits(f32x8 v) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
    return m;
}
// What a row of largest magnitude `top` is multiplied by to give its codes, and its scale.  A row that
// holds an infinity or a NaN has codes of 0 and a scale of NaN, so that what is made of it is NaN.
__device__ __forceinline__ float int8_factor(uint32_t top, float &scale) {
    const float amax = fmaxf(__uint_as_float(top), kMinAmax);
    scale = top >= kInfBits ? __builtin_nanf("") : amax / kInt8Max;
    return kInt8Max / amax;
}
// Codes of a chunk of such a row; top: the row's.
__device__ __forceinline__ u32x2 row_codes8(f32x8 v, uint32_t top, float inv) {
    return top >= kInfBits ? u32x2{0, 0} : codes8_int(v, inv);
}

// Largest over a team of THREADS threads; see team_sum.
template <int THREADS> __device__ __forceinline__ uint32_t team_max(uint32_t v, float *red, int set) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
    if (THREADS == 64) return v;
    constexpr int W = THREADS / 64;
    float *r = red + set * W;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = __uint_as_float(v);
    __syncthreads();
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) t = max(t, __float_as_uint(r[w]));
    return t;
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

// How a row of N values is shared out: a wave with two chunks a lane, teams of four and of sixteen
// waves with one or two, or sixteen waves that walk it.
enum Shape { kWave2, kFour2, kSixteen1, kSixteen2, kLong };
inline Shape shape_of(int64_t N) {
    return N <= 1024 ? kWave2 : N <= 4096 ? kFour2 : N <= 8192 ? kSixteen1 : N <= 16384 ? kSixteen2 : kLong;
}

}  // namespace
}  // namespace gemm

#endif
