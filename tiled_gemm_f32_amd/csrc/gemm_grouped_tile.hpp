// Tile kernel of the grouped and block-scaled products: instantiated in
// gemm_grouped_f32.hip, gemm_grouped_bf16.hip and gemm_grouped_fp8.hip.
//
// A workgroup makes a tile of BM x BN outputs of one group, walking k in
// slabs of 128 bytes a row (32 fp32, 64 bf16 or 128 fp8 values: for fp8
// exactly one scale block).  A ring of NS LDS stages holds a slab each: while
// one is multiplied the next NS - 1 land in the others.  WM x WN waves each
// hold 32*FM x 32*FN outputs; a wave keeps the slab's B fragments and two
// sets of A fragments in registers, so every LDS byte of A is read once a
// wave and the reads of A fragment i + 1 (or of the next slab) run under the
// products of fragment i.
//
// Measured, and what bounds it: 8192^3 fp8 in 256 x 256 takes 455 to 500 us
// over boxes (2.2 to 2.4 PF; profiled, 484 at least and 594 in the median): a
// slab takes 1.6 us, of which its matrix instructions alone would take 0.93
// and its 64 KB 0.55 to 0.68 to land with every compute unit loading.  8
// uneven groups of 8192 x 4096 x 2048 bf16, inputs changing from call to call:
// 165 us (0.83 PF; a library's product of 8192^3 reaches 1.1 to 1.5 here).
// The matrix cores are 0.47 busy in it: 353 MB come for operands of 168, a
// wave's tile of 128 x 64 reads more of LDS than 128 x 128 would, a workgroup
// stores its tile with the matrix cores idle, and groups cut tiles.  It is not
// the power limit: zeros take 161.  fp32 is bound by the matrix cores, 0.84 to
// 0.87 busy (a slab of 128 x 128 takes 1.75 us of them, 0.6 of loads; 8 uneven
// groups of 8192 x 2048 x 1024 285 us, 121 TF; 8192 x 4096 x 4096 1.88 ms, 146).
//
// fp8 with block scales: the matrix core sums a block of 128 k into a partial
// tile of its own (two v_mfma_f32_32x32x64_f8f6f4, the first with a zero
// addend), which is then added to the accumulators times the block's scale,
// a(row) * b(column block): 16 fused multiply-adds a fragment (64 cycles)
// beside 128 matrix cycles, issued while the other wave of the SIMD has the
// matrix core.  The accumulators must be architectural registers for that,
// which is why a wave's tile is 128 x 64 and two waves share a SIMD (the
// 128 x 128 wave tile of the per-tensor fp8 kernels fills the accumulation
// registers, which only matrix instructions can add to).
//
// LDS layouts, in 16-byte chunks:
//   k-contiguous operand: [rows][8 chunks]; chunk c of row r at
//     c ^ ((r >> 1) & 7): 32 rows at one chunk touch every bank group of the
//     256-byte period twice a half-wave.
//   bf16 stored the other way: [64-column block][64 k][8 chunks], chunk c of
//     k row r at c ^ 4*((r >> 1) & 1), read with ds_read_b64_tr_b16.
//   fp8 stored the other way: [128-column block][128 k][8 chunks], chunk c of
//     k row r at c ^ (r & 7), read with ds_read_b64_tr_b8.
//   fp32 stored the other way: [32-column block][32 k][8 chunks], read a value a
//     lane (a fragment pair's 16 instructions take 1024 cycles, its reads some
//     100).
//
// DMA: operands whose rows start on 16 bytes come by direct-to-LDS buffer
// loads.  Rows past the ends fall outside the buffer resource and read as
// zero; where K ends inside a slab, what the loads brought past it is zeroed
// in LDS before it is read.  Otherwise (REG) chunks go through registers with
// unaligned 16-byte loads, and the last slab is put in order in LDS.
#pragma once

#include <algorithm>
#include <cmath>

#include "gemm_grouped.hpp"

#if defined(__HIPCC__)

namespace gemm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v2i lds_v2i;
typedef unsigned __int128 u128;

constexpr int kSlab = 128;              // bytes of k a slab holds of every row

// A vector at any alignment of its elements, which the hardware's global accesses take.
template <class V> struct __attribute__((packed, aligned(1))) Anywhere {
    V v;
};

template <int DT_, int FM_, int FN_, int WM_, int WN_, bool AKN_, bool BKN_, bool DMA_, int NS_ = 2>
struct TileConfig {
    static constexpr int DT = DT_, FM = FM_, FN = FN_, WM = WM_, WN = WN_;
    static constexpr bool AKN = AKN_, BKN = BKN_, DMA = DMA_;
    static constexpr int NS = DMA ? NS_ : 2;          // LDS stages
    static constexpr int NW = WM * WN, BM = 32 * FM * WM, BN = 32 * FN * WN;
    static constexpr int esz = DT == GEMM_DTYPE_FP8F32 ? 1 : DT == GEMM_DTYPE_BF16F32 ? 2 : 4;
    static constexpr int BK = kSlab / esz;            // k a slab
    // REG: slabs under way in registers.  Two where there is room: a small tile's products
    // of one slab do not cover a load.
    static constexpr int kSets = DMA ? 1 : FM == 1 || (FM == 2 && !AKN) ? 2 : 1;
    static constexpr int kA = BM * kSlab, kB = BN * kSlab, kStage = kA + kB;
};

// One operand of a tile as the loads see it: KN false: `rows` rows of
// `len` k at base (row stride ld); KN true: `len` rows of k, `rows` columns.
template <class C, bool KN, int ROWS>
struct Loader {
    static constexpr int esz = C::esz;
    static constexpr int kLoads = ROWS * 8 / (64 * C::NW);    // 16-byte chunks a thread and slab
    static constexpr int kGroups = C::BK / 8;                 // KN: groups of 8 k rows a slab
    static_assert(!KN || kGroups % C::NW == 0, "a load of all waves stays in one block of columns");
    const char *base;
    int64_t ld;          // bytes
    int rows, len;       // elements
    uint32_t off;        // this lane's offset in load 0
    uint32_t odd;        // NW == 1: in load 1, whose rows are swizzled as rows 8 .. 15 of 16
    u32x4 reg[C::DMA ? 1 : C::kSets][C::DMA ? 1 : kLoads];

    static __device__ __forceinline__ int swizzle(int r) {
        return !KN ? (r >> 1) & 7 : esz == 4 ? 0 : esz == 2 ? 4 * ((r >> 1) & 1) : r & 7;
    }
    __device__ __forceinline__ void init(int wave, int lane) {
        const int r = 8 * wave + (lane >> 3);
        off = (uint32_t)(r * (int)ld + 16 * ((lane & 7) ^ swizzle(r)));
        odd = (uint32_t)(r * (int)ld + 16 * ((lane & 7) ^ swizzle(r + 8)));
    }
    __device__ __forceinline__ uint32_t offset(int j) const { return !KN && C::NW == 1 && j % 2 == 1 ? odd : off; }
    // First row (KN: k row) and first byte along the row of load j, over all waves.
    static __device__ __forceinline__ constexpr int row_of(int j) {
        return KN ? 8 * ((j * C::NW) % kGroups) : 8 * C::NW * j;
    }
    static __device__ __forceinline__ constexpr int byte_of(int j) { return KN ? kSlab * ((j * C::NW) / kGroups) : 0; }

    // DMA: the buffer resource of slab t.  Bounds in 32 bits and without branches, which would
    // cut the loop's schedule: a panel of 256 rows is below 2^31 bytes (checked on the host).
    __device__ __forceinline__ rsrc_t source(int t) const {
        const int step = (int)ld;
        const int left = KN ? slab_left(t, C::BK, len) : len * esz - t * kSlab;          // KN: rows, else bytes
        const char *src = base + (KN ? (int64_t)t * C::BK * ld : (int64_t)t * kSlab);
        const int wide = ((KN ? rows * esz : max(left, 0)) + 15) & ~15;         // whole chunks
        const int deep = KN ? min(left, C::BK) : rows;
        const int bytes = (int)((uint32_t)deep * (uint32_t)step - (uint32_t)(step - wide));      // past the end: any
        return make_rsrc(src, (uint32_t)(max(bytes, 0) & ~((left - 1) >> 31)));
    }
    __device__ __forceinline__ void load(const rsrc_t &r, char *stage, int wave, int j) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(stage + (j * C::NW + wave) * 1024), 16,
                                                 offset(j) + (uint32_t)(row_of(j) * (int)ld + byte_of(j)), 0, 0, 0);
    }
    // REG: slab t into staging set `set`, at offsets that the panel's last 16 bytes bound.  Where
    // a row (or, KN, a row of the last columns) ends inside a chunk, what follows it in memory
    // comes too; the panel's last chunk comes too early.  Both are put right by cut, in the last slab.
    __device__ __forceinline__ void hold(int t, int set) {
        if constexpr (!C::DMA) {
            const int step = (int)ld, wide = (KN ? rows : len) * esz;
            const int first = KN ? slab_first(t, C::BK, len) : 0;
            const int limit = KN ? slab_limit(len - first, C::BK, step, wide) : (rows - 1) * step + wide - 16;
            // From 16 bytes before: the last tile's columns may be fewer than a chunk.
            const char *src = base + (int64_t)first * ld - 16;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int at = min((int)offset(j) + row_of(j) * step + (KN ? byte_of(j) : t * kSlab), limit);
                reg[set][j] = reinterpret_cast<const Anywhere<u32x4> *>(src + (uint32_t)(at + 16))->v;
            }
        }
    }
    __device__ __forceinline__ void stash(char *stage, int set, int wave, int lane) const {
        if constexpr (!C::DMA) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                *reinterpret_cast<u32x4 *>(stage + (j * C::NW + wave) * 1024 + lane * 16) = reg[set][j];
        }
    }
    // Slab t, the last one, in LDS: zero what lies past K, and (REG) move the panel's last chunk
    // to its place.  tid: of the 64 * NW threads whose loads it was.
    __device__ __forceinline__ void cut(int t, char *stage, int tid) const {
        if (KN && C::DMA) return;                                // k rows past the last were read as zero
        const int left = KN ? len - t * C::BK : len * esz - t * kSlab;
        const int wide = KN ? rows * esz : left;
        for (int i = tid; i < ROWS * 8; i += 64 * C::NW) {
            const int r = KN ? (i >> 3) % C::BK : i >> 3;
            const int byte = 16 * ((i & 7) ^ swizzle(r)) + (KN ? kSlab * ((i >> 3) / C::BK) : 0);
            const int past = byte + 16 - wide;                   // bytes of the chunk past the row's end
            const bool moved = !C::DMA && r == (KN ? left : rows) - 1 && past > 0 && past < 16;
            if (!moved && (KN ? r < left : past <= 0)) continue;
            u32x4 *at = reinterpret_cast<u32x4 *>(stage + 16 * i);
            u32x4 v = *at;
            if (moved)
                v = __builtin_bit_cast(u32x4, __builtin_bit_cast(u128, v) >> (8 * past));
            if (KN) {
                if (r >= left) v = u32x4{};
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int n = 16 - past - 4 * d;             // valid bytes from here on
                    v[d] &= n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1;
                }
            }
            *at = v;
        }
    }
};

// One 32-row fragment of a slab: 16 registers a lane, grouped as the matrix
// instruction takes them (fp8: two of 64 k; bf16: four of 16 k), so that they
// are read into place.
template <int ESZ> struct FragOf {
    u32x4 q[4];
};
template <> struct FragOf<1> {
    i32x8 h[2];
};

// Offset in a panel of this lane's first read of the fragment at row (column) 32 * f.
template <class C, bool KN> __device__ __forceinline__ uint32_t frag_base(int f, int lane) {
    const int h = lane >> 5, l32 = lane & 31;
    if constexpr (!KN) {
        const int c = C::esz == 1 ? 2 * h : h;
        return (uint32_t)((32 * f + l32) * kSlab + 16 * (c ^ ((l32 >> 1) & 7)));
    } else if constexpr (C::esz == 2) {
        const int q = lane >> 4, j16 = lane & 15;
        const int row = 8 * (q >> 1) + (j16 >> 2);
        const int c = 2 * (q & 1) + ((j16 & 3) >> 1) + 4 * ((f & 1) ^ ((row >> 1) & 1));
        return (uint32_t)((f >> 1) * (C::BK * kSlab) + row * kSlab + 16 * c + 8 * (j16 & 1));
    } else if constexpr (C::esz == 4) {
        return (uint32_t)((32 * f + 4 * h) * kSlab + 4 * l32);
    } else {
        const int s16 = lane & 15;
        const int e = ((s16 >> 1) & 3) + 4 * (s16 >> 3);
        const int c = (2 * f + (l32 >> 4)) & 7;
        return (uint32_t)((f >> 2) * (C::BK * kSlab) + (32 * h + e) * kSlab + 16 * (c ^ e) + 8 * (s16 & 1));
    }
}
// Fragment i after the one `base` is for (a multiple of the wave's number of
// them), all 128 bytes of k.  Further chunks are the first one's offset with
// bits flipped, the swizzles being exclusive ors.
template <class C, bool KN>
__device__ __forceinline__ FragOf<C::esz> read_frag(const char *panel, uint32_t base, int i) {
    FragOf<C::esz> v;
    if constexpr (!KN) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // fp8: 32 consecutive bytes of each half; bf16 and fp32: 16 bytes of each 32.
            const uint32_t flip = 16u * (C::esz == 1 ? 4 * (q >> 1) + (q & 1) : 2 * q);
            const u32x4 w = *reinterpret_cast<const u32x4 *>(panel + ((base ^ flip) + 32 * kSlab * i));
            if constexpr (C::esz == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v.h[q >> 1][4 * (q & 1) + e] = (int)w[e];
            } else {
                v.q[q] = w;
            }
        }
    } else if constexpr (C::esz == 2) {
        const char *at = panel + ((base ^ (64u * (i & 1))) + (i >> 1) * (C::BK * kSlab));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(at + 16 * kSlab * q));
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(at + 16 * kSlab * q + 4 * kSlab));
            v.q[q] = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    } else if constexpr (C::esz == 4) {
        const uint32_t *at = reinterpret_cast<const uint32_t *>(panel + (base + 32 * kSlab * i));
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) v.q[q][e] = at[(8 * q + e) * (kSlab / 4)];
    } else {
        const char *at = panel + (base ^ (32u * i));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const v2i w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(at + (64 * (q >> 2) + 8 * (q & 3)) * kSlab));
            v.h[q >> 2][2 * (q & 3)] = w[0];
            v.h[q >> 2][2 * (q & 3) + 1] = w[1];
        }
    }
    return v;
}

// B^T as the first operand and A^T as the second: register 4g + t of lane
// (h, l32) is row l32, column 8g + 4h + t of the fragment.
__device__ __forceinline__ f32x16 product_fp8(const FragOf<1> &a, const FragOf<1> &b, int half, f32x16 part) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b.h[half], a.h[half], part, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x16 product_bf16(const FragOf<2> &a, const FragOf<2> &b, int half, f32x16 acc) {
#pragma unroll
    for (int i = 2 * half; i < 2 * half + 2; ++i)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b.q[i]),
                                                      __builtin_bit_cast(bf16x8, a.q[i]), acc, 0, 0, 0);
    return acc;
}

// The two lane halves' k of one instruction lie four apart (their 16 bytes), in both operands.
__device__ __forceinline__ f32x16 product_f32(const FragOf<4> &a, const FragOf<4> &b, int half, f32x16 acc) {
#pragma unroll
    for (int i = 2 * half; i < 2 * half + 2; ++i) {
        const f32x4 av = __builtin_bit_cast(f32x4, a.q[i]), bv = __builtin_bit_cast(f32x4, b.q[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bv[e], av[e], acc, 0, 0, 0);
    }
    return acc;
}
template <int ESZ>
__device__ __forceinline__ f32x16 product(const FragOf<ESZ> &a, const FragOf<ESZ> &b, int half, f32x16 acc) {
    if constexpr (ESZ == 1) return product_fp8(a, b, half, acc);
    else if constexpr (ESZ == 2) return product_bf16(a, b, half, acc);
    else return product_f32(a, b, half, acc);
}

// Where a tile's operands and results are.
struct Place {
    const char *a, *b;
    int64_t out;                  // elements
    int rows, cols, len;          // of the tile, and its k
    int group, row0, n0;
};

// A tile of one group, for all waves of a workgroup.  st, scale: LDS for NS stages and their scales, an
// array each: the compiler can then tell that a read of one does not depend on loads still landing in
// another.
template <class C>
__device__ __forceinline__ void make_tile(const GroupedParams &p, const Place &at, char *st0, char *st1, char *st2,
                                          char *st3, float *scale0, float *scale1, float *scale2, float *scale3) {
    constexpr int FM = C::FM, FN = C::FN, NW = C::NW, BM = C::BM, BN = C::BN;
    constexpr bool FP8 = C::DT == GEMM_DTYPE_FP8F32, WGRAD = C::AKN;
    constexpr int NS = C::NS;
    static_assert(NS == 2 || (NS <= 4 && C::DMA), "");
    auto stage = [&](int i) __attribute__((always_inline)) -> char * {
        return i == 0 ? st0 : i == 1 ? st1 : i == 2 ? st2 : st3;
    };

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int out_rows = at.rows, out_cols = at.cols, group = at.group, row0 = at.row0, n0 = at.n0;
    const int64_t out_at = at.out;

    Loader<C, C::AKN, BM> a;
    Loader<C, C::BKN, BN> b;
    a.base = at.a;
    b.base = at.b;
    a.rows = out_rows;
    b.rows = out_cols;
    a.len = b.len = at.len;
    a.ld = p.lda * C::esz;
    b.ld = p.ldb * C::esz;
    a.init(wave, lane);
    b.init(wave, lane);

    // Slabs that are read as they land; the last one is put in order first where K ends inside it
    // (always, if it came through registers).
    const int len = a.len;
    const bool cut = !C::DMA || ((!C::AKN || !C::BKN) && len % C::BK != 0);
    const int nk = cut ? (len - 1) / C::BK : slabs_of(len, C::BK);

    const int l32 = lane & 31;
    // Scales of the block that slab t is go to LDS as the slab does, into its
    // stage's set: wave w < kScaleA loads those
    // of 64 rows, the next wave those of the tile's column blocks, the others
    // nothing; five loads a wave and slab from global memory instead cost a
    // tenth of the whole call.
    constexpr int kScaleA = (BM + 63) / 64;
    static_assert(!FP8 || kScaleA < NW, "a wave for each 64 rows and one for the columns");
    auto scale_set = [&](int i) __attribute__((always_inline)) -> float * {
        return i == 0 ? scale0 : i == 1 ? scale1 : i == 2 ? scale2 : scale3;
    };
    const float *sc_base = nullptr;
    int64_t sc_step = 0;
    uint32_t sc_bytes = 0, sc_off = 0;
    if constexpr (FP8) {
        const bool of_a = wave < kScaleA, of_b = wave == kScaleA;
        const int col_blocks = (out_cols + GEMM_SCALE_BLOCK - 1) / GEMM_SCALE_BLOCK;
        const int64_t each = of_a ? p.sc.a_row : p.sc.b_n;
        const int count = of_a ? out_rows : col_blocks;
        sc_base = of_a ? p.sc.a + (int64_t)row0 * p.sc.a_row
                       : p.sc.b + (int64_t)group * p.sc.b_group + (int64_t)(n0 / GEMM_SCALE_BLOCK) * p.sc.b_n;
        sc_step = of_a ? p.sc.a_block : p.sc.b_k;
        sc_bytes = of_a || of_b ? (uint32_t)((count - 1) * (int)each + 1) * 4u : 0u;
        sc_off = (uint32_t)min(of_a ? 64 * wave + lane : lane, count - 1) * (uint32_t)each * 4u;
    }
    const int blocks = slabs_of(len, GEMM_SCALE_BLOCK);
    auto load_scales = [&](int t, float *set) __attribute__((always_inline)) {
        if constexpr (FP8) {
            const rsrc_t r = make_rsrc(sc_base + min(t, blocks - 1) * sc_step, sc_bytes);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(set + 64 * wave), 4, sc_off, 0, 0, 0);
        }
    };
    // a(row) * b(column block) for this lane's rows of fragment i, from a slab's set.
    auto scale_of = [&](const float *set, int i) __attribute__((always_inline)) {
        return FP8 ? set[(wm * FM + i) * 32 + l32] * set[64 * kScaleA + wn * 32 * FN / GEMM_SCALE_BLOCK] : 0.0f;
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
    FragOf<C::esz> fa[2], fb[FN];
    static_assert(FM <= 2 || !C::AKN || C::esz == 2, "");
    uint32_t a_base = frag_base<C, C::AKN>(wm * FM, lane), b_base = frag_base<C, C::BKN>(wn * FN, lane);
    auto read_a = [&](const char *st, int i) { return read_frag<C, C::AKN>(st, a_base, i); };
    auto read_b = [&](const char *st, int j) { return read_frag<C, C::BKN>(st + C::kA, b_base, j); };
    constexpr int NA = Loader<C, C::AKN, BM>::kLoads, NB = Loader<C, C::BKN, BN>::kLoads;
    // Loads from..to-1 of a slab's NA + NB, from its two resources.
    auto load = [&](const rsrc_t &ra, const rsrc_t &rb, char *st, int from, int to) __attribute__((always_inline)) {
#pragma unroll
        for (int l = from; l < to; ++l) {
            if (l < NB) b.load(rb, st + C::kA, wave, l);
            else a.load(ra, st, wave, l - NB);
        }
    };
    auto fetch = [&](int t, char *st, int set) __attribute__((always_inline)) {
        if constexpr (C::DMA) {
            load(a.source(t), b.source(t), st, 0, NA + NB);
        } else {
            a.hold(t, set);
            b.hold(t, set);
        }
    };
    auto stash = [&](char *st, int set) __attribute__((always_inline)) {
        a.stash(st, set, wave, lane);
        b.stash(st + C::kA, set, wave, lane);
    };
    constexpr int kSets = C::kSets;

    // fp8: the partial tile of one product is added while the next one is
    // multiplied, half of it behind each matrix instruction, so that a wave
    // keeps the matrix core busy by itself.  The last product's of a slab is
    // added by the next slab (kCarry: an even number of products, so that it is
    // always in part[1]); s_due is the scale it takes.
    constexpr int kProducts = FM * FN;
    constexpr bool kCarry = kProducts % 2 == 0;
    f32x16 part[2] = {};
    float s_due = 0.0f;
    // Half of the partial tile of product n (modulo their number).
    auto add = [&](int n, int half) __attribute__((always_inline)) {
        if constexpr (FP8) {
            const int m = (n + kProducts) % kProducts;
#pragma unroll
            for (int e = 8 * half; e < 8 * half + 8; ++e)
                acc[m / FN][m % FN][e] = fmaf(part[m & 1][e], s_due, acc[m / FN][m % FN][e]);
        }
    };
    // Products of slab t, whose fragments (B's, and A's first) are in
    // registers, from stage `cur`; meanwhile slab t + 1 lands in `next`, whose
    // first fragments are read at the end, and slab t + 2 is sent for.
    // `first`: the set that holds A's first fragment; `scales`: the slab's; `turn`: t modulo the
    // loop's turn.
    //
    // With four steps a slab (kSpread) the loads go out one between two matrix
    // instructions, half of them behind the barrier and the rest in the next
    // slab's first step: sent in a row they hold up the matrix instructions
    // behind them (8192^3 fp8: 500 us; 480 spread over the last step, 465 so).
    // Tiles of fewer steps wait for memory rather than for the matrix cores,
    // and send them at once.
    constexpr bool kSpread = C::DMA && NW == 8;
    constexpr int kFirst = NS == 2 ? (NA + NB) / 2 : NA + NB, kRest = NA + NB - kFirst;
    constexpr int kSlabLoads = NA + NB + (FP8 ? 1 : 0);
    auto slab = [&](int t, char *cur, char *next, int first, float *scales, int turn) __attribute__((always_inline)) {
        // Addresses are made again from these in every slab: kept across the loop they would
        // take more registers than there are.
        asm volatile("" : "+v"(a_base), "+v"(b_base), "+v"(a.off), "+v"(b.off));
        rsrc_t ra, rb;
        if (kSpread && kRest > 0) {
            ra = a.source(t + 1);
            rb = b.source(t + 1);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int s = (first + i) & 1;
            const float s_ab = scale_of(scales, i);
            if (i + 1 < FM) {
                fa[s ^ 1] = read_a(cur, i + 1);
            } else {
                stash(next, (turn + 1) % kSets);
                // Slab t + 1 (and its scales) has landed; of three stages or more, or two sets of
                // staging registers, later slabs' loads may be under way.
                __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(C::DMA ? (NS - 2) * kSlabLoads : (kSets - 1) * (NA + NB)));
                __builtin_amdgcn_s_barrier();
                fa[s ^ 1] = read_a(next, 0);
                load_scales(t + NS, scales);
                __builtin_amdgcn_sched_barrier(0);        // the waits count what was sent after the scales
                if constexpr (kSpread) {
                    ra = a.source(t + NS);
                    rb = b.source(t + NS);
                } else if constexpr (C::DMA) {
                    fetch(t + NS, cur, 0);
                } else {
                    fetch(t + 1 + kSets, cur, (turn + 1) % kSets);     // the set that was put away
                }
            }
            // The loads that go out in gap g (0 .. 2 * FN - 1) of this step.
            auto send = [&](int g) __attribute__((always_inline)) {
                if (kSpread && i + 1 == FM) load(ra, rb, cur, g * kFirst / (2 * FN), (g + 1) * kFirst / (2 * FN));
                if (kSpread && i == 0)
                    load(ra, rb, next, kFirst + g * kRest / (2 * FN), kFirst + (g + 1) * kRest / (2 * FN));
            };
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int n = i * FN + j;
                if constexpr (FP8) part[n & 1] = product<C::esz>(fa[s], fb[j], 0, f32x16{});
                else acc[i][j] = product<C::esz>(fa[s], fb[j], 0, acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
                if (kCarry || n > 0) add(n - 1, 0);
                send(2 * j);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (FP8) part[n & 1] = product<C::esz>(fa[s], fb[j], 1, part[n & 1]);
                else acc[i][j] = product<C::esz>(fa[s], fb[j], 1, acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
                if (i + 1 == FM) fb[j] = read_b(next, j);
                if (kCarry || n > 0) add(n - 1, 1);
                send(2 * j + 1);
                s_due = s_ab;
            }
            if (!kCarry && i + 1 == FM) {
                add(-1, 0);
                add(-1, 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (len > 0) {
        // In this order: the waits count on it.
        load_scales(0, scale0);
        fetch(0, st0, 0);
        if constexpr (C::DMA) {
#pragma unroll
            for (int i = 1; i < NS; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                load_scales(i, scale_set(i));
                __builtin_amdgcn_sched_barrier(0);
                if (kSpread) load(a.source(i), b.source(i), stage(i), 0, kFirst);
                else fetch(i, stage(i), 0);
            }
        } else {
            // Every set's loads go out before the first is waited for.
            __builtin_amdgcn_sched_barrier(0);
            load_scales(1, scale_set(1));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 1; i < kSets; ++i) fetch(i, st0, i);
            __builtin_amdgcn_sched_barrier(0);
            stash(st0, 0);
            fetch(kSets, st0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        // Slab 0 has landed when only the others' loads are left.
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(
            C::DMA ? (NS - 1) * ((kSpread ? kFirst : NA + NB) + (FP8 ? 1 : 0)) : kSets * (NA + NB) + (FP8 ? 1 : 0)));
        __builtin_amdgcn_s_barrier();
        fa[0] = read_a(st0, 0);
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = read_b(st0, j);
        int t = 0;
        // Whole turns of the stages as straight-line code, then the rest.
        constexpr int kRound = FM * NS % 2 == 0 ? NS : 2 * NS;
        for (; t + kRound <= nk; t += kRound) {
#pragma unroll
            for (int u = 0; u < kRound; ++u)
                slab(t + u, stage(u % NS), stage((u + 1) % NS), (u * FM) & 1, scale_set(u % NS), u);
        }
#pragma unroll
        for (int u = 0; u < kRound - 1; ++u)
            if (t + u < nk) slab(t + u, stage(u % NS), stage((u + 1) % NS), (u * FM) & 1, scale_set(u % NS), u);
        if (cut) {
            // Slab nk ends K.  It has landed (slab 0: the wait above), every
            // wave has read what it will of it, and it is read again.
            const int at = nk % NS;
            char *cur = stage(at), *next = stage((at + 1) % NS);
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
            __builtin_amdgcn_s_barrier();
            a.cut(nk, cur, threadIdx.x);
            b.cut(nk, cur + C::kA, threadIdx.x);
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
            __builtin_amdgcn_s_barrier();
            fa[0] = read_a(cur, 0);
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[j] = read_b(cur, j);
            slab(nk, cur, next, 0, scale_set(at), 0);
        }
        if (kCarry) {
            add(-1, 0);
            add(-1, 1);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(C::DMA || FP8 ? 0 : 63));       // (what is under way to LDS)
        __builtin_amdgcn_s_barrier();
    }

    // Epilogue: 32 rows of the wave's columns at a time through its own piece
    // of LDS, so that a store instruction writes whole runs of a row.
    constexpr int kPiece = 32 * FN * 128, kFit = C::kStage / kPiece;
    constexpr int kChunks = 8 * FN;                  // 16-byte chunks (4 columns) of a row
    char *piece = wave < kFit ? st0 + wave * kPiece : st1 + (wave - kFit) * kPiece;
    float *of = static_cast<float *>(p.out) + out_at;
    uint16_t *oh = static_cast<uint16_t *>(p.out) + out_at;
    const bool bf16_out = !WGRAD && p.out_type == GEMM_OUT_BF16;
    // The lane again, opaque: what is made of it stays out of the loop's registers.
    int elane = threadIdx.x & 63;
    asm volatile("" : "+v"(elane));
    const int el32 = elane & 31;
    const int cc = elane % kChunks;
    const int col = wn * 32 * FN + 4 * cc;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = (8 * j + 2 * g + (elane >> 5)) ^ (el32 & (kChunks - 1));
                *reinterpret_cast<f32x4 *>(piece + el32 * (kChunks * 16) + 16 * c) =
                    f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            }
        constexpr int kRows = 64 / kChunks;          // rows an instruction takes
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += kRows) {
            const int r = r0 + elane / kChunks;
            f32x4 v = *reinterpret_cast<const f32x4 *>(piece + r * (kChunks * 16) + 16 * (cc ^ (r & (kChunks - 1))));
            const int row = (wm * FM + i) * 32 + r;
            if (row >= out_rows || col >= out_cols) continue;
            const int64_t o = (int64_t)row * p.ldo + col;
            const bool whole = col + 4 <= out_cols;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= p.alpha;
            if (bf16_out) {
                const uint32_t h0 = to_bf16(v[0]), h1 = to_bf16(v[1]), h2 = to_bf16(v[2]), h3 = to_bf16(v[3]);
                if (whole) {
                    reinterpret_cast<Anywhere<u32x2> *>(oh + o)->v = u32x2{h0 | (h1 << 16), h2 | (h3 << 16)};
                } else {
                    const uint32_t hs[4] = {h0, h1, h2, h3};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < out_cols) oh[o + e] = (uint16_t)hs[e];
                }
            } else {
                if (WGRAD && p.beta != 0.0f) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < out_cols) v[e] = fmaf(p.beta, of[o + e], v[e]);
                }
                if (whole) {
                    reinterpret_cast<Anywhere<f32x4> *>(of + o)->v = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < out_cols) of[o + e] = v[e];
                }
            }
        }
    }
}

// The place of a tile that find_tile found, `shift` columns into its own.  Integer divisions are vector
// code: their results are made scalar again, so that the buffer resources made of them are.
template <class C>
__device__ __forceinline__ Place place_of(const GroupedParams &p, const GroupTile &t, int tile_cols, int shift) {
    Place at;
    const int owner = __builtin_amdgcn_readfirstlane(t.group);
    at.group = max(owner, 0);
    at.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    at.rows = __builtin_amdgcn_readfirstlane(t.rows);
    at.n0 = __builtin_amdgcn_readfirstlane(t.tn) * tile_cols + shift;
    at.cols = min(C::BN, p.N - at.n0);
    at.len = owner < 0 ? 0 : p.K;
    at.a = static_cast<const char *>(p.A) + (int64_t)at.row0 * p.lda * C::esz;
    at.b = static_cast<const char *>(p.B) +
           ((int64_t)at.group * p.stride_b + (C::BKN ? (int64_t)at.n0 : (int64_t)at.n0 * p.ldb)) * C::esz;
    at.out = (int64_t)at.row0 * p.ldo + at.n0;
    return at;
}

template <class C>
__global__ void __launch_bounds__(64 * C::NW, 2)
grouped_tile_kernel(GroupedParams p, int tiles_m, int tiles_n) {
    constexpr int NS = C::NS, kScales = C::DT == GEMM_DTYPE_FP8F32 ? C::NW * 64 : 1;
    __shared__ __attribute__((aligned(1024))) char st0[C::kStage], st1[C::kStage];
    __shared__ __attribute__((aligned(1024))) char st2[NS > 2 ? C::kStage : 16], st3[NS > 3 ? C::kStage : 16];
    __shared__ float scale0[kScales], scale1[kScales], scale2[NS > 2 ? kScales : 1], scale3[NS > 3 ? kScales : 1];
    Place at;
    if constexpr (C::AKN) {
        int tm, tn, lo, hi;
        tile_coords(blockIdx.x, tiles_m, tiles_n, 4, tm, tn);
        at.group = find_group(p, blockIdx.y, lo, hi);
        at.row0 = __builtin_amdgcn_readfirstlane(tm) * C::BM;
        at.n0 = __builtin_amdgcn_readfirstlane(tn) * C::BN;
        at.rows = min(C::BM, p.N - at.row0);
        at.cols = min(C::BN, p.K - at.n0);
        at.len = hi - lo;
        at.a = static_cast<const char *>(p.A) + ((int64_t)lo * p.lda + at.row0) * C::esz;
        at.b = static_cast<const char *>(p.B) + ((int64_t)lo * p.ldb + at.n0) * C::esz;
        at.out = (int64_t)at.group * p.stride_out + (int64_t)at.row0 * p.ldo + at.n0;
    } else {
        at = place_of<C>(p, find_tile(p, blockIdx.x, C::BM, tiles_n, 4), C::BN, 0);
        if (at.rows <= 0) return;
    }
    make_tile<C>(p, at, st0, st1, st2, st3, scale0, scale1, scale2, scale3);
}

// The same, where the tiles past the last whole turn of the compute units are
// shared out: 128 x 256 to each of two workgroups, or 128 x 128 to each of
// four.  Tiles of at most 128 rows, groups' last ones, are made as 128 x 256.
// (8 groups of 8192 x 2048 x 4096 bf16, 1.1 turns: 159 us in whole tiles of 192 x
// 256, 151 so; 16 groups of 8192 x 4096 x 4096 fp8, 2.5 turns: 187 to 204 and 179
// to 193.)
template <class C, class HALF, class QUARTER>
__global__ void __launch_bounds__(64 * C::NW, 2)
grouped_shared_kernel(GroupedParams p, int tiles_n) {
    constexpr int kScales = C::DT == GEMM_DTYPE_FP8F32 ? C::NW * 64 : 1;
    static_assert(C::NS == 2 && HALF::NS == 2 && QUARTER::NS == 2 && C::BM == 256 && C::BN == 256, "");
    __shared__ __attribute__((aligned(1024))) char st0[C::kStage], st1[C::kStage];
    __shared__ float scale0[kScales], scale1[kScales];
    GroupTile t = find_tile<true>(p, blockIdx.x, C::BM, tiles_n, 4);
    t.parts = __builtin_amdgcn_readfirstlane(t.parts);
    t.part = __builtin_amdgcn_readfirstlane(t.part);
    if (t.parts > 1) {
        const int below = (t.parts == 4 ? t.part >> 1 : t.part) * 128;
        t.row0 += below;
        t.rows = min(t.rows - below, 128);
    }
    if (t.parts == 4) {
        const Place at = place_of<QUARTER>(p, t, C::BN, 128 * (t.part & 1));
        if (at.rows > 0 && at.cols > 0) make_tile<QUARTER>(p, at, st0, st1, st1, st1, scale0, scale1, scale1, scale1);
        return;
    }
    Place at = place_of<C>(p, t, C::BN, 0);
    if (at.rows <= 0) return;
    if (at.rows <= 128) make_tile<HALF>(p, at, st0, st1, st1, st1, scale0, scale1, scale1, scale1);
    else make_tile<C>(p, at, st0, st1, st1, st1, scale0, scale1, scale1, scale1);
}

constexpr int kComputeUnits = 256;

template <class C> hipError_t launch_grouped_tile(const GroupedParams &p, hipStream_t stream) {
    GroupedParams args = p;
    int tiles_m, tiles_n;
    dim3 grid;
    if (C::AKN) {
        tiles_m = (p.N + C::BM - 1) / C::BM;
        tiles_n = (p.K + C::BN - 1) / C::BN;
        grid = dim3((unsigned)(tiles_m * tiles_n), (unsigned)p.groups);
    } else {
        tiles_m = (int)most_row_tiles(p.M, p.groups, C::BM, p.ends != nullptr);
        tiles_n = (p.N + C::BN - 1) / C::BN;
        grid = dim3((unsigned)(tiles_m * tiles_n));
    }
    void *argv[] = {&args, &tiles_m, &tiles_n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&grouped_tile_kernel<C>), grid, dim3(64 * C::NW), argv, 0,
                           stream);
}

template <int DT, bool BKN> hipError_t launch_grouped_shared(const GroupedParams &p, hipStream_t stream) {
    typedef TileConfig<DT, 4, 2, 2, 4, false, BKN, true> C;
    typedef TileConfig<DT, 2, 2, 2, 4, false, BKN, true> HALF;
    typedef TileConfig<DT, 2, 1, 2, 4, false, BKN, true> QUARTER;
    GroupedParams args = p;
    int tiles_n = (p.N + C::BN - 1) / C::BN;
    const int64_t tiles = most_row_tiles(p.M, p.groups, C::BM, p.ends != nullptr) * tiles_n;
    void *argv[] = {&args, &tiles_n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&grouped_shared_kernel<C, HALF, QUARTER>),
                           dim3((unsigned)(tiles + kShareTurn)), dim3(64 * C::NW), argv, 0, stream);
}

// Tiles and how long they take: 256 x 256, 192 x 256 and 128 x 256 (eight
// waves, the last on three stages), 128 x 128, 64 x 128 and 32 x 128 (four waves).
enum TileSize { kTile256, kTile192, kTileWide, kTile128, kTile64, kTile32 };

struct TileCost {
    int bm, bn;
    // us: a slab's and a tile's share of a busy compute unit's time, and a slab of a lone
    // workgroup (measured at 64 .. 8192 rows of K = 777 .. 16384, fp8 and bf16 alike since a slab
    // has the same bytes and matrix cycles).
    double slab, tile, alone;
};
constexpr TileCost kTileCosts[] = {
    {256, 256, 1.6, 8.0, 1.2},  {192, 256, 1.26, 7.5, 0.95}, {128, 256, 1.0, 7.0, 0.7},
    {128, 128, 0.59, 4.5, 0.6}, {64, 128, 0.40, 2.5, 0.38},
    {32, 128, 0.33, 1.2, 0.25}};

// `turn`: every compute unit gets one workgroup at most, and nothing hides
// its loads but loads of its own: the small tiles then take four stages
// (1024 x 2048 x 4096 bf16 in 64 x 128: 41 us on two stages, 27.5 on four; 64 x
// 4096 x 4096 in 32 x 128: 36.6 and 18.2), which otherwise cost more in
// workgroups a compute unit than they bring.
struct TileChoice {
    TileSize size;
    bool turn;
    double time;
};

// Time of `turns` turns of tiles that are `slabs` slabs deep.  tile_factor: of a tile's own time; `matrix`: us of
// matrix instructions that a slab of 128 x 128 takes, where they take longer than its loads (fp32);
// `staged`: us that a lone workgroup's slab takes longer through registers, a busy one's half as much.
inline double tile_time(const TileCost &c, double turns, double slabs, double tile_factor, double matrix,
                        double staged) {
    const double least_slab = matrix * c.bm * c.bn / (128 * 128);
    return std::max(turns * (slabs * (std::max(c.slab, least_slab) + staged / 2) + c.tile * tile_factor),
                    slabs * (std::max(c.alone, least_slab) + staged) + 6.0);
}

// The tile of the least time over `rows` rows of an output of `cols` columns,
// `slabs` slabs deep, in `groups` groups: large ones move the fewest bytes a
// product.  In 128 x 256, 128 x 128 and 256 x 256 (these with their last turn
// shared out), us: 2048 x 4096 x 4096 fp8 39, 43 and 42; 8192^3 510, 586 and
// 458; 16 uneven groups of 8192 x 4096 x 4096 210 to 220, 229 to 240 and 175 to
// 183; 64 rows of 4096 x 4096 27, 23 and 26, but 13 in 32 x 128.  192 x 256 is
// for numbers of tiles that 256 x 256 makes a poor last turn of: 32 uneven
// groups of 8192 x 2048 x 1024 bf16 66 to 69, and 69 to 72 in 256 x 256; the
// estimate takes it for 8 uneven groups of 8192 x 4096 x 2048 too, 164 to 172
// where 256 x 256 takes 153 to 163.
// Groups are taken to be alike, with half an empty tile each at their ends.
// `first`: the largest to consider.  256 x 256 tiles past the last whole turn go to two or four
// workgroups each.
inline TileChoice tile_choice(double rows, double cols, double slabs, double groups, TileSize first, double matrix,
                              double staged) {
    TileChoice best = {};
    double least = 0.0;
    for (int i = first; i <= kTile32; ++i) {
        const TileCost &c = kTileCosts[i];
        const double each = rows / groups / c.bm + 0.5;
        const double high = groups > 1 ? groups * std::max(1.0, each) : std::ceil(rows / c.bm);
        const double tiles = high * std::ceil(cols / c.bn);
        const double turns = std::ceil(tiles / kComputeUnits);
        double t = tile_time(c, turns, slabs, 1.0, matrix, staged);
        if (i == kTile256) {
            const double whole = std::floor(tiles / kComputeUnits), left = tiles - kComputeUnits * whole;
            const double rest = left <= 0.0                  ? 0.0
                                : left <= kComputeUnits / 4 ? slabs * 0.65 + 6.0
                                : left <= kComputeUnits / 2 ? slabs * 1.15 + 7.0
                                                            : slabs * c.slab + c.tile;
            t = std::max(whole * (slabs * c.slab + c.tile) + rest, slabs * 0.65 + 6.0);
        }
        if (i == first || t < least) {
            least = t;
            best = {static_cast<TileSize>(i), turns <= 1.0, t};
        }
    }
    return best;
}

// Time of the kernel whose waves share out k (gemm_grouped_deep.hip) in tiles of 32 x bn: `each` us
// for a wave's slab, eight slabs at a time.  Tiles of 32 columns share a compute unit by two, others
// take it in turns; groups are unlike each other, so a tenth is added to the number of tiles.  (On the
// same inputs in every call, 16 x 4096 x 4096 fp8 against K x N weights: 13.0 us in 32 x 128, 9.9 so;
// 128 x 2000 x 8000 fp8: 23.2 and 11.3; 64 x 1000 x 1024 fp32: 21.4 and 8.1; but 300 x 2000 x 4000 fp8,
// 630 tiles: 15.8 and 17.3.)
inline double deep_time(double rows, double cols, double slabs, double groups, int bn, double each) {
    const double high = groups > 1 ? 1.1 * groups * std::max(1.0, rows / groups / 32 + 0.5) : std::ceil(rows / 32);
    const double tiles = high * std::ceil(cols / bn);
    const double turns = tiles / kComputeUnits;
    return (bn == 32 ? std::max(1.0, turns) : std::ceil(turns)) * (std::ceil(slabs / 8) * each + 4.0) + 2.5;
}

// 16 instructions of 64 cycles for each of 4 x 4 fragment pairs, on four matrix cores.
constexpr double kMatrixF32 = 1.75;

template <int DT, bool BKN, bool DMA> hipError_t launch_sized(const GroupedParams &p, hipStream_t s) {
    constexpr bool FP8 = DT == GEMM_DTYPE_FP8F32, F32 = DT == GEMM_DTYPE_F32;
    const double slabs = std::ceil((double)p.K * (FP8 ? 1 : F32 ? 4 : 2) / kSlab);
    const double groups = p.ends != nullptr ? std::max(1, std::min(p.groups, p.M)) : 1;
    // Staging registers leave room for fewer accumulators, partial tiles for fewer still; fp32 is
    // bound by the matrix cores at 128 x 128 already.  (8 groups of 8000 x 4095 x 2047 bf16 through
    // registers: 217 us in 128 x 128, 187 in 192 x 256.)
    constexpr TileSize first = F32 ? kTile128 : DMA ? kTile256 : FP8 ? kTile64 : kTile192;
    const TileChoice c = tile_choice(p.M, p.N, slabs, groups, first, F32 ? kMatrixF32 : 0.0, DMA ? 0.0 : 0.15);
    constexpr int32_t op = BKN ? GEMM_OP_N : GEMM_OP_T;
    if (deep_time(p.M, p.N, slabs, groups, deep_columns(DT, BKN), F32 || BKN || !DMA ? 0.9 : 0.6) < c.time &&
        deep_takes(DT, op, DMA, p))
        return launch_grouped_deep(DT, op, DMA, p, s);
    switch (c.size) {
        case kTile256:
            if constexpr (first == kTile256) return launch_grouped_shared<DT, BKN>(p, s);
        case kTile192:
            if constexpr (first <= kTile192)
                return launch_grouped_tile<TileConfig<DT, 3, 2, 2, 4, false, BKN, DMA>>(p, s);
        case kTileWide:
            if constexpr (first <= kTileWide)
                return launch_grouped_tile<TileConfig<DT, 2, 2, 2, 4, false, BKN, DMA, DMA ? 3 : 2>>(p, s);
        case kTile128:
            // (The others' products of a 128 x 128 slab cover its loads.)
            if constexpr (DMA && DT == GEMM_DTYPE_BF16F32)
                if (c.turn) return launch_grouped_tile<TileConfig<DT, 2, 2, 2, 2, false, BKN, DMA, 4>>(p, s);
            if constexpr (first != kTile64)
                return launch_grouped_tile<TileConfig<DT, 2, 2, 2, 2, false, BKN, DMA>>(p, s);
        case kTile64:
            // (fp32 comes past here: twice 32 x 128 costs as much and starts sooner.)
            if constexpr (DMA && !F32)
                if (c.turn) return launch_grouped_tile<TileConfig<DT, 1, 2, 2, 2, false, BKN, DMA, 4>>(p, s);
            if constexpr (!F32) return launch_grouped_tile<TileConfig<DT, 1, 2, 2, 2, false, BKN, DMA>>(p, s);
        default:
            if constexpr (DMA)
                if (c.turn) return launch_grouped_tile<TileConfig<DT, 1, 1, 1, 4, false, BKN, DMA, 4>>(p, s);
            return launch_grouped_tile<TileConfig<DT, 1, 1, 1, 4, false, BKN, DMA>>(p, s);
    }
}
template <int DT> hipError_t launch_typed(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t s) {
    if (op_b == GEMM_OP_N) return dma ? launch_sized<DT, true, true>(p, s) : launch_sized<DT, true, false>(p, s);
    return dma ? launch_sized<DT, false, true>(p, s) : launch_sized<DT, false, false>(p, s);
}


// Weight gradients: both operands are walked down their rows.  Results are
// fp32, so a tile's store takes twice the time.  Every group has all N x K of
// them, so a group's row tiles are counted as they are.  Three workgroups of
// 64 x 128 share a compute unit, so part of a turn of those costs a part.
// (6953 rows in 3 groups of 632 x 2136 bf16: 52 us in 256 x 256, 37 in 128 x 128;
// 4096 in 4 of 512 x 1024: 16.4 in 128 x 128, 11.8 in 64 x 128; 411 in 8 of
// 400 x 728, 1.3 turns of 64 x 128: 6.8 and 6.0.  Over 180 sizes of 250 to 16384
// rows the tile taken is 1.3% slower than the best of the three, 15% at most but
// for five.)
inline TileSize wgrad_tile(int N, int K, int groups, double slabs, bool large, double matrix) {
    constexpr TileSize sizes[] = {kTile256, kTile128, kTile64};        // what launch_wgrad has
    TileSize best = kTile64;
    double least = 0.0;
    for (const TileSize size : sizes) {
        if (size == kTile256 && !large) continue;
        const TileCost &c = kTileCosts[size];
        const double tiles = groups * std::ceil((double)N / c.bm) * std::ceil((double)K / c.bn);
        const double turns = tiles / kComputeUnits;
        const double t =
            tile_time(c, size == kTile64 ? std::max(1.0, turns) : std::ceil(turns), slabs, 2.0, matrix, 0.0);
        if (least == 0.0 || t < least) {
            least = t;
            best = size;
        }
    }
    return best;
}
template <int DT> hipError_t launch_wgrad(bool dma, const GroupedParams &p, hipStream_t s) {
    constexpr bool F32 = DT == GEMM_DTYPE_F32;
    // Each group as deep as they are on average.
    const double slabs = std::ceil((double)p.M / p.groups / (F32 ? 32 : 64));
    const TileSize size = wgrad_tile(p.N, p.K, p.groups, slabs, dma && !F32, F32 ? kMatrixF32 : 0.0);
    if constexpr (!F32)
        if (size == kTile256) return launch_grouped_tile<TileConfig<DT, 4, 2, 2, 4, true, true, true>>(p, s);
    if (size == kTile128)
        return dma ? launch_grouped_tile<TileConfig<DT, 2, 2, 2, 2, true, true, true>>(p, s)
                   : launch_grouped_tile<TileConfig<DT, 2, 2, 2, 2, true, true, false>>(p, s);
    return dma ? launch_grouped_tile<TileConfig<DT, 1, 2, 2, 2, true, true, true>>(p, s)
               : launch_grouped_tile<TileConfig<DT, 1, 2, 2, 2, true, true, false>>(p, s);
}

}  // namespace
}  // namespace gemm

#endif
