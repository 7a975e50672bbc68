// Shared by the grouped and block-scaled products (gemm_grouped, gemm_block_scaled,
// gemm_grouped_wgrad): their arguments, and the map from a workgroup to a tile
// of a group.
//
// The rows of A are sorted by group and only the device knows where groups
// end.  A launch therefore covers the most row tiles that any division of M
// rows can need, and each workgroup finds its tile itself: every wave reads
// the ends 64 at a time, turns them into tile counts, and scans those across
// its lanes.  Workgroups past the real count leave at once.
#pragma once

#include "gemm_device.hpp"

namespace gemm {

// One launch, already validated (gemm_experts_api.cpp): sizes below 2^31,
// pointers aligned to their elements.
struct GroupedParams {
    const void *A;
    const void *B;
    void *out;
    const int32_t *ends;       // null: one group of all M rows
    int32_t M, N, K, groups;
    int64_t lda, ldb, stride_b, ldo;
    int64_t stride_out;        // weight gradients: elements between groups' results
    float alpha, beta;         // beta: weight gradients only
    int32_t out_type;          // GEMM_OUT_F32 or GEMM_OUT_BF16
    gemm_block_scales sc;      // fp8 only
    bool by_size;              // weight gradients of at most 64 groups: in the order of their rows
};

// Most row tiles of `tile_m` rows that M rows in `groups` groups can make,
// the rows past the last end counted as one group more: each of c groups
// that have rows adds at most one tile to the M / tile_m whole ones.
inline int64_t most_row_tiles(int64_t M, int64_t groups, int64_t tile_m, bool grouped) {
    if (!grouped) return (M + tile_m - 1) / tile_m;
    const int64_t c = groups + 1 < M ? groups + 1 : M;
    return c + (M - c) / tile_m;
}

// Operands walked down k that come through registers: the last offset, from a slab's first row on,
// that one of its 16-byte loads may start at.  left: rows from there to the panel's end (1 at least);
// step, wide: bytes between rows and of one.  The panel's end bounds its last slab; every other slab is
// bounded by the row after its own bk, which a load that starts inside it reaches at most, so that the
// offset stays in 32 bits however deep the panel is.
constexpr int slab_limit(int left, int bk, int step, int wide) {
    return (left <= bk ? left - 1 : bk) * step + wide - 16;
}

// Slabs of bk that len takes, the first row of slab t (of one past the end: the last row), and the rows
// from slab t's first one on (zero or less past the end), of len up to 2^31 - 1 and a few slabs more.
constexpr int slabs_of(int len, int bk) { return (int)(((int64_t)len + bk - 1) / bk); }
constexpr int slab_first(int t, int bk, int len) {
    return (int)((uint32_t)t * (uint32_t)bk < (uint32_t)len ? (uint32_t)t * (uint32_t)bk : (uint32_t)len - 1);
}
constexpr int slab_left(int t, int bk, int len) { return (int)((uint32_t)len - (uint32_t)t * (uint32_t)bk); }

#if defined(__HIPCC__)

// A tile's rows: `rows` of them from row0; group is -1 for the rows past the
// last end, which are zeroed; rows <= 0: nothing to do.  tn: tile column.
// parts: 1, or 2 or 4 where the tile is shared out, of which this is `part`.
struct GroupTile {
    int group, row0, rows, tn, part, parts;
};

// Workgroups of tiles that come after the last whole turn of the compute
// units: each tile goes to two of them, or to four, where all are then in one
// turn.  wg becomes the tile's number.
constexpr int kShareTurn = 256;
__device__ __forceinline__ void share_out(int64_t tiles, int &wg, GroupTile &t) {
    const int left = (int)(tiles % kShareTurn);
    const int64_t past = wg - (tiles - left);
    t.parts = left <= kShareTurn / 4 ? 4 : left <= kShareTurn / 2 ? 2 : 1;
    if (past < 0) t.parts = 1;
    t.part = past < 0 ? 0 : (int)past % t.parts;
    if (past >= 0) wg = (int)(tiles - left + past / t.parts);
}

// Inclusive scans over the 64 lanes.
__device__ __forceinline__ int wave_scan_max(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v = max(v, o);
    }
    return v;
}
__device__ __forceinline__ int wave_scan_add(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// First row and past-the-last row of group `lane + 64 * chunk` (the group
// after the last one: the rows past every end), from the ends clamped to
// their running maximum and to M.  `carry` is the running maximum of the
// chunks before and is moved on.
__device__ __forceinline__ void group_bounds(const GroupedParams &p, int chunk, int lane, int &carry, int &lo,
                                             int &hi) {
    const int g = 64 * chunk + lane;
    int e = g < p.groups ? min(max(p.ends[g], 0), p.M) : g == p.groups ? p.M : 0;
    e = max(wave_scan_max(e, lane), carry);
    const int before = __shfl_up(e, 1);
    lo = lane == 0 ? carry : before;
    hi = e;
    carry = __shfl(e, 63);
}

// The tile of workgroup `wg`, for tiles of tile_m rows and tiles_n columns of
// tiles.  Tiles are walked in the order of tile_coords over the real number
// of row tiles, so the dead workgroups of the launch are its last ones.
template <bool SHARE = false>
__device__ __forceinline__ GroupTile find_tile(const GroupedParams &p, int wg, int tile_m, int tiles_n, int group_m) {
    GroupTile t;
    t.part = 0;
    t.parts = 1;
    if (p.ends == nullptr) {
        int tm;
        const int tiles_m = (p.M + tile_m - 1) / tile_m;
        t.group = t.row0 = t.rows = t.tn = 0;
        if (SHARE) {
            share_out((int64_t)tiles_m * tiles_n, wg, t);
            if (wg >= (int64_t)tiles_m * tiles_n) return t;
        }
        tile_coords(wg, tiles_m, tiles_n, group_m, tm, t.tn);
        t.group = 0;
        t.row0 = tm * tile_m;
        t.rows = min(tile_m, p.M - t.row0);
        return t;
    }
    const int lane = threadIdx.x & 63;
    const int chunks = p.groups / 64 + 1;
    int carry = 0, total = 0, lo, hi, upto = 0, mine = 0;
    for (int c = 0; c < chunks; ++c) {
        group_bounds(p, c, lane, carry, lo, hi);
        mine = (hi - lo + tile_m - 1) / tile_m;
        upto = wave_scan_add(mine, lane) + total;
        total = __builtin_amdgcn_readlane(upto, 63);      // scalar, so that no lane seems to differ
    }
    t.group = 0;
    t.row0 = t.rows = t.tn = 0;
    if (SHARE) share_out((int64_t)total * tiles_n, wg, t);
    if ((int64_t)wg >= (int64_t)total * tiles_n) return t;
    int tm;
    tile_coords(wg, total, tiles_n, group_m, tm, t.tn);
    int last = chunks - 1;
    if (chunks > 1) {         // find the chunk of 64 groups again that holds tile tm
        carry = 0;
        total = 0;
        for (last = 0; last < chunks; ++last) {
            group_bounds(p, last, lane, carry, lo, hi);
            mine = (hi - lo + tile_m - 1) / tile_m;
            upto = wave_scan_add(mine, lane) + total;
            total = __builtin_amdgcn_readlane(upto, 63);
            if (tm < total) break;
        }
    }
    const int src = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(upto > tm)) - 1);
    const int first = __shfl(upto - mine, src), row = __shfl(lo, src), end = __shfl(hi, src);
    const int g = 64 * last + src;
    t.group = g < p.groups ? g : -1;
    t.row0 = row + (tm - first) * tile_m;
    t.rows = min(tile_m, end - t.row0);
    return t;
}

// Rows [lo, hi) of the group that takes turn `turn` (weight gradients: one group a workgroup), and
// that group.  by_size: those with the most rows go first, so that what is left for the launch's end
// is short, a tile's time being its group's rows.
__device__ __forceinline__ int find_group(const GroupedParams &p, int turn, int &lo, int &hi) {
    const int lane = threadIdx.x & 63;
    int carry = 0, g = turn;
    if (p.by_size) {
        group_bounds(p, 0, lane, carry, lo, hi);
        const int rows = lane < p.groups ? hi - lo : -1;
        int before = 0;                                    // groups that go before this lane's
        for (int i = 0; i < p.groups; ++i) {
            const int other = __builtin_amdgcn_readlane(rows, i);
            before += other > rows || (other == rows && i < lane);
        }
        g = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(before == turn)) - 1);
    } else {
        for (int c = 0;; ++c) {
            group_bounds(p, c, lane, carry, lo, hi);
            if (g < 64 * (c + 1)) break;
        }
    }
    lo = __builtin_amdgcn_readfirstlane(__shfl(lo, g & 63));
    hi = __builtin_amdgcn_readfirstlane(__shfl(hi, g & 63));
    return g;
}

#endif  // __HIPCC__

// Launchers.  The general ones run every type, layout and alignment; the
// others the tiles of gemm_grouped_tile.hpp.  dma: rows of both operands
// start on 16 bytes.
hipError_t launch_grouped_fp8(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream);
hipError_t launch_grouped_bf16(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream);
hipError_t launch_grouped_f32(int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream);
// Few rows (on average 64 a group at most) and weights stored N x K, rows on
// 16 bytes: the rows of the tile that suits, or 0 for calls that are not its.
int skinny_rows(int32_t dtype, int32_t op_b, const GroupedParams &p);
hipError_t launch_grouped_skinny(int32_t dtype, int rows, const GroupedParams &p, hipStream_t stream);
// Few output tiles: whether the kernel whose waves share out k can run the call, and that kernel.
constexpr int deep_columns(int32_t dtype, bool kn) {         // of its tiles of 32 rows
    return !kn || dtype == GEMM_DTYPE_F32 ? 32 : dtype == GEMM_DTYPE_BF16F32 ? 64 : 128;
}
bool deep_takes(int32_t dtype, int32_t op_b, bool dma, const GroupedParams &p);
hipError_t launch_grouped_deep(int32_t dtype, int32_t op_b, bool dma, const GroupedParams &p, hipStream_t stream);
hipError_t launch_wgrad_bf16(bool dma, const GroupedParams &p, hipStream_t stream);
hipError_t launch_wgrad_f32(bool dma, const GroupedParams &p, hipStream_t stream);
hipError_t launch_grouped_general(int32_t dtype, int32_t op_b, const GroupedParams &p, hipStream_t stream);
hipError_t launch_wgrad_general(int32_t dtype, const GroupedParams &p, hipStream_t stream);

}  // namespace gemm
