// Layer norm with the residual's addition, its backward pass, and the quantiser to 8-bit integers with a
// scale a row: passes over rows, bound by HBM.
//
// As in gemm_norm.hip a row is read once and kept in registers, 8 consecutive values (a chunk) a lane at a
// time: s = x + residual, mean(s), then the mean of (s - mean)^2 from the registers, which costs a second
// trip around the team but no memory and does not cancel as mean(s^2) - mean(s)^2 would where a row's mean
// is large beside its deviation.  y = (s - mean) * r * weight + bias.  Codes with a scale a row take a third
// trip, for the row's largest magnitude.  Rows past 16384 values are walked once for each of these, from the
// caches after the first.
//
// Measured (a copy reaches 5.2 TB/s here): 8192 x 4096 bf16 in training, 268 MB each way, forward 47 us (5.7 TB/s),
// backward 50 (5.3) and 5 for the last sum over partial rows; 8192 x 8192 bf16 with a residual to codes with a scale a
// row, 470 MB, 86 to 91 us (5.2 to 5.5), to fp8 97 (4.9); 5366 x 8176 fp32 135 and 150 us (5.2 and 4.7).  1000 x 777
// fp32: 6.7, 6.5 and 3.3 us: a launch each, the trips to memory of a row's operands, which wait for one another in
// the forward pass, and two around a wave.  Codes of 8192 x 4096 bf16 18 us (5.6 TB/s).
//
// Widths off 8 and between the powers of two are slower: lanes past a row's end idle, and a row's last chunk takes
// longer (gemm_rows.hpp).  8192 rows bf16, forward and backward with the last sum: 4500 columns (off 8) 121 and 118 us
// (2.4 and 2.5 TB/s), 6000 86 and 87 (4.6 and 4.5), 9000 129 and 162 (4.6 and 3.7); 5000 x 5000 48 and 58 (4.2 and
// 3.5), 5000 x 5001 68 and 78.
#include "gemm_norm.hpp"
#include "gemm_rows.hpp"

namespace gemm {
namespace {

// A chunk's codes with a scale a row out.
__device__ __forceinline__ void put_codes(const LayerNormParams &p, int64_t row, int64_t col, f32x8 y, int n,
                                          uint32_t top, float inv) {
    store_codes(static_cast<uint8_t *>(p.out) + row * p.ldo + col, row_codes8(y, top, inv), n);
}

// s - mean of a chunk, zero past the row's end.
__device__ __forceinline__ f32x8 centred(f32x8 s, float mean, int n) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) s[e] = e < n ? s[e] - mean : 0.0f;
    return s;
}
__device__ __forceinline__ float sum8(f32x8 v) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}
__device__ __forceinline__ float squares8(f32x8 v, float sq) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) sq = fmaf(v[e], v[e], sq);
    return sq;
}
__device__ __forceinline__ f32x8 unit_to_y(f32x8 c, float r, f32x8 w, f32x8 b) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) c[e] = fmaf(c[e] * r, w[e], b[e]);
    return c;
}

template <int DT, int THREADS, int PER, bool LARGE>
__global__ void __launch_bounds__(THREADS == 64 ? 256 : THREADS)
layer_norm_kernel(LayerNormParams p) {
    constexpr int TEAMS = THREADS == 64 ? 4 : 1;
    __shared__ float red[3 * (THREADS / 64)];
    const int64_t row = folded_block() * TEAMS + (TEAMS > 1 ? threadIdx.x / THREADS : 0);
    const int t = threadIdx.x % THREADS;
    if (row >= p.M) return;                    // the whole team together
    const int N = (int)p.N;
    f32x8 s[PER];
    typename Io<DT>::Raw w[PER], b[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        s[i] = norm_sum<DT>(p, row, col, N - col);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        w[i] = load_raw<DT>(p.weight, col, N - col);
        b[i] = {};
        if (p.bias != nullptr) b[i] = load_raw<DT>(p.bias, col, N - col);
    }
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        total += sum8(s[i]);
        const int col = kChunk * (t + i * THREADS);
        if (p.sum != nullptr) store8<DT, LARGE>(p.sum, row * p.ld_sum + col, s[i], N - col);
    }
    const float mean = team_sum<THREADS>(total, red, 0) / (float)N;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        s[i] = centred(s[i], mean, N - col);
        sq = squares8(s[i], sq);
    }
    const float r = 1.0f / sqrtf(team_sum<THREADS>(sq, red, 1) / (float)N + p.eps);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        s[i] = unit_to_y(s[i], r, Io<DT>::values(w[i]), Io<DT>::values(b[i]));
        if (p.out_type == GEMM_OUT_INT8) top = max(top, max_bits(s[i]));     // (zero past the row's end)
        else put_norm<LARGE>(p, row, col, s[i], N - col);
    }
    if (p.out_type != GEMM_OUT_INT8) return;
    top = team_max<THREADS>(top, red, 2);
    float scale;
    const float inv = int8_factor(top, scale);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        if (col < N) put_codes(p, row, col, s[i], N - col, top, inv);
    }
    if (t == 0) p.scales[row * p.ld_scales] = scale;
}

// Rows of any length: sixteen waves walk the row.
template <int DT>
__global__ void __launch_bounds__(1024)
layer_norm_long_kernel(LayerNormParams p) {
    __shared__ float red[3 * 16];
    const int64_t row = folded_block();
    if (row >= p.M) return;
    float total = 0.0f, sq = 0.0f;
    for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024)
        total += sum8(norm_sum<DT>(p, row, col, (int)min((int64_t)kChunk, p.N - col)));
    const float mean = team_sum<1024>(total, red, 0) / (float)p.N;
    for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024) {
        const int n = (int)min((int64_t)kChunk, p.N - col);
        sq = squares8(centred(norm_sum<DT>(p, row, col, n), mean, n), sq);
    }
    const float r = 1.0f / sqrtf(team_sum<1024>(sq, red, 1) / (float)p.N + p.eps);
    auto y_of = [&](f32x8 s, int64_t col, int n) __attribute__((always_inline)) {
        f32x8 b = {};
        if (p.bias != nullptr) b = load8<DT>(p.bias, col, n);
        return unit_to_y(centred(s, mean, n), r, load8<DT>(p.weight, col, n), b);
    };
    uint32_t top = 0;
    float scale = 0.0f, inv = 0.0f;
    if (p.out_type == GEMM_OUT_INT8) {
        for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024) {
            const int n = (int)min((int64_t)kChunk, p.N - col);
            top = max(top, max_bits(y_of(norm_sum<DT>(p, row, col, n), col, n)));
        }
        top = team_max<1024>(top, red, 2);
        inv = int8_factor(top, scale);
        if (threadIdx.x == 0) p.scales[row * p.ld_scales] = scale;
    }
    // Every lane runs every round: a block's maximum goes over 16 of them.
    for (int64_t c0 = 0; c0 < p.N; c0 += kChunk * 1024) {
        const int64_t col = c0 + kChunk * threadIdx.x;
        const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.N - col));
        f32x8 y = {};
        if (n > 0) {
            const f32x8 s = norm_sum<DT>(p, row, col, n);
            if (p.sum != nullptr) store8<DT>(p.sum, row * p.ld_sum + col, s, n);
            y = y_of(s, col, n);
            if (p.out_type == GEMM_OUT_INT8) put_codes(p, row, col, y, n, top, inv);
        }
        if (p.out_type != GEMM_OUT_INT8) put_norm(p, row, col, y, n);
    }
}

// Sums of two values over a team, in both: `red` holds two floats a wave for each of two sets.
template <int THREADS> __device__ __forceinline__ void team_sum2(float &a, float &b, float *red, int set) {
    a = sum64(a);
    b = sum64(b);
    if (THREADS == 64) return;
    constexpr int W = THREADS / 64;
    float *r = red + 2 * set * W;
    if ((threadIdx.x & 63) == 0) {
        r[2 * (threadIdx.x >> 6)] = a;
        r[2 * (threadIdx.x >> 6) + 1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        a += r[2 * w];
        b += r[2 * w + 1];
    }
}

// Backward pass.  With c = s - mean, r = (mean(c^2) + eps)^-1/2, n = c * r and g = dy * weight:
//     dx = r * (g - mean(g) - n * mean(g * n)) + ds      dweight = sum of dy * n      dbias = sum of dy
// A first trip around the team sums s and g, a second c^2 and g * c.  As in gemm_norm.hip a team takes rows
// team, team + teams, ... and keeps its columns' weights and both gradient sums in registers; they go to a
// row of `partials` each (N of dweight, then N of dbias), which layer_dweight_kernel adds.
template <int DT, int THREADS, int PER, bool LARGE>
__global__ void __launch_bounds__(THREADS == 64 ? 256 : THREADS)
layer_norm_backward_kernel(LayerNormGradParams p) {
    constexpr int TEAMS = THREADS == 64 ? 4 : 1;
    typedef typename Io<DT>::Raw Raw;
    __shared__ float red[4 * (THREADS / 64)];
    const int team = blockIdx.x * TEAMS + (TEAMS > 1 ? threadIdx.x / THREADS : 0), teams = gridDim.x * TEAMS;
    const int t = threadIdx.x % THREADS;
    const int N = (int)p.N;
    const float inv_n = 1.0f / (float)N;
    f32x8 w[PER], dw[PER], db[PER];
    Raw dy[PER], s[PER], ds[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        w[i] = load8<DT>(p.weight, col, N - col);
        dw[i] = db[i] = f32x8{};
        ds[i] = Raw{};
    }
    for (int64_t row = team; row < p.M; row += teams) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int col = kChunk * (t + i * THREADS);
            s[i] = load_raw<DT, LARGE>(p.s, row * p.lds + col, N - col);
            dy[i] = load_raw<DT, LARGE>(p.dy, row * p.lddy + col, N - col);
            if (p.ds != nullptr) ds[i] = load_raw<DT, LARGE>(p.ds, row * p.ldds + col, N - col);
        }
        float total = 0.0f, g_sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const f32x8 yv = Io<DT>::values(dy[i]);
            total += sum8(Io<DT>::values(s[i]));
#pragma unroll
            for (int e = 0; e < kChunk; ++e) g_sum = fmaf(yv[e], w[i][e], g_sum);
        }
        // A wave that is a trip ahead writes the other set, and it cannot be two ahead past the next barrier.
        team_sum2<THREADS>(total, g_sum, red, 0);
        const float mean = total * inv_n;
        float sq = 0.0f, gc = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const f32x8 c = centred(Io<DT>::values(s[i]), mean, N - kChunk * (t + i * THREADS));
            const f32x8 yv = Io<DT>::values(dy[i]);
            sq = squares8(c, sq);
#pragma unroll
            for (int e = 0; e < kChunk; ++e) gc = fmaf(yv[e] * w[i][e], c[e], gc);
        }
        team_sum2<THREADS>(sq, gc, red, 1);
        const float r = 1.0f / sqrtf(sq * inv_n + p.eps);
        const float g_mean = g_sum * inv_n, along = r * (gc * inv_n);      // of the size of g
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int col = kChunk * (t + i * THREADS);
            const f32x8 c = centred(Io<DT>::values(s[i]), mean, N - col);
            const f32x8 yv = Io<DT>::values(dy[i]), dv = Io<DT>::values(ds[i]);
            f32x8 dx;
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                const float n = c[e] * r;
                dx[e] = fmaf(r, fmaf(-along, n, fmaf(yv[e], w[i][e], -g_mean)), dv[e]);
                dw[i][e] = fmaf(yv[e], n, dw[i][e]);
                db[i][e] += yv[e];
            }
            store8<DT, LARGE>(p.dx, row * p.lddx + col, dx, N - col);
        }
    }
    if (p.partials == nullptr) return;
    if constexpr (TEAMS > 1) {
        // One partial row a workgroup: its teams' sums are added through LDS, in order.
        __shared__ __attribute__((aligned(16))) float sums[TEAMS][2][PER * THREADS * kChunk];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            *reinterpret_cast<f32x8 *>(&sums[threadIdx.x / THREADS][0][kChunk * (t + i * THREADS)]) = dw[i];
            *reinterpret_cast<f32x8 *>(&sums[threadIdx.x / THREADS][1][kChunk * (t + i * THREADS)]) = db[i];
        }
        __syncthreads();
        for (int at = threadIdx.x; at < 2 * N; at += TEAMS * THREADS) {
            const int of = at >= N, col = at - of * N;
            double v = 0.0;
#pragma unroll
            for (int i = 0; i < TEAMS; ++i) v += sums[i][of][col];
            p.partials[(int64_t)blockIdx.x * 2 * N + at] = (float)v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int col = kChunk * (t + i * THREADS);
            store8<GEMM_DTYPE_F32>(p.partials, (int64_t)team * 2 * N + col, dw[i], N - col);
            store8<GEMM_DTYPE_F32>(p.partials, ((int64_t)team * 2 + 1) * N + col, db[i], N - col);
        }
    }
}

// Rows past 16384 values: the sums first, then the row again from the caches.  The gradients' running sums
// live in `partials`.
template <int DT>
__global__ void __launch_bounds__(1024)
layer_norm_backward_long_kernel(LayerNormGradParams p) {
    __shared__ float red[4 * 16];
    const int team = blockIdx.x, teams = gridDim.x;
    const float inv_n = 1.0f / (float)p.N;
    for (int64_t row = team; row < p.M; row += teams) {
        float total = 0.0f, g_sum = 0.0f;
        for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024) {
            const int n = (int)min((int64_t)kChunk, p.N - col);
            const f32x8 yv = load8<DT>(p.dy, row * p.lddy + col, n), w = load8<DT>(p.weight, col, n);
            total += sum8(load8<DT>(p.s, row * p.lds + col, n));
#pragma unroll
            for (int e = 0; e < kChunk; ++e) g_sum = fmaf(yv[e], w[e], g_sum);
        }
        team_sum2<1024>(total, g_sum, red, 0);
        const float mean = total * inv_n;
        float sq = 0.0f, gc = 0.0f;
        for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024) {
            const int n = (int)min((int64_t)kChunk, p.N - col);
            const f32x8 c = centred(load8<DT>(p.s, row * p.lds + col, n), mean, n);
            const f32x8 yv = load8<DT>(p.dy, row * p.lddy + col, n), w = load8<DT>(p.weight, col, n);
            sq = squares8(c, sq);
#pragma unroll
            for (int e = 0; e < kChunk; ++e) gc = fmaf(yv[e] * w[e], c[e], gc);
        }
        team_sum2<1024>(sq, gc, red, 1);
        const float r = 1.0f / sqrtf(sq * inv_n + p.eps);
        const float g_mean = g_sum * inv_n, along = r * (gc * inv_n);
        for (int64_t col = kChunk * threadIdx.x; col < p.N; col += kChunk * 1024) {
            const int n = (int)min((int64_t)kChunk, p.N - col);
            const f32x8 c = centred(load8<DT>(p.s, row * p.lds + col, n), mean, n);
            const f32x8 yv = load8<DT>(p.dy, row * p.lddy + col, n), w = load8<DT>(p.weight, col, n);
            f32x8 dv = {}, dx, unit;
            if (p.ds != nullptr) dv = load8<DT>(p.ds, row * p.ldds + col, n);
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                unit[e] = c[e] * r;
                dx[e] = fmaf(r, fmaf(-along, unit[e], fmaf(yv[e], w[e], -g_mean)), dv[e]);
            }
            if (p.partials != nullptr) {
                const int64_t of_w = (int64_t)team * 2 * p.N + col, of_b = of_w + p.N;
                f32x8 dw = {}, db = {};
                if (row != team) {
                    dw = load8<GEMM_DTYPE_F32>(p.partials, of_w, n);
                    db = load8<GEMM_DTYPE_F32>(p.partials, of_b, n);
                }
#pragma unroll
                for (int e = 0; e < kChunk; ++e) {
                    dw[e] = fmaf(yv[e], unit[e], dw[e]);
                    db[e] += yv[e];
                }
                store8<GEMM_DTYPE_F32>(p.partials, of_w, dw, n);
                store8<GEMM_DTYPE_F32>(p.partials, of_b, db, n);
            }
            store8<DT>(p.dx, row * p.lddx + col, dx, n);
        }
    }
}

// dweight and dbias: sums of `parts` partial rows of 2 * N in a fixed order.  32 columns a workgroup, 32
// threads a column each adding every 32nd row, eight rows in flight, then the threads' sums in turn.  These
// sums and those of a workgroup's teams above are in 64 bits, for 0.1 to 0.2 us: fp32 rounds the sum over a
// team's own rows (a single one, up to 2048 rows of at most 2048 columns or 512 wider ones) and each partial
// sum.  1000 x 777 fp32: dweight and dbias off by 7e-8 and 4e-8 of their norms, in fp32 alone 1.4e-7 and 1.2e-7.
__global__ void __launch_bounds__(1024)
layer_dweight_kernel(const float *partials, float *dweight, float *dbias, int parts, int64_t N) {
    __shared__ double part[32][32];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t at = folded_block() * 32 + c;
    double s[8] = {};
    if (at < 2 * N)
        for (int i = g; i < parts; i += 256) {
            float v[8];            // (rows past the last one: that again, so that no load waits for a branch)
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = partials[(int64_t)min(i + 32 * u, parts - 1) * 2 * N + at];
#pragma unroll
            for (int u = 0; u < 8; ++u) s[u] += i + 32 * u < parts ? v[u] : 0.0f;
        }
    part[g][c] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    if (g == 0 && at < 2 * N) {
        double t = 0.0;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += part[i][c];
        float *to = at < N ? dweight : dbias;
        if (to != nullptr) to[at < N ? at : at - N] = (float)t;
    }
}

// Codes of rows with a scale each.
template <int DT, int THREADS, int PER>
__global__ void __launch_bounds__(THREADS == 64 ? 256 : THREADS)
quantize_int8_kernel(Int8Params p) {
    constexpr int TEAMS = THREADS == 64 ? 4 : 1;
    __shared__ float red[THREADS / 64];
    const int64_t row = folded_block() * TEAMS + (TEAMS > 1 ? threadIdx.x / THREADS : 0);
    const int t = threadIdx.x % THREADS;
    if (row >= p.M) return;                    // the whole team together
    const int K = (int)p.K;
    f32x8 v[PER];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        v[i] = load8<DT>(p.x, row * p.ldx + col, K - col);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) top = max(top, max_bits(v[i]));
    top = team_max<THREADS>(top, red, 0);
    float scale;
    const float inv = int8_factor(top, scale);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = kChunk * (t + i * THREADS);
        if (col < K) store_codes(p.q + row * p.ldq + col, row_codes8(v[i], top, inv), K - col);
    }
    if (t == 0) p.scales[row] = scale;
}
template <int DT>
__global__ void __launch_bounds__(1024)
quantize_int8_long_kernel(Int8Params p) {
    __shared__ float red[16];
    const int64_t row = folded_block();
    if (row >= p.M) return;
    uint32_t top = 0;
    for (int64_t col = kChunk * threadIdx.x; col < p.K; col += kChunk * 1024)
        top = max(top, max_bits(load8<DT>(p.x, row * p.ldx + col, (int)min((int64_t)kChunk, p.K - col))));
    top = team_max<1024>(top, red, 0);
    float scale;
    const float inv = int8_factor(top, scale);
    for (int64_t col = kChunk * threadIdx.x; col < p.K; col += kChunk * 1024) {
        const int n = (int)min((int64_t)kChunk, p.K - col);
        store_codes(p.q + row * p.ldq + col, row_codes8(load8<DT>(p.x, row * p.ldx + col, n), top, inv), n);
    }
    if (threadIdx.x == 0) p.scales[row] = scale;
}

// A chunk a lane keeps the most rows' loads under way.  8192 rows in 512 threads and one chunk, and in 256 and
// two: 4096 bf16 50 us and 53; in 1024 and one, and 512 and two: 8192 bf16 92 and 97, but 94 and 86 to codes with
// a scale a row, which take another trip around the team.
template <int DT, bool LARGE> hipError_t norm_type(const LayerNormParams &p, hipStream_t s) {
    if (p.N <= 1024) return go(&layer_norm_kernel<DT, 64, 2, LARGE>, fold((p.M + 3) / 4), 256, s, p);
    if (p.N <= 2048) return go(&layer_norm_kernel<DT, 256, 1, LARGE>, fold(p.M), 256, s, p);
    if (p.N <= 4096) return go(&layer_norm_kernel<DT, 512, 1, LARGE>, fold(p.M), 512, s, p);
    if (p.N <= 8192 && p.out_type == GEMM_OUT_INT8) return go(&layer_norm_kernel<DT, 512, 2, LARGE>, fold(p.M), 512, s, p);
    if (p.N <= 8192) return go(&layer_norm_kernel<DT, 1024, 1, LARGE>, fold(p.M), 1024, s, p);
    if (p.N <= 16384) return go(&layer_norm_kernel<DT, 1024, 2, LARGE>, fold(p.M), 1024, s, p);
    return go(&layer_norm_long_kernel<DT>, fold(p.M), 1024, s, p);
}

// Workgroups of the backward pass: enough to fill the compute units.  Their partial sums, 16 bytes a column and
// workgroup written and read again, are a small part of what is moved from some 4000 rows on.  Of fewer they are
// more: twice the operator's own bytes for bf16 up to 512 rows of more than 2048 columns (512 x 8192: 67 MB
// beside 34, 23 us; 1024 x 8192 27, 2048 x 8192 39).
int grad_workgroups(int64_t M, int64_t N) {
    const int64_t rows = N <= 2048 ? (M + 3) / 4 : M;        // rows a workgroup takes at once: 4, or 1
    return (int)(rows < 512 ? rows : 512);
}

// Here more chunks a lane pay, as a row's two trips around the team cost more than its loads.  8192 rows bf16 of 2048
// in 64 threads and four chunks 28 us, in 256 and two 40; of 8192 in 256 and four 96, in 512 and two 101, in 1024 and
// one 115; 5366 x 8176 fp32 150, 154 and 164.
template <int DT, bool LARGE> hipError_t grad_type(const LayerNormGradParams &p, hipStream_t s) {
    const dim3 grid((unsigned)grad_workgroups(p.M, p.N));
    if (p.N <= 1024) return go(&layer_norm_backward_kernel<DT, 64, 2, LARGE>, grid, 256, s, p);
    if (p.N <= 2048) return go(&layer_norm_backward_kernel<DT, 64, 4, LARGE>, grid, 256, s, p);
    if (p.N <= 4096) return go(&layer_norm_backward_kernel<DT, 256, 2, LARGE>, grid, 256, s, p);
    if (p.N <= 8192) return go(&layer_norm_backward_kernel<DT, 256, 4, LARGE>, grid, 256, s, p);
    if (p.N <= 16384) return go(&layer_norm_backward_kernel<DT, 512, 4, LARGE>, grid, 512, s, p);
    return go(&layer_norm_backward_long_kernel<DT>, grid, 1024, s, p);
}

template <int DT> hipError_t quantize_type(const Int8Params &p, hipStream_t s) {
    switch (shape_of(p.K)) {
        case kWave2: return go(&quantize_int8_kernel<DT, 64, 2>, fold((p.M + 3) / 4), 256, s, p);
        case kFour2: return go(&quantize_int8_kernel<DT, 256, 2>, fold(p.M), 256, s, p);
        case kSixteen1: return go(&quantize_int8_kernel<DT, 1024, 1>, fold(p.M), 1024, s, p);
        case kSixteen2: return go(&quantize_int8_kernel<DT, 1024, 2>, fold(p.M), 1024, s, p);
        default: return go(&quantize_int8_long_kernel<DT>, fold(p.M), 1024, s, p);
    }
}

}  // namespace

int layer_norm_grad_partials(int64_t M, int64_t N) {
    if (M <= 0 || N <= 0) return 0;
    return grad_workgroups(M, N);
}

// A pass whose operands of this many bytes each cannot stay in the L2s accesses them non-temporally.  Without and with,
// 4096 columns bf16, inputs in turn: 64 MB forward 49 us and 48, backward 55 and 49; 32 MB 28 and 23, 32 and 29; 16 MB
// 14.7 and 13.4, 16.7 and 17.9.
static bool large(int64_t M, int64_t N, int32_t dtype) { return (double)M * N * (dtype == GEMM_DTYPE_F32 ? 4 : 2) >= 32 << 20; }

hipError_t launch_layer_norm(const LayerNormParams &p, hipStream_t s) {
    if (large(p.M, p.N, p.dtype))
        return p.dtype == GEMM_DTYPE_F32 ? norm_type<GEMM_DTYPE_F32, true>(p, s)
                                         : norm_type<GEMM_DTYPE_BF16F32, true>(p, s);
    return p.dtype == GEMM_DTYPE_F32 ? norm_type<GEMM_DTYPE_F32, false>(p, s)
                                     : norm_type<GEMM_DTYPE_BF16F32, false>(p, s);
}

hipError_t launch_layer_norm_backward(const LayerNormGradParams &p, hipStream_t s) {
    const bool sums = p.dweight != nullptr || p.dbias != nullptr;
    hipError_t err = hipSuccess;
    if (p.M > 0) {
        if (large(p.M, p.N, p.dtype))
            err = p.dtype == GEMM_DTYPE_F32 ? grad_type<GEMM_DTYPE_F32, true>(p, s)
                                            : grad_type<GEMM_DTYPE_BF16F32, true>(p, s);
        else
            err = p.dtype == GEMM_DTYPE_F32 ? grad_type<GEMM_DTYPE_F32, false>(p, s)
                                            : grad_type<GEMM_DTYPE_BF16F32, false>(p, s);
    }
    if (err != hipSuccess || !sums) return err;
    return go(&layer_dweight_kernel, fold((2 * p.N + 31) / 32), 1024, s, (const float *)p.partials, p.dweight, p.dbias,
              layer_norm_grad_partials(p.M, p.N), p.N);
}

hipError_t launch_quantize_int8(const Int8Params &p, hipStream_t s) {
    return p.dtype == GEMM_DTYPE_F32 ? quantize_type<GEMM_DTYPE_F32>(p, s) : quantize_type<GEMM_DTYPE_BF16F32>(p, s);
}

}  // namespace gemm
