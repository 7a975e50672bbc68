// Tokens sorted by expert and back: the plan (a stable counting sort of the router's choices), the rows
// handed out to the experts, their results put together with the choices' weights, and the gradients.
//
// The plan is bound by latency: a few bytes a choice.  A workgroup counts its choices by expert in LDS, a
// table a wave; the tables' prefixes over waves (and over workgroups) and the experts' starts then give
// every wave the next row of each expert, and it walks its choices again, 64 at a time, each lane's rank
// among those of its expert being the set bits below its own in the lanes that share it.  Nothing depends
// on the order that waves run in.
//
// The others are passes over rows, bound by HBM.  All go by token, not by row: a token's row is read once
// and written to each of its experts' rows, or its experts' rows are read and it is written once, so that
// no sum needs an atomic and none is made in an order that could change.
//
// Measured (a copy reaches 5.2 TB/s here): 8192 tokens x 4096 bf16, top 2: handed out 34 to 39 us (201 MB, 5.1 to 5.9
// TB/s), together again with a residual 44 (268 MB, 6.1), gradients 60 (335 MB, 5.6), the plan 10 in two launches.
// 8192 x 2048 bf16, top 8 with half of the choices here: 59 and 33 us (302 and 201 MB).  16 tokens x 4096, top 4: 3.2,
// 4 and 3.4 us for the plan, out and together, a launch and two trips to memory each.
#include <algorithm>

#include "gemm_route.hpp"
#include "gemm_rows.hpp"

namespace gemm {
namespace {

// ---------------------------------------------------------------- the plan

// Expert of choice i, or -1 for numbers that are no group's.
__device__ __forceinline__ int expert_of(const PlanParams &p, int i) {
    const int64_t at = p.ld == p.top ? (int64_t)i : (int64_t)(i / p.top) * p.ld + i % p.top;
    if (p.wide) {
        const int64_t e = static_cast<const int64_t *>(p.experts)[at];
        return e >= 0 && e < p.groups ? (int)e : -1;
    }
    const int e = static_cast<const int32_t *>(p.experts)[at];
    return e >= 0 && e < p.groups ? e : -1;
}

// Choices of each workgroup by expert.
__global__ void __launch_bounds__(1024)
plan_count_kernel(PlanParams p) {
    extern __shared__ __attribute__((aligned(16))) int lds[];
    for (int e = threadIdx.x; e < p.groups; e += blockDim.x) lds[e] = 0;
    __syncthreads();
    const int first = blockIdx.x * p.per, past = min(p.choices - first, p.per);
    for (int i = threadIdx.x; i < past; i += blockDim.x) {
        const int e = expert_of(p, first + i);
        if (e >= 0) atomicAdd(&lds[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.groups; e += blockDim.x) p.counts[(int64_t)blockIdx.x * p.groups + e] = lds[e];
}

// Lanes that hold the same value as this one, of 0 .. 2^bits - 1.
__device__ __forceinline__ uint64_t same_lanes(int v, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((v >> b) & 1);
        m &= (v >> b) & 1 ? set : ~set;
    }
    return m;
}

// `waves`: those that have a table of counts, and choices; with more workgroups than one, the others help to
// add up their counts.
__global__ void __launch_bounds__(1024)
plan_place_kernel(PlanParams p, int bits, int waves) {
    extern __shared__ __attribute__((aligned(16))) int lds[];
    __shared__ int used;
    const int E = p.groups, tid = threadIdx.x, threads = blockDim.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    volatile int *count = lds;                 // [waves][E]: choices, then the next row of each expert
    volatile int *start = lds + waves * E;     // [E]
    int *before = lds + (waves + 1) * E;       // [E]: choices of the workgroups before (more than one only)
    const int tables = (p.blocks > 1 ? waves + 2 : waves + 1) * E;
    for (int i = tid; i < tables; i += threads) count[i] = 0;
    __syncthreads();
    if (p.blocks > 1) {
        // Threads share out an expert's column of the counts where there are fewer experts than threads.
        const int wide = bits < 10 ? 1 << bits : 1024, part = tid / wide, parts = threads / wide;
        for (int e = tid & (wide - 1); e < E; e += wide) {
            int all = 0, run = 0;
#pragma unroll 8
            for (int b = part; b < p.blocks; b += parts) {
                const int c = p.counts[(int64_t)b * E + e];
                all += c;
                run += b < (int)blockIdx.x ? c : 0;
            }
            atomicAdd(&lds[waves * E + e], all);
            atomicAdd(&before[e], run);
        }
    }

    const int first = blockIdx.x * p.per, mine = max(0, min(p.choices - first, p.per));
    const int each = ((mine + waves - 1) / waves + 63) / 64 * 64;
    const int lo = first + min(mine, wave * each), hi = wave < waves ? first + min(mine, (wave + 1) * each) : lo;
    for (int i = lo + lane; i < hi; i += 64) {
        const int e = expert_of(p, i);
        if (e >= 0) atomicAdd(&lds[wave * E + e], 1);
    }
    __syncthreads();

    // A wave's first row of an expert, counted from the expert's start: the choices of the workgroups and
    // of the waves before.
    for (int e = tid; e < E; e += threads) {
        int run = p.blocks > 1 ? before[e] : 0;
        for (int w = 0; w < waves; ++w) {
            const int c = count[w * E + e];
            count[w * E + e] = run;
            run += c;
        }
        if (p.blocks == 1) start[e] = run;
    }
    __syncthreads();
    if (wave == 0) {
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane, c = e < E ? start[e] : 0;
            int upto = c;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(upto, d);
                if (lane >= d) upto += o;
            }
            upto += carry;
            if (e < E) {
                start[e] = upto - c;
                if (blockIdx.x == 0) p.ends[e] = upto;
            }
            carry = __shfl(upto, 63);
        }
        if (lane == 0) used = carry;
    }
    __syncthreads();

    for (int i0 = lo; i0 < hi; i0 += 64) {
        const int i = i0 + lane;
        const int e = i < hi ? expert_of(p, i) : -1;
        const uint64_t same = same_lanes(e < 0 ? E : e, bits);
        if (e >= 0) {
            const uint64_t before = same & ((1ull << lane) - 1);
            const int next = count[wave * E + e], row = start[e] + next + __popcll(before);
            if (before == 0) count[wave * E + e] = next + __popcll(same);
            p.place[i] = row;
            if (p.order != nullptr) p.order[row] = i;
        } else if (i < hi) {
            p.place[i] = -1;
        }
    }
    if (p.order != nullptr)
        for (int64_t r = used + (int64_t)blockIdx.x * threads + tid; r < p.choices; r += (int64_t)p.blocks * threads)
            p.order[r] = -1;
}

// ---------------------------------------------------------------- rows

// First row past the groups' (all of them, if the caller does not say).
__device__ __forceinline__ int64_t rows_used(const int32_t *last, int64_t rows) {
    return last == nullptr ? rows : min(max((int64_t)*last, (int64_t)0), rows);
}
// Token and slab of unit u.  32-bit division where it will do: the 64-bit one is some hundred instructions.
__device__ __forceinline__ void split_unit(int64_t u, int slabs, int64_t &token, int &slab) {
    token = u >> 32 == 0 ? (int64_t)((uint32_t)u / (uint32_t)slabs) : u / slabs;
    slab = (int)(u - token * slabs);
}
__device__ __forceinline__ int64_t wave_unit(int64_t first) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return first * 4 + wave;
}

// A wave holds 1024 * U bytes of a token's row and stores them to each of its rows.  A row's last 16 bytes
// end where it does, over what the 16 before hold: the bytes in both are the same.  `teams`: tokens, or as
// many waves as clear the rows past the last group's where there are none.
template <int U, bool LARGE>
__global__ void __launch_bounds__(256)
dispatch_kernel(DispatchParams p, int64_t teams, int slabs) {
    const int64_t u = wave_unit(folded_block());
    if (u >= teams * slabs) return;
    int64_t token;
    int slab;
    split_unit(u, slabs, token, slab);
    const int lane = threadIdx.x & 63;
    const int64_t used = rows_used(p.last, p.rows);
    const int64_t first = (int64_t)slab * 1024 * U;
    u32x4 v[U];
    auto put_row = [&](int64_t row) __attribute__((always_inline)) {
        char *to = p.out + row * p.ldo;
        if (p.wide >= 16) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t at = first + 1024 * i + 16 * lane;
                if (at >= p.wide) continue;
                if (LARGE) put_nt(to + min(at, p.wide - 16), v[i]);
                else put(to + min(at, p.wide - 16), v[i]);
            }
        } else if (lane < p.wide) {
            to[lane] = (char)v[0][0];
        }
    };
    if (token < p.tokens) {
        const char *from = p.x + token * p.ldx;
        if (p.wide >= 16) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t at = first + 1024 * i + 16 * lane;
                if (at < p.wide) v[i] = get<u32x4>(from + min(at, p.wide - 16));
            }
        } else if (lane < p.wide) {
            v[0][0] = (uint32_t)(uint8_t)from[lane];
        }
        for (int k = 0; k < p.top; ++k) {
            const int row = p.place[token * p.top + k];
            if (row < 0 || row >= used) continue;
            put_row(row);
            if (slab == 0)
                for (int c = lane; c < p.scale_cols; c += 64)
                    p.out_scales[row * p.ldos + c] = p.scales[token * p.lds + c];
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) v[i] = u32x4{};
    for (int64_t row = used + token; row < p.rows; row += teams) {
        put_row(row);
        if (slab == 0)
            for (int c = lane; c < p.scale_cols; c += 64) p.out_scales[row * p.ldos + c] = 0.0f;
    }
}

// A wave makes 512 values of a token: the residual's, then each choice's in turn times its weight, in fp32.
// Its lanes read the places and weights of up to 64 choices at once; of those that have a row, four rows'
// loads are under way at a time, but in a row's last wave, if N is no multiple of 512: there a chunk that the
// row ends in or before waits at each load (8192 tokens, top 2, bf16: 43 us at 4096 columns, 70 at 4095).
template <int DT, bool LARGE>
__global__ void __launch_bounds__(256)
combine_kernel(CombineParams p, int slabs) {
    typedef typename Io<DT>::Raw Raw;
    const int64_t u = wave_unit(folded_block());
    if (u >= p.tokens * slabs) return;
    int64_t token;
    int slab;
    split_unit(u, slabs, token, slab);
    const int lane = threadIdx.x & 63;
    const int64_t col = (int64_t)slab * 512 + kChunk * lane;
    const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.N - col));
    f32x8 acc = {};
    if (p.residual != nullptr) acc = load8<DT>(p.residual, token * p.ld_res + col, n);
    for (int k0 = 0; k0 < p.top; k0 += 64) {
        int place = -1;
        float share = 1.0f;
        if (k0 + lane < p.top) {
            place = p.place[token * p.top + k0 + lane];
            if (p.weights != nullptr) share = p.weights[token * p.ldw + k0 + lane];
        }
        uint64_t left = __ballot(place >= 0 && place < p.n_rows);
        while (left != 0) {
            Raw v[4];
            float w[4];
            const int many = min(__popcll(left), 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= many) continue;
                const int k = __ffsll((unsigned long long)left) - 1;
                left &= left - 1;
                w[j] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, share), k));
                v[j] = load_raw<DT, LARGE>(p.rows, (int64_t)__builtin_amdgcn_readlane(place, k) * p.ldr + col, n);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= many) continue;
                const f32x8 f = Io<DT>::values(v[j]);
#pragma unroll
                for (int e = 0; e < kChunk; ++e) acc[e] = fmaf(w[j], f[e], acc[e]);
            }
        }
    }
    store8<DT, LARGE>(p.out, token * p.ldo + col, acc, n);
}

// Gradients of combine: a team of threads holds a token's dout, and for each of its choices stores weight *
// dout to the choice's row and sums dout * the row.  LONG: rows that the team walks.
constexpr int kGradChoices = 64;          // choices whose sums wait in LDS
template <int DT, int THREADS, int PER, bool LONG, bool LARGE>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS)
combine_backward_kernel(CombineGradParams p, int64_t teams) {
    constexpr int TEAMS = THREADS < 256 ? 256 / THREADS : 1, W = THREADS / 64;
    typedef typename Io<DT>::Raw Raw;
    __shared__ float red[W > 1 ? kGradChoices * W : 1];
    const int64_t token = folded_block() * TEAMS + (TEAMS > 1 ? threadIdx.x / THREADS : 0);
    if (token >= teams) return;                // the whole team together
    const int t = threadIdx.x % THREADS;
    const int64_t used = rows_used(p.last, p.n_rows);
    const int64_t span = LONG ? p.N : 1;       // (one trip otherwise)
    Raw d[PER];
    auto load_dout = [&](int64_t c0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t col = c0 + kChunk * (t + i * THREADS);
            const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.N - col));
            d[i] = load_raw<DT, LARGE>(p.dout, token * p.lddo + col, n);
        }
    };
    if (token < p.tokens) {
        if (!LONG) load_dout(0);
        for (int k0 = 0; k0 < p.top; k0 += kGradChoices) {
            const int ks = min(p.top - k0, kGradChoices);
            for (int k = 0; k < ks; ++k) {
                const int64_t choice = token * p.top + k0 + k;
                const int row = p.place[choice];
                float s = 0.0f;
                if (row >= 0 && row < used) {
                    const float w = p.weights[token * p.ldw + k0 + k];
                    for (int64_t c0 = 0; c0 < span; c0 += (int64_t)kChunk * THREADS * PER) {
                        if (LONG) load_dout(c0);
                        Raw v[PER];
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const int64_t col = c0 + kChunk * (t + i * THREADS);
                            const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.N - col));
                            v[i] = Raw{};
                            if (p.dweights != nullptr) v[i] = load_raw<DT, LARGE>(p.rows, row * p.ldr + col, n);
                        }
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const int64_t col = c0 + kChunk * (t + i * THREADS);
                            const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.N - col));
                            f32x8 g = Io<DT>::values(d[i]);
                            const f32x8 f = Io<DT>::values(v[i]);
#pragma unroll
                            for (int e = 0; e < kChunk; ++e) {
                                s = fmaf(g[e], f[e], s);
                                g[e] *= w;
                            }
                            store8<DT, LARGE>(p.drows, row * p.lddr + col, g, n);
                        }
                    }
                }
                if (p.dweights != nullptr) {
                    s = sum64(s);
                    if (W == 1) {
                        if (t == 0) p.dweights[token * p.lddw + k0 + k] = s;
                    } else if ((threadIdx.x & 63) == 0) {
                        red[k * W + (threadIdx.x >> 6)] = s;
                    }
                }
            }
            if (W > 1 && p.dweights != nullptr) {
                __syncthreads();
                for (int k = threadIdx.x; k < ks; k += THREADS) {
                    float s = 0.0f;
#pragma unroll
                    for (int w = 0; w < W; ++w) s += red[k * W + w];
                    p.dweights[token * p.lddw + k0 + k] = s;
                }
                __syncthreads();
            }
        }
    }
    for (int64_t row = used + token; row < p.n_rows; row += teams)
        for (int64_t c0 = 0; c0 < span; c0 += (int64_t)kChunk * THREADS * PER) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int64_t col = c0 + kChunk * (t + i * THREADS);
                const int n = (int)max((int64_t)0, min((int64_t)kChunk, p.N - col));
                store8<DT, LARGE>(p.drows, row * p.lddr + col, f32x8{}, n);
            }
        }
}

// Tokens, or where rows past the last group's are cleared and there are no tokens, some teams for that.  (With
// few tokens those teams clear a large buffer's rows one after the other: into 8192 rows of 4096 bf16 1 token
// takes 630 us, its gradients 700, 16 tokens 45 and 54; into 64 rows 5.4 and 5.7.)
int64_t teams_for(int64_t tokens, int64_t rows, bool clears) {
    return tokens > 0 || !clears ? tokens : rows < 1024 ? rows : 1024;
}

// Rows of so many bytes in all cannot stay in the L2s: they are read and written non-temporally.  Measured with
// inputs in turn, without and with, bf16, top 2: 64 MB of rows handed out 23 and 18 us, together again 26 and 24,
// gradients 35 and 30; 32 MB 10.7 and 10, 12.3 and 13.8, 14 and 17; 16 MB 7.6 and 5.6, 7.5 and 8.1, 8.7 and 10.
bool large(int64_t rows, int64_t bytes) { return (double)rows * bytes >= 32 << 20; }

template <int DT, bool LARGE> hipError_t combine_type(const CombineParams &p, hipStream_t s) {
    const int slabs = (int)((p.N + 511) / 512);
    return go(&combine_kernel<DT, LARGE>, fold((p.tokens * slabs + 3) / 4), 256, s, p, slabs);
}

template <int DT, bool LARGE> hipError_t combine_grad_type(const CombineGradParams &p, hipStream_t s) {
    const int64_t teams = teams_for(p.tokens, p.n_rows, p.last != nullptr);
    if (teams == 0) return hipSuccess;
    switch (shape_of(p.N)) {
        case kWave2: return go(&combine_backward_kernel<DT, 64, 2, false, LARGE>, fold((teams + 3) / 4), 256, s, p, teams);
        case kFour2: return go(&combine_backward_kernel<DT, 256, 2, false, LARGE>, fold(teams), 256, s, p, teams);
        case kSixteen1: return go(&combine_backward_kernel<DT, 1024, 1, false, LARGE>, fold(teams), 1024, s, p, teams);
        default: return go(&combine_backward_kernel<DT, 1024, 1, true, LARGE>, fold(teams), 1024, s, p, teams);
    }
}

}  // namespace

// One workgroup for few choices: a second launch costs the GPU as much as five steps of its waves (2400 choices of
// 64 groups 7.05 us in one workgroup, 6.95 in five; 8192 of 128 groups 14.0 and 8.2).  Each of several then adds up
// the counts of all, which bounds how many pay (65536 of 64: 8.4 us in 64, 7.9 in 128; 524288: 18.2 and 13.4).
int plan_blocks(int64_t choices) {
    return choices <= 2560 ? 1 : (int)std::min((choices + 511) / 512, (int64_t)128);
}

hipError_t launch_plan(const PlanParams &p, hipStream_t s) {
    PlanParams q = p;
    q.blocks = plan_blocks(p.choices);
    q.per = (p.choices + q.blocks - 1) / q.blocks;
    // As many waves as have 64 choices, and as their tables leave room for.
    int waves = 16;
    while (waves > 1 && (waves * p.groups > kPlanCounters || 32 * waves >= q.per)) waves /= 2;
    int bits = 1;
    while (p.groups >> bits != 0) ++bits;
    if (q.blocks > 1) {
        void *argv[] = {&q};
        const hipError_t err = hipLaunchKernel(reinterpret_cast<const void *>(&plan_count_kernel), dim3((unsigned)q.blocks),
                                               dim3(1024), argv, (size_t)q.groups * 4, s);
        if (err != hipSuccess) return err;
    }
    void *argv[] = {&q, &bits, &waves};
    return hipLaunchKernel(reinterpret_cast<const void *>(&plan_place_kernel), dim3((unsigned)q.blocks),
                           dim3((unsigned)(q.blocks > 1 ? 1024 : 64 * waves)), argv,
                           (size_t)(q.blocks > 1 ? waves + 2 : waves + 1) * q.groups * 4, s);
}

hipError_t launch_dispatch(const DispatchParams &p, hipStream_t s) {
    const int64_t teams = teams_for(p.tokens, p.rows, p.last != nullptr);
    if (teams == 0) return hipSuccess;
    // 4 KB a wave where that leaves waves for every compute unit, else 1 KB.
    const int big = (int)((p.wide + 4095) / 4096), small = (int)((p.wide + 1023) / 1024);
    const bool wide = teams * big >= 4096;
    const dim3 grid = fold((teams * (wide ? big : small) + 3) / 4);
    if (large(p.rows, p.wide))
        return wide ? go(&dispatch_kernel<4, true>, grid, 256, s, p, teams, big)
                    : go(&dispatch_kernel<1, true>, grid, 256, s, p, teams, small);
    return wide ? go(&dispatch_kernel<4, false>, grid, 256, s, p, teams, big)
                : go(&dispatch_kernel<1, false>, grid, 256, s, p, teams, small);
}

hipError_t launch_combine(const CombineParams &p, hipStream_t s) {
    if (large(p.n_rows, p.N * (p.dtype == GEMM_DTYPE_F32 ? 4 : 2)))
        return p.dtype == GEMM_DTYPE_F32 ? combine_type<GEMM_DTYPE_F32, true>(p, s)
                                         : combine_type<GEMM_DTYPE_BF16F32, true>(p, s);
    return p.dtype == GEMM_DTYPE_F32 ? combine_type<GEMM_DTYPE_F32, false>(p, s)
                                     : combine_type<GEMM_DTYPE_BF16F32, false>(p, s);
}

hipError_t launch_combine_backward(const CombineGradParams &p, hipStream_t s) {
    if (large(p.n_rows, p.N * (p.dtype == GEMM_DTYPE_F32 ? 4 : 2)))
        return p.dtype == GEMM_DTYPE_F32 ? combine_grad_type<GEMM_DTYPE_F32, true>(p, s)
                                         : combine_grad_type<GEMM_DTYPE_BF16F32, true>(p, s);
    return p.dtype == GEMM_DTYPE_F32 ? combine_grad_type<GEMM_DTYPE_F32, false>(p, s)
                                     : combine_grad_type<GEMM_DTYPE_BF16F32, false>(p, s);
}

}  // namespace gemm
