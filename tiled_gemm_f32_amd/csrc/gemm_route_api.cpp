// Entry points of the routing around the experts: argument checks (all before any HIP call) and launch.
#include <cstdint>

#include "gemm.h"
#include "gemm_kernels.hpp"
#include "gemm_route.hpp"

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;

int64_t at_least_1(int64_t n) { return n > 1 ? n : 1; }
// A pointer that is read or written: there, and on its elements.
bool bad_ptr(const void *p, uintptr_t esz) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % esz != 0; }
bool bad_opt(const void *p, uintptr_t esz) { return p != nullptr && bad_ptr(p, esz); }
bool float_type(int32_t dtype) { return dtype == GEMM_DTYPE_F32 || dtype == GEMM_DTYPE_BF16F32; }
uintptr_t size_of(int32_t dtype) { return dtype == GEMM_DTYPE_F32 ? 4 : 2; }
bool past(int64_t a, int64_t b, int64_t c, int64_t d) { return a > kMaxDim || b > kMaxDim || c > kMaxDim || d > kMaxDim; }
// A token's choices and its scales are walked 64 at a time in 32-bit numbers, which go that far past the last one.
constexpr int64_t kMostWalked = kMaxDim - 63;
// Choices of a call are numbered in 32 bits.
bool many_choices(int64_t tokens, int32_t top) {
    return tokens > kMaxDim || top > kMostWalked || (top > 0 && tokens > kMaxDim / top);
}

gemm_status launched(hipError_t err) { return err == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

}  // namespace

extern "C" {

GEMM_API int64_t gemm_expert_plan_workspace_size(int64_t tokens, int32_t top, int32_t groups) {
    if (tokens <= 0 || top <= 0 || groups <= 0 || groups > gemm::kPlanGroups || tokens > gemm::kPlanChoices / top) return 0;
    const int blocks = gemm::plan_blocks(tokens * top);
    return blocks > 1 ? (int64_t)blocks * groups * 4 : 0;
}

GEMM_API gemm_status gemm_expert_plan(int32_t id_bytes, int64_t tokens, int32_t top, int32_t groups,
                                      const void *experts, int64_t ld, int32_t *order, int32_t *place, int32_t *ends,
                                      void *workspace, int64_t workspace_bytes, gemm_stream_t stream) {
    if ((id_bytes != 4 && id_bytes != 8) || tokens < 0 || top < 1 || groups < 1 || ld < top || workspace_bytes < 0)
        return GEMM_ERR_INVALID_ARG;
    if (bad_ptr(ends, 4)) return GEMM_ERR_INVALID_ARG;
    if (tokens > 0 && (bad_ptr(experts, (uintptr_t)id_bytes) || bad_ptr(place, 4) || bad_opt(order, 4)))
        return GEMM_ERR_INVALID_ARG;
    if (groups > gemm::kPlanGroups || tokens > gemm::kPlanChoices / top || ld > kMaxDim) return GEMM_ERR_UNSUPPORTED;
    const int64_t need = gemm_expert_plan_workspace_size(tokens, top, groups);
    if (bad_opt(workspace, 4)) return GEMM_ERR_INVALID_ARG;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GEMM_ERR_SCRATCH;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    gemm::PlanParams p = {};
    p.experts = experts;
    p.ld = tokens > 1 ? ld : top;
    p.wide = id_bytes == 8;
    p.top = top;
    p.groups = groups;
    p.choices = (int32_t)(tokens * top);
    p.order = order;
    p.place = place;
    p.ends = ends;
    p.counts = static_cast<int32_t *>(workspace);
    return launched(gemm::launch_plan(p, static_cast<hipStream_t>(stream)));
}

GEMM_API gemm_status gemm_dispatch(int32_t elem_bytes, int64_t tokens, int32_t top, int64_t N, const void *X,
                                   int64_t ldx, const int32_t *place, const int32_t *last, int64_t rows, void *out,
                                   int64_t ldo, int64_t scale_cols, const float *scales, int64_t lds,
                                   float *out_scales, int64_t ldos, gemm_stream_t stream) {
    if ((elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) || tokens < 0 || top < 1 || N < 0 || rows < 0 ||
        scale_cols < 0)
        return GEMM_ERR_INVALID_ARG;
    if (ldx < at_least_1(N) || ldo < at_least_1(N) || (scale_cols > 0 && (lds < scale_cols || ldos < scale_cols)))
        return GEMM_ERR_INVALID_ARG;
    const bool reads = tokens > 0 && rows > 0 && N > 0;
    if (reads && (bad_ptr(X, (uintptr_t)elem_bytes) || bad_ptr(place, 4) || (scale_cols > 0 && bad_ptr(scales, 4))))
        return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && N > 0 &&
        (bad_ptr(out, (uintptr_t)elem_bytes) || bad_opt(last, 4) || (scale_cols > 0 && bad_ptr(out_scales, 4))))
        return GEMM_ERR_INVALID_ARG;
    if (many_choices(tokens, top) || past(N, ldx, ldo, rows) || scale_cols > kMostWalked ||
        (scale_cols > 0 && past(0, lds, ldos, 0)))
        return GEMM_ERR_UNSUPPORTED;
    if (rows == 0 || N == 0 || (tokens == 0 && last == nullptr)) return GEMM_OK;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    gemm::DispatchParams p = {};
    p.x = static_cast<const char *>(X);
    p.out = static_cast<char *>(out);
    p.place = place;
    p.last = last;
    p.scales = scales;
    p.out_scales = out_scales;
    p.tokens = tokens;
    p.rows = rows;
    p.ldx = ldx * elem_bytes;
    p.ldo = ldo * elem_bytes;
    p.wide = N * elem_bytes;
    p.lds = lds;
    p.ldos = ldos;
    p.top = top;
    p.scale_cols = (int32_t)scale_cols;
    return launched(gemm::launch_dispatch(p, static_cast<hipStream_t>(stream)));
}

GEMM_API gemm_status gemm_combine(int32_t dtype, int64_t tokens, int32_t top, int64_t N, const void *rows,
                                  int64_t ldr, int64_t n_rows, const int32_t *place, const float *weights,
                                  int64_t ldw, const void *residual, int64_t ld_res, void *out, int64_t ldo,
                                  gemm_stream_t stream) {
    if (!float_type(dtype) || tokens < 0 || top < 1 || N < 0 || n_rows < 0) return GEMM_ERR_INVALID_ARG;
    const int64_t row = at_least_1(N);
    if (ldr < row || ldo < row || (residual != nullptr && ld_res < row) || (weights != nullptr && ldw < top))
        return GEMM_ERR_INVALID_ARG;
    const uintptr_t esz = size_of(dtype);
    const bool writes = tokens > 0 && N > 0;
    if (writes && (bad_ptr(out, esz) || bad_opt(residual, esz))) return GEMM_ERR_INVALID_ARG;
    if (writes && n_rows > 0 && (bad_ptr(rows, esz) || bad_ptr(place, 4) || bad_opt(weights, 4)))
        return GEMM_ERR_INVALID_ARG;
    if (many_choices(tokens, top) || past(N, ldr, ldo, n_rows) || (residual != nullptr && ld_res > kMaxDim) ||
        (weights != nullptr && ldw > kMaxDim))
        return GEMM_ERR_UNSUPPORTED;
    if (!writes) return GEMM_OK;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    gemm::CombineParams p = {};
    p.rows = rows;
    p.residual = residual;
    p.out = out;
    p.place = place;
    p.weights = weights;
    p.tokens = tokens;
    p.n_rows = n_rows;
    p.N = N;
    p.ldr = ldr;
    p.ld_res = ld_res;
    p.ldo = ldo;
    p.ldw = ldw;
    p.dtype = dtype;
    p.top = n_rows > 0 ? top : 0;              // no row: no place is looked at
    return launched(gemm::launch_combine(p, static_cast<hipStream_t>(stream)));
}

GEMM_API gemm_status gemm_combine_backward(int32_t dtype, int64_t tokens, int32_t top, int64_t N, const void *dout,
                                           int64_t lddo, const void *rows, int64_t ldr, int64_t n_rows,
                                           const int32_t *place, const int32_t *last, const float *weights,
                                           int64_t ldw, void *drows, int64_t lddr, float *dweights, int64_t lddw,
                                           gemm_stream_t stream) {
    if (!float_type(dtype) || tokens < 0 || top < 1 || N < 0 || n_rows < 0) return GEMM_ERR_INVALID_ARG;
    const int64_t row = at_least_1(N);
    const bool sums = dweights != nullptr;
    if (lddo < row || lddr < row || ldw < top || (sums && (ldr < row || lddw < top))) return GEMM_ERR_INVALID_ARG;
    const uintptr_t esz = size_of(dtype);
    if (bad_opt(dweights, 4)) return GEMM_ERR_INVALID_ARG;
    if (tokens > 0 && (n_rows > 0 || sums) && (bad_ptr(place, 4) || bad_ptr(weights, 4))) return GEMM_ERR_INVALID_ARG;
    if (tokens > 0 && n_rows > 0 && N > 0 && (bad_ptr(dout, esz) || (sums && bad_ptr(rows, esz))))
        return GEMM_ERR_INVALID_ARG;
    if (n_rows > 0 && N > 0 && (bad_ptr(drows, esz) || bad_opt(last, 4))) return GEMM_ERR_INVALID_ARG;
    if (many_choices(tokens, top) || past(N, lddo, lddr, n_rows) || ldw > kMaxDim ||
        (sums && (ldr > kMaxDim || lddw > kMaxDim)))
        return GEMM_ERR_UNSUPPORTED;
    if (tokens == 0 && (last == nullptr || n_rows == 0 || N == 0)) return GEMM_OK;
    if ((n_rows == 0 || N == 0) && !sums) return GEMM_OK;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    gemm::CombineGradParams p = {};
    p.dout = dout;
    p.rows = rows;
    p.drows = drows;
    p.place = place;
    p.last = last;
    p.weights = weights;
    p.dweights = dweights;
    p.tokens = tokens;
    p.n_rows = n_rows;
    p.N = N;
    p.lddo = lddo;
    p.ldr = ldr;
    p.lddr = lddr;
    p.ldw = ldw;
    p.lddw = lddw;
    p.dtype = dtype;
    p.top = top;
    return launched(gemm::launch_combine_backward(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
