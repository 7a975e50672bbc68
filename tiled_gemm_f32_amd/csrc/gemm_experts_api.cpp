// Entry points of the sparse expert layer's operators: argument checks (all
// before any HIP call), kernel choice and launch.
#include <cmath>
#include <cstdint>

#include "gemm.h"
#include "gemm_grouped.hpp"
#include "gemm_kernels.hpp"
#include "gemm_norm.hpp"

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr int64_t kMaxGroups = 65535;          // a grid dimension
constexpr int64_t kMaxInt8K = 131071;          // products of -128 and -128 that a 32-bit sum holds
// Workgroups of one launch: their threads along x (512 each at most) are counted in 32 bits.
constexpr int64_t kMaxTiles = (int64_t(1) << 32) / 512 - 1;

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }
int64_t at_least_1(int64_t n) { return n > 1 ? n : 1; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A pointer that is read or written: there, and on its elements.
bool bad_ptr(const void *p, uintptr_t esz) { return p == nullptr || !aligned(p, esz); }
bool bad_opt(const void *p, uintptr_t esz) { return p != nullptr && !aligned(p, esz); }
bool float_type(int32_t dtype) { return dtype == GEMM_DTYPE_F32 || dtype == GEMM_DTYPE_BF16F32; }
uintptr_t size_of(int32_t dtype) { return dtype == GEMM_DTYPE_F32 ? 4 : dtype == GEMM_DTYPE_BF16F32 ? 2 : 1; }

bool rows_on16(const void *p, int64_t ld, int64_t esz) { return aligned(p, 16) && ld * esz % 16 == 0; }
// Offsets inside a tile's panel of 256 rows (and of their scales) are 32-bit.
constexpr int64_t kMaxTileRow = (int64_t(1) << 31) / 256 - 256;

gemm_status launched(hipError_t err) { return err == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

struct Product {
    int32_t dtype, op_b, groups;
    const int32_t *ends;
    bool grouped;
    int64_t M, N, K;
    float alpha;
    const void *A, *B;
    int64_t lda, ldb, stride_b;
    const gemm_block_scales *sc;
    int32_t out_type;
    void *out;
    int64_t ldo;
};

gemm_status run(const Product &c, gemm_stream_t stream) {
    if (!float_type(c.dtype) && c.dtype != GEMM_DTYPE_FP8F32) return GEMM_ERR_INVALID_ARG;
    if (c.op_b != GEMM_OP_N && c.op_b != GEMM_OP_T) return GEMM_ERR_INVALID_ARG;
    if (c.out_type < GEMM_OUT_F32 || c.out_type > GEMM_OUT_FP8) return GEMM_ERR_INVALID_ARG;
    if (c.M < 0 || c.N < 0 || c.K < 0 || c.groups < 0) return GEMM_ERR_INVALID_ARG;
    const int64_t b_len = c.op_b == GEMM_OP_N ? c.N : c.K;       // a stored row of B
    if (c.lda < at_least_1(c.K) || c.ldb < at_least_1(b_len) || c.ldo < at_least_1(c.N) || c.stride_b < 0)
        return GEMM_ERR_INVALID_ARG;
    const bool reads = c.M > 0 && c.N > 0 && c.K > 0 && c.alpha != 0.0f && c.groups > 0;
    const uintptr_t esz = size_of(c.dtype);
    if (reads && (bad_ptr(c.A, esz) || bad_ptr(c.B, esz))) return GEMM_ERR_INVALID_ARG;
    if (c.M > 0 && c.N > 0 && bad_ptr(c.out, c.out_type == GEMM_OUT_F32 ? 4 : 2)) return GEMM_ERR_INVALID_ARG;
    if (c.grouped && c.groups > 0 && c.M > 0 && c.N > 0 && bad_ptr(c.ends, 4)) return GEMM_ERR_INVALID_ARG;
    if (c.dtype == GEMM_DTYPE_FP8F32) {
        if (c.sc == nullptr) return GEMM_ERR_INVALID_ARG;
        if (c.sc->a_row < 0 || c.sc->a_block < 0 || c.sc->b_n < 0 || c.sc->b_k < 0 || c.sc->b_group < 0)
            return GEMM_ERR_INVALID_ARG;
        if (reads && (bad_ptr(c.sc->a, 4) || bad_ptr(c.sc->b, 4))) return GEMM_ERR_INVALID_ARG;
    } else if (c.sc != nullptr) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (c.out_type == GEMM_OUT_FP8) return GEMM_ERR_UNSUPPORTED;
    if (c.M > kMaxDim || c.N > kMaxDim || c.K > kMaxDim || c.lda > kMaxDim || c.ldb > kMaxDim || c.ldo > kMaxDim ||
        c.groups > kMaxGroups)
        return GEMM_ERR_UNSUPPORTED;
    if (c.M == 0 || c.N == 0) return GEMM_OK;
    // Bounds every launch: tiles of 32 x 128, the most there are, are at most twice these and of 256
    // threads.  (The kernels of smaller tiles take fewer, and leave the others.)
    if (gemm::most_row_tiles(c.M, c.groups, 64, c.grouped) * ceil_div(c.N, 64) > kMaxTiles)
        return GEMM_ERR_UNSUPPORTED;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    gemm::GroupedParams p = {};
    p.A = c.A;
    p.B = c.B;
    p.out = c.out;
    p.ends = c.grouped ? c.ends : nullptr;
    p.M = (int32_t)c.M;
    p.N = (int32_t)c.N;
    p.K = reads ? (int32_t)c.K : 0;            // alpha == 0 reads no operand
    p.groups = c.groups;
    p.lda = c.lda;
    p.ldb = c.ldb;
    p.stride_b = c.stride_b;
    p.ldo = c.ldo;
    p.alpha = c.alpha;
    p.out_type = c.out_type;
    if (c.sc != nullptr) p.sc = *c.sc;
    // A row's bytes must hold one 16-byte load, whatever their alignment.
    const int64_t sz = (int64_t)esz;
    const bool tiles = c.K * sz >= 16 && b_len * sz >= 16 && c.lda * sz < kMaxTileRow &&
                       c.ldb * sz < kMaxTileRow && (c.sc == nullptr || (c.sc->a_row < kMaxTileRow / 4 && c.sc->b_n < kMaxTileRow));
    const auto s = static_cast<hipStream_t>(stream);
    if (!tiles) return launched(gemm::launch_grouped_general(c.dtype, c.op_b, p, s));
    if (c.M == 1) p.lda = ceil_div(c.K * sz, 16) * 16 / sz;          // the stride of a single row is not used
    const bool dma = rows_on16(c.A, p.lda, sz) && rows_on16(c.B, c.ldb, sz) && c.stride_b * sz % 16 == 0;
    if (c.dtype == GEMM_DTYPE_F32) return launched(gemm::launch_grouped_f32(c.op_b, dma, p, s));
    if (dma)
        if (const int rows = gemm::skinny_rows(c.dtype, c.op_b, p))
            return launched(gemm::launch_grouped_skinny(c.dtype, rows, p, s));
    return launched(c.dtype == GEMM_DTYPE_FP8F32 ? gemm::launch_grouped_fp8(c.op_b, dma, p, s)
                                                 : gemm::launch_grouped_bf16(c.op_b, dma, p, s));
}

}  // namespace

extern "C" {

GEMM_API gemm_status gemm_block_scaled(int32_t op_b, int64_t M, int64_t N, int64_t K, float alpha, const uint8_t *A,
                                       int64_t lda, const uint8_t *B, int64_t ldb, const gemm_block_scales *scales,
                                       int32_t out_type, void *out, int64_t ldo, gemm_stream_t stream) {
    return run(Product{GEMM_DTYPE_FP8F32, op_b, 1, nullptr, false, M, N, K, alpha, A, B, lda, ldb, 0, scales, out_type,
                       out, ldo},
               stream);
}

GEMM_API gemm_status gemm_grouped(int32_t dtype, int32_t op_b, int32_t groups, const int32_t *ends, int64_t M,
                                  int64_t N, int64_t K, float alpha, const void *A, int64_t lda, const void *B,
                                  int64_t ldb, int64_t stride_b, const gemm_block_scales *scales, int32_t out_type,
                                  void *out, int64_t ldo, gemm_stream_t stream) {
    return run(Product{dtype, op_b, groups, ends, true, M, N, K, alpha, A, B, lda, ldb, stride_b, scales, out_type,
                       out, ldo},
               stream);
}

GEMM_API gemm_status gemm_grouped_wgrad(int32_t dtype, int32_t groups, const int32_t *ends, int64_t M, int64_t N,
                                        int64_t K, float alpha, const void *dY, int64_t lddy, const void *X,
                                        int64_t ldx, float beta, float *dW, int64_t ldw, int64_t stride_w,
                                        gemm_stream_t stream) {
    if (!float_type(dtype) && dtype != GEMM_DTYPE_FP8F32) return GEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0 || groups < 0) return GEMM_ERR_INVALID_ARG;
    if (lddy < at_least_1(N) || ldx < at_least_1(K) || ldw < at_least_1(K) || stride_w < 0) return GEMM_ERR_INVALID_ARG;
    const bool writes = groups > 0 && N > 0 && K > 0;
    const bool reads = writes && M > 0 && alpha != 0.0f;
    if (writes && (bad_ptr(dW, 4) || bad_ptr(ends, 4))) return GEMM_ERR_INVALID_ARG;
    const uintptr_t esz = size_of(dtype);
    if (reads && (bad_ptr(dY, esz) || bad_ptr(X, esz))) return GEMM_ERR_INVALID_ARG;
    if (!float_type(dtype)) return GEMM_ERR_UNSUPPORTED;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim || lddy > kMaxDim || ldx > kMaxDim || ldw > kMaxDim ||
        groups > kMaxGroups || ceil_div(N, 64) * ceil_div(K, 64) > kMaxTiles)
        return GEMM_ERR_UNSUPPORTED;
    if (!writes) return GEMM_OK;
    // Groups' results must not overlap: each starts past the one before, or row n of all of them lies
    // before row n + 1 of the first.
    const bool apart = stride_w >= (N - 1) * ldw + K;
    const bool between = stride_w >= K && stride_w <= ldw && (groups - 1) * stride_w + K <= ldw;
    if (groups > 1 && !apart && !between) return GEMM_ERR_INVALID_ARG;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    gemm::GroupedParams p = {};
    p.A = dY;
    p.B = X;
    p.out = dW;
    p.ends = ends;
    p.M = reads ? (int32_t)M : 0;              // alpha == 0 reads no operand
    p.N = (int32_t)N;
    p.K = (int32_t)K;
    p.groups = groups;
    p.lda = lddy;
    p.ldb = ldx;
    p.ldo = ldw;
    p.stride_out = stride_w;
    p.alpha = alpha;
    p.beta = beta;
    const int64_t sz = (int64_t)esz;
    // Deep groups are bound by their products, and the launch's end by the last of them (8 groups of
    // 8192 x 4096 x 2048 bf16: 178 us in the order of their numbers, 165 so); shallow ones by the
    // results' stores, which the larger groups' products hide if they come between (40 groups of
    // 2000 x 1024 x 1024 bf16: 37 and 40).  Twelve slabs of 128 bytes a group's column.
    p.by_size = groups <= 64 && M * sz >= 1536 * (int64_t)groups;
    const auto s = static_cast<hipStream_t>(stream);
    if (N * sz < 16 || K * sz < 16 || lddy * sz >= kMaxTileRow || ldx * sz >= kMaxTileRow)
        return launched(gemm::launch_wgrad_general(dtype, p, s));
    const bool dma = rows_on16(dY, lddy, sz) && rows_on16(X, ldx, sz);
    return launched(dtype == GEMM_DTYPE_F32 ? gemm::launch_wgrad_f32(dma, p, s) : gemm::launch_wgrad_bf16(dma, p, s));
}

GEMM_API gemm_status gemm_quantize(int32_t dtype, int32_t block_rows, int64_t M, int64_t K, const void *X, int64_t ldx,
                                   uint8_t *Q, int64_t ldq, float *scales, int64_t lds, gemm_stream_t stream) {
    if (!float_type(dtype) || (block_rows != 1 && block_rows != GEMM_SCALE_BLOCK) || M < 0 || K < 0)
        return GEMM_ERR_INVALID_ARG;
    if (ldx < at_least_1(K) || ldq < at_least_1(K) || lds < at_least_1(ceil_div(K, GEMM_SCALE_BLOCK)))
        return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || K > kMaxDim || ldx > kMaxDim || ldq > kMaxDim || lds > kMaxDim) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return GEMM_OK;
    if (bad_ptr(X, size_of(dtype)) || bad_ptr(Q, 1) || bad_ptr(scales, 4)) return GEMM_ERR_INVALID_ARG;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    const gemm::QuantParams p = {X, Q, scales, M, K, ldx, ldq, lds, dtype, block_rows};
    return launched(gemm::launch_quantize(p, static_cast<hipStream_t>(stream)));
}

GEMM_API gemm_status gemm_rms_norm(int32_t dtype, int64_t M, int64_t N, const void *X, int64_t ldx,
                                   const void *residual, int64_t ldr, const void *weight, float eps, void *sum,
                                   int64_t ld_sum, int32_t out_type, void *out, int64_t ldo, float *scales,
                                   int64_t ld_scales, gemm_stream_t stream) {
    if (!float_type(dtype) || out_type < GEMM_OUT_F32 || out_type > GEMM_OUT_FP8 || M < 0 || N < 0)
        return GEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps)) return GEMM_ERR_INVALID_ARG;
    const int64_t row = at_least_1(N);
    if (ldx < row || ldo < row || (residual != nullptr && ldr < row) || (sum != nullptr && ld_sum < row))
        return GEMM_ERR_INVALID_ARG;
    const bool fp8 = out_type == GEMM_OUT_FP8;
    if (fp8 && ld_scales < at_least_1(ceil_div(N, GEMM_SCALE_BLOCK))) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || N > kMaxDim || ldx > kMaxDim || ldo > kMaxDim || (residual != nullptr && ldr > kMaxDim) ||
        (sum != nullptr && ld_sum > kMaxDim) || (fp8 && ld_scales > kMaxDim))
        return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    const uintptr_t esz = size_of(dtype);
    if (bad_ptr(X, esz) || bad_ptr(weight, esz) || bad_opt(residual, esz) || bad_opt(sum, esz) ||
        bad_ptr(out, fp8 ? 1 : out_type == GEMM_OUT_BF16 ? 2 : 4) || (fp8 && bad_ptr(scales, 4)))
        return GEMM_ERR_INVALID_ARG;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    const gemm::NormParams p = {X,   residual, weight, sum, out,       scales, M,     N,
                                ldx, ldr,      ld_sum, ldo, ld_scales, eps,    dtype, out_type};
    return launched(gemm::launch_rms_norm(p, static_cast<hipStream_t>(stream)));
}

GEMM_API int64_t gemm_rms_norm_workspace_size(int64_t M, int64_t N) {
    if (M <= 0 || N <= 0 || M > kMaxDim || N > kMaxDim) return 0;
    return (int64_t)gemm::norm_grad_partials(M, N) * N * 4;
}

GEMM_API gemm_status gemm_rms_norm_backward(int32_t dtype, int64_t M, int64_t N, const void *dY, int64_t lddy,
                                            const void *S, int64_t lds, const void *weight, float eps, const void *dS,
                                            int64_t ldds, void *dX, int64_t lddx, float *dweight, void *workspace,
                                            int64_t workspace_bytes, gemm_stream_t stream) {
    if (!float_type(dtype) || M < 0 || N < 0 || workspace_bytes < 0) return GEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps)) return GEMM_ERR_INVALID_ARG;
    const int64_t row = at_least_1(N);
    if (lddy < row || lds < row || lddx < row || (dS != nullptr && ldds < row)) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || N > kMaxDim || lddy > kMaxDim || lds > kMaxDim || lddx > kMaxDim ||
        (dS != nullptr && ldds > kMaxDim))
        return GEMM_ERR_UNSUPPORTED;
    if (N == 0 || (M == 0 && dweight == nullptr)) return GEMM_OK;
    const uintptr_t esz = size_of(dtype);
    if (bad_opt(dweight, 4)) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && (bad_ptr(dY, esz) || bad_ptr(S, esz) || bad_ptr(weight, esz) || bad_ptr(dX, esz) || bad_opt(dS, esz)))
        return GEMM_ERR_INVALID_ARG;
    if (M > 0 && dweight != nullptr) {
        if (bad_opt(workspace, 4)) return GEMM_ERR_INVALID_ARG;
        if (workspace == nullptr || workspace_bytes < gemm_rms_norm_workspace_size(M, N)) return GEMM_ERR_SCRATCH;
    }
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    const gemm::NormGradParams p = {dY, S, weight, dS, dX, dweight, static_cast<float *>(workspace), M, N, lddy, lds,
                                    ldds, lddx, eps, dtype};
    return launched(gemm::launch_rms_norm_backward(p, static_cast<hipStream_t>(stream)));
}

GEMM_API gemm_status gemm_layer_norm(int32_t dtype, int64_t M, int64_t N, const void *X, int64_t ldx,
                                     const void *residual, int64_t ldr, const void *weight, const void *bias,
                                     float eps, void *sum, int64_t ld_sum, int32_t out_type, void *out, int64_t ldo,
                                     float *scales, int64_t ld_scales, gemm_stream_t stream) {
    if (!float_type(dtype) || out_type < GEMM_OUT_F32 || out_type > GEMM_OUT_INT8 || M < 0 || N < 0)
        return GEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps)) return GEMM_ERR_INVALID_ARG;
    const int64_t row = at_least_1(N);
    if (ldx < row || ldo < row || (residual != nullptr && ldr < row) || (sum != nullptr && ld_sum < row))
        return GEMM_ERR_INVALID_ARG;
    const bool codes = out_type == GEMM_OUT_FP8 || out_type == GEMM_OUT_INT8;
    const int64_t per_row = out_type == GEMM_OUT_FP8 ? at_least_1(ceil_div(N, GEMM_SCALE_BLOCK)) : 1;
    if (codes && ld_scales < per_row) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || N > kMaxDim || ldx > kMaxDim || ldo > kMaxDim || (residual != nullptr && ldr > kMaxDim) ||
        (sum != nullptr && ld_sum > kMaxDim) || (codes && ld_scales > kMaxDim))
        return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    const uintptr_t esz = size_of(dtype);
    if (bad_ptr(X, esz) || bad_ptr(weight, esz) || bad_opt(bias, esz) || bad_opt(residual, esz) || bad_opt(sum, esz) ||
        bad_ptr(out, codes ? 1 : out_type == GEMM_OUT_BF16 ? 2 : 4) || (codes && bad_ptr(scales, 4)))
        return GEMM_ERR_INVALID_ARG;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    const gemm::LayerNormParams p = {X,   residual, weight, bias, sum,       out, scales, M,       N,
                                     ldx, ldr,      ld_sum, ldo,  ld_scales, eps, dtype,  out_type};
    return launched(gemm::launch_layer_norm(p, static_cast<hipStream_t>(stream)));
}

GEMM_API int64_t gemm_layer_norm_workspace_size(int64_t M, int64_t N) {
    if (M <= 0 || N <= 0 || M > kMaxDim || N > kMaxDim) return 0;
    return (int64_t)gemm::layer_norm_grad_partials(M, N) * N * 8;
}

GEMM_API gemm_status gemm_layer_norm_backward(int32_t dtype, int64_t M, int64_t N, const void *dY, int64_t lddy,
                                              const void *S, int64_t lds, const void *weight, float eps,
                                              const void *dS, int64_t ldds, void *dX, int64_t lddx, float *dweight,
                                              float *dbias, void *workspace, int64_t workspace_bytes,
                                              gemm_stream_t stream) {
    if (!float_type(dtype) || M < 0 || N < 0 || workspace_bytes < 0) return GEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps)) return GEMM_ERR_INVALID_ARG;
    const int64_t row = at_least_1(N);
    if (lddy < row || lds < row || lddx < row || (dS != nullptr && ldds < row)) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || N > kMaxDim || lddy > kMaxDim || lds > kMaxDim || lddx > kMaxDim ||
        (dS != nullptr && ldds > kMaxDim))
        return GEMM_ERR_UNSUPPORTED;
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (N == 0 || (M == 0 && !sums)) return GEMM_OK;
    const uintptr_t esz = size_of(dtype);
    if (bad_opt(dweight, 4) || bad_opt(dbias, 4)) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && (bad_ptr(dY, esz) || bad_ptr(S, esz) || bad_ptr(weight, esz) || bad_ptr(dX, esz) || bad_opt(dS, esz)))
        return GEMM_ERR_INVALID_ARG;
    if (M > 0 && sums) {
        if (bad_opt(workspace, 4)) return GEMM_ERR_INVALID_ARG;
        if (workspace == nullptr || workspace_bytes < gemm_layer_norm_workspace_size(M, N)) return GEMM_ERR_SCRATCH;
    }
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    const gemm::LayerNormGradParams p = {dY, S, weight, dS, dX, dweight, dbias,
                                         sums ? static_cast<float *>(workspace) : nullptr, M, N, lddy, lds, ldds, lddx,
                                         eps, dtype};
    return launched(gemm::launch_layer_norm_backward(p, static_cast<hipStream_t>(stream)));
}

GEMM_API gemm_status gemm_quantize_int8(int32_t dtype, int64_t M, int64_t K, const void *X, int64_t ldx, int8_t *Q,
                                        int64_t ldq, float *scales, gemm_stream_t stream) {
    if (!float_type(dtype) || M < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (ldx < at_least_1(K) || ldq < at_least_1(K)) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || K > kMaxDim || ldx > kMaxDim || ldq > kMaxDim) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return GEMM_OK;
    if (bad_ptr(X, size_of(dtype)) || bad_ptr(Q, 1) || bad_ptr(scales, 4)) return GEMM_ERR_INVALID_ARG;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    const gemm::Int8Params p = {X, reinterpret_cast<uint8_t *>(Q), scales, M, K, ldx, ldq, dtype};
    return launched(gemm::launch_quantize_int8(p, static_cast<hipStream_t>(stream)));
}

GEMM_API gemm_status gemm_int8(int32_t op_b, int32_t groups, const int32_t *ends, int64_t M, int64_t N, int64_t K,
                               const int8_t *A, int64_t lda, const int8_t *B, int64_t ldb, int64_t stride_b,
                               const gemm_int8_scales *scales, int32_t out_type, void *out, int64_t ldo,
                               gemm_stream_t stream) {
    if (op_b != GEMM_OP_N && op_b != GEMM_OP_T) return GEMM_ERR_INVALID_ARG;
    if (out_type < GEMM_OUT_F32 || out_type > GEMM_OUT_INT8) return GEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0 || groups < 0 || (ends == nullptr && groups > 1))
        return GEMM_ERR_INVALID_ARG;
    const int64_t b_len = op_b == GEMM_OP_N ? N : K;       // a stored row of B
    if (lda < at_least_1(K) || ldb < at_least_1(b_len) || ldo < at_least_1(N) || stride_b < 0)
        return GEMM_ERR_INVALID_ARG;
    if (scales == nullptr || scales->a_row < 0 || scales->b_col < 0 || scales->b_group < 0 || scales->bias_group < 0)
        return GEMM_ERR_INVALID_ARG;
    const bool writes = M > 0 && N > 0, reads = writes && K > 0 && groups > 0;
    if (reads && (bad_ptr(A, 1) || bad_ptr(B, 1) || bad_ptr(scales->a, 4) || bad_ptr(scales->b, 4)))
        return GEMM_ERR_INVALID_ARG;
    if (writes && (bad_ptr(out, out_type == GEMM_OUT_F32 ? 4 : 2) || bad_opt(scales->bias, 4) || bad_opt(ends, 4)))
        return GEMM_ERR_INVALID_ARG;
    if (out_type != GEMM_OUT_F32 && out_type != GEMM_OUT_BF16) return GEMM_ERR_UNSUPPORTED;
    if (M > kMaxDim || N > kMaxDim || K > kMaxInt8K || lda > kMaxDim || ldb > kMaxDim || ldo > kMaxDim ||
        groups > kMaxGroups)
        return GEMM_ERR_UNSUPPORTED;
    if (!writes) return GEMM_OK;
    if (gemm::most_row_tiles(M, groups, 64, ends != nullptr) * ceil_div(N, 64) > kMaxTiles) return GEMM_ERR_UNSUPPORTED;
    gemm_status st = gemm::check_device();
    if (st != GEMM_OK) return st;
    gemm::GroupedParams p = {};
    p.A = A;
    p.B = B;
    p.out = out;
    p.ends = ends;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.K = (int32_t)K;
    p.groups = groups;
    p.lda = lda;
    p.ldb = ldb;
    p.stride_b = stride_b;
    p.ldo = ldo;
    p.alpha = 1.0f;
    p.out_type = out_type;
    p.ts = *scales;
    if (groups == 0) {                         // all rows are past the last end
        p.ends = nullptr;
        p.groups = 1;
        p.K = 0;
        p.ts.bias = nullptr;
    }
    const auto s = static_cast<hipStream_t>(stream);
    // A row must hold one 16-byte load, whatever its alignment.
    if (p.K < 16 || b_len < 16 || lda >= kMaxTileRow || ldb >= kMaxTileRow)
        return launched(gemm::launch_int8_general(op_b, p, s));
    if (M == 1) p.lda = ceil_div(K, 16) * 16;                        // the stride of a single row is not used
    const bool dma = rows_on16(A, p.lda, 1) && rows_on16(B, ldb, 1) && stride_b % 16 == 0;
    return launched(gemm::launch_grouped_int8(op_b, dma, p, s));
}

}  // extern "C"
