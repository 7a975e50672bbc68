// Arguments of the norm and quantiser launches (gemm_norm.hip), validated by
// gemm_experts_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.h"

namespace gemm {

struct QuantParams {
    const void *x;
    uint8_t *q;
    float *scales;
    int64_t M, K, ldx, ldq, lds;
    int32_t dtype, block_rows;
};

struct NormParams {
    const void *x, *residual, *weight;
    void *sum, *out;
    float *scales;
    int64_t M, N, ldx, ldr, ld_sum, ldo, ld_scales;
    float eps;
    int32_t dtype, out_type;
};

struct NormGradParams {
    const void *dy, *s, *weight, *ds;
    void *dx;
    float *dweight, *partials;
    int64_t M, N, lddy, lds, ldds, lddx;
    float eps;
    int32_t dtype;
};

// Rows of partial weight gradients the backward pass leaves (each N floats).
int norm_grad_partials(int64_t M, int64_t N);

hipError_t launch_quantize(const QuantParams &p, hipStream_t stream);
hipError_t launch_rms_norm(const NormParams &p, hipStream_t stream);
hipError_t launch_rms_norm_backward(const NormGradParams &p, hipStream_t stream);

}  // namespace gemm
