// Arguments of the routing launches (gemm_route.hip), validated by gemm_route_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.h"

namespace gemm {

struct PlanParams {
    const void *experts;        // tokens x top, rows ld apart
    int64_t ld;
    int32_t wide, top, groups;  // wide: 64-bit numbers
    int32_t choices;            // tokens * top
    int32_t *order, *place, *ends, *counts;       // order: may be null
    int32_t blocks, per;        // workgroups, choices of each
};

struct DispatchParams {
    const char *x;
    char *out;
    const int32_t *place, *last;       // last: where the last group ends, or null
    const float *scales;
    float *out_scales;
    int64_t tokens, rows, ldx, ldo, wide, lds, ldos;       // ldx, ldo, wide: bytes
    int32_t top, scale_cols;
};

struct CombineParams {
    const void *rows, *residual;
    void *out;
    const int32_t *place;
    const float *weights;
    int64_t tokens, n_rows, N, ldr, ld_res, ldo, ldw;
    int32_t dtype, top;
};

struct CombineGradParams {
    const void *dout, *rows;
    void *drows;
    const int32_t *place, *last;
    const float *weights;
    float *dweights;
    int64_t tokens, n_rows, N, lddo, ldr, lddr, ldw, lddw;
    int32_t dtype, top;
};

constexpr int64_t kPlanGroups = 4096, kPlanChoices = int64_t(1) << 30;
// Counters of a workgroup's waves, a table of the groups each: with two tables more they fit 64 KB of LDS.
constexpr int kPlanCounters = 8000;
// Workgroups that sort so many choices (1: one launch and no workspace).
int plan_blocks(int64_t choices);

hipError_t launch_plan(const PlanParams &p, hipStream_t stream);
hipError_t launch_dispatch(const DispatchParams &p, hipStream_t stream);
hipError_t launch_combine(const CombineParams &p, hipStream_t stream);
hipError_t launch_combine_backward(const CombineGradParams &p, hipStream_t stream);

}  // namespace gemm
