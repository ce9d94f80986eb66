// cm_norm.cuh -- launch entries of the layer norm's kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cm.h"

namespace cm {

struct NormParams {
    const void *x;
    const void *gamma, *beta;   // either may be null (1 and 0)
    const void *dy, *res;       // backward; res may be null
    void *out;                  // y, or dx
    float *mean, *rstd;         // forward: written if non-null; backward: read
    int64_t ldx, lddy, ldr, ldo;
    int64_t rows, h;
    float eps;
    int p_f32;                  // type of gamma and beta
    // backward: per-CTA partial sums [parts][2][h] of dgamma and dbeta, then the sums
    float *partial;
    void *dgamma, *dbeta;
    int g_f32, accumulate;
};

cudaError_t launch_layer_norm(const NormParams &p, cm_dtype x, cm_dtype y, cudaStream_t stream);
int64_t norm_backward_parts(int64_t rows, int64_t h);
cudaError_t launch_layer_norm_backward(const NormParams &p, cm_dtype x, cm_dtype y, cudaStream_t stream);

}  // namespace cm
