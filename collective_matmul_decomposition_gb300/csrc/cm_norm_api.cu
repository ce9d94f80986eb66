// cm_norm_api.cu -- the C ABI of the layer norm: argument checks and launches.
#include <nvtx3/nvToolsExt.h>

#include <algorithm>

#include "cm_internal.h"
#include "cm_norm.cuh"

namespace cm {
namespace {

constexpr int64_t kMaxExtent = int64_t(1) << 30;

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

bool bad_dtype(cm_dtype t) { return t != CM_BF16 && t != CM_F32; }
bool misaligned(const void *p, cm_dtype t) { return (reinterpret_cast<uintptr_t>(p) & (t == CM_F32 ? 3u : 1u)) != 0; }

cm_status check_rows(const void *p, cm_dtype t, int64_t ld, int64_t h) {
    if (!p) return CM_ERR_INVALID_ARG;
    if (ld < h || ld > kMaxExtent) return CM_ERR_SHAPE;
    return misaligned(p, t) ? CM_ERR_ALIGNMENT : CM_OK;
}

cm_status check_extents(int64_t rows, int64_t h) {
    return rows < 0 || h <= 0 || rows > kMaxExtent || h > kMaxExtent ? CM_ERR_SHAPE : CM_OK;
}

size_t backward_workspace(int64_t rows, int64_t h) {
    return size_t(norm_backward_parts(rows, h)) * 2 * size_t(h) * sizeof(float);
}

}  // namespace
}  // namespace cm

using namespace cm;

#define CM_TRY(x)                        \
    do {                                 \
        const cm_status st_ = (x);       \
        if (st_ != CM_OK) return st_;    \
    } while (0)

extern "C" {

cm_status cm_layer_norm(const void *x, cm_dtype x_dtype, int64_t ldx, const void *gamma, const void *beta,
                        cm_dtype param_dtype, float eps, void *y, cm_dtype y_dtype, int64_t ldy, float *mean,
                        float *rstd, int64_t rows, int64_t h, cm_stream_t stream) {
    NvtxRange range("cm_layer_norm");
    if (bad_dtype(x_dtype) || bad_dtype(y_dtype) || bad_dtype(param_dtype) || !(eps >= 0.0f))
        return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(rows, h));
    if (rows == 0) return CM_OK;
    CM_TRY(check_rows(x, x_dtype, ldx, h));
    CM_TRY(check_rows(y, y_dtype, ldy, h));
    if (misaligned(gamma, param_dtype) || misaligned(beta, param_dtype) || misaligned(mean, CM_F32) ||
        misaligned(rstd, CM_F32))
        return CM_ERR_ALIGNMENT;
    NormParams p = {};
    p.x = x;
    p.ldx = ldx;
    p.gamma = gamma;
    p.beta = beta;
    p.p_f32 = param_dtype == CM_F32;
    p.eps = eps;
    p.out = y;
    p.ldo = ldy;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.h = h;
    return launch_layer_norm(p, x_dtype, y_dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? CM_OK
                                                                                                         : CM_ERR_CUDA;
}

size_t cm_layer_norm_backward_workspace_size(int64_t rows, int64_t h) {
    return check_extents(rows, h) == CM_OK ? std::max<size_t>(256, backward_workspace(rows, h)) : 0;
}

cm_status cm_layer_norm_backward(const void *x, cm_dtype x_dtype, int64_t ldx, const void *dy, cm_dtype dy_dtype,
                                 int64_t lddy, const void *gamma, cm_dtype param_dtype, const float *mean,
                                 const float *rstd, const void *residual, int64_t ldr, void *dx, int64_t lddx,
                                 void *dgamma, void *dbeta, cm_dtype grad_dtype, int accumulate, int64_t rows,
                                 int64_t h, void *ws, size_t ws_bytes, cm_stream_t stream_) {
    NvtxRange range("cm_layer_norm_backward");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (bad_dtype(x_dtype) || bad_dtype(dy_dtype) || bad_dtype(param_dtype) || bad_dtype(grad_dtype))
        return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(rows, h));
    if (misaligned(gamma, param_dtype) || misaligned(dgamma, grad_dtype) || misaligned(dbeta, grad_dtype))
        return CM_ERR_ALIGNMENT;
    if (rows == 0) {   // the sums over no rows
        const size_t bytes = size_t(h) * (grad_dtype == CM_F32 ? 4 : 2);
        if (!accumulate && ((dgamma && cudaMemsetAsync(dgamma, 0, bytes, stream) != cudaSuccess) ||
                            (dbeta && cudaMemsetAsync(dbeta, 0, bytes, stream) != cudaSuccess)))
            return CM_ERR_CUDA;
        return CM_OK;
    }
    CM_TRY(check_rows(x, x_dtype, ldx, h));
    CM_TRY(check_rows(dy, dy_dtype, lddy, h));
    CM_TRY(check_rows(dx, x_dtype, lddx, h));
    if (residual) CM_TRY(check_rows(residual, x_dtype, ldr, h));
    if (!mean || !rstd) return CM_ERR_INVALID_ARG;
    if (misaligned(mean, CM_F32) || misaligned(rstd, CM_F32) || (reinterpret_cast<uintptr_t>(ws) & 15u) != 0)
        return CM_ERR_ALIGNMENT;
    if ((dgamma || dbeta) && (!ws || ws_bytes < backward_workspace(rows, h))) return CM_ERR_WORKSPACE;
    NormParams p = {};
    p.x = x;
    p.ldx = ldx;
    p.dy = dy;
    p.lddy = lddy;
    p.gamma = gamma;
    p.p_f32 = param_dtype == CM_F32;
    p.mean = const_cast<float *>(mean);
    p.rstd = const_cast<float *>(rstd);
    p.res = residual;
    p.ldr = ldr;
    p.out = dx;
    p.ldo = lddx;
    p.rows = rows;
    p.h = h;
    p.partial = static_cast<float *>(ws);
    p.dgamma = dgamma;
    p.dbeta = dbeta;
    p.g_f32 = grad_dtype == CM_F32;
    p.accumulate = accumulate != 0;
    return launch_layer_norm_backward(p, x_dtype, dy_dtype, stream) == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

}  // extern "C"
