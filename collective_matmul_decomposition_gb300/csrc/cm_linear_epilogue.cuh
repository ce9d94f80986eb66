// cm_linear_epilogue.cuh -- the activations and their derivatives, in fp32,
// for the epilogues of the linear layer's kernels.
#pragma once

#include <cuda_bf16.h>

#include "cm_linear.cuh"

namespace cm {
namespace lin {
namespace {

// 2^a and 1 / a by the special-function unit, within two units of the last
// place of fp32; 2^a overflows to infinity, whose reciprocal is 0.
__device__ __forceinline__ float exp2_fast(float a) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
__device__ __forceinline__ float rcp_fast(float a) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
// 1 / (1 + exp(-t)), given a = -t log2(e).  The rounding of a costs |a| 2^-24
// of the result at most: below 2^-19 where the result is not itself below
// 2^-24, which a bf16 output (2^-8) does not see.
__device__ __forceinline__ float sigmoid_of(float a) { return rcp_fast(1.0f + exp2_fast(a)); }
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid(float t) { return sigmoid_of(-kLog2e * t); }

// The normal distribution's integral up to v, and exp(-v^2 / 2).  By formula
// 7.1.26 of Abramowitz and Stegun's Handbook of Mathematical Functions, whose
// error is at most 1.5e-7: erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2) with
// t = 1 / (1 + p x), for x = |v| / sqrt 2.  A third of erff's instructions.
__device__ __forceinline__ float normal_cdf(float v, float &e) {
    const float x = fabsf(v) * 0.7071067811865476f;
    e = exp2_fast(-0.5f * kLog2e * (v * v));
    const float t = rcp_fast(fmaf(0.3275911f, x, 1.0f));
    const float q = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
    const float half = 0.5f * q * e;   // of erfc
    return v < 0.0f ? half : 1.0f - half;
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float act1(float v, int act) {
    switch (act) {
        case CM_ACT_RELU: return v > 0.0f || v != v ? v : 0.0f;
        case CM_ACT_GELU: {
            float e;
            return v * normal_cdf(v, e);
        }
        // (1 + tanh u) / 2 = sigmoid(2u)
        case CM_ACT_GELU_TANH:
            return v * sigmoid_of(v * (-2.0f * kLog2e * kGeluC + -2.0f * kLog2e * kGeluC * kGeluA * (v * v)));
        case CM_ACT_SILU: return v * sigmoid(v);
        default: return v;
    }
}

// the activation's derivative at z
__device__ __forceinline__ float dact1(float z, int act) {
    switch (act) {
        case CM_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case CM_ACT_GELU: {
            float e;
            const float cdf = normal_cdf(z, e);
            return cdf + z * e * 0.3989422804014327f;
        }
        case CM_ACT_GELU_TANH: {
            const float s = sigmoid_of(z * (-2.0f * kLog2e * kGeluC + -2.0f * kLog2e * kGeluC * kGeluA * (z * z)));
            return s + 2.0f * z * s * (1.0f - s) * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
        }
        case CM_ACT_SILU: {
            const float s = sigmoid(z);
            return s * (1.0f + z * (1.0f - s));
        }
        default: return 1.0f;
    }
}

// The same over a slice, the choice outside the loop.
template <int N>
__device__ __forceinline__ void apply_act(float (&f)[N], int act) {
    switch (act) {
        case CM_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = act1(f[i], CM_ACT_RELU);
            break;
        case CM_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = act1(f[i], CM_ACT_GELU);
            break;
        case CM_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = act1(f[i], CM_ACT_GELU_TANH);
            break;
        case CM_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = act1(f[i], CM_ACT_SILU);
            break;
        default: break;
    }
}
template <int N>
__device__ __forceinline__ void mul_dact(float (&f)[N], const float (&z)[N], int act) {
    switch (act) {
        case CM_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] *= dact1(z[i], CM_ACT_RELU);
            break;
        case CM_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] *= dact1(z[i], CM_ACT_GELU);
            break;
        case CM_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] *= dact1(z[i], CM_ACT_GELU_TANH);
            break;
        case CM_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] *= dact1(z[i], CM_ACT_SILU);
            break;
        default: break;
    }
}

__device__ __forceinline__ float load_bias(const LinearEpilogue &e, int64_t c) {
    if (!e.bias) return 0.0f;
    return e.bias_f32 ? static_cast<const float *>(e.bias)[c]
                      : __bfloat162float(static_cast<const __nv_bfloat16 *>(e.bias)[c]);
}

}  // namespace
}  // namespace lin
}  // namespace cm
