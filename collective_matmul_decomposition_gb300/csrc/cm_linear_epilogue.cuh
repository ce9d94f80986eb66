// cm_linear_epilogue.cuh -- the activations and their derivatives, in fp32,
// for the epilogues of the linear layer's kernels.
#pragma once

#include <cuda_bf16.h>

#include "cm_linear.cuh"

namespace cm {
namespace lin {
namespace {

// 1 / (1 + exp(-t)): exp's overflow to infinity gives 0, its underflow 1.
// __expf is off by at most 2 + 1.2 |t| units of the last place and the fast
// division by 2: below 2^-20 where 1 / (1 + exp(-t)) is not itself below 2^-8,
// which a bf16 output (2^-9) does not see.
__device__ __forceinline__ float sigmoid(float t) {
    const float d = 1.0f + __expf(-t);
    return d > 1e38f ? 0.0f : __fdividef(1.0f, d);
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float act1(float v, int act) {
    switch (act) {
        case CM_ACT_RELU: return v > 0.0f || v != v ? v : 0.0f;
        case CM_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.7071067811865476f));
        // (1 + tanh u) / 2 = sigmoid(2u)
        case CM_ACT_GELU_TANH: return v * sigmoid(2.0f * kGeluC * (v + kGeluA * v * v * v));
        case CM_ACT_SILU: return v * sigmoid(v);
        default: return v;
    }
}

// the activation's derivative at z
__device__ __forceinline__ float dact1(float z, int act) {
    switch (act) {
        case CM_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case CM_ACT_GELU:
            return 0.5f * (1.0f + erff(z * 0.7071067811865476f)) + z * __expf(-0.5f * z * z) * 0.3989422804014327f;
        case CM_ACT_GELU_TANH: {
            const float s = sigmoid(2.0f * kGeluC * (z + kGeluA * z * z * z));
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
