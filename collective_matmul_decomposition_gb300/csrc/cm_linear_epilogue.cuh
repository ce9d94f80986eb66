// cm_linear_epilogue.cuh -- the activations and their derivatives, in fp32,
// for the epilogues of the linear layer's kernels.
#pragma once

#include <cuda_bf16.h>

#include "cm_linear.cuh"
#include "cm_vec.cuh"

namespace cm {
namespace lin {
namespace {

using namespace vec;

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
__device__ __forceinline__ F2 exp2_fast(F2 a) {
    const float2 p = parts(a);
    return pair(exp2_fast(p.x), exp2_fast(p.y));
}
__device__ __forceinline__ F2 rcp_fast(F2 a) {
    const float2 p = parts(a);
    return pair(rcp_fast(p.x), rcp_fast(p.y));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + exp(-t)), given a = -t log2(e).  The rounding of a costs |a| 2^-24
// of the result at most: below 2^-19 where the result is not itself below
// 2^-24, which a bf16 output (2^-8) does not see.
__device__ __forceinline__ F2 sigmoid_of(F2 a) { return rcp_fast(add(both(1.0f), exp2_fast(a))); }
// (1 + tanh u) / 2 = sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3); v2 = v^2
__device__ __forceinline__ F2 gelu_tanh_gate(F2 v, F2 v2) {
    constexpr float k = -2.0f * kLog2e * kGeluC;
    return sigmoid_of(mul(v, fma(v2, both(k * kGeluA), both(k))));
}
// The normal distribution's integral up to v, and e = exp(-v^2 / 2).  The near
// tail is t q(t) e with t = 1 / (1 + p |v|), the form of formula 7.1.26 of
// Abramowitz and Stegun's Handbook of Mathematical Functions, with eight
// coefficients instead of its five, fitted here for the least relative error
// (linear programming over 0 <= |v| <= 14): 9.5e-8, so that GELU keeps its
// accuracy where it is small, which the handbook's absolute 1.5e-7 does not
// (5e-4 of the value at v = -4, 1e-2 at -8).  What is left is the rounding of
// the exponent, at most 1.5 v^2 2^-24.
__device__ __forceinline__ F2 normal_cdf(F2 v, F2 &e) {
    const float2 s = parts(v);
    constexpr float p = 0.30405593f;
    const F2 t = rcp_fast(pair(fmaf(p, fabsf(s.x), 1.0f), fmaf(p, fabsf(s.y), 1.0f)));
    e = exp2_fast(mul(mul(v, v), both(-0.5f * kLog2e)));
    F2 q = fma(t, both(0.036636885f), both(-0.15430708f));
    q = fma(t, q, both(0.19037811f));
    q = fma(t, q, both(-0.0415411f));
    q = fma(t, q, both(0.122740515f));
    q = fma(t, q, both(0.102677226f));
    q = fma(t, q, both(0.12215613f));
    q = fma(t, q, both(0.12125933f));
    const float2 h = parts(mul(mul(q, t), e));
    return pair(s.x < 0.0f ? h.x : 1.0f - h.x, s.y < 0.0f ? h.y : 1.0f - h.y);
}

// act(v) of a pair
template <int ACT>
__device__ __forceinline__ F2 act2(F2 v) {
    if constexpr (ACT == CM_ACT_RELU) {
        const float2 s = parts(v);
        return pair(s.x > 0.0f || s.x != s.x ? s.x : 0.0f, s.y > 0.0f || s.y != s.y ? s.y : 0.0f);
    } else if constexpr (ACT == CM_ACT_GELU) {
        F2 e;
        return mul(v, normal_cdf(v, e));
    } else if constexpr (ACT == CM_ACT_GELU_TANH) {
        return mul(v, gelu_tanh_gate(v, mul(v, v)));
    } else if constexpr (ACT == CM_ACT_SILU) {
        return mul(v, sigmoid_of(mul(v, both(-kLog2e))));
    } else {
        return v;
    }
}

// act'(z) of a pair
template <int ACT>
__device__ __forceinline__ F2 dact2(F2 z) {
    if constexpr (ACT == CM_ACT_RELU) {
        const float2 s = parts(z);
        return pair(s.x > 0.0f ? 1.0f : 0.0f, s.y > 0.0f ? 1.0f : 0.0f);
    } else if constexpr (ACT == CM_ACT_GELU) {
        F2 e;
        const F2 cdf = normal_cdf(z, e);
        return fma(mul(z, both(0.3989422804014327f)), e, cdf);
    } else if constexpr (ACT == CM_ACT_GELU_TANH) {
        // s + z s (1 - s) 2u'.  Past |z| = 2^32, where s is 0 or 1 and the second
        // term nothing, z^2 is held: it must not overflow to meet 1 - s = 0
        const float2 sq = parts(mul(z, z));
        const F2 z2 = pair(fminf(sq.x, 0x1p64f), fminf(sq.y, 0x1p64f)), s = gelu_tanh_gate(z, z2);
        const F2 du = fma(z2, both(6.0f * kGeluC * kGeluA), both(2.0f * kGeluC));
        return fma(mul(z, s), mul(fma(s, both(-1.0f), both(1.0f)), du), s);
    } else if constexpr (ACT == CM_ACT_SILU) {
        const F2 s = sigmoid_of(mul(z, both(-kLog2e)));
        return mul(s, fma(z, fma(s, both(-1.0f), both(1.0f)), both(1.0f)));
    } else {
        return both(1.0f);
    }
}

template <int ACT, int N>
__device__ __forceinline__ void act_loop(float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 r = parts(act2<ACT>(pair(f[i], f[i + 1])));
        f[i] = r.x;
        f[i + 1] = r.y;
    }
}
template <int ACT, int N>
__device__ __forceinline__ void dact_loop(float (&f)[N], const float (&z)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 r = parts(mul(pair(f[i], f[i + 1]), dact2<ACT>(pair(z[i], z[i + 1]))));
        f[i] = r.x;
        f[i + 1] = r.y;
    }
}

// f = act(f), and f *= act'(z); the choice of activation outside the loop.
template <int N>
__device__ __forceinline__ void apply_act(float (&f)[N], int act) {
    switch (act) {
        case CM_ACT_RELU: act_loop<CM_ACT_RELU>(f); break;
        case CM_ACT_GELU: act_loop<CM_ACT_GELU>(f); break;
        case CM_ACT_GELU_TANH: act_loop<CM_ACT_GELU_TANH>(f); break;
        case CM_ACT_SILU: act_loop<CM_ACT_SILU>(f); break;
        default: break;
    }
}
template <int N>
__device__ __forceinline__ void mul_dact(float (&f)[N], const float (&z)[N], int act) {
    switch (act) {
        case CM_ACT_RELU: dact_loop<CM_ACT_RELU>(f, z); break;
        case CM_ACT_GELU: dact_loop<CM_ACT_GELU>(f, z); break;
        case CM_ACT_GELU_TANH: dact_loop<CM_ACT_GELU_TANH>(f, z); break;
        case CM_ACT_SILU: dact_loop<CM_ACT_SILU>(f, z); break;
        default: break;
    }
}

// act(z) and act'(z) of a pair, by the same steps as act2 and dact2 but with their common
// exponential and reciprocal taken once.
template <int ACT>
__device__ __forceinline__ F2 act_and_slope(F2 z, F2 &slope) {
    if constexpr (ACT == CM_ACT_GELU) {
        F2 e;
        const F2 cdf = normal_cdf(z, e);
        slope = fma(mul(z, both(0.3989422804014327f)), e, cdf);
        return mul(z, cdf);
    } else if constexpr (ACT == CM_ACT_GELU_TANH) {
        const float2 sq = parts(mul(z, z));   // held as in dact2
        const F2 z2 = pair(fminf(sq.x, 0x1p64f), fminf(sq.y, 0x1p64f)), s = gelu_tanh_gate(z, z2);
        const F2 du = fma(z2, both(6.0f * kGeluC * kGeluA), both(2.0f * kGeluC)), zs = mul(z, s);
        slope = fma(zs, mul(fma(s, both(-1.0f), both(1.0f)), du), s);
        return zs;
    } else if constexpr (ACT == CM_ACT_SILU) {
        const F2 s = sigmoid_of(mul(z, both(-kLog2e)));
        slope = mul(s, fma(z, fma(s, both(-1.0f), both(1.0f)), both(1.0f)));
        return mul(z, s);
    } else {
        slope = dact2<ACT>(z);
        return act2<ACT>(z);
    }
}

// g becomes act(g) u.
template <int ACT, int N>
__device__ __forceinline__ void gate_loop(float (&g)[N], const float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 r = parts(mul(act2<ACT>(pair(g[i], g[i + 1])), pair(u[i], u[i + 1])));
        g[i] = r.x;
        g[i + 1] = r.y;
    }
}
template <int N>
__device__ __forceinline__ void apply_gate(float (&g)[N], const float (&u)[N], int act) {
    switch (act) {
        case CM_ACT_RELU: gate_loop<CM_ACT_RELU>(g, u); break;
        case CM_ACT_GELU: gate_loop<CM_ACT_GELU>(g, u); break;
        case CM_ACT_GELU_TANH: gate_loop<CM_ACT_GELU_TANH>(g, u); break;
        case CM_ACT_SILU: gate_loop<CM_ACT_SILU>(g, u); break;
        default: gate_loop<CM_ACT_NONE>(g, u); break;
    }
}
// From d, the gradient of act(g) u: g becomes d u act'(g), its own gradient, and u becomes d act(g).
template <int ACT, int N>
__device__ __forceinline__ void gate_grad_loop(const float (&d)[N], float (&g)[N], float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const F2 dd = pair(d[i], d[i + 1]);
        F2 slope;
        const F2 a = act_and_slope<ACT>(pair(g[i], g[i + 1]), slope);
        const float2 dg = parts(mul(mul(dd, pair(u[i], u[i + 1])), slope)), du = parts(mul(dd, a));
        g[i] = dg.x, g[i + 1] = dg.y;
        u[i] = du.x, u[i + 1] = du.y;
    }
}
template <int N>
__device__ __forceinline__ void gate_grad(const float (&d)[N], float (&g)[N], float (&u)[N], int act) {
    switch (act) {
        case CM_ACT_RELU: gate_grad_loop<CM_ACT_RELU>(d, g, u); break;
        case CM_ACT_GELU: gate_grad_loop<CM_ACT_GELU>(d, g, u); break;
        case CM_ACT_GELU_TANH: gate_grad_loop<CM_ACT_GELU_TANH>(d, g, u); break;
        case CM_ACT_SILU: gate_grad_loop<CM_ACT_SILU>(d, g, u); break;
        default: gate_grad_loop<CM_ACT_NONE>(d, g, u); break;
    }
}

__device__ __forceinline__ float load_bias(const void *bias, int f32, int64_t c) {
    if (!bias) return 0.0f;
    return f32 ? static_cast<const float *>(bias)[c] : __bfloat162float(static_cast<const __nv_bfloat16 *>(bias)[c]);
}
__device__ __forceinline__ float load_bias(const LinearEpilogue &e, int64_t c) {
    if (!e.bias) return 0.0f;
    return e.bias_f32 ? static_cast<const float *>(e.bias)[c]
                      : __bfloat162float(static_cast<const __nv_bfloat16 *>(e.bias)[c]);
}

}  // namespace
}  // namespace lin
}  // namespace cm
