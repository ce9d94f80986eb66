// cm_adamw.cu -- one AdamW step over many tensors in one launch.
//
//   g = scale grad
//   m = b1 m + (1 - b1) g;   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr decay) - lr/(1 - b1^t) m / (sqrt(v/(1 - b2^t)) + eps)
//
// p is the fp32 master copy where there is one (the bf16 parameter is then its
// rounding), else the parameter itself.  All arithmetic is fp32; b^t and the
// factors made of it come from the host in fp64.
//
// States in 8 bits: m and sqrt(v) in blocks of 256 elements, each an e4m3 code
// times the block's fp32 scale (largest magnitude / 448).  The root is kept
// instead of v because it spans half the powers of two; a positive root never
// gets code 0, which would turn its next update into m / eps.  The update of
// this step uses the unrounded m and v.  Elements that are not finite get the
// NaN code and do not count for the scale; a block whose largest magnitude is
// below 2^-100 is stored as zeros.
//
// Rounding to the nearest code leaves a state where it was when a step moves
// it by less than half a code (3 to 6 % of it), which a slow average (b2 near
// 1) mostly does; only its block's scale then follows the gradients.  With a
// seed the codes are rounded up or down with the chances that keep their
// mean, from a hash of the seed, the tensor's place in the list and the
// element's index, so that averages move however small the steps.
//
// Bound by memory: 28 bytes an element with bf16 gradients and parameters, a
// master copy and fp32 states, 16.06 with 8-bit states.  A warp takes a block
// of 256 elements, a thread 8 neighbours of it, all its loads before the first
// use.  The tensors' addresses are kernel parameters, so a step needs no copy
// of a table to the device.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cm_internal.h"

namespace cm {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kBlock = CM_ADAMW_BLOCK;
constexpr int kAdamThreads = 256;
constexpr int64_t kAdamChunk = int64_t(kAdamThreads) * 8;   // elements a CTA updates
constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100

struct Entry {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    float *ms, *vs;
    int64_t numel;
    float keep;           // 1 - lr * weight_decay
    int32_t first_chunk;  // of this launch
    uint32_t index;       // in the caller's list
    uint8_t param_f32, grad_f32, bits8, vec;
};

// The launch with few tensors copies a small table.
template <int CAP>
struct Table {
    Entry e[CAP];
    int count;
    float b1, b2, c1, c2;   // betas and 1 - beta
    float step, root_scale, eps;   // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    const float *grad_scale;
    uint32_t seed_lo, seed_hi;
    bool seeded;
};

__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void load8(const bf16 *p, float (&f)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(bf16 *p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float decode(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
// The code nearest to v (already divided by the scale), ties to even; |v| <= 448.
__device__ __forceinline__ uint8_t encode(float v) {
    return uint8_t(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}

// Whether the thread's 8 elements can go in whole vectors.
struct Span {
    int64_t i0;
    int n;      // 0..8 elements of the tensor
    bool vec;
};

template <typename T>
__device__ __forceinline__ void get(const T *p, const Span &s, float (&f)[8]) {
    if (s.vec) {
        load8(p + s.i0, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < s.n ? float(p[s.i0 + i]) : 0.0f;
    }
}
__device__ __forceinline__ void put(float *p, const Span &s, const float (&f)[8]) {
    if (s.vec) {
        store8(p + s.i0, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < s.n) p[s.i0 + i] = f[i];
    }
}
__device__ __forceinline__ void put(bf16 *p, const Span &s, const float (&f)[8]) {
    if (s.vec) {
        store8(p + s.i0, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < s.n) p[s.i0 + i] = __float2bfloat16_rn(f[i]);
    }
}
__device__ __forceinline__ void get_codes(const uint8_t *p, const Span &s, uint8_t (&c)[8]) {
    if (s.vec) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p + s.i0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = uint8_t(w.x >> (8 * i));
            c[4 + i] = uint8_t(w.y >> (8 * i));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = i < s.n ? p[s.i0 + i] : uint8_t(0);
    }
}

// 32 mixed bits of a counter (the finalizer of MurmurHash3).
__device__ __forceinline__ uint32_t mix(uint32_t h) {
    h ^= h >> 16;
    h *= 0x85ebca6bu;
    h ^= h >> 13;
    h *= 0xc2b2ae35u;
    return h ^ (h >> 16);
}

// The neighbouring e4m3 values of v (finite, |v| <= 448), the upper one with the chance
// that keeps the mean; u: 16 random bits.  Normal values keep 3 bits of fp32's
// 23; below 2^-6 the step is 2^-9.
__device__ __forceinline__ float dither(float v, uint32_t u) {
    if (fabsf(v) >= 0.015625f) {
        const uint32_t b = __float_as_uint(v);
        return __uint_as_float((b + (u << 4)) & 0xfff00000u);
    }
    return copysignf(floorf(fabsf(v) * 512.0f + float(u) * 0x1p-16f) * 0x1p-9f, v);
}

// Quantise the warp's block: codes and scale of the 256 values its threads
// hold.  `bits`: 16 random bits an element where the rounding is seeded.
template <bool ROOT>
__device__ __forceinline__ void put_codes(uint8_t *p, float *scale, const Span &s, const float (&f)[8], bool seeded,
                                          const uint32_t (&bits)[8]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < s.n && isfinite(f[i])) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const bool live = amax >= kTiny;
    const float inv = live ? __fmul_rn(1.0f / amax, kE4m3Max) : 0.0f;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // the block's largest value times inv may end one unit above 448; the codes end there
        float x = fminf(fmaxf(f[i] * inv, -kE4m3Max), kE4m3Max);
        if (seeded) x = dither(x, ROOT ? bits[i] >> 16 : bits[i] & 0xffffu);
        uint8_t c = isfinite(f[i]) ? encode(x) : uint8_t(0x7f);
        if (ROOT && live && c == 0 && f[i] > 0.0f) c = 1;
        w[i >> 2] |= uint32_t(c) << (8 * (i & 3));
    }
    if (s.vec) {
        *reinterpret_cast<uint2 *>(p + s.i0) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < s.n) p[s.i0 + i] = uint8_t(w[i >> 2] >> (8 * (i & 3)));
    }
    if ((threadIdx.x & 31) == 0 && s.n > 0) *scale = live ? amax * (1.0f / kE4m3Max) : 0.0f;
}

template <int CAP>
__global__ void __launch_bounds__(kAdamThreads) cm_adamw_kernel(const __grid_constant__ Table<CAP> t) {
    // the tensor of this chunk: the last one that starts at or before it
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].first_chunk <= int(blockIdx.x)) lo = mid; else hi = mid - 1;
    }
    const Entry &e = t.e[lo];
    Span s;
    s.i0 = int64_t(int(blockIdx.x) - e.first_chunk) * kAdamChunk + int64_t(threadIdx.x) * 8;
    s.n = int(max(int64_t(0), min(int64_t(8), e.numel - s.i0)));
    s.vec = e.vec && s.n == 8;
    const int64_t block = s.i0 / kBlock;
    const float scale = t.grad_scale ? *t.grad_scale : 1.0f;

    float g[8], p[8], m[8], v[8], root[8];
    if (e.grad_f32) get(static_cast<const float *>(e.grad), s, g);
    else get(static_cast<const bf16 *>(e.grad), s, g);
    if (e.master) get(e.master, s, p);
    else if (e.param_f32) get(static_cast<const float *>(e.param), s, p);
    else get(static_cast<const bf16 *>(e.param), s, p);
    if (e.bits8) {
        uint8_t cm[8], cv[8];
        get_codes(static_cast<const uint8_t *>(e.m), s, cm);
        get_codes(static_cast<const uint8_t *>(e.v), s, cv);
        const float sm = s.n ? e.ms[block] : 0.0f, sv = s.n ? e.vs[block] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = decode(cm[i]) * sm;
            const float r = decode(cv[i]) * sv;
            v[i] = r * r;
        }
    } else {
        get(static_cast<const float *>(e.m), s, m);
        get(static_cast<const float *>(e.v), s, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gi = g[i] * scale;
        // rounded one by one, not contracted: a code must not depend on how
        // the compiler groups a sum that lies on the border between two
        m[i] = __fadd_rn(__fmul_rn(t.b1, m[i]), __fmul_rn(t.c1, gi));
        v[i] = __fadd_rn(__fmul_rn(t.b2, v[i]), __fmul_rn(__fmul_rn(t.c2, gi), gi));
        root[i] = sqrtf(v[i]);
        p[i] = p[i] * e.keep - t.step * m[i] / (root[i] * t.root_scale + t.eps);
    }
    if (e.master) put(e.master, s, p);
    if (e.param_f32) put(static_cast<float *>(e.param), s, p);
    else put(static_cast<bf16 *>(e.param), s, p);
    if (e.bits8) {
        __syncwarp();   // every lane has read the block's old scales
        uint32_t bits[8];
        if (t.seeded) {
            const uint32_t key = mix(mix(uint32_t(s.i0 >> 32) + t.seed_hi) ^ (e.index + t.seed_lo));
#pragma unroll
            for (int i = 0; i < 8; ++i) bits[i] = mix((uint32_t(s.i0) + uint32_t(i)) ^ key);
        }
        put_codes<false>(static_cast<uint8_t *>(e.m), e.ms + block, s, m, t.seeded, bits);
        put_codes<true>(static_cast<uint8_t *>(e.v), e.vs + block, s, root, t.seeded, bits);
    } else {
        put(static_cast<float *>(e.m), s, m);
        put(static_cast<float *>(e.v), s, v);
    }
}

constexpr int kSmallTable = 32, kLargeTable = 360;
static_assert(sizeof(Table<kLargeTable>) <= 32764, "kernel parameters");

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int CAP>
cudaError_t launch(const Table<kLargeTable> &all, int64_t chunks, cudaStream_t stream) {
    Table<CAP> t;
    std::copy(all.e, all.e + all.count, t.e);
    t.count = all.count;
    t.b1 = all.b1, t.b2 = all.b2, t.c1 = all.c1, t.c2 = all.c2;
    t.step = all.step, t.root_scale = all.root_scale, t.eps = all.eps;
    t.grad_scale = all.grad_scale;
    t.seed_lo = all.seed_lo, t.seed_hi = all.seed_hi, t.seeded = all.seeded;
    cm_adamw_kernel<CAP><<<unsigned(chunks), kAdamThreads, 0, stream>>>(t);
    return cudaGetLastError();
}

cm_status check_tensor(const cm_adamw_tensor &x) {
    if ((x.param_dtype != CM_BF16 && x.param_dtype != CM_F32) || (x.grad_dtype != CM_BF16 && x.grad_dtype != CM_F32) ||
        (x.state_bits != 32 && x.state_bits != 8))
        return CM_ERR_INVALID_ARG;
    if (x.numel < 0 || x.numel > (int64_t(1) << 42)) return CM_ERR_SHAPE;
    if (x.numel == 0) return CM_OK;
    if (!x.param || !x.grad || !x.exp_avg || !x.exp_avg_sq) return CM_ERR_INVALID_ARG;
    if (x.state_bits == 8 && (!x.exp_avg_scale || !x.exp_avg_sq_scale)) return CM_ERR_INVALID_ARG;
    if (!aligned(x.param, x.param_dtype == CM_F32 ? 4 : 2) || !aligned(x.grad, x.grad_dtype == CM_F32 ? 4 : 2) ||
        !aligned(x.master, 4) || (x.state_bits == 32 && (!aligned(x.exp_avg, 4) || !aligned(x.exp_avg_sq, 4))) ||
        !aligned(x.exp_avg_scale, 4) || !aligned(x.exp_avg_sq_scale, 4))
        return CM_ERR_ALIGNMENT;
    return CM_OK;
}

}  // namespace
}  // namespace cm

using namespace cm;

extern "C" cm_status cm_adamw(const cm_adamw_tensor *tensors, int count, double lr, double beta1, double beta2,
                              double eps, int64_t step, const float *grad_scale, uint64_t seed,
                              cm_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    nvtxRangePushA("cm_adamw");
    struct Pop {
        ~Pop() { nvtxRangePop(); }
    } pop;
    if (count < 0 || (count > 0 && !tensors) || step < 1 || !std::isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) ||
        !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(eps) || !aligned(grad_scale, 4))
        return CM_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const cm_status st = check_tensor(tensors[i]);
        if (st != CM_OK) return st;
    }
    Table<kLargeTable> t;
    t.b1 = float(beta1), t.b2 = float(beta2), t.c1 = float(1.0 - beta1), t.c2 = float(1.0 - beta2);
    t.step = float(lr / (1.0 - std::pow(beta1, double(step))));
    t.root_scale = float(1.0 / std::sqrt(1.0 - std::pow(beta2, double(step))));
    t.eps = float(eps);
    t.grad_scale = grad_scale;
    t.seed_lo = uint32_t(seed), t.seed_hi = uint32_t(seed >> 32), t.seeded = seed != 0;
    int i = 0;
    while (i < count) {
        int64_t chunks = 0;
        t.count = 0;
        for (; i < count && t.count < kLargeTable; ++i) {
            const cm_adamw_tensor &x = tensors[i];
            if (x.numel == 0) continue;
            const int64_t c = (x.numel + kAdamChunk - 1) / kAdamChunk;
            if (chunks + c > 0x7fffffff) break;
            Entry &e = t.e[t.count++];
            e = {x.param, x.grad, x.master, x.exp_avg, x.exp_avg_sq, x.exp_avg_scale, x.exp_avg_sq_scale, x.numel};
            e.keep = float(1.0 - lr * double(x.weight_decay));
            e.first_chunk = int32_t(chunks);
            e.index = uint32_t(i);
            e.param_f32 = x.param_dtype == CM_F32;
            e.grad_f32 = x.grad_dtype == CM_F32;
            e.bits8 = x.state_bits == 8;
            const uintptr_t state = x.state_bits == 8 ? 8 : 16;
            e.vec = aligned(x.param, 16) && aligned(x.grad, 16) && aligned(x.master, 16) && aligned(x.exp_avg, state) &&
                    aligned(x.exp_avg_sq, state);
            chunks += c;
        }
        if (t.count == 0) continue;
        const cudaError_t err = t.count <= kSmallTable ? launch<kSmallTable>(t, chunks, stream)
                                                       : launch<kLargeTable>(t, chunks, stream);
        if (err != cudaSuccess) return CM_ERR_CUDA;
    }
    return CM_OK;
}
