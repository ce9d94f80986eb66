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
// element's index, so that averages move however small the steps.  It costs 8 %
// (50 M elements: 183 us).
//
// Bound by memory: 28 bytes an element with bf16 gradients and parameters, a
// master copy and fp32 states (59 M elements: 239 us, the rate of a copy), 16.06
// with 8-bit states (50 M with fp32 gradients, 18.06: 168 us, 5.4 TB/s; there the
// passes' arithmetic is not wholly under other warps' loads).  A warp takes a block
// of 256 elements, a thread 8 neighbours of it, all its loads before the first
// use.  The tensors' addresses are kernel parameters, so a step needs no copy
// of a table to the device.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cm_internal.h"
#include "cm_launch.cuh"
#include "cm_vec.cuh"

namespace cm {
namespace {

constexpr int kBlock = CM_ADAMW_BLOCK;
constexpr int kAdamThreads = 256;
constexpr int kAdamPass = kAdamThreads * 8;             // elements a CTA updates at a time
// Passes of a CTA.  Four with codes, whose passes are long on arithmetic: finding
// the tensor is paid once for them (50 M elements: 168 us, with one pass 180);
// one without, where four would only put loads behind stores (59 M elements:
// 4 % slower).
constexpr int kCodePasses = 4;
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
    uint32_t seed_key;   // of the seed's two halves
    bool seeded;
};

using namespace vec;

// A thread's 8 elements: the first one's index, how many belong to the tensor,
// and whether they can go in whole vectors.
struct Span {
    int64_t i0;
    int n;
    bool vec;
};

template <typename T>
__device__ __forceinline__ V8 get(const T *p, const Span &s) {
    if (s.vec) return load8(p + s.i0);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < s.n ? to_f(p[s.i0 + i]) : 0.0f;
    return {{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
}
template <typename T>
__device__ __forceinline__ void put(T *p, const Span &s, const V8 &v) {
    if (s.vec) {
        store8(p + s.i0, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = parts(v.p[i]);
        if (2 * i < s.n) from_f(p + s.i0 + 2 * i, q.x);
        if (2 * i + 1 < s.n) from_f(p + s.i0 + 2 * i + 1, q.y);
    }
}

// The values of 8 codes times their scale.
__device__ __forceinline__ V8 get_codes(const uint8_t *p, const Span &s, float scale) {
    uint2 w = make_uint2(0u, 0u);
    if (s.vec) {
        w = *reinterpret_cast<const uint2 *>(p + s.i0);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < s.n) (i < 4 ? w.x : w.y) |= uint32_t(p[s.i0 + i]) << (8 * (i & 3));
    }
    V8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t q = (i < 2 ? w.x : w.y) >> (16 * (i & 1));
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(q & 0xffffu), __NV_E4M3)));
        v.p[i] = mul(pair(f.x, f.y), both(scale));
    }
    return v;
}
// The two nearest codes, ties to even; beyond 448 the largest, not a number the NaN code.
__device__ __forceinline__ uint32_t encode2(float a, float b) {
    return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// 32 mixed bits of a counter (the finalizer of MurmurHash3).  The random bits of
// an element come from the seed, the tensor's place in the list and the index
// in turn, each added to what the one before was mixed to: were they added up
// unmixed, a tensor would get the bits that its neighbour had a seed earlier.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t h) {
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
// hold (zeros behind the tensor's end).  ROOT: a positive value keeps a code
// above zero.  `bits`: 16 random bits an element where the rounding is seeded.
template <bool ROOT>
__device__ __forceinline__ void put_codes(uint8_t *p, float *scale, const Span &s, const V8 &v, bool seeded,
                                          const uint32_t (&bits)[8]) {
    float f[8];
    // magnitudes order as their bits do, and what is not finite lies above them
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = parts(v.p[i]);
        f[2 * i] = q.x;
        f[2 * i + 1] = q.y;
        top = max(top, max(__float_as_uint(q.x) & 0x7fffffffu, __float_as_uint(q.y) & 0x7fffffffu));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const bool odd = top >= 0x7f800000u;   // somewhere in the block
    if (odd) {
        top = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (isfinite(f[i])) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
    }
    const float amax = __uint_as_float(top);
    const bool live = amax >= kTiny;
    const float inv = live ? __fmul_rn(1.0f / amax, kE4m3Max) : 0.0f;
    const float least = live ? 0x1p-9f : 0.0f;   // the smallest code's value
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float a = f[2 * i + k];
            x[k] = a * inv;
            if (seeded) x[k] = dither(fminf(fmaxf(x[k], -kE4m3Max), kE4m3Max), ROOT ? bits[2 * i + k] >> 16 : bits[2 * i + k] & 0xffffu);
            if (ROOT) x[k] = a > 0.0f ? fmaxf(x[k], least) : 0.0f;
            if (odd && !isfinite(a)) x[k] = __uint_as_float(0x7fffffffu);
        }
        w[i] = encode2(x[0], x[1]);
    }
    const uint2 c = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    if (s.vec) {
        *reinterpret_cast<uint2 *>(p + s.i0) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < s.n) p[s.i0 + i] = uint8_t((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
    if ((threadIdx.x & 31) == 0 && s.n > 0) *scale = live ? amax * (1.0f / kE4m3Max) : 0.0f;
}

// CODES: some tensor of the table has 8-bit states, each by its own flag.  A
// table without any runs without that path's registers (59 M elements with fp32
// states: 2 % slower with the path).  Five CTAs an SM: with
// four or six, 8-bit steps were 10 and 4 % slower.
template <int CAP, bool CODES>
__global__ void __launch_bounds__(kAdamThreads, 5) cm_adamw_kernel(const __grid_constant__ Table<CAP> t) {
    let_next_start();
    wait_for_previous();
    // the tensor of this chunk: the last one that starts at or before it
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].first_chunk <= int(blockIdx.x)) lo = mid; else hi = mid - 1;
    }
    const std::conditional_t<CODES, Entry, const Entry &> e = t.e[lo];
    const F2 scale = both(t.grad_scale ? *t.grad_scale : 1.0f);
    Span s;
    constexpr int kPasses = CODES ? kCodePasses : 1;
    s.i0 = int64_t(int(blockIdx.x) - e.first_chunk) * (kPasses * kAdamPass) + int64_t(threadIdx.x) * 8;
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass, s.i0 += kAdamPass) {
        if (s.i0 - int64_t(threadIdx.x & 31) * 8 >= e.numel) break;   // by warps: a block's threads stay together
        s.n = int(max(int64_t(0), min(int64_t(8), e.numel - s.i0)));
        s.vec = e.vec && s.n == 8;
        const int64_t block = s.i0 / kBlock;
        V8 g = e.grad_f32 ? get(static_cast<const float *>(e.grad), s) : get(static_cast<const bf16 *>(e.grad), s);
        V8 p = e.master ? get(e.master, s)
               : e.param_f32 ? get(static_cast<const float *>(e.param), s) : get(static_cast<const bf16 *>(e.param), s);
        V8 m, v, root;
        if (CODES && e.bits8) {
            m = get_codes(static_cast<const uint8_t *>(e.m), s, s.n ? e.ms[block] : 0.0f);
            v = get_codes(static_cast<const uint8_t *>(e.v), s, s.n ? e.vs[block] : 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) v.p[i] = mul(v.p[i], v.p[i]);
        } else {
            m = get(static_cast<const float *>(e.m), s);
            v = get(static_cast<const float *>(e.v), s);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 gi = mul(g.p[i], scale);
            // rounded one by one, not fused (which pairs would be): a code must not
            // depend on how a sum that lies on the border between two is grouped
            const float2 gs = parts(gi), ms = parts(m.p[i]), vs = parts(v.p[i]);
            m.p[i] = pair(__fadd_rn(__fmul_rn(t.b1, ms.x), __fmul_rn(t.c1, gs.x)),
                          __fadd_rn(__fmul_rn(t.b1, ms.y), __fmul_rn(t.c1, gs.y)));
            v.p[i] = pair(__fadd_rn(__fmul_rn(t.b2, vs.x), __fmul_rn(__fmul_rn(t.c2, gs.x), gs.x)),
                          __fadd_rn(__fmul_rn(t.b2, vs.y), __fmul_rn(__fmul_rn(t.c2, gs.y), gs.y)));
            const float2 q = parts(v.p[i]), num = parts(mul(both(t.step), m.p[i]));
            const float2 r = make_float2(sqrtf(q.x), sqrtf(q.y));
            root.p[i] = pair(r.x, r.y);
            // the fast division is off by two units of the update's last place
            const float2 den = parts(fma(root.p[i], both(t.root_scale), both(t.eps)));
            p.p[i] = fma(p.p[i], both(e.keep), pair(-__fdividef(num.x, den.x), -__fdividef(num.y, den.y)));
        }
        if (e.master) put(e.master, s, p);
        if (e.param_f32) put(static_cast<float *>(e.param), s, p);
        else put(static_cast<bf16 *>(e.param), s, p);
        if (CODES && e.bits8) {
            __syncwarp();   // every lane has read the block's old scales
            uint32_t bits[8] = {};
            if (t.seeded) {
                const uint32_t key = mix(mix(t.seed_key + e.index) + uint32_t(s.i0 >> 32));
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
}

constexpr int kSmallTable = 32, kLargeTable = 360;
static_assert(sizeof(Table<kLargeTable>) <= 32764, "kernel parameters");

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int CAP>
cudaError_t launch(const Table<kLargeTable> &all, bool codes, int64_t chunks, cudaStream_t stream) {
    Table<CAP> t;
    std::copy(all.e, all.e + all.count, t.e);
    t.count = all.count;
    t.b1 = all.b1, t.b2 = all.b2, t.c1 = all.c1, t.c2 = all.c2;
    t.step = all.step, t.root_scale = all.root_scale, t.eps = all.eps;
    t.grad_scale = all.grad_scale;
    t.seed_key = all.seed_key, t.seeded = all.seeded;
    return launch_after(codes ? cm_adamw_kernel<CAP, true> : cm_adamw_kernel<CAP, false>, dim3(unsigned(chunks)),
                        kAdamThreads, 0, 1, stream, t);
}

cm_status check_tensor(const cm_adamw_tensor &x) {
    if ((x.param_dtype != CM_BF16 && x.param_dtype != CM_F32) || (x.grad_dtype != CM_BF16 && x.grad_dtype != CM_F32) ||
        (x.state_bits != 32 && x.state_bits != 8))
        return CM_ERR_INVALID_ARG;
    if (x.numel < 0 || x.numel > (int64_t(1) << 41)) return CM_ERR_SHAPE;
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
    bool codes = false;
    for (int i = 0; i < count; ++i) {
        const cm_status st = check_tensor(tensors[i]);
        if (st != CM_OK) return st;
        codes = codes || (tensors[i].state_bits == 8 && tensors[i].numel > 0);
    }
    const int64_t chunk = int64_t(codes ? kCodePasses : 1) * kAdamPass;
    Table<kLargeTable> t;
    t.b1 = float(beta1), t.b2 = float(beta2), t.c1 = float(1.0 - beta1), t.c2 = float(1.0 - beta2);
    t.step = float(lr / (1.0 - std::pow(beta1, double(step))));
    t.root_scale = float(1.0 / std::sqrt(1.0 - std::pow(beta2, double(step))));
    t.eps = float(eps);
    t.grad_scale = grad_scale;
    t.seed_key = mix(mix(uint32_t(seed)) + uint32_t(seed >> 32)), t.seeded = seed != 0;
    int i = 0;
    while (i < count) {
        int64_t chunks = 0;
        t.count = 0;
        for (; i < count && t.count < kLargeTable; ++i) {
            const cm_adamw_tensor &x = tensors[i];
            if (x.numel == 0) continue;
            const int64_t c = (x.numel + chunk - 1) / chunk;
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
        const cudaError_t err = t.count <= kSmallTable ? launch<kSmallTable>(t, codes, chunks, stream)
                                                       : launch<kLargeTable>(t, codes, chunks, stream);
        if (err != cudaSuccess) return CM_ERR_CUDA;
    }
    return CM_OK;
}
