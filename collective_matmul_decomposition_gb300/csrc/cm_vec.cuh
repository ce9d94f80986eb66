// cm_vec.cuh -- vectors of eight neighbouring elements (bf16 or fp32) as four
// pairs of fp32, and the arithmetic on pairs: sm_103a adds, multiplies and
// fuses two fp32 in one instruction.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace cm {
namespace vec {
namespace {

using bf16 = __nv_bfloat16;

// Two fp32 in one 64-bit register pair.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 pair(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 both(float a) { return pair(a, a); }
__device__ __forceinline__ float2 parts(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum(F2 a) {
    const float2 p = parts(a);
    return p.x + p.y;
}

struct V8 {
    F2 p[4];
};
__device__ __forceinline__ V8 fill(float a) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = both(a);
    return r;
}
// 16-byte aligned
__device__ __forceinline__ V8 load8(const float *p) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    return {{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
}
__device__ __forceinline__ F2 unpack(uint32_t w) {
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ V8 load8(const bf16 *p) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    return {{unpack(a.x), unpack(a.y), unpack(a.z), unpack(a.w)}};
}
__device__ __forceinline__ void store8(float *p, const V8 &v) {
    const float2 a = parts(v.p[0]), b = parts(v.p[1]), c = parts(v.p[2]), d = parts(v.p[3]);
    reinterpret_cast<float4 *>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
}
__device__ __forceinline__ uint32_t pack(F2 a) {
    const float2 p = parts(a);
    const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ void store8(bf16 *p, const V8 &v) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack(v.p[0]), pack(v.p[1]), pack(v.p[2]), pack(v.p[3]));
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float *p, float v) { *p = v; }
__device__ __forceinline__ void from_f(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }

// The vector at column c of a row of h elements; past the end: zeros.  The
// last vector of a ragged row goes element by element.
template <typename T>
__device__ __forceinline__ V8 load_row8(const T *row, int c, int h) {
    if (c + 8 <= h) return load8(row + c);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < h ? to_f(row[c + i]) : 0.0f;
    return {{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
}
template <typename T>
__device__ __forceinline__ void store_row8(T *row, int c, int h, const V8 &v) {
    if (c + 8 <= h) {
        store8(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = parts(v.p[i]);
            if (c + 2 * i < h) from_f(row + c + 2 * i, p.x);
            if (c + 2 * i + 1 < h) from_f(row + c + 2 * i + 1, p.y);
        }
    }
}

// Asynchronous copy of up to 16 bytes to shared memory; bytes beyond `n` are
// zeros there and not read.
__device__ __forceinline__ void copy16(void *dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src),
                 "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The vector at column c of a row of h, to its place in `dst`.
template <typename T>
__device__ __forceinline__ void copy_row8(T *dst, const T *row, int c, int h) {
    constexpr int kPer = 16 / int(sizeof(T));
#pragma unroll
    for (int k = 0; k < 8 / kPer; ++k) {
        const int left = h - c - k * kPer;
        const int n = left >= kPer ? 16 : left > 0 ? left * int(sizeof(T)) : 0;
        copy16(dst + c + k * kPer, n ? row + c + k * kPer : row, n);
    }
}

}  // namespace
}  // namespace vec
}  // namespace cm
