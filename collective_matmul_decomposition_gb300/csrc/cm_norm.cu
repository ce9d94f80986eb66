// cm_norm.cu -- layer norm, forward and backward, and column sums.
//
//   forward   mean = sum(x)/h, var = sum((x - mean)^2)/h, rstd = 1/sqrt(var + eps)
//             y = (x - mean) rstd gamma + beta
//   backward  xh = (x - mean) rstd, t = dy gamma
//             dx = rstd (t - sum(t)/h - xh sum(t xh)/h) + res
//             dgamma = sum_rows dy xh, dbeta = sum_rows dy
//
// Statistics and sums are fp32.  The variance is that of the centred values
// (two passes over registers), so a row far from zero loses nothing.
#include "cm_norm.cuh"

#include <cuda_bf16.h>

#include <algorithm>

#include "cm_linear.cuh"

namespace cm {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float *p, float v) { *p = v; }
__device__ __forceinline__ void from_f(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }

// 8 neighbouring elements, 16-byte aligned
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
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
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
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
// The vector at column c of a row of h elements; past the end: zeros.  The
// last vector of a ragged row goes element by element.
template <typename T>
__device__ __forceinline__ void load_row8(const T *row, int64_t c, int64_t h, float (&f)[8]) {
    if (c + 8 <= h) {
        load8(row + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < h ? to_f(row[c + i]) : 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void store_row8(T *row, int64_t c, int64_t h, const float (&f)[8]) {
    if (c + 8 <= h) {
        store8(row + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < h) from_f(row + c + i, f[i]);
    }
}
__device__ __forceinline__ void load_param8(const void *p, int f32, float null_value, int64_t c, int64_t h, float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = null_value;
    } else if (f32) {
        load_row8(static_cast<const float *>(p), c, h, f);
    } else {
        load_row8(static_cast<const bf16 *>(p), c, h, f);
    }
}
__device__ __forceinline__ float param1(const void *p, int f32, float null_value, int64_t c) {
    return !p ? null_value : f32 ? static_cast<const float *>(p)[c] : to_f(static_cast<const bf16 *>(p)[c]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the `width` threads (a multiple of 32) that share a row.  `buf`
// holds one value a warp and is used once.
__device__ __forceinline__ float row_sum(float v, int width, float *buf) {
    v = warp_sum(v);
    if (width == 32) return v;
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    const int nw = width >> 5, first = warp / nw * nw;
    return warp_sum(lane < nw ? buf[first + lane] : 0.0f);
}

// ---- forward ------------------------------------------------------------------

// `width` threads hold a row in registers, R vectors of 8 each.
template <typename X, typename Y, int R>
__global__ void __launch_bounds__(1024) cm_layer_norm_kernel(NormParams p, int width) {
    __shared__ float buf[2][32];
    const int per = int(blockDim.x) / width, group = int(threadIdx.x) / width, t = int(threadIdx.x) - group * width;
    const int64_t row = int64_t(blockIdx.x) * per + group;
    const bool live = row < p.rows;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    float f[R][8];
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t c = (int64_t(r) * width + t) * 8;
        if (live && c < p.h) {
            load_row8(x, c, p.h, f[r]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[r][i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += f[r][i];
    }
    const float inv_h = 1.0f / float(p.h);
    const float mean = row_sum(s, width, buf[0]) * inv_h;
    float q = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t c = (int64_t(r) * width + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < p.h) q += (f[r][i] - mean) * (f[r][i] - mean);
    }
    const float rstd = 1.0f / sqrtf(row_sum(q, width, buf[1]) * inv_h + p.eps);
    if (!live) return;
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    Y *y = static_cast<Y *>(p.out) + row * p.ldo;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t c = (int64_t(r) * width + t) * 8;
        if (c >= p.h) break;
        float g[8], b[8];
        load_param8(p.gamma, p.p_f32, 1.0f, c, p.h, g);
        load_param8(p.beta, p.p_f32, 0.0f, c, p.h, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[r][i] = (f[r][i] - mean) * rstd * g[i] + b[i];
        store_row8(y, c, p.h, f[r]);
    }
}

// Any extent, stride and alignment: one CTA a row, element by element, the
// row read three times (the second and third time from L2).
template <typename X, typename Y>
__global__ void __launch_bounds__(512) cm_layer_norm_any_kernel(NormParams p) {
    __shared__ float buf[2][32];
    const int64_t row = blockIdx.x;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < p.h; c += blockDim.x) s += to_f(x[c]);
    const float mean = row_sum(s, int(blockDim.x), buf[0]) / float(p.h);
    float q = 0.0f;
    for (int64_t c = threadIdx.x; c < p.h; c += blockDim.x) q += (to_f(x[c]) - mean) * (to_f(x[c]) - mean);
    const float rstd = 1.0f / sqrtf(row_sum(q, int(blockDim.x), buf[1]) / float(p.h) + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    Y *y = static_cast<Y *>(p.out) + row * p.ldo;
    for (int64_t c = threadIdx.x; c < p.h; c += blockDim.x)
        from_f(y + c, (to_f(x[c]) - mean) * rstd * param1(p.gamma, p.p_f32, 1.0f, c) + param1(p.beta, p.p_f32, 0.0f, c));
}

// ---- backward: input gradient -----------------------------------------------------

// X: type of x, res and dx; Y: type of dy.
template <typename X, typename Y>
__global__ void __launch_bounds__(512) cm_layer_norm_dx_any_kernel(NormParams p) {
    __shared__ float buf[2][32];
    const int64_t row = blockIdx.x;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    const Y *dy = static_cast<const Y *>(p.dy) + row * p.lddy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < p.h; c += blockDim.x) {
        const float t = to_f(dy[c]) * param1(p.gamma, p.p_f32, 1.0f, c);
        s1 += t;
        s2 += t * ((to_f(x[c]) - mean) * rstd);
    }
    s1 = row_sum(s1, int(blockDim.x), buf[0]) / float(p.h);
    s2 = row_sum(s2, int(blockDim.x), buf[1]) / float(p.h);
    X *dx = static_cast<X *>(p.out) + row * p.ldo;
    const X *res = static_cast<const X *>(p.res) + row * p.ldr;
    for (int64_t c = threadIdx.x; c < p.h; c += blockDim.x) {
        const float t = to_f(dy[c]) * param1(p.gamma, p.p_f32, 1.0f, c);
        float v = (t - s1 - (to_f(x[c]) - mean) * rstd * s2) * rstd;
        if (p.res) v += to_f(res[c]);
        from_f(dx + c, v);
    }
}

// ---- column sums: dgamma and dbeta, or the plain sum of a matrix's rows ---------------

constexpr int kColY = 8;   // row lanes of a CTA; its 32 column lanes hold V columns each

// Partial sums over the rows of chunk blockIdx.y.  STATS: [chunk][2][h] of
// dy xh and dy; otherwise [chunk][h] of dy.
template <typename X, typename Y, int V, bool STATS>
__global__ void __launch_bounds__(32 * kColY) cm_colsum_kernel(NormParams p) {
    __shared__ float sm[STATS ? 2 : 1][kColY][32 * V];
    const int tx = int(threadIdx.x) & 31, ty = int(threadIdx.x) >> 5;
    const int64_t c = (int64_t(blockIdx.x) * 32 + tx) * V;
    const int64_t r0 = p.rows * blockIdx.y / gridDim.y, r1 = p.rows * (blockIdx.y + 1) / gridDim.y;
    float a[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = b[i] = 0.0f;
    if (c < p.h) {
#pragma unroll 4
        for (int64_t r = r0 + ty; r < r1; r += kColY) {
            float d[V], f[V];
            const Y *dy = static_cast<const Y *>(p.dy) + r * p.lddy;
            const X *x = static_cast<const X *>(p.x) + r * p.ldx;
            if constexpr (V == 8) {
                load_row8(dy, c, p.h, d);
                if constexpr (STATS) load_row8(x, c, p.h, f);
            } else {
                d[0] = to_f(dy[c]);
                if constexpr (STATS) f[0] = to_f(x[c]);
            }
            if constexpr (STATS) {
                const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
                for (int i = 0; i < V; ++i) a[i] += d[i] * ((f[i] - mean) * rstd);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) b[i] += d[i];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (STATS) sm[1][ty][tx * V + i] = a[i];
        sm[0][ty][tx * V + i] = b[i];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 32 * V; j += 32 * kColY) {
        const int64_t cc = int64_t(blockIdx.x) * 32 * V + j;
        if (cc >= p.h) continue;
        float sb = 0.0f, sa = 0.0f;
        for (int k = 0; k < kColY; ++k) {
            sb += sm[0][k][j];
            if constexpr (STATS) sa += sm[1][k][j];
        }
        if constexpr (STATS) {
            p.partial[(int64_t(blockIdx.y) * 2) * p.h + cc] = sa;
            p.partial[(int64_t(blockIdx.y) * 2 + 1) * p.h + cc] = sb;
        } else {
            p.partial[int64_t(blockIdx.y) * p.h + cc] = sb;
        }
    }
}

// out[c] (+)= sum over parts, in their order, of partial[part * stride + c]
__device__ __forceinline__ void sum_parts(const float *partial, int64_t parts, int64_t stride, void *out, int f32,
                                          int accumulate, int64_t c) {
    if (!out) return;
    float s = 0.0f;
#pragma unroll 8
    for (int64_t k = 0; k < parts; ++k) s += partial[k * stride + c];
    if (f32) {
        float *o = static_cast<float *>(out) + c;
        *o = accumulate ? *o + s : s;
    } else {
        bf16 *o = static_cast<bf16 *>(out) + c;
        from_f(o, accumulate ? to_f(*o) + s : s);
    }
}

__global__ void __launch_bounds__(128) cm_sum_parts_kernel(const float *partial, int64_t parts, int64_t h, void *out0,
                                                           void *out1, int f32, int accumulate) {
    const int64_t c = int64_t(blockIdx.x) * 128 + threadIdx.x;
    if (c >= h) return;
    const int64_t stride = out1 || gridDim.y > 1 ? 2 * h : h;
    if (blockIdx.y == 0)
        sum_parts(partial, parts, stride, out0, f32, accumulate, c);
    else
        sum_parts(partial + h, parts, stride, out1, f32, accumulate, c);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return n;
}

// Chunks of rows for the column sums: enough CTAs for two rounds of the SMs,
// at least 32 rows each.
int64_t chunks_for(int64_t rows, int64_t cols) {
    const int64_t blocks = (cols + 255) / 256;
    return std::max<int64_t>(1, std::min<int64_t>((rows + 31) / 32, std::max<int64_t>(1, 608 / blocks)));
}

template <typename X, typename Y>
cudaError_t forward(const NormParams &p, cudaStream_t stream) {
    const int64_t vecs = (p.h + 7) / 8;
    const bool vec = aligned16(p.x) && aligned16(p.out) && aligned16(p.gamma) && aligned16(p.beta) && p.ldx % 8 == 0 &&
                     p.ldo % 8 == 0 && vecs <= 4096;
    if (!vec) {
        if (p.rows > 0x7fffffff) return cudaErrorInvalidValue;
        cm_layer_norm_any_kernel<X, Y><<<unsigned(p.rows), 512, 0, stream>>>(p);
        return cudaGetLastError();
    }
    // few rows: all of a row's loads at once; many: fewer, busier threads
    const int sms = sm_count();
    int R = p.rows < 4 * sms ? (vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4) : (vecs >= 128 ? 4 : vecs >= 64 ? 2 : 1);
    const int width = int((vecs + 32 * R - 1) / (32 * R)) * 32;
    const int per = std::max(1, 128 / width);
    const int64_t grid = (p.rows + per - 1) / per;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 g(static_cast<unsigned>(grid)), b(static_cast<unsigned>(width * per));
    if (R == 1)
        cm_layer_norm_kernel<X, Y, 1><<<g, b, 0, stream>>>(p, width);
    else if (R == 2)
        cm_layer_norm_kernel<X, Y, 2><<<g, b, 0, stream>>>(p, width);
    else
        cm_layer_norm_kernel<X, Y, 4><<<g, b, 0, stream>>>(p, width);
    return cudaGetLastError();
}

template <typename X, typename Y>
cudaError_t backward(const NormParams &p, cudaStream_t stream) {
    if (p.rows > 0x7fffffff) return cudaErrorInvalidValue;
    if (p.rows > 0) cm_layer_norm_dx_any_kernel<X, Y><<<unsigned(p.rows), 512, 0, stream>>>(p);
    if (!p.dgamma && !p.dbeta) return cudaGetLastError();
    const bool vec = aligned16(p.x) && aligned16(p.dy) && p.ldx % 8 == 0 && p.lddy % 8 == 0;
    const int64_t chunks = chunks_for(p.rows, p.h);
    if (vec)
        cm_colsum_kernel<X, Y, 8, true><<<dim3(unsigned((p.h + 255) / 256), unsigned(chunks)), 32 * kColY, 0, stream>>>(p);
    else
        cm_colsum_kernel<X, Y, 1, true><<<dim3(unsigned((p.h + 31) / 32), unsigned(chunks)), 32 * kColY, 0, stream>>>(p);
    cm_sum_parts_kernel<<<dim3(unsigned((p.h + 127) / 128), 2), 128, 0, stream>>>(p.partial, chunks, p.h, p.dgamma,
                                                                                 p.dbeta, p.g_f32, p.accumulate);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const NormParams &p, cm_dtype x, cm_dtype y, cudaStream_t stream) {
    if (x == CM_BF16) return y == CM_BF16 ? forward<bf16, bf16>(p, stream) : forward<bf16, float>(p, stream);
    return y == CM_BF16 ? forward<float, bf16>(p, stream) : forward<float, float>(p, stream);
}

int64_t norm_backward_parts(int64_t rows, int64_t h) { return chunks_for(rows, h); }

cudaError_t launch_layer_norm_backward(const NormParams &p, cm_dtype x, cm_dtype y, cudaStream_t stream) {
    if (x == CM_BF16) return y == CM_BF16 ? backward<bf16, bf16>(p, stream) : backward<bf16, float>(p, stream);
    return y == CM_BF16 ? backward<float, bf16>(p, stream) : backward<float, float>(p, stream);
}

int64_t colsum_chunks(int64_t rows, int64_t cols) { return chunks_for(rows, cols); }

cudaError_t launch_colsum(const void *x, int64_t ldx, int64_t rows, int64_t cols, float *partial, void *out,
                          bool out_f32, bool accumulate, cudaStream_t stream) {
    NormParams p = {};
    p.dy = x;
    p.lddy = ldx;
    p.rows = rows;
    p.h = cols;
    p.partial = partial;
    const int64_t chunks = chunks_for(rows, cols);
    cm_colsum_kernel<bf16, bf16, 8, false>
        <<<dim3(unsigned((cols + 255) / 256), unsigned(chunks)), 32 * kColY, 0, stream>>>(p);
    cm_sum_parts_kernel<<<dim3(unsigned((cols + 127) / 128), 1), 128, 0, stream>>>(partial, chunks, cols, out, nullptr,
                                                                                  out_f32 ? 1 : 0, accumulate ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace cm
