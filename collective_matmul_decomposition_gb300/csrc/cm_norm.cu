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
#include "cm_vec.cuh"

namespace cm {
namespace {

using namespace vec;

__device__ __forceinline__ V8 load_param8(const void *p, int f32, float null_value, int c, int h) {
    if (!p) return fill(null_value);
    return f32 ? load_row8(static_cast<const float *>(p), c, h) : load_row8(static_cast<const bf16 *>(p), c, h);
}
__device__ __forceinline__ float param1(const void *p, int f32, float null_value, int64_t c) {
    return !p ? null_value : f32 ? static_cast<const float *>(p)[c] : to_f(static_cast<const bf16 *>(p)[c]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The `width` threads (a multiple of 32) that share a row, one group of several
// in a CTA.  Groups meet at a barrier of their own, so that they drift apart
// and one's arithmetic fills another's waits.
struct Group {
    int width, index, warps, lane, warp;   // warp: in the group
    __device__ Group(int w) {
        width = w;
        index = int(threadIdx.x) / w;
        warps = w >> 5;
        lane = int(threadIdx.x) & 31;
        warp = (int(threadIdx.x) >> 5) - index * warps;
    }
    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(width) : "memory");
    }
};

// Sum over a group.  `buf` has a slot a warp of the group, rounded up to a
// multiple of four; the caller alternates between buffers, so that one barrier
// a call suffices.
__device__ __forceinline__ float row_sum(float v, const Group &g, float *buf) {
    v = warp_sum(v);
    if (g.warps == 1) return v;
    if (g.lane == 0) buf[g.warp] = v;
    g.sync();
    v = 0.0f;
    for (int k = 0; k < g.warps; k += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(buf + k);
        v += q.x;
        if (k + 1 < g.warps) v += q.y;
        if (k + 2 < g.warps) v += q.z;
        if (k + 3 < g.warps) v += q.w;
    }
    return v;
}
// Two sums at once; `buf` holds two floats a warp.
__device__ __forceinline__ float2 row_sum2(float a, float b, const Group &g, float *buf) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (g.warps == 1) return make_float2(a, b);
    if (g.lane == 0) *reinterpret_cast<float2 *>(buf + 2 * g.warp) = make_float2(a, b);
    g.sync();
    a = b = 0.0f;
    for (int k = 0; k < g.warps; k += 2) {
        const float4 q = *reinterpret_cast<const float4 *>(buf + 2 * k);
        a += q.x;
        b += q.y;
        if (k + 1 < g.warps) a += q.z, b += q.w;
    }
    return make_float2(a, b);
}
// Slots of a group in a shared buffer of kRowBuf floats (32 warps at most, 16 groups).
constexpr int kRowBuf = 128;
__device__ __forceinline__ float *row_buf(float *buf, const Group &g, int floats) {
    return buf + g.index * ((g.warps * floats + 3) & ~3);
}

// A parameter vector to shared memory as fp32, 1 (or 0) where there is none.
__device__ __forceinline__ void stage_param(float *dst, const void *p, int f32, float null_value, int h) {
    for (int c = int(threadIdx.x) * 8; c < h; c += int(blockDim.x) * 8)
        store8(dst + c, load_param8(p, f32, null_value, c, h));
}
// Asynchronous copy of the vector at column c of a row of h to its place in `dst`.
template <typename T>
__device__ __forceinline__ void copy_vec(T *dst, const T *row, int c, int h) {
    constexpr int kPer = 16 / int(sizeof(T));
    if (c + 8 <= h) {
#pragma unroll
        for (int k = 0; k < 8 / kPer; ++k) copy16(dst + c + k * kPer, row + c + k * kPer);
    } else if (c < h) {
        copy_row8(dst, row, c, h);
    }
}

// ---- forward ------------------------------------------------------------------

constexpr int kRingThreads = 512;   // of a persistent CTA, as whole rows

// A thread's share of a row: R vectors, vector r at column (r width + t) 8,
// t = its place in the group.
template <int R>
struct Share {
    V8 x[R];
};

// sum of the elements; those past the row's end are zeros
template <int R>
__device__ __forceinline__ float total(const Share<R> &s) {
    F2 q[2] = {both(0.0f), both(0.0f)};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i & 1] = add(q[i & 1], s.x[r].p[i]);
    return sum(add(q[0], q[1]));
}
// sum of the squares of the elements less `mean`
template <int R>
__device__ __forceinline__ float squares(const Share<R> &s, float mean, int width, int t, int h) {
    F2 q[2] = {both(0.0f), both(0.0f)};
    const F2 m = both(-mean);
    float tail = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        if (c + 8 <= h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 d = add(s.x[r].p[i], m);
                q[i & 1] = fma(d, d, q[i & 1]);
            }
        } else if (c < h) {   // a ragged end
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 d = parts(add(s.x[r].p[i], m));
                if (c + 2 * i < h) tail += d.x * d.x;
                if (c + 2 * i + 1 < h) tail += d.y * d.y;
            }
        }
    }
    return sum(add(q[0], q[1])) + tail;
}
// (x - mean) rstd g + b; the difference first, so that a constant row gives b
__device__ __forceinline__ V8 scaled(const V8 &x, float mean, float rstd, const V8 &g, const V8 &b) {
    V8 y;
    const F2 rs = both(rstd), m = both(-mean);
#pragma unroll
    for (int i = 0; i < 4; ++i) y.p[i] = fma(mul(add(x.p[i], m), rs), g.p[i], b.p[i]);
    return y;
}

// Many rows: persistent CTAs stream their rows through a ring of S row buffers
// in shared memory, filled by asynchronous copies S - 1 rows ahead, so that
// DRAM stays busy through the two reductions of a row.  A thread copies just
// the vectors that it reads itself: the ring needs no barrier.  gamma and beta
// stay in shared memory as fp32.  What is left bounds the kernel by instructions
// as much as by memory: hence four vectors a thread, pairs of fp32, and no
// test for missing parameters in the loop.
template <typename X, typename Y, int R, int S>
__global__ void __launch_bounds__(kRingThreads, 1) cm_layer_norm_ring_kernel(const __grid_constant__ NormParams p, int width) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float sums[2][2][kRowBuf];
    const Group g(width);
    const int t = int(threadIdx.x) - g.index * width, per = int(blockDim.x) / width;
    const int h = int(p.h), h8 = (h + 7) / 8 * 8;
    float *const gamma = reinterpret_cast<float *>(smem), *const beta = gamma + h8;
    X *const ring = reinterpret_cast<X *>(beta + h8) + g.index * h8;
    const int stage = per * h8;
    const int64_t step = int64_t(gridDim.x) * per;
    int64_t ask_row = int64_t(blockIdx.x) * per + g.index;
    const X *ask_x = static_cast<const X *>(p.x) + ask_row * p.ldx;
    auto ask = [&](int st) {
        if (ask_row < p.rows) {
#pragma unroll
            for (int r = 0; r < R; ++r) copy_vec(ring + st * stage, ask_x, (r * width + t) * 8, h);
        }
        copy_commit();
        ask_row += step;
        ask_x += step * p.ldx;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) ask(k);
    stage_param(gamma, p.gamma, p.p_f32, 1.0f, h);
    stage_param(beta, p.beta, p.p_f32, 0.0f, h);
    __syncthreads();
    const float inv_h = 1.0f / float(h);
    int st = 0, flip = 0;
    Y *y = static_cast<Y *>(p.out) + (int64_t(blockIdx.x) * per + g.index) * p.ldo;
    for (int64_t row = int64_t(blockIdx.x) * per + g.index; row < p.rows; row += step) {
        ask(st == 0 ? S - 1 : st - 1);
        copy_wait<S - 1>();
        Share<R> f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            f.x[r] = c < h ? load8(ring + st * stage + c) : fill(0.0f);
        }
        const float mean = row_sum(total(f), g, row_buf(sums[flip][0], g, 1)) * inv_h;
        const float var = row_sum(squares(f, mean, width, t, h), g, row_buf(sums[flip][1], g, 1)) * inv_h;
        const float rstd = rsqrtf(var + p.eps);
        if (t == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            if (c >= h) break;
            store_row8(y, c, h, scaled(f.x[r], mean, rstd, load8(gamma + c), load8(beta + c)));
        }
        y += step * p.ldo;
        st = st + 1 == S ? 0 : st + 1;
        flip ^= 1;
    }
    copy_wait<0>();
}

// Few rows: `width` threads hold a row in registers.
template <typename X, typename Y, int R>
__global__ void __launch_bounds__(1024) cm_layer_norm_kernel(NormParams p, int width) {
    __shared__ __align__(16) float sums[2][kRowBuf];
    const Group g(width);
    const int per = int(blockDim.x) / width, t = int(threadIdx.x) - g.index * width;
    const int64_t row = int64_t(blockIdx.x) * per + g.index;
    const int h = int(p.h);
    const bool live = row < p.rows;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    Share<R> f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        f.x[r] = live && c < h ? load_row8(x, c, h) : fill(0.0f);
    }
    const float inv_h = 1.0f / float(h);
    const float mean = row_sum(total(f), g, row_buf(sums[0], g, 1)) * inv_h;
    const float rstd = rsqrtf(row_sum(squares(f, mean, width, t, h), g, row_buf(sums[1], g, 1)) * inv_h + p.eps);
    if (!live) return;
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    Y *y = static_cast<Y *>(p.out) + row * p.ldo;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        if (c >= h) break;
        store_row8(y, c, h, scaled(f.x[r], mean, rstd, load_param8(p.gamma, p.p_f32, 1.0f, c, h),
                                   load_param8(p.beta, p.p_f32, 0.0f, c, h)));
    }
}

// Any extent, stride and alignment: one CTA a row, element by element, the
// row read three times (the second and third time from L2).
template <typename X, typename Y>
__global__ void __launch_bounds__(512) cm_layer_norm_any_kernel(NormParams p) {
    __shared__ __align__(16) float sums[2][kRowBuf];
    const Group g{int(blockDim.x)};
    const int64_t row = blockIdx.x;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < p.h; c += blockDim.x) s += to_f(x[c]);
    const float mean = row_sum(s, g, sums[0]) / float(p.h);
    float q = 0.0f;
    for (int64_t c = threadIdx.x; c < p.h; c += blockDim.x) q += (to_f(x[c]) - mean) * (to_f(x[c]) - mean);
    const float rstd = rsqrtf(row_sum(q, g, sums[1]) / float(p.h) + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    Y *y = static_cast<Y *>(p.out) + row * p.ldo;
    for (int64_t c = threadIdx.x; c < p.h; c += blockDim.x)
        from_f(y + c, (to_f(x[c]) - mean) * rstd * param1(p.gamma, p.p_f32, 1.0f, c) + param1(p.beta, p.p_f32, 0.0f, c));
}

// ---- backward -------------------------------------------------------------------

// X: type of x, res and dx; Y: type of dy.
//
// One pass over x, dy and res gives dx and the sums over rows: persistent CTAs
// stream rows through a ring of S row buffers as the forward kernel does.  A
// thread owns the same R vectors of columns in every row, so dgamma and dbeta
// collect in its registers; after the row's sums the row is read again from the
// ring, not held in registers, which leaves those to the sums.  At the end the
// groups of a CTA are added in order and written as its part.
template <typename X, typename Y, int R, int S>
__global__ void __launch_bounds__(kRingThreads, 1) cm_layer_norm_backward_ring_kernel(const __grid_constant__ NormParams p,
                                                                                      int width) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float sums[2][kRowBuf];
    const Group g(width);
    const int t = int(threadIdx.x) - g.index * width, per = int(blockDim.x) / width;
    const int h = int(p.h), h8 = (h + 7) / 8 * 8;
    float *const gamma = reinterpret_cast<float *>(smem);
    uint8_t *const ring = smem + h8 * 4;
    const int xs = h8 * int(sizeof(X)), ys = h8 * int(sizeof(Y));
    const int row_bytes = xs + ys + (p.res ? xs : 0);
    const int64_t step = int64_t(gridDim.x) * per, row0 = int64_t(blockIdx.x) * per + g.index;
    auto slot = [&](int st) { return ring + (st * per + g.index) * row_bytes; };
    int64_t ask_row = row0;
    const X *ask_x = static_cast<const X *>(p.x) + row0 * p.ldx, *ask_r = static_cast<const X *>(p.res) + row0 * p.ldr;
    const Y *ask_y = static_cast<const Y *>(p.dy) + row0 * p.lddy;
    auto ask = [&](int st) {
        if (ask_row < p.rows) {
            uint8_t *d = slot(st);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (r * width + t) * 8;
                copy_vec(reinterpret_cast<X *>(d), ask_x, c, h);
                copy_vec(reinterpret_cast<Y *>(d + xs), ask_y, c, h);
                if (p.res) copy_vec(reinterpret_cast<X *>(d + xs + ys), ask_r, c, h);
            }
        }
        copy_commit();
        ask_row += step;
        ask_x += step * p.ldx;
        ask_y += step * p.lddy;
        ask_r += step * p.ldr;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) ask(k);
    stage_param(gamma, p.gamma, p.p_f32, 1.0f, h);
    V8 a[R], b[R];
#pragma unroll
    for (int r = 0; r < R; ++r) a[r] = b[r] = fill(0.0f);
    __syncthreads();
    const float inv_h = 1.0f / float(h);
    float mean = 0.0f, rstd = 0.0f;
    if (row0 < p.rows) {
        mean = p.mean[row0];
        rstd = p.rstd[row0];
    }
    int st = 0, flip = 0;
    X *dx = static_cast<X *>(p.out) + row0 * p.ldo;
    for (int64_t row = row0; row < p.rows; row += step) {
        ask(st == 0 ? S - 1 : st - 1);
        float next_mean = 0.0f, next_rstd = 0.0f;
        if (row + step < p.rows) {
            next_mean = p.mean[row + step];
            next_rstd = p.rstd[row + step];
        }
        copy_wait<S - 1>();
        const uint8_t *d = slot(st);
        const F2 rs = both(rstd), m = both(-mean);
        F2 q1 = both(0.0f), q2 = both(0.0f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            if (c >= h) break;
            const V8 x = load8(reinterpret_cast<const X *>(d) + c), y = load8(reinterpret_cast<const Y *>(d + xs) + c);
            const V8 w = load8(gamma + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // past a ragged end dy is zero: nothing is added
                const F2 xh = mul(add(x.p[i], m), rs), u = mul(y.p[i], w.p[i]);
                q1 = add(q1, u);
                q2 = fma(u, xh, q2);
                a[r].p[i] = fma(y.p[i], xh, a[r].p[i]);
                b[r].p[i] = add(b[r].p[i], y.p[i]);
            }
        }
        const float2 rowsum = row_sum2(sum(q1), sum(q2), g, row_buf(sums[flip], g, 2));
        // dx = rstd u - (x - mean) k - rstd s1 + res, k = rstd^2 s2
        const float s1 = rowsum.x * inv_h, s2 = rowsum.y * inv_h;
        const F2 k = both(-rstd * rstd * s2), off = both(-rstd * s1);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            if (c >= h) break;
            const V8 x = load8(reinterpret_cast<const X *>(d) + c), y = load8(reinterpret_cast<const Y *>(d + xs) + c);
            const V8 w = load8(gamma + c);
            V8 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o.p[i] = fma(mul(y.p[i], w.p[i]), rs, fma(add(x.p[i], m), k, off));
            if (p.res) {
                const V8 z = load8(reinterpret_cast<const X *>(d + xs + ys) + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) o.p[i] = add(o.p[i], z.p[i]);
            }
            store_row8(dx, c, h, o);
        }
        dx += step * p.ldo;
        mean = next_mean;
        rstd = next_rstd;
        flip ^= 1;
        st = st + 1 == S ? 0 : st + 1;
    }
    copy_wait<0>();
    if (!p.partial) return;
    float *const mine = p.partial + int64_t(blockIdx.x) * 2 * h;
    if (per == 1) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = parts(a[r].p[i]), v = parts(b[r].p[i]);
                if (c + 2 * i < h) mine[c + 2 * i] = u.x, mine[h + c + 2 * i] = v.x;
                if (c + 2 * i + 1 < h) mine[c + 2 * i + 1] = u.y, mine[h + c + 2 * i + 1] = v.y;
            }
        }
        return;
    }
    // [group][2][h8] over the ring, which nobody uses any more: 8 bytes a
    // column and group, of the S (2 + 2) at least that the ring has
    __syncthreads();
    float *const parts_of = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        if (c >= h) break;
        store8(parts_of + g.index * 2 * h8 + c, a[r]);
        store8(parts_of + (g.index * 2 + 1) * h8 + c, b[r]);
    }
    __syncthreads();
    for (int c = int(threadIdx.x); c < 2 * h; c += int(blockDim.x)) {
        const int o = c < h ? c : c - h + h8;
        float v = 0.0f;
        for (int i = 0; i < per; ++i) v += parts_of[i * 2 * h8 + o];
        mine[c] = v;
    }
}

__device__ __forceinline__ void spread(const V8 &v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = parts(v.p[i]);
        f[2 * i] = a.x;
        f[2 * i + 1] = a.y;
    }
}
__device__ __forceinline__ V8 gather(const float (&f)[8]) {
    return {{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
}

// Any extent, stride and alignment (V = 1), or rows too long for the ring
// (V = 8): one CTA a row, x and dy read a second time from L2.  The sums over
// rows are then the column kernel's.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(512) cm_layer_norm_dx_any_kernel(NormParams p) {
    __shared__ __align__(16) float sums[kRowBuf];
    const Group gr{int(blockDim.x)};
    const int64_t row = blockIdx.x;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    const Y *dy = static_cast<const Y *>(p.dy) + row * p.lddy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    auto fetch = [&](int64_t c, float (&xh)[V], float (&u)[V]) {
        float g[V];
        if constexpr (V == 8) {
            spread(load_row8(x, int(c), int(p.h)), xh);
            spread(load_row8(dy, int(c), int(p.h)), u);
            spread(load_param8(p.gamma, p.p_f32, 1.0f, int(c), int(p.h)), g);
        } else {
            xh[0] = to_f(x[c]);
            u[0] = to_f(dy[c]);
            g[0] = param1(p.gamma, p.p_f32, 1.0f, c);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            xh[i] = (xh[i] - mean) * rstd;
            u[i] *= g[i];
        }
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = int64_t(threadIdx.x) * V; c < p.h; c += int64_t(blockDim.x) * V) {
        float xh[V], u[V];
        fetch(c, xh, u);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s1 += u[i];
            s2 += u[i] * xh[i];
        }
    }
    const float2 sum = row_sum2(s1, s2, gr, sums);
    s1 = sum.x / float(p.h);
    s2 = sum.y / float(p.h);
    X *dx = static_cast<X *>(p.out) + row * p.ldo;
    const X *res = static_cast<const X *>(p.res) + row * p.ldr;
    for (int64_t c = int64_t(threadIdx.x) * V; c < p.h; c += int64_t(blockDim.x) * V) {
        float xh[V], u[V], f[V];
        fetch(c, xh, u);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 0.0f;
        if (p.res) {
            if constexpr (V == 8)
                spread(load_row8(res, int(c), int(p.h)), f);
            else
                f[0] = to_f(res[c]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += (u[i] - s1 - xh[i] * s2) * rstd;
        if constexpr (V == 8)
            store_row8(dx, int(c), int(p.h), gather(f));
        else
            from_f(dx + c, f[0]);
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
                spread(load_row8(dy, int(c), int(p.h)), d);
                if constexpr (STATS) spread(load_row8(x, int(c), int(p.h)), f);
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

// out[c] (+)= sum over parts of partial[part * stride + c]: eight lanes take
// every eighth part, then their sums are added in order.
__global__ void __launch_bounds__(256) cm_sum_parts_kernel(const float *partial, int64_t parts, int64_t h, int64_t stride,
                                                           void *out0, void *out1, int f32, int accumulate) {
    __shared__ float sm[8][32];
    const int tx = int(threadIdx.x) & 31, ty = int(threadIdx.x) >> 5;
    const int64_t c = int64_t(blockIdx.x) * 32 + tx;
    void *out = blockIdx.y ? out1 : out0;
    if (!out) return;
    const float *src = partial + (blockIdx.y ? h : 0);
    float s = 0.0f;
    if (c < h) {
#pragma unroll 8
        for (int64_t k = ty; k < parts; k += 8) s += src[k * stride + c];
    }
    sm[ty][tx] = s;
    __syncthreads();
    if (ty || c >= h) return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sm[k][tx];
    if (f32) {
        float *o = static_cast<float *>(out) + c;
        *o = accumulate ? *o + s : s;
    } else {
        bf16 *o = static_cast<bf16 *>(out) + c;
        from_f(o, accumulate ? to_f(*o) + s : s);
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMostSms = 160;

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return std::min(n, kMostSms);
}

// Chunks of rows for the column sums: enough CTAs for two rounds of the SMs,
// at least 32 rows each.
int64_t chunks_for(int64_t rows, int64_t cols) {
    const int64_t blocks = (cols + 255) / 256;
    return std::max<int64_t>(1, std::min<int64_t>((rows + 31) / 32, std::max<int64_t>(1, 608 / blocks)));
}

constexpr int64_t kSmemCta = 227 * 1024;

// The sums over rows of the partial sums of `parts` CTAs.
void sum_parts(const float *partial, int64_t parts, int64_t h, int64_t stride, void *out0, void *out1, int f32,
               int accumulate, cudaStream_t stream) {
    cm_sum_parts_kernel<<<dim3(unsigned((h + 31) / 32), stride > h ? 2 : 1), 256, 0, stream>>>(
        partial, parts, h, stride, out0, out1, f32, accumulate);
}

template <typename K>
cudaError_t opt_in(K kernel, int64_t smem) {
    return smem > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemCta - 3 * 1024))
                            : cudaSuccess;
}

int row_width(int64_t vecs, int R) { return int((vecs + 32 * R - 1) / (32 * R)) * 32; }

// Geometry of a persistent launch over rows of h elements: R vectors a thread,
// `per` rows at a time of `width` threads each, S row buffers a group.  As many
// rows as 512 threads and shared memory hold with two buffers each, then a third
// buffer if it fits; one CTA an SM.  ctas = 0 where a row is too long.
struct RingPlan {
    int R = 0, S = 0, width = 0, per = 1;
    int64_t ctas = 0, smem = 0;
};

RingPlan ring_plan(int64_t rows, int64_t h, int64_t row_bytes, int64_t fixed_bytes, int sms) {
    RingPlan r;
    const int64_t vecs = (h + 7) / 8, limit = kSmemCta - 3 * 1024 /* the kernels' own buffers */;
    r.R = vecs < 64 ? 1 : vecs < 128 ? 2 : 4;
    r.width = row_width(vecs, r.R);
    if (r.width > kRingThreads) return r;
    const int64_t row = vecs * 8 * row_bytes, fixed = vecs * 8 * fixed_bytes;
    for (r.per = std::min(kRingThreads / r.width, kRingThreads / 32 - 1); r.per > 1 && fixed + 2 * r.per * row > limit;)
        --r.per;
    r.S = fixed + 3 * r.per * row <= limit ? 3 : 2;
    r.smem = fixed + r.S * r.per * row;
    if (r.smem > limit) return r;
    r.ctas = std::min<int64_t>(sms, (rows + r.per - 1) / r.per);
    return r;
}

template <typename X, typename Y, int R, int S>
cudaError_t forward_ring(const NormParams &p, const RingPlan &r, cudaStream_t stream) {
    cudaError_t e = opt_in(cm_layer_norm_ring_kernel<X, Y, R, S>, r.smem);
    if (e != cudaSuccess) return e;
    cm_layer_norm_ring_kernel<X, Y, R, S>
        <<<unsigned(r.ctas), unsigned(r.width * r.per), size_t(r.smem), stream>>>(p, r.width);
    return cudaGetLastError();
}

template <typename X, typename Y>
cudaError_t forward(const NormParams &p, cudaStream_t stream) {
    const int64_t vecs = (p.h + 7) / 8;
    const bool vec = aligned16(p.x) && aligned16(p.out) && aligned16(p.gamma) && aligned16(p.beta) && p.ldx % 8 == 0 &&
                     p.ldo % 8 == 0 && vecs <= 4096;
    if (p.rows > 0x7fffffff) return cudaErrorInvalidValue;
    if (!vec) {
        cm_layer_norm_any_kernel<X, Y><<<unsigned(p.rows), 512, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const RingPlan r = ring_plan(p.rows, p.h, sizeof(X), 8, sm_count());
    // the ring pays once a group has a few rows to run ahead on
    if (r.ctas > 0 && p.rows >= 4 * r.ctas * r.per) {
        if (r.S == 3)
            return r.R == 1   ? forward_ring<X, Y, 1, 3>(p, r, stream)
                   : r.R == 2 ? forward_ring<X, Y, 2, 3>(p, r, stream)
                              : forward_ring<X, Y, 4, 3>(p, r, stream);
        if (r.R == 4) return forward_ring<X, Y, 4, 2>(p, r, stream);   // shorter rows leave room for three
    }
    // all of a row's loads at once
    const int R = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
    const int width = row_width(vecs, R), per = std::max(1, 128 / width);
    const unsigned grid = unsigned((p.rows + per - 1) / per), threads = unsigned(width * per);
    if (R == 1)
        cm_layer_norm_kernel<X, Y, 1><<<grid, threads, 0, stream>>>(p, width);
    else if (R == 2)
        cm_layer_norm_kernel<X, Y, 2><<<grid, threads, 0, stream>>>(p, width);
    else
        cm_layer_norm_kernel<X, Y, 4><<<grid, threads, 0, stream>>>(p, width);
    return cudaGetLastError();
}

template <typename X, typename Y, int R, int S>
cudaError_t backward_ring(const NormParams &p, const RingPlan &r, cudaStream_t stream) {
    cudaError_t e = opt_in(cm_layer_norm_backward_ring_kernel<X, Y, R, S>, r.smem);
    if (e != cudaSuccess) return e;
    cm_layer_norm_backward_ring_kernel<X, Y, R, S>
        <<<unsigned(r.ctas), unsigned(r.width * r.per), size_t(r.smem), stream>>>(p, r.width);
    return cudaGetLastError();
}

template <typename X, typename Y>
cudaError_t backward(NormParams p, cudaStream_t stream) {
    if (p.rows > 0x7fffffff) return cudaErrorInvalidValue;
    const bool sums = p.dgamma || p.dbeta;
    if (!sums) p.partial = nullptr;
    const bool in_vec = aligned16(p.x) && aligned16(p.dy) && p.ldx % 8 == 0 && p.lddy % 8 == 0;
    const bool vec = in_vec && aligned16(p.out) && aligned16(p.gamma) && p.ldo % 8 == 0 &&
                     (!p.res || (aligned16(p.res) && p.ldr % 8 == 0));
    if (vec) {
        const RingPlan r = ring_plan(p.rows, p.h, int64_t(sizeof(X)) * (p.res ? 2 : 1) + int64_t(sizeof(Y)), 4, sm_count());
        if (r.ctas > 0) {
            const cudaError_t e = r.S == 3 ? (r.R == 1   ? backward_ring<X, Y, 1, 3>(p, r, stream)
                                              : r.R == 2 ? backward_ring<X, Y, 2, 3>(p, r, stream)
                                                         : backward_ring<X, Y, 4, 3>(p, r, stream))
                                           : (r.R == 1   ? backward_ring<X, Y, 1, 2>(p, r, stream)
                                              : r.R == 2 ? backward_ring<X, Y, 2, 2>(p, r, stream)
                                                         : backward_ring<X, Y, 4, 2>(p, r, stream));
            if (e != cudaSuccess || !sums) return e;
            sum_parts(p.partial, r.ctas, p.h, 2 * p.h, p.dgamma, p.dbeta, p.g_f32, p.accumulate, stream);
            return cudaGetLastError();
        }
    }
    if (vec)
        cm_layer_norm_dx_any_kernel<X, Y, 8><<<unsigned(p.rows), 512, 0, stream>>>(p);
    else
        cm_layer_norm_dx_any_kernel<X, Y, 1><<<unsigned(p.rows), 512, 0, stream>>>(p);
    if (!sums) return cudaGetLastError();
    const int64_t chunks = chunks_for(p.rows, p.h);
    if (in_vec)
        cm_colsum_kernel<X, Y, 8, true><<<dim3(unsigned((p.h + 255) / 256), unsigned(chunks)), 32 * kColY, 0, stream>>>(p);
    else
        cm_colsum_kernel<X, Y, 1, true><<<dim3(unsigned((p.h + 31) / 32), unsigned(chunks)), 32 * kColY, 0, stream>>>(p);
    sum_parts(p.partial, chunks, p.h, 2 * p.h, p.dgamma, p.dbeta, p.g_f32, p.accumulate, stream);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const NormParams &p, cm_dtype x, cm_dtype y, cudaStream_t stream) {
    if (x == CM_BF16) return y == CM_BF16 ? forward<bf16, bf16>(p, stream) : forward<bf16, float>(p, stream);
    return y == CM_BF16 ? forward<float, bf16>(p, stream) : forward<float, float>(p, stream);
}

// The most parts that a call with these extents makes, whatever its types: a
// persistent launch has one CTA an SM, at most as many as there are rows.  The
// SM count is an upper bound, so that the size can be asked for without a device.
int64_t norm_backward_parts(int64_t rows, int64_t h) {
    return std::max(chunks_for(rows, h), std::min<int64_t>(kMostSms, std::max<int64_t>(1, rows)));
}

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
    sum_parts(partial, chunks, cols, cols, out, nullptr, out_f32 ? 1 : 0, accumulate ? 1 : 0, stream);
    return cudaGetLastError();
}

}  // namespace cm
