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

__device__ __forceinline__ void copy_param8(uint8_t *dst, const void *p, int f32, int c, int h) {
    if (!p) return;
    if (f32)
        copy_row8(reinterpret_cast<float *>(dst), static_cast<const float *>(p), c, h);
    else
        copy_row8(reinterpret_cast<bf16 *>(dst), static_cast<const bf16 *>(p), c, h);
}
// The same vector back from shared memory.
__device__ __forceinline__ V8 get_param8(const uint8_t *src, const void *p, int f32, float null_value, int c) {
    if (!p) return fill(null_value);
    return f32 ? load8(reinterpret_cast<const float *>(src) + c) : load8(reinterpret_cast<const bf16 *>(src) + c);
}

// Two row_sum()s at once.  `buf` holds a pair a warp; the caller alternates
// between two of them, so that one barrier a call suffices.
__device__ __forceinline__ float2 row_sum2(float a, float b, int width, float2 *buf) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (width == 32) return make_float2(a, b);
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    if (lane == 0) buf[warp] = make_float2(a, b);
    __syncthreads();
    const int nw = width >> 5, first = warp / nw * nw;
    const float2 v = lane < nw ? buf[first + lane] : make_float2(0.0f, 0.0f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// ---- forward ------------------------------------------------------------------

constexpr int kRingThreads = 512;   // of a persistent CTA, as whole rows

// A thread's share of a row: R vectors, vector r at column (r width + t) 8.
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
// stay in shared memory.
template <typename X, typename Y, int R, int S>
__global__ void __launch_bounds__(kRingThreads, 2) cm_layer_norm_ring_kernel(NormParams p, int width) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float buf[2][2][32];
    const int per = int(blockDim.x) / width, group = int(threadIdx.x) / width, t = int(threadIdx.x) - group * width;
    const int h = int(p.h), h8 = (h + 7) / 8 * 8, ps = p.p_f32 ? 4 : 2;
    uint8_t *const sg = smem, *const sb = sg + (p.gamma ? h8 * ps : 0);
    X *const ring = reinterpret_cast<X *>(sb + (p.beta ? h8 * ps : 0)) + group * h8;
    const int stage = per * h8;
    const int64_t first = int64_t(blockIdx.x) * per, step = int64_t(gridDim.x) * per;
    auto ask = [&](int64_t base, int st) {
        const int64_t row = base + group;
        if (row < p.rows) {
            const X *x = static_cast<const X *>(p.x) + row * p.ldx;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (r * width + t) * 8;
                if (c < h) copy_row8(ring + st * stage, x, c, h);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        if (group == 0 && c < h) {
            copy_param8(sg, p.gamma, p.p_f32, c, h);
            copy_param8(sb, p.beta, p.p_f32, c, h);
        }
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) ask(first + k * step, k);
    if (per > 1) {   // the other groups read what group 0 has copied
        copy_wait<0>();
        __syncthreads();
    }
    const float inv_h = 1.0f / float(h);
    int st = 0, flip = 0;
    for (int64_t base = first; base < p.rows; base += step) {
        ask(base + (S - 1) * step, (st + S - 1) % S);
        copy_wait<S - 1>();
        const int64_t row = base + group;
        const bool live = row < p.rows;
        Share<R> f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            f.x[r] = live && c < h ? load8(ring + st * stage + c) : fill(0.0f);
        }
        const float mean = row_sum(total(f), width, buf[flip][0]) * inv_h;
        const float rstd =
            1.0f / sqrtf(row_sum(squares(f, mean, width, t, h), width, buf[flip][1]) * inv_h + p.eps);
        if (live) {
            if (t == 0) {
                if (p.mean) p.mean[row] = mean;
                if (p.rstd) p.rstd[row] = rstd;
            }
            Y *y = static_cast<Y *>(p.out) + row * p.ldo;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (r * width + t) * 8;
                if (c >= h) break;
                store_row8(y, c, h, scaled(f.x[r], mean, rstd, get_param8(sg, p.gamma, p.p_f32, 1.0f, c),
                                           get_param8(sb, p.beta, p.p_f32, 0.0f, c)));
            }
        }
        st = st + 1 == S ? 0 : st + 1;
        flip ^= 1;
    }
    copy_wait<0>();
}

// Few rows: `width` threads hold a row in registers.
template <typename X, typename Y, int R>
__global__ void __launch_bounds__(1024) cm_layer_norm_kernel(NormParams p, int width) {
    __shared__ float buf[2][32];
    const int per = int(blockDim.x) / width, group = int(threadIdx.x) / width, t = int(threadIdx.x) - group * width;
    const int64_t row = int64_t(blockIdx.x) * per + group;
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
    const float mean = row_sum(total(f), width, buf[0]) * inv_h;
    const float rstd = 1.0f / sqrtf(row_sum(squares(f, mean, width, t, h), width, buf[1]) * inv_h + p.eps);
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

// ---- backward -------------------------------------------------------------------

// X: type of x, res and dx; Y: type of dy.
//
// One pass over x, dy and res gives dx and the sums over rows: persistent CTAs
// stream rows through a ring of S row buffers as the forward kernel does.  A
// thread owns the same R vectors of columns in every row, so dgamma and dbeta
// collect in its registers; after the rows' sums the row is read again from the
// ring, not held in registers, which leaves those to the sums.  At the end the
// groups of a CTA are added in order and written as its part.
template <typename X, typename Y, int R, int S>
__global__ void __launch_bounds__(kRingThreads, 1) cm_layer_norm_backward_ring_kernel(NormParams p, int width) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 buf[2][32];
    const int per = int(blockDim.x) / width, group = int(threadIdx.x) / width, t = int(threadIdx.x) - group * width;
    const int h = int(p.h), h8 = (h + 7) / 8 * 8;
    uint8_t *const sg = smem;
    uint8_t *const ring = sg + (p.gamma ? h8 * (p.p_f32 ? 4 : 2) : 0);
    const int xs = h8 * int(sizeof(X)), ys = h8 * int(sizeof(Y));
    const int row_bytes = xs + ys + (p.res ? xs : 0);
    const int64_t first = int64_t(blockIdx.x) * per, step = int64_t(gridDim.x) * per;
    auto slot = [&](int st) { return ring + (st * per + group) * row_bytes; };
    auto ask = [&](int64_t base, int st) {
        const int64_t row = base + group;
        if (row < p.rows) {
            uint8_t *d = slot(st);
            const X *x = static_cast<const X *>(p.x) + row * p.ldx, *res = static_cast<const X *>(p.res) + row * p.ldr;
            const Y *dy = static_cast<const Y *>(p.dy) + row * p.lddy;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (r * width + t) * 8;
                if (c >= h) break;
                copy_row8(reinterpret_cast<X *>(d), x, c, h);
                copy_row8(reinterpret_cast<Y *>(d + xs), dy, c, h);
                if (p.res) copy_row8(reinterpret_cast<X *>(d + xs + ys), res, c, h);
            }
        }
        copy_commit();
    };
    V8 a[R], b[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        if (group == 0 && c < h) copy_param8(sg, p.gamma, p.p_f32, c, h);
        a[r] = b[r] = fill(0.0f);
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) ask(first + k * step, k);
    if (per > 1) {
        copy_wait<0>();
        __syncthreads();
    }
    const float inv_h = 1.0f / float(h);
    float mean = 0.0f, rstd = 0.0f;
    if (first + group < p.rows) {
        mean = p.mean[first + group];
        rstd = p.rstd[first + group];
    }
    int st = 0, flip = 0;
    for (int64_t base = first; base < p.rows; base += step) {
        ask(base + (S - 1) * step, (st + S - 1) % S);
        const int64_t row = base + group;
        const bool live = row < p.rows;
        float next_mean = 0.0f, next_rstd = 0.0f;
        if (row + step < p.rows) {
            next_mean = p.mean[row + step];
            next_rstd = p.rstd[row + step];
        }
        copy_wait<S - 1>();
        const uint8_t *d = slot(st);
        float s1 = 0.0f, s2 = 0.0f;
        if (live) {
            const F2 rs = both(rstd), m = both(-mean);
            F2 q1 = both(0.0f), q2 = both(0.0f);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (r * width + t) * 8;
                if (c >= h) break;
                const V8 x = load8(reinterpret_cast<const X *>(d) + c), y = load8(reinterpret_cast<const Y *>(d + xs) + c);
                const V8 g = get_param8(sg, p.gamma, p.p_f32, 1.0f, c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // past a ragged end dy is zero: nothing is added
                    const F2 xh = mul(add(x.p[i], m), rs), u = mul(y.p[i], g.p[i]);
                    q1 = add(q1, u);
                    q2 = fma(u, xh, q2);
                    a[r].p[i] = fma(y.p[i], xh, a[r].p[i]);
                    b[r].p[i] = add(b[r].p[i], y.p[i]);
                }
            }
            s1 = sum(q1);
            s2 = sum(q2);
        }
        const float2 rowsum = row_sum2(s1, s2, width, buf[flip]);
        if (live) {
            // dx = rstd u - (x - mean) k - rstd s1 + res, k = rstd^2 s2
            s1 = rowsum.x * inv_h;
            s2 = rowsum.y * inv_h;
            const F2 rs = both(rstd), m = both(-mean), k = both(-rstd * rstd * s2), off = both(-rstd * s1);
            X *dx = static_cast<X *>(p.out) + row * p.ldo;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (r * width + t) * 8;
                if (c >= h) break;
                const V8 x = load8(reinterpret_cast<const X *>(d) + c), y = load8(reinterpret_cast<const Y *>(d + xs) + c);
                const V8 g = get_param8(sg, p.gamma, p.p_f32, 1.0f, c);
                V8 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o.p[i] = fma(mul(y.p[i], g.p[i]), rs, fma(add(x.p[i], m), k, off));
                if (p.res) {
                    const V8 z = load8(reinterpret_cast<const X *>(d + xs + ys) + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o.p[i] = add(o.p[i], z.p[i]);
                }
                store_row8(dx, c, h, o);
            }
        }
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
    float *const sums = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        if (c >= h) break;
        store8(sums + group * 2 * h8 + c, a[r]);
        store8(sums + (group * 2 + 1) * h8 + c, b[r]);
    }
    __syncthreads();
    for (int c = int(threadIdx.x); c < 2 * h; c += int(blockDim.x)) {
        const int o = c < h ? c : c - h + h8;
        float v = 0.0f;
        for (int g = 0; g < per; ++g) v += sums[g * 2 * h8 + o];
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
    __shared__ float2 buf[32];
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
    const float2 sum = row_sum2(s1, s2, int(blockDim.x), buf);
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

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return std::min(n, 160);
}

// Chunks of rows for the column sums: enough CTAs for two rounds of the SMs,
// at least 32 rows each.
int64_t chunks_for(int64_t rows, int64_t cols) {
    const int64_t blocks = (cols + 255) / 256;
    return std::max<int64_t>(1, std::min<int64_t>((rows + 31) / 32, std::max<int64_t>(1, 608 / blocks)));
}

constexpr int64_t kSmemCta = 227 * 1024, kSmemSm = 228 * 1024;

// CTAs of a persistent launch: at most `most` an SM, if shared memory has room.
int64_t resident(int sms, int64_t smem, int most) {
    return int64_t(sms) * std::max<int64_t>(1, std::min<int64_t>(most, kSmemSm / (smem + 1024 + 512)));
}

// The sums over rows of the partial sums of `parts` CTAs.
void sum_parts(const float *partial, int64_t parts, int64_t h, int64_t stride, void *out0, void *out1, int f32,
               int accumulate, cudaStream_t stream) {
    cm_sum_parts_kernel<<<dim3(unsigned((h + 31) / 32), stride > h ? 2 : 1), 256, 0, stream>>>(
        partial, parts, h, stride, out0, out1, f32, accumulate);
}

template <typename K>
cudaError_t opt_in(K kernel, int64_t smem) {
    return smem > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemCta - 1024))
                            : cudaSuccess;
}

int rows_per_cta(int width) { return std::max(1, kRingThreads / width); }

template <typename X, typename Y, int R>
cudaError_t forward_ring(const NormParams &p, int width, int per, int64_t smem, int64_t ctas, cudaStream_t stream) {
    cudaError_t e = opt_in(cm_layer_norm_ring_kernel<X, Y, R, 3>, smem);
    if (e != cudaSuccess) return e;
    cm_layer_norm_ring_kernel<X, Y, R, 3><<<unsigned(ctas), unsigned(width * per), size_t(smem), stream>>>(p, width);
    return cudaGetLastError();
}

int row_width(int64_t vecs, int R) { return int((vecs + 32 * R - 1) / (32 * R)) * 32; }

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
    const int sms = sm_count();
    {
        const int R = vecs < 64 ? 1 : vecs <= 1024 ? 2 : 4;
        const int width = row_width(vecs, R), per = rows_per_cta(width);
        const int64_t ps = (p.p_f32 ? 4 : 2) * ((p.gamma ? 1 : 0) + (p.beta ? 1 : 0));
        const int64_t smem = vecs * 8 * (ps + int64_t(sizeof(X)) * 3 * per);
        const int64_t ctas = resident(sms, smem, 2);
        // the ring pays once a CTA has a few rows to run ahead on
        if (width <= kRingThreads && smem <= kSmemCta - 1024 && p.rows >= 4 * ctas * per)
            return R == 1   ? forward_ring<X, Y, 1>(p, width, per, smem, ctas, stream)
                   : R == 2 ? forward_ring<X, Y, 2>(p, width, per, smem, ctas, stream)
                            : forward_ring<X, Y, 4>(p, width, per, smem, ctas, stream);
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

// Launch geometry of the one-pass backward kernel; ctas = 0 where a row is
// too long for it.  Alignment aside, it depends on extents and types only, so
// that the workspace's size can follow it.
struct RingPlan {
    int R = 0, S = 0, width = 0, per = 1;
    int64_t ctas = 0, smem = 0;
};

RingPlan ring_plan(int64_t rows, int64_t h, int64_t xs, int64_t ys, bool res, int64_t gamma_bytes, int sms) {
    RingPlan r;
    const int64_t vecs = (h + 7) / 8;
    if (vecs > 2048) return r;
    r.R = vecs < 64 ? 1 : vecs <= 1024 ? 2 : 4;
    r.width = row_width(vecs, r.R);
    r.per = rows_per_cta(r.width);
    const int64_t row = vecs * 8 * (xs + ys + (res ? xs : 0)) * r.per, fixed = vecs * 8 * gamma_bytes;
    for (r.S = 3; r.S >= 2; --r.S) {
        r.smem = fixed + r.S * row;
        if (r.smem <= kSmemCta - 1024) break;
    }
    if (r.S < 2) return r;
    r.ctas = std::min<int64_t>(resident(sms, r.smem, 1), (rows + r.per - 1) / r.per);
    return r;
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
        const RingPlan r = ring_plan(p.rows, p.h, sizeof(X), sizeof(Y), p.res != nullptr,
                                     p.gamma ? (p.p_f32 ? 4 : 2) : 0, sm_count());
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

// The most parts that any types of a call with these extents make: a
// persistent launch has one CTA an SM, and no more than rows need.  The SM count is an upper bound, so that the size can be asked
// for without a device.
int64_t norm_backward_parts(int64_t rows, int64_t h) {
    constexpr int kMostSms = 160;
    const RingPlan r = ring_plan(rows, h, 2, 2, false, 0, kMostSms);
    return std::max(chunks_for(rows, h), r.ctas);
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
