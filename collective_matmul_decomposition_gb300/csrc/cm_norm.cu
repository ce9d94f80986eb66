// cm_norm.cu -- layer norm, forward and backward, and column sums.
//
//   forward   mean = sum(x)/h, var = sum((x - mean)^2)/h, rstd = 1/sqrt(var + eps)
//             y = (x - mean) rstd gamma + beta
//   backward  xh = (x - mean) rstd, t = dy gamma
//             dx = rstd (t - sum(t)/h - xh sum(t xh)/h) + res
//             dgamma = sum_rows dy xh, dbeta = sum_rows dy
//
// All are bound by memory, and short of it by the latency of a row's reductions:
// 8192 x 8192 in bf16 takes 52 us forward (5.2 TB/s) and 97 us backward with
// residual and parameter gradients (5.5 TB/s); 65536 x 512: 26.3 and 48.6 us.
//
// Statistics and sums are fp32.  The variance is that of the centred values
// (two passes over registers), so a row far from zero loses nothing.
#include "cm_norm.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "cm_device.cuh"
#include "cm_launch.cuh"
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
// The sum of one row, or the sums of two.
__device__ __forceinline__ void rows_sum(float a, float, const Group &g, float *buf, float (&v)[1]) {
    v[0] = row_sum(a, g, row_buf(buf, g, 1));
}
__device__ __forceinline__ void rows_sum(float a, float b, const Group &g, float *buf, float (&v)[2]) {
    const float2 q = row_sum2(a, b, g, row_buf(buf, g, 2));
    v[0] = q.x;
    v[1] = q.y;
}

// The columns of a CTA: all, or its half of them in a cluster of two.
struct Columns {
    int half, first, count, rank, cta, ctas;
    __device__ Columns(int64_t h, bool split) {
        half = split ? int((h + 15) / 16 * 8) : int(h);
        rank = split ? int(blockIdx.x & 1) : 0;
        first = rank * half;
        count = split ? min(half, int(h) - first) : half;
        cta = split ? int(blockIdx.x >> 1) : int(blockIdx.x);
        ctas = split ? int(gridDim.x >> 1) : int(gridDim.x);
    }
};
__device__ __forceinline__ float of_other(const float *slot, int rank) {
    float o;
    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                 : "=f"(o)
                 : "r"(dev::mapa_shared(dev::smem_u32(slot), uint32_t(rank ^ 1)))
                 : "memory");
    return o;
}
// The sum of a row from the sums of its halves, in their order, so that both
// CTAs have the same.  All threads of both call it; `slot` is one of two that
// take turns, so that the next sum is not written before this one is read.
__device__ __forceinline__ float with_other(float v, float *slot, int rank) {
    if (threadIdx.x == 0) *slot = v;
    dev::cluster_sync();
    const float o = of_other(slot, rank);
    return rank == 0 ? v + o : o + v;
}

// A parameter vector to shared memory as fp32, 1 (or 0) where there is none.
// The first and second halves of the vectors lie in two planes of h8 / 2, so
// that neighbouring threads read neighbouring 16 bytes.
// A group of `width` threads, t its place in it, covers the row with R vectors
// a thread; all loads before the first store.
template <int R>
__device__ __forceinline__ void stage_param(float *dst, const void *p, int f32, float null_value, int h, int h8, int width,
                                            int t) {
    V8 v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        v[r] = c < h ? load_param8(p, f32, null_value, c, h) : fill(0.0f);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * width + t) * 8;
        if (c >= h) break;
        const float2 a0 = parts(v[r].p[0]), a1 = parts(v[r].p[1]), b0 = parts(v[r].p[2]), b1 = parts(v[r].p[3]);
        *reinterpret_cast<float4 *>(dst + c / 2) = make_float4(a0.x, a0.y, a1.x, a1.y);
        *reinterpret_cast<float4 *>(dst + (h8 + c) / 2) = make_float4(b0.x, b0.y, b1.x, b1.y);
    }
}
__device__ __forceinline__ V8 staged_param(const float *src, int c, int h8) {
    const float4 a = *reinterpret_cast<const float4 *>(src + c / 2);
    const float4 b = *reinterpret_cast<const float4 *>(src + (h8 + c) / 2);
    return {{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
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

constexpr int kRingThreads = 512;   // of a persistent CTA at most, as whole groups

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
// s / h from inv = 1 / h: the product, which is off by a unit of the last place
// for many h, and its remainder's part, so that exact quotients come out exact.
// The compiler's division costs 1 to 8 % of the ring kernel (65536 x 512 in bf16:
// 27.1 us for 26.0, 100000 x 64: 27.1 for 25.1).
__device__ __forceinline__ float quotient(float s, float h, float inv) {
    const float q = s * inv, rest = fmaf(-q, h, s);
    return rest == rest ? fmaf(rest, inv, q) : q;   // a sum that is not finite has no remainder
}
// (x - mean) rstd g + b; the difference first, so that a row of one value gives b
// wherever the row's sum is exact (and the mean its quotient, rounded once)
__device__ __forceinline__ V8 scaled(const V8 &x, float mean, float rstd, const V8 &g, const V8 &b) {
    V8 y;
    const F2 rs = both(rstd), m = both(-mean);
#pragma unroll
    for (int i = 0; i < 4; ++i) y.p[i] = fma(mul(add(x.p[i], m), rs), g.p[i], b.p[i]);
    return y;
}

// Many rows: persistent CTAs stream their rows through a ring of S buffers in
// shared memory, filled by asynchronous copies S - 1 steps ahead, so that DRAM
// stays busy through the reductions.  A thread copies just the vectors that it
// reads itself: the ring needs no barrier.  A group takes NR rows a step: what
// bounds it is the latency of the two reductions, one after the other, and two
// rows share that, and the reads of gamma and beta (8192 x 8192 in bf16: 50 us
// with two, 68 with one).  Rows longer than 8192 go one by one, to keep the
// registers.  gamma and beta stay in shared memory as fp32.
template <typename X, typename Y, int R, int NR, int S>
__global__ void __launch_bounds__(kRingThreads, 1) cm_layer_norm_ring_kernel(const __grid_constant__ NormParams p, int width) {
    let_next_start();
    wait_for_previous();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float sums[2][2][kRowBuf];
    const Group g(width);
    const int t = int(threadIdx.x) - g.index * width, per = int(blockDim.x) / width;
    const int h = int(p.h), h8 = (h + 7) / 8 * 8;
    float *const gamma = reinterpret_cast<float *>(smem), *const beta = gamma + h8;
    X *const ring = reinterpret_cast<X *>(beta + h8) + g.index * NR * h8;
    const int stage = per * NR * h8;
    const int64_t step = int64_t(gridDim.x) * per * NR, row0 = (int64_t(blockIdx.x) * per + g.index) * NR;
    int64_t ask_row = row0;
    const X *ask_x = static_cast<const X *>(p.x) + row0 * p.ldx;
    auto ask = [&](int st) {
#pragma unroll
        for (int k = 0; k < NR; ++k)
            if (ask_row + k < p.rows) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    copy_vec(ring + st * stage + k * h8, ask_x + k * p.ldx, (r * width + t) * 8, h);
            }
        copy_commit();
        ask_row += step;
        ask_x += step * p.ldx;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) ask(k);
    if (g.index == 0) {
        stage_param<R>(gamma, p.gamma, p.p_f32, 1.0f, h, h8, width, t);
        stage_param<R>(beta, p.beta, p.p_f32, 0.0f, h, h8, width, t);
    }
    __syncthreads();
    const float inv_h = 1.0f / float(h);
    int st = 0, flip = 0;
    Y *y = static_cast<Y *>(p.out) + row0 * p.ldo;
    for (int64_t row = row0; row < p.rows; row += step) {
        ask(st == 0 ? S - 1 : st - 1);
        copy_wait<S - 1>();
        const bool second = NR > 1 && row + 1 < p.rows;   // its buffer holds an older row if not
        Share<R> f[NR];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
#pragma unroll
            for (int k = 0; k < NR; ++k) f[k].x[r] = c < h ? load8(ring + st * stage + k * h8 + c) : fill(0.0f);
        }
        float mean[NR], rstd[NR];
        rows_sum(total(f[0]), NR > 1 ? total(f[NR - 1]) : 0.0f, g, sums[flip][0], mean);
#pragma unroll
        for (int k = 0; k < NR; ++k) mean[k] = quotient(mean[k], float(h), inv_h);
        rows_sum(squares(f[0], mean[0], width, t, h), NR > 1 ? squares(f[NR - 1], mean[NR - 1], width, t, h) : 0.0f, g,
                 sums[flip][1], rstd);
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            rstd[k] = rsqrtf(rstd[k] * inv_h + p.eps);
            if (t == 0 && (k == 0 || second)) {
                if (p.mean) p.mean[row + k] = mean[k];
                if (p.rstd) p.rstd[row + k] = rstd[k];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            if (c >= h) break;
            const V8 w = staged_param(gamma, c, h8), b = staged_param(beta, c, h8);
            store_row8(y, c, h, scaled(f[0].x[r], mean[0], rstd[0], w, b));
            if (second) store_row8(y + p.ldo, c, h, scaled(f[NR - 1].x[r], mean[NR - 1], rstd[NR - 1], w, b));
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
    let_next_start();
    wait_for_previous();
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
    const float mean = quotient(row_sum(total(f), g, row_buf(sums[0], g, 1)), float(h), inv_h);
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
    let_next_start();
    wait_for_previous();
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
//
// G: type of the staged gamma, fp32, or bf16 where that is what it came as and
// the longer rows leave no room for more.
//
// SPLIT: rows too long for one CTA are shared by a cluster of two, the first
// half of the columns in one and the second in the other; they exchange a
// row's two sums through shared memory.
template <typename X, typename Y, typename G, int R, int S, bool SPLIT>
__global__ void __launch_bounds__(kRingThreads, 1) cm_layer_norm_backward_ring_kernel(const __grid_constant__ NormParams p,
                                                                                      int width) {
    let_next_start();
    wait_for_previous();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float sums[2][kRowBuf];
    __shared__ float other[SPLIT ? 4 : 1];
    const Group g(width);
    const int t = int(threadIdx.x) - g.index * width, per = int(blockDim.x) / width;
    const Columns cols(p.h, SPLIT);
    const int h = cols.count, h8 = (cols.half + 7) / 8 * 8, c0 = cols.first;
    G *const gamma = reinterpret_cast<G *>(smem);
    uint8_t *const ring = smem + h8 * int(sizeof(G));
    const int xs = h8 * int(sizeof(X)), ys = h8 * int(sizeof(Y));
    const int row_bytes = xs + ys + (p.res ? xs : 0);
    const int64_t step = int64_t(cols.ctas) * per, row0 = int64_t(cols.cta) * per + g.index;
    auto slot = [&](int st) { return ring + (st * per + g.index) * row_bytes; };
    int64_t ask_row = row0;
    const X *ask_x = static_cast<const X *>(p.x) + row0 * p.ldx + c0;
    const X *ask_r = static_cast<const X *>(p.res) + row0 * p.ldr + c0;
    const Y *ask_y = static_cast<const Y *>(p.dy) + row0 * p.lddy + c0;
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
    V8 a[R], b[R];
    if (g.index == 0) {   // all loads before the first store
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            a[r] = c < h ? load_param8(p.gamma, p.p_f32, 1.0f, c0 + c, c0 + h) : fill(0.0f);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            if (c < h) store8(gamma + c, a[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) a[r] = b[r] = fill(0.0f);
    __syncthreads();
    const float inv_h = 1.0f / float(p.h);
    float mean = 0.0f, rstd = 0.0f;
    if (row0 < p.rows) {
        mean = p.mean[row0];
        rstd = p.rstd[row0];
    }
    int st = 0, flip = 0;
    X *dx = static_cast<X *>(p.out) + row0 * p.ldo + c0;
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
        float2 rowsum = row_sum2(sum(q1), sum(q2), g, row_buf(sums[flip], g, 2));
        if constexpr (SPLIT) {   // one row a step (per = 1): both CTAs make the same steps
            if (threadIdx.x == 0) other[2 * flip + 1] = rowsum.y;
            const float x = with_other(rowsum.x, &other[2 * flip], cols.rank), o = of_other(&other[2 * flip + 1], cols.rank);
            rowsum = make_float2(x, cols.rank == 0 ? rowsum.y + o : o + rowsum.y);
        }
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
    if constexpr (SPLIT) dev::cluster_sync();   // the other CTA has read this one's last sums
    if (!p.partial) return;
    float *const mine = p.partial + int64_t(cols.cta) * 2 * p.h + c0;
    if (per == 1) {
        const bool whole = p.h % 8 == 0;   // every part's row starts on 16 bytes
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * width + t) * 8;
            if (whole && c < h) {
                store8(mine + c, a[r]);
                store8(mine + p.h + c, b[r]);
                continue;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = parts(a[r].p[i]), v = parts(b[r].p[i]);
                if (c + 2 * i < h) mine[c + 2 * i] = u.x, mine[p.h + c + 2 * i] = v.x;
                if (c + 2 * i + 1 < h) mine[c + 2 * i + 1] = u.y, mine[p.h + c + 2 * i + 1] = v.y;
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
    let_next_start();
    wait_for_previous();
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

constexpr int kColY = 8;   // row lanes of a CTA, or 32 for few rows; its 32 column lanes hold V columns each

// out[c] (+)= s, if there is an output
__device__ __forceinline__ void put_sum(void *out, int f32, int accumulate, int64_t c, float s) {
    if (!out) return;
    if (f32) {
        float *o = static_cast<float *>(out) + c;
        *o = accumulate ? *o + s : s;
    } else {
        bf16 *o = static_cast<bf16 *>(out) + c;
        from_f(o, accumulate ? to_f(*o) + s : s);
    }
}

// Bound by memory for long sums, by the launch for short ones: a CTA takes a
// chunk of rows and 256 columns, so that a row's reads are 512 neighbouring bytes.
// A weight gradient without the bias's sums and with them: rows 300, 1024 x 1024
// 4.9 and 9.4 us; 65536, 256 x 256 33 and 50; 1813, 483 x 24629 46 and 74; whether
// the sums come before the product or after it is one.
// Partial sums over the rows of chunk blockIdx.y.  STATS: [chunk][2][h] of
// dy xh and dy; otherwise [chunk][h] of dy.
template <typename X, typename Y, int V, bool STATS, int kY>
__global__ void __launch_bounds__(32 * kY) cm_colsum_kernel(NormParams p) {
    let_next_start();
    wait_for_previous();
    __shared__ float sm[STATS ? 2 : 1][kY][32 * V];
    const int tx = int(threadIdx.x) & 31, ty = int(threadIdx.x) >> 5;
    const int64_t c = (int64_t(blockIdx.x) * 32 + tx) * V;
    const int64_t r0 = p.rows * blockIdx.y / gridDim.y, r1 = p.rows * (blockIdx.y + 1) / gridDim.y;
    float a[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = b[i] = 0.0f;
    if (c < p.h) {
#pragma unroll 8
        for (int64_t r = r0 + ty; r < r1; r += kY) {
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
    for (int j = threadIdx.x; j < 32 * V; j += 32 * kY) {
        const int64_t cc = int64_t(blockIdx.x) * 32 * V + j;
        if (cc >= p.h) continue;
        float sb = 0.0f, sa = 0.0f;
        for (int k = 0; k < kY; ++k) {
            sb += sm[0][k][j];
            if constexpr (STATS) sa += sm[1][k][j];
        }
        if (gridDim.y == 1) {   // a chunk that is all rows: the result itself
            put_sum(p.dgamma, p.g_f32, p.accumulate, cc, sa);
            put_sum(p.dbeta, p.g_f32, p.accumulate, cc, sb);
        } else if constexpr (STATS) {
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
    let_next_start();
    wait_for_previous();
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
    put_sum(out, f32, accumulate, c, s);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMostSms = 160;

constexpr int kDevices = 64;

// SMs of the current device and its number (looked up once a device).
int sm_count(int *device = nullptr) {
    static std::atomic<int> cached[kDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) dev = 0;
    if (device) *device = dev;
    if (const int c = cached[dev].load(std::memory_order_relaxed)) return c;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    n = std::min(n, kMostSms);
    cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Chunks of rows for the column sums: enough CTAs for two rounds of the SMs, at
// least 64 rows each, and no more than 304, whose sums the second launch adds;
// few rows are one chunk, whose sum is the result.  65536 x 256: 18 us, with
// 128 chunks at most 25.
int64_t chunks_for(int64_t rows, int64_t cols) {
    if (rows <= 128) return 1;
    const int64_t blocks = (cols + 255) / 256;
    return std::max<int64_t>(1, std::min({(rows + 63) / 64, std::max<int64_t>(1, 608 / blocks), int64_t(304)}));
}

constexpr int64_t kRingSmem = 224 * 1024;   // of 227 KB; the kernels' own buffers take up to 2

// The sums over rows of the partial sums of `parts` CTAs.
cudaError_t sum_parts(const float *partial, int64_t parts, int64_t h, int64_t stride, void *out0, void *out1, int f32,
                      int accumulate, cudaStream_t stream) {
    return launch_after(cm_sum_parts_kernel, dim3(unsigned((h + 31) / 32), stride > h ? 2 : 1), 256, 0, 1, stream, partial,
                        parts, h, stride, out0, out1, f32, accumulate);
}

int row_width(int64_t vecs, int R) { return int((vecs + 32 * R - 1) / (32 * R)) * 32; }

// Geometry of a persistent launch over rows of h elements: R vectors a thread,
// `per` rows at a time of `width` threads each, S row buffers a group.  As many
// rows as the threads and shared memory hold with two buffers each, then a third
// buffer if it fits; one CTA an SM.  ctas = 0 where a row is too long.
struct RingPlan {
    int R = 0, S = 0, width = 0, per = 1;
    int64_t ctas = 0, smem = 0;
};

// rows: how many there are for the groups to share; row_bytes: ring bytes a
// column and buffer; fixed_bytes: bytes a column outside the ring; most_per:
// groups at most (15 have a barrier each).
RingPlan ring_plan(int64_t rows, int64_t h, int64_t row_bytes, int64_t fixed_bytes, int most_r, int most_per, int sms) {
    RingPlan r;
    const int64_t vecs = (h + 7) / 8, limit = kRingSmem;
    r.R = vecs < 64 ? 1 : vecs < 128 ? 2 : most_r;
    r.width = row_width(vecs, r.R);
    if (r.width > kRingThreads) return r;
    const int64_t row = vecs * 8 * row_bytes, fixed = vecs * 8 * fixed_bytes;
    for (r.per = std::min(kRingThreads / r.width, most_per); r.per > 1 && fixed + 2 * r.per * row > limit;)
        --r.per;
    r.S = fixed + 3 * r.per * row <= limit ? 3 : 2;
    r.smem = fixed + r.S * r.per * row;
    if (r.smem > limit) return r;
    r.ctas = std::min<int64_t>(sms, (rows + r.per - 1) / r.per);
    return r;
}

// Launches a persistent kernel, in clusters of two CTAs a row if `split`.
template <auto kernel>
cudaError_t launch_ring(const NormParams &p, const RingPlan &r, bool split, cudaStream_t stream) {
    static std::atomic<bool> prepared[kDevices];   // setting it twice does no harm
    int dev = 0;
    sm_count(&dev);
    if (!prepared[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kRingSmem));
        if (e != cudaSuccess) return e;
        prepared[dev].store(true, std::memory_order_release);
    }
    return launch_after(kernel, dim3(unsigned(split ? 2 * r.ctas : r.ctas)), unsigned(r.width * r.per), size_t(r.smem),
                        split ? 2 : 1, stream, p, r.width);
}

template <typename X, typename Y, int R, int NR, int S>
cudaError_t forward_ring(const NormParams &p, const RingPlan &r, cudaStream_t stream) {
    return launch_ring<cm_layer_norm_ring_kernel<X, Y, R, NR, S>>(p, r, false, stream);
}

template <typename X, typename Y>
cudaError_t forward(const NormParams &p, cudaStream_t stream) {
    const int64_t vecs = (p.h + 7) / 8;
    const bool vec = aligned16(p.x) && aligned16(p.out) && aligned16(p.gamma) && aligned16(p.beta) && p.ldx % 8 == 0 &&
                     p.ldo % 8 == 0 && vecs <= 4096;
    if (p.rows > 0x7fffffff) return cudaErrorInvalidValue;
    if (!vec) {
        return launch_after(cm_layer_norm_any_kernel<X, Y>, dim3(unsigned(p.rows)), 512, 0, 1, stream, p);
    }
    const int sms = sm_count();
    // the register kernel: all of a row's loads at once
    const int R = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
    const int width = row_width(vecs, R), per = std::max(1, 128 / width);
    // The ring pays once that kernel would take more than two rounds of CTAs
    // (1024 threads an SM).  Rows of 8192 in bf16: 152 rows 3.6 us in registers
    // and 6.4 in the ring, 304 6.6 and 6.5, 600 12.3 and 6.6; rows of 2048:
    // 1200 5.0 and 6.5, 2400 9.0 and 6.7.  Rows longer than 16384 fit no ring;
    // 2000 of 28672 take 93 us.
    if (p.rows > 2 * int64_t(sms) * std::max(1, 1024 / (width * per)) * per) {
        if (vecs <= 1024) {
            const RingPlan r = ring_plan((p.rows + 1) / 2, p.h, 2 * sizeof(X), 8, 4, 15, sms);
            if (r.ctas > 0 && r.R == 4)
                return r.S == 3 ? forward_ring<X, Y, 4, 2, 3>(p, r, stream) : forward_ring<X, Y, 4, 2, 2>(p, r, stream);
            if (r.ctas > 0 && r.S == 3)   // rows this short leave room for three
                return r.R == 1 ? forward_ring<X, Y, 1, 2, 3>(p, r, stream) : forward_ring<X, Y, 2, 2, 3>(p, r, stream);
        } else {
            const RingPlan r = ring_plan(p.rows, p.h, sizeof(X), 8, 4, 15, sms);
            if (r.ctas > 0)
                return r.S == 3 ? forward_ring<X, Y, 4, 1, 3>(p, r, stream) : forward_ring<X, Y, 4, 1, 2>(p, r, stream);
        }
    }
    const unsigned grid = unsigned((p.rows + per - 1) / per), threads = unsigned(width * per);
    return launch_after(R == 1   ? cm_layer_norm_kernel<X, Y, 1>
                        : R == 2 ? cm_layer_norm_kernel<X, Y, 2>
                                 : cm_layer_norm_kernel<X, Y, 4>,
                        dim3(grid), threads, 0, 1, stream, p, width);
}

template <typename X, typename Y, int R, int S, bool SPLIT = false, typename G = float>
cudaError_t backward_ring(const NormParams &p, const RingPlan &r, cudaStream_t stream) {
    return launch_ring<cm_layer_norm_backward_ring_kernel<X, Y, G, R, S, SPLIT>>(p, r, SPLIT, stream);
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
        const int64_t bytes = int64_t(sizeof(X)) * (p.res ? 2 : 1) + int64_t(sizeof(Y));
        const int sms = sm_count();
        RingPlan r = ring_plan(p.rows, p.h, bytes, 4, 4, 15, sms);
        cudaError_t e = cudaErrorInvalidValue;
        if (r.ctas > 0) {
            e = r.S == 3 ? (r.R == 1   ? backward_ring<X, Y, 1, 3>(p, r, stream)
                            : r.R == 2 ? backward_ring<X, Y, 2, 3>(p, r, stream)
                                       : backward_ring<X, Y, 4, 3>(p, r, stream))
                         : (r.R == 1   ? backward_ring<X, Y, 1, 2>(p, r, stream)
                            : r.R == 2 ? backward_ring<X, Y, 2, 2>(p, r, stream)
                                       : backward_ring<X, Y, 4, 2>(p, r, stream));
        } else if (r = ring_plan(p.rows, p.h, bytes, 2, 4, 1, sms); r.ctas > 0 && !(p.gamma && p.p_f32)) {
            e = r.S == 3 ? backward_ring<X, Y, 4, 3, false, bf16>(p, r, stream)
                         : backward_ring<X, Y, 4, 2, false, bf16>(p, r, stream);
        } else if (r = ring_plan(p.rows, (p.h + 15) / 16 * 8, bytes, 4, 4, 1, sms / 2); r.ctas > 0) {
            e = r.S == 3 ? backward_ring<X, Y, 4, 3, true>(p, r, stream) : backward_ring<X, Y, 4, 2, true>(p, r, stream);
        }
        if (r.ctas > 0 && (e != cudaSuccess || !sums)) return e;
        if (r.ctas > 0) {
            return sum_parts(p.partial, r.ctas, p.h, 2 * p.h, p.dgamma, p.dbeta, p.g_f32, p.accumulate, stream);
        }
    }
    cudaError_t e = launch_after(vec ? cm_layer_norm_dx_any_kernel<X, Y, 8> : cm_layer_norm_dx_any_kernel<X, Y, 1>,
                                 dim3(unsigned(p.rows)), 512, 0, 1, stream, p);
    if (e != cudaSuccess || !sums) return e;
    const int64_t chunks = chunks_for(p.rows, p.h);
    const int per_cta = in_vec ? 256 : 32;   // columns
    e = launch_after(in_vec ? cm_colsum_kernel<X, Y, 8, true, kColY> : cm_colsum_kernel<X, Y, 1, true, kColY>,
                     dim3(unsigned((p.h + per_cta - 1) / per_cta), unsigned(chunks)), 32 * kColY, 0, 1, stream, p);
    if (e != cudaSuccess || chunks == 1) return e;
    return sum_parts(p.partial, chunks, p.h, 2 * p.h, p.dgamma, p.dbeta, p.g_f32, p.accumulate, stream);
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
    p.dbeta = out;
    p.g_f32 = out_f32;
    p.accumulate = accumulate;
    const int64_t chunks = chunks_for(rows, cols);
    const cudaError_t e = launch_after(chunks == 1 ? cm_colsum_kernel<bf16, bf16, 8, false, 32>
                                                   : cm_colsum_kernel<bf16, bf16, 8, false, kColY>,
                                       dim3(unsigned((cols + 255) / 256), unsigned(chunks)),
                                       32 * (chunks == 1 ? 32 : kColY), 0, 1, stream, p);
    if (e != cudaSuccess || chunks == 1) return e;
    return sum_parts(partial, chunks, cols, cols, out, nullptr, out_f32 ? 1 : 0, accumulate ? 1 : 0, stream);
}

}  // namespace cm
