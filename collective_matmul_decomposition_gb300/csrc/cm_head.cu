// cm_head.cu -- around the products of the loss over a vocabulary: the rows that
// have a target are gathered in front of them, the parts' statistics joined and the
// input's gradient put back in its rows behind them.
//
// Rows without a target cost nothing in the products, whose tiles end at the last
// slot, and whatever they hold (infinities, NaN) meets no sum.
#include <cuda_bf16.h>

#include <algorithm>

#include "cm_launch.cuh"
#include "cm_linear.cuh"
#include "cm_vec.cuh"

namespace cm {
namespace {

using namespace vec;

constexpr int kRowsThreads = 256, kRowsMost = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int64_t target_of(const HeadRows &p, int64_t row) {
    return p.target_bits == 64 ? static_cast<const int64_t *>(p.targets)[row]
                               : int64_t(static_cast<const int32_t *>(p.targets)[row]);
}

// The largest of the magnitudes that are finite.
__device__ __forceinline__ float larger(float a, float b) {
    b = fabsf(b);
    return b <= 3.0e38f ? fmaxf(a, b) : a;
}

// A CTA places 4 to 64 rows (`per`: 1003 rows of 4101 elements in 64s 86 us, on 16
// SMs, now 15).  It counts all rows' targets itself, which costs a pass over them from L2
// (rows^2 / per of them in all, little beside the products' rows K n), and saves a
// launch and a scan across CTAs.
//
// The gradients' factors are kept relative to the largest of them (scale), by which the
// results are multiplied at the end in fp32: the bf16 gradient of a logit then does not
// carry the rounding of a common factor such as 1 / rows.
__global__ void __launch_bounds__(kRowsThreads) cm_head_rows_kernel(const HeadRows p, int per) {
    __shared__ int counts[2][kRowsThreads / 32];
    __shared__ float tops[kRowsThreads / 32];
    __shared__ int slots[kRowsMost];
    let_next_start();
    wait_for_previous();
    const int64_t r0 = int64_t(blockIdx.x) * per, r1 = min(p.rows, r0 + per);
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    int before = 0, all = 0;
    float top = 0.0f;
#pragma unroll 4
    for (int64_t r = threadIdx.x; r < p.rows; r += kRowsThreads) {
        const int64_t t = target_of(p, r);
        const float a = p.dloss ? p.dloss[r] : 0.0f, b = p.dlse ? p.dlse[r] : 0.0f;   // read whether it counts or not
        if (t < 0) continue;
        ++all;
        before += r < r0;
        top = larger(larger(top, a), a + b);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (lane == 0) counts[0][warp] = before, counts[1][warp] = all, tops[warp] = top;
    __syncthreads();
    before = all = 0, top = 0.0f;
#pragma unroll
    for (int i = 0; i < kRowsThreads / 32; ++i) before += counts[0][i], all += counts[1][i], top = fmaxf(top, tops[i]);
    const float scale = top > 0.0f ? top : 1.0f;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.count = all;
        if (p.scale) *p.scale = scale;
    }
    if (warp == 0) {   // the CTA's rows, in order
        for (int i = 0; i < per; i += 32) {
            const int64_t r = r0 + i + lane;
            const int64_t t = r < r1 ? target_of(p, r) : -1;
            const uint32_t live = __ballot_sync(0xffffffffu, t >= 0);
            const int slot = t >= 0 ? before + __popc(live & ((1u << lane) - 1)) : -1;
            before += __popc(live);
            if (r >= r1) continue;
            slots[i + lane] = slot;
            if (p.slot_of) p.slot_of[r] = slot;
            if (slot < 0) {
                if (p.loss) p.loss[r] = 0.0f;
                if (p.lse_out) p.lse_out[r] = 0.0f;
                if (p.picked_out) p.picked_out[r] = 0.0f;
                continue;
            }
            p.target[slot] = t >= p.vocab ? kNoToken : t >= p.first && t - p.first < p.n ? int32_t(t - p.first) : kNotHere;
            if (p.row_of) p.row_of[slot] = int32_t(r);
            if (p.picked) p.picked[slot] = 0.0f;
            if (p.dloss) {
                // a target beyond the vocabulary: NaN, as its loss
                const float a = t >= p.vocab ? __int_as_float(0x7fffffff) : p.dloss[r];
                p.hit[slot] = a / scale;
                p.grad[slot] = (p.dlse ? a + p.dlse[r] : a) / scale;
                p.lse2[slot] = p.lse[r] * kLog2e;
            }
        }
    }
    if (all == p.rows && !p.always) return;   // the products read x itself
    __syncthreads();
    const int K = int(p.K), nv = (K + 7) / 8;
    const bf16 *x = static_cast<const bf16 *>(p.x);
    bf16 *xs = static_cast<bf16 *>(p.xs);
    const int total = int(r1 - r0) * nv;
    for (int at = int(threadIdx.x); at < total; at += 4 * kRowsThreads) {   // four loads before the first store
        V8 f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = at + k * kRowsThreads, i = j / nv;
            if (j < total && slots[i] >= 0) f[k] = load_row8(x + (r0 + i) * p.ldx, (j - i * nv) * 8, K);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = at + k * kRowsThreads, i = j / nv;
            if (j < total && slots[i] >= 0) store_row8(xs + int64_t(slots[i]) * p.ldxs, (j - i * nv) * 8, K, f[k]);
        }
    }
    // zeros behind the last slot: where a product's contraction reads on to its slice's end
    const int64_t end = p.always ? p.rows : min(p.rows, int64_t(max(all, 1) + 63) / 64 * 64);
    const V8 zero = fill(0.0f);
    for (int64_t s = max(r0, int64_t(all)) + warp; s < min(r1, end); s += kRowsThreads / 32)
        for (int v = lane; v < nv; v += 32) store_row8(xs + s * p.ldxs, v * 8, K, zero);
}

// {m, s}: m the largest in powers of two, s the sum of 2^(. - m).
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x), base = m == -INFINITY ? 0.0f : m;
    return make_float2(m, a.y * exp2f(a.x - base) + b.y * exp2f(b.x - base));
}

// A CTA joins the parts of eight slots: eight lanes of a warp read one part of them (64
// neighbouring bytes), its four groups of lanes four parts, its 16 warps 64; a thread
// has eight loads under way.  Then the groups' and the warps' results are joined in order.
// 8192 rows of 1024 parts take 27 us, one row of 256 3 (32 slots a CTA, one to a lane: 39
// and 8).
constexpr int kJoinWarps = 16, kJoinSlots = 8, kJoinAtOnce = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) cm_head_join_kernel(const HeadJoin p) {
    __shared__ float2 part[kJoinWarps][kJoinSlots];
    let_next_start();
    wait_for_previous();
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    const int64_t slot = int64_t(blockIdx.x) * kJoinSlots + lane % kJoinSlots;
    const int count = *p.count;
    if (int64_t(blockIdx.x) * kJoinSlots >= count) return;
    constexpr int kStep = kJoinWarps * (32 / kJoinSlots);
    float2 a = make_float2(-INFINITY, 0.0f);
    if (slot < count)
        for (int64_t k = warp * (32 / kJoinSlots) + lane / kJoinSlots; k < p.parts; k += kStep * kJoinAtOnce) {
            float2 b[kJoinAtOnce];
#pragma unroll
            for (int i = 0; i < kJoinAtOnce; ++i)
                b[i] = k + i * kStep < p.parts ? p.stat[(k + i * kStep) * p.stride + slot] : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int i = 0; i < kJoinAtOnce; ++i) a = join(a, b[i]);
        }
#pragma unroll
    for (int o = kJoinSlots; o < 32; o *= 2) {
        const float2 b = make_float2(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o));
        a = join(a, b);   // the same in both lanes: a sum of two
    }
    if (lane < kJoinSlots) part[warp][lane] = a;
    __syncthreads();
    if (warp || lane >= kJoinSlots || slot >= count) return;
#pragma unroll
    for (int i = 1; i < kJoinWarps; ++i) a = join(a, part[i][lane]);
    const float lse = (a.x + log2f(a.y)) * kLn2, picked = p.picked[slot];
    const int32_t row = p.row_of[slot];
    if (p.loss) p.loss[row] = p.target[slot] == kNoToken ? __int_as_float(0x7fffffff) : lse - picked;
    if (p.lse) p.lse[row] = lse;
    if (p.picked_out) p.picked_out[row] = picked;
}

// Half a CTA a row, four vectors a thread under way.  Bound by memory and, at 8.7 us for
// 2048 x 2048, by its launch.
template <typename T>
__global__ void __launch_bounds__(256) cm_head_scatter_kernel(const HeadScatter p) {
    let_next_start();
    wait_for_previous();
    const int half = int(threadIdx.x) >> 7, at = int(threadIdx.x) & 127, K = int(p.K);
    const int64_t row = int64_t(blockIdx.x) * 2 + half;
    if (row >= p.rows) return;
    const int32_t slot = p.slot_of[row];
    const float scale = *p.scale;
    T *to = static_cast<T *>(p.dx) + row * p.lddx;
    const float *from = p.sum + int64_t(max(slot, 0)) * p.ld;
    for (int c = at * 8; c < K; c += 4096) {
        V8 f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = fill(0.0f);
            if (slot >= 0 && c + 1024 * k < K) f[k] = load_row8(from, c + 1024 * k, K);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[k].p[i] = mul(f[k].p[i], both(scale));
            if (c + 1024 * k < K) store_row8(to, c + 1024 * k, K, f[k]);
        }
    }
}

}  // namespace

cudaError_t launch_head_rows(const HeadRows &p, cudaStream_t stream) {
    const int per = int(std::max<int64_t>(4, std::min<int64_t>(kRowsMost, p.rows / 512 / 4 * 4)));
    return launch_after(cm_head_rows_kernel, dim3(unsigned((p.rows + per - 1) / per)), kRowsThreads, 0, 1, stream, p, per);
}
cudaError_t launch_head_join(const HeadJoin &p, cudaStream_t stream) {
    return launch_after(cm_head_join_kernel, dim3(unsigned((p.stride + kJoinSlots - 1) / kJoinSlots)), 32 * kJoinWarps, 0, 1, stream, p);
}
cudaError_t launch_head_scatter(const HeadScatter &p, cudaStream_t stream) {
    return launch_after(p.dx_f32 ? cm_head_scatter_kernel<float> : cm_head_scatter_kernel<bf16>, dim3(unsigned((p.rows + 1) / 2)), 256, 0,
                        1, stream, p);
}

}  // namespace cm
