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

constexpr int kRowsThreads = 256, kRowsWarps = kRowsThreads / 32, kRowsMost = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int64_t target_of(const HeadRows &p, int64_t row) {
    return p.target_bits == 64 ? static_cast<const int64_t *>(p.targets)[row]
                               : int64_t(static_cast<const int32_t *>(p.targets)[row]);
}

// The largest of the magnitudes that are finite.
__device__ __forceinline__ float larger(float a, float b) {
    b = fabsf(b);
    return b < INFINITY ? fmaxf(a, b) : a;
}

// Counts of a CTA's threads, summed; the same in all of them.
struct Counted {
    int before, all;
    float top;
};
__device__ __forceinline__ Counted over_cta(Counted c) {
    __shared__ Counted warps[kRowsWarps];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        c.before += __shfl_xor_sync(0xffffffffu, c.before, o);
        c.all += __shfl_xor_sync(0xffffffffu, c.all, o);
        c.top = fmaxf(c.top, __shfl_xor_sync(0xffffffffu, c.top, o));
    }
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = c;
    __syncthreads();
    c = {0, 0, 0.0f};
#pragma unroll
    for (int i = 0; i < kRowsWarps; ++i) c = {c.before + warps[i].before, c.all + warps[i].all, fmaxf(c.top, warps[i].top)};
    return c;
}

// The rows r0 .. r1 - 1 that have a target: those in front of row `split`, all, and the
// largest of their factors.
__device__ __forceinline__ Counted count_rows(const HeadRows &p, int64_t r0, int64_t r1, int64_t split) {
    Counted c = {0, 0, 0.0f};
#pragma unroll 4
    for (int64_t r = r0 + threadIdx.x; r < r1; r += kRowsThreads) {
        const int64_t t = target_of(p, r);
        const float a = p.dloss ? p.dloss[r] : 0.0f, b = p.dlse ? p.dlse[r] : 0.0f;   // read whether it counts or not
        if (t < 0) continue;
        ++c.all;
        c.before += r < split;
        c.top = larger(larger(c.top, a), a + b);
    }
    return over_cta(c);
}

// Many rows: a CTA counts a group of `per` of them.
__global__ void __launch_bounds__(kRowsThreads) cm_head_count_kernel(const HeadRows p, int64_t per) {
    let_next_start();
    wait_for_previous();
    const int64_t r0 = int64_t(blockIdx.x) * per;
    const Counted c = count_rows(p, r0, min(p.rows, r0 + per), r0);
    if (threadIdx.x == 0) p.groups[blockIdx.x] = {c.all, c.top};
}

// A CTA places a group of `per` rows, `step` (4 to 64) at a time; up to kHeadRowsOnce rows
// in one step (1003 rows of 4101 elements in 64s 86 us, on 16 SMs, in 4s 15).  Then
// it counts all rows' targets itself, which costs a pass over them from L2, and saves a
// launch and a scan across CTAs; beyond that the passes would cost more (rows^2 / per
// targets in all: 2^20 rows of 8 elements over 8 columns took 7.2 ms, now 0.55), and it adds up the
// groups' counts instead.
//
// The gradients' factors are kept relative to the largest of them (scale), by which the
// results are multiplied at the end in fp32: the bf16 gradient of a logit then does not
// carry the rounding of a common factor such as 1 / rows.
template <bool GROUPS>
__global__ void __launch_bounds__(kRowsThreads, 4) cm_head_rows_kernel(const HeadRows p, int64_t per, int step) {
    __shared__ int slots[kRowsMost];
    let_next_start();
    wait_for_previous();
    const int64_t g0 = int64_t(blockIdx.x) * per, g1 = min(p.rows, g0 + per);
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    Counted counted = {0, 0, 0.0f};
    if constexpr (!GROUPS) {
        counted = count_rows(p, 0, p.rows, g0);
    } else {
        for (int i = int(threadIdx.x); i < int(gridDim.x); i += kRowsThreads) {
            const HeadGroup g = p.groups[i];
            counted = {counted.before + (i < int(blockIdx.x) ? g.count : 0), counted.all + g.count, fmaxf(counted.top, g.top)};
        }
        counted = over_cta(counted);
    }
    const int all = counted.all;
    int before = counted.before;   // of warp 0: rows with a target in front of the step
    const float scale = counted.top > 0.0f ? counted.top : 1.0f;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.count = all;
        if (p.scale) *p.scale = scale;
    }
    const int K = int(p.K), nv = (K + 7) / 8;
    const bf16 *x = static_cast<const bf16 *>(p.x);
    bf16 *xs = static_cast<bf16 *>(p.xs);
    // zeros behind the last slot: where a product's contraction reads on to its slice's end
    const int64_t end = p.always ? p.rows : min(p.rows, int64_t(max(all, 1) + 63) / 64 * 64);
    for (int64_t r0 = g0; r0 < g1; r0 += step) {
        const int64_t r1 = GROUPS ? min(g1, r0 + step) : g1;
        if (warp == 0) {   // the step's rows, in order
            for (int i = 0; i < step; i += 32) {
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
        if (all == p.rows && !p.always) {   // the products read x itself
            if (GROUPS) continue;
            return;
        }
        __syncthreads();
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
        const V8 zero = fill(0.0f);
        for (int64_t s = max(r0, int64_t(all)) + warp; s < min(r1, end); s += kRowsWarps)
            for (int v = lane; v < nv; v += 32) store_row8(xs + s * p.ldxs, v * 8, K, zero);
        if constexpr (!GROUPS) return;
        __syncthreads();   // the slots have been read
    }
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
    const int step = int(std::max<int64_t>(4, std::min<int64_t>(kRowsMost, p.rows / 512 / 4 * 4)));
    int64_t per = step;
    if (p.rows > kHeadRowsOnce) {   // whole steps a group
        per = (p.rows + kHeadGroups * step - 1) / (kHeadGroups * step) * step;
        const cudaError_t e = launch_after(cm_head_count_kernel, dim3(unsigned((p.rows + per - 1) / per)), kRowsThreads, 0, 1, stream, p, per);
        if (e != cudaSuccess) return e;
    }
    return launch_after(p.rows > kHeadRowsOnce ? cm_head_rows_kernel<true> : cm_head_rows_kernel<false>, dim3(unsigned((p.rows + per - 1) / per)), kRowsThreads, 0, 1, stream, p, per, step);
}
cudaError_t launch_head_join(const HeadJoin &p, cudaStream_t stream) {
    return launch_after(cm_head_join_kernel, dim3(unsigned((p.stride + kJoinSlots - 1) / kJoinSlots)), 32 * kJoinWarps, 0, 1, stream, p);
}
cudaError_t launch_head_scatter(const HeadScatter &p, cudaStream_t stream) {
    return launch_after(p.dx_f32 ? cm_head_scatter_kernel<float> : cm_head_scatter_kernel<bf16>, dim3(unsigned((p.rows + 1) / 2)), 256, 0,
                        1, stream, p);
}

}  // namespace cm
