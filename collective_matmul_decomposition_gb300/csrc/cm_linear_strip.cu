// cm_linear_strip.cu -- the linear layer's kernel for few rows (tokens).
//
// D[row][col] = sum_k B[row][k] A[col][k], with the weights' columns on the
// tensor core's 128-row side and 16 to 256 tokens on its column side: a call
// with one token wastes 15 of 16 accumulator columns but none of the weights'
// bandwidth, which bounds it (K*n*2 bytes are read for 2*K*n flops a token).
// One CTA computes one tile.  Where there are fewer tiles than SMs, the K
// slices of a tile are split over a cluster of up to eight CTAs: each leaves
// its fp32 partial tile in its own shared memory, and the cluster's CTAs add
// them in rank order, each for its share of the tokens, so one launch does it,
// nothing passes through global memory, and the result does not depend on timing.
//
// Bound by HBM where the weights are large: one token through 28672 x 8192 takes
// 69.7 us, 6738 GB/s.  A small call is bound by latency: one token through 4096 x
// 2048 takes 6.6 to 7.0 us, of which 2.5 are its bytes; the rest is starting, the first
// loads, and the sum over the cluster.  45 tokens through 8190 x 3579: 14.7 us for
// 8.8 us of bytes.
//
// Roles (128 threads): a thread of warp 0 issues the TMA loads, one of warp 1 the
// MMAs; then all four warps run the epilogue (a thread owns one column, so a
// warp's loads and stores are 32 neighbouring elements of one row).  Two CTAs
// fit on an SM: one's epilogue runs under the other's loads.
//
// Every wait is bounded by p.timeout_ns; on expiry the first failing thread
// records {code, tile, CTA, site}, and the CTA drains its loads, frees its
// tensor memory and returns.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "cm_device.cuh"
#include "cm_kernel.cuh"
#include "cm_launch.cuh"
#include "cm_linear.cuh"
#include "cm_linear_epilogue.cuh"

namespace cm {
namespace {

using namespace dev;

constexpr int kThreadsL = 128;
constexpr int kTileCols = 128;
constexpr int kStripA = kTileCols * kBK * 2;   // 16 KB of the column operand per slice
constexpr int kStripMaxStages = 12;

struct StripSmem {
    uint8_t *ring;
    uint64_t *full, *empty, *acc, *drain;
    uint32_t *tmem_slot;
    volatile int *abort;
};

__device__ __noinline__ void report_linear(LinearStatus *s, uint32_t site, uint32_t tile) {
    if (atomicCAS(&s->w[0], 0u, uint32_t(CM_ERR_TIMEOUT)) == 0u) {
        s->w[1] = tile;
        s->w[2] = blockIdx.x;
        s->w[3] = site;
        __threadfence();
    }
}

__device__ bool wait_l(const LinearStripParams &p, const StripSmem &s, uint64_t *bar, uint32_t parity, uint32_t site) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0u) {
            if (*s.abort) return false;
            if (globaltimer() - t0 > p.timeout_ns) {
                report_linear(p.status, site, blockIdx.x);
                *s.abort = 1;
                return false;
            }
        }
    }
}

__device__ void drain_l(const LinearStripParams &p, uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer() - t0 > p.timeout_ns) break;
}

// Sum over the cluster's partial tiles of one element, in rank order.
__device__ __forceinline__ float cluster_sum(uint32_t addr, int splits) {
    float f[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        f[r] = 0.0f;
        if (r < splits)
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f[r]) : "r"(mapa_shared(addr, uint32_t(r))) : "memory");
    }
    float v = f[0];
#pragma unroll
    for (int r = 1; r < 8; ++r)
        if (r < splits) v += f[r];
    return v;
}

// The epilogue of kBatch rows (row0 + k * step, those below `end`) of one
// column: every load of the batch before the first store, so that their
// latencies overlap.
constexpr int kBatch = 8;
__device__ __forceinline__ void finish(const LinearEpilogue &e, float (&v)[kBatch], float bias, int64_t row0, int64_t step,
                                       int64_t end, int64_t col) {
    float in[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) v[k] += bias;
    if (e.z) {
        __nv_bfloat16 *z = static_cast<__nv_bfloat16 *>(e.z) + row0 * e.ldz + col;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (row0 + k * step < end) z[k * step * e.ldz] = __float2bfloat16_rn(v[k]);
    }
    auto read = [&](const void *m, int64_t ld) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(m) + row0 * ld + col;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) in[k] = row0 + k * step < end ? __bfloat162float(p[k * step * ld]) : 0.0f;
    };
    if (e.dact) {
        read(e.zin, e.ldzin);
        lin::mul_dact(v, in, e.act);
    } else {
        lin::apply_act(v, e.act);
    }
    if (e.res) {
        read(e.res, e.ldr);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) v[k] += in[k];
    }
    if (e.y_f32) {
        float *y = static_cast<float *>(e.y) + row0 * e.ldy + col;
        if (e.accumulate) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) in[k] = row0 + k * step < end ? y[k * step * e.ldy] : 0.0f;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) v[k] += in[k];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (row0 + k * step < end) y[k * step * e.ldy] = v[k];
    } else {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(e.y) + row0 * e.ldy + col;
        if (e.accumulate) {
            read(e.y, e.ldy);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) v[k] += in[k];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (row0 + k * step < end) y[k * step * e.ldy] = __float2bfloat16_rn(v[k]);
    }
}

// The same for the gate's gradients: v is the gradient of act(g) u.
__device__ __forceinline__ void finish_gate_grad(const LinearEpilogue &e, float (&v)[kBatch], int64_t row0, int64_t step,
                                                 int64_t end, int64_t col) {
    float g[kBatch], u[kBatch];
    const int64_t in = row0 * e.ldzin + col;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const bool live = row0 + k * step < end;
        g[k] = live ? __bfloat162float(static_cast<const __nv_bfloat16 *>(e.zin)[in + k * step * e.ldzin]) : 0.0f;
        u[k] = live ? __bfloat162float(static_cast<const __nv_bfloat16 *>(e.zin2)[in + k * step * e.ldzin]) : 0.0f;
    }
    lin::gate_grad(v, g, u, e.act);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        if (row0 + k * step >= end) continue;
        static_cast<__nv_bfloat16 *>(e.z)[(row0 + k * step) * e.ldz + col] = __float2bfloat16_rn(g[k]);
        static_cast<__nv_bfloat16 *>(e.y)[(row0 + k * step) * e.ldy + col] = __float2bfloat16_rn(u[k]);
    }
}

// The gated product of the rows t, t + step, ... below `end` of a tile: the partial
// tiles of `splits` CTAs, [token][64 gate columns, 64 up columns], are summed in
// rank order; a thread takes one column of every other of those rows.  Bound as the plain
// strips: one token through 4096 x 2 2048 takes 7.5 us, 64 through 8192 x 2 3584 25 us.
__device__ __forceinline__ void finish_gated(const LinearEpilogue &e, const float *part, int splits, int t0, int step, int end,
                                             int64_t row0, int64_t col0, int64_t cols) {
    constexpr int kPairs = 4;
    const int j = int(threadIdx.x) & 63;
    const int64_t col = col0 + j;
    if (col >= cols) return;
    const float bg = lin::load_bias(e.bias, e.bias_f32, col), bu = lin::load_bias(e.bias2, e.bias_f32, col);
    for (int t = t0 + (int(threadIdx.x) >> 6) * step; t < end; t += 2 * kPairs * step) {
        float g[kPairs], u[kPairs];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            const int at = (t + 2 * k * step) * kTileCols + j;
            const bool live = t + 2 * k * step < end;
            g[k] = u[k] = 0.0f;
            if (!live) continue;
            g[k] = (splits > 1 ? cluster_sum(smem_u32(part + at), splits) : part[at]) + bg;
            u[k] = (splits > 1 ? cluster_sum(smem_u32(part + at + 64), splits) : part[at + 64]) + bu;
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            const int64_t row = row0 + t + 2 * k * step;
            if (!e.z || t + 2 * k * step >= end) continue;
            static_cast<__nv_bfloat16 *>(e.z)[row * e.ldz + col] = __float2bfloat16_rn(g[k]);
            static_cast<__nv_bfloat16 *>(e.z2)[row * e.ldz + col] = __float2bfloat16_rn(u[k]);
        }
        lin::apply_gate(g, u, e.act);
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
            if (t + 2 * k * step < end)
                static_cast<__nv_bfloat16 *>(e.y)[(row0 + t + 2 * k * step) * e.ldy + col] = __float2bfloat16_rn(g[k]);
    }
}

// The same for the logits' gradients: exp(v - lse) grad, less hit in the target's
// column; zeros behind the last slot.  One row, 4096 x 131072: 169 us, the weights' bytes.
__device__ __forceinline__ void finish_softgrad(const LinearEpilogue &e, const LinearHead &h, int count, float (&v)[kBatch],
                                                int64_t row0, int64_t step, int64_t end, int64_t col) {
    float lse2[kBatch], grad[kBatch], hit[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t row = row0 + k * step;
        lse2[k] = grad[k] = hit[k] = 0.0f;
        if (row >= end || row >= count) continue;
        lse2[k] = h.lse2[row];
        grad[k] = h.grad[row];
        hit[k] = h.target[row] == h.first + col ? h.hit[row] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t row = row0 + k * step;
        if (row >= end) continue;
        const float p = row < count ? lin::exp2_fast(fmaf(v[k], lin::kLog2e, -lse2[k])) * grad[k] - hit[k] : 0.0f;
        static_cast<__nv_bfloat16 *>(e.y)[row * e.ldy + col] = __float2bfloat16_rn(p);
    }
}

// The softmax statistics of a tile's 128 columns for the rows t0, t0 + step, ... below
// `end`: a warp takes every fourth of those rows, a lane four neighbouring columns.  The
// partial tiles are summed as above.  One row, 4096 x 32768: 42 us, 6.4 TB/s.
__device__ __forceinline__ void finish_stats(const LinearHead &h, int count, const float *part, int splits, int t0, int step,
                                             int end, int64_t row0, int64_t col0, int64_t cols) {
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    for (int t = t0 + warp * step; t < end && row0 + t < count; t += 4 * step) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = t * kTileCols + lane * 4 + i;
            f[i] = splits > 1 ? cluster_sum(smem_u32(part + at), splits) : part[at];
        }
        const int64_t row = row0 + t, col = col0 + lane * 4, target = h.target[row];
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (target == col + i && col + i < cols) h.picked[row] = f[i];
            if (col + i >= cols) f[i] = -INFINITY;
            top = fmaxf(top, f[i]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float m = top * lin::kLog2e, base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += lin::exp2_fast(fmaf(f[i], lin::kLog2e, -base));
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) h.stat[col0 / kTileCols * h.stride + row] = make_float2(m, sum);
    }
}

// The sums of accumulators 1 .. used - 1 added to the first one's, as bits of fp32.
__device__ __forceinline__ void add_parts(uint32_t taddr, uint32_t acc_cols, int used, uint32_t (&v)[32]) {
    for (int k = 1; k < used; ++k) {
        uint32_t u[32];
        tmem_ld32(taddr + uint32_t(k) * acc_cols, u);
        tmem_wait_ld_regs(u);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
    }
}

// The products of the loss's logits, in parts of at most kStatSlices slices, an accumulator
// each.  Where there are more parts than accumulators they are multiplied in rounds:
// behind each round the accumulators' sum goes to the first one, and the others take the
// next parts.  The ring is filled again meanwhile, and an SM's other CTA goes on.
// 64 rows, 8192 x 32768 (three rounds): the loss takes 124 us; 128 rows (seven) 130, as with one.
// Leaves how many accumulators hold a part or a sum in `used`; false after an expired wait,
// with the loader's place in the ring for what it has to wait for.
template <bool A_MN>
__device__ __forceinline__ bool multiply_parts(const LinearStripMore &p, const StripSmem &s, uint32_t tmem, uint32_t acc_cols, int accs,
                                               int col0, int row0, int nrows, int kb0, int kb1, int &used, int &stage, int &issued,
                                               uint32_t &phase) {
    const int warp = int(threadIdx.x) >> 5;
    const uint32_t stage_bytes = uint32_t(kStripA + p.tok * kBK * 2), taddr = tmem + (uint32_t(warp * 32) << 16);
    const int per_part = min(kStatSlices, (kb1 - kb0 + accs - 1) / accs);
    bool good = true;
    int next = kb0;   // the first slice that is not on its way yet
    for (int first = kb0, round = 0;; ++round) {
        const int kept = round ? 1 : 0, last = min(kb1, first + per_part * (accs - kept)), until = min(kb1, last + p.stages);
        used = kept + (last - first + per_part - 1) / per_part;
        if (warp == 0) {
            if (elect_one()) {
                for (int kb = next; kb < until; ++kb) {
                    if (!mbar_try_wait(&s.empty[stage], phase ^ 1u) && !wait_l(p, s, &s.empty[stage], phase ^ 1u, kLinSiteEmpty))
                        break;
                    uint8_t *sa = s.ring + uint32_t(stage) * stage_bytes, *sb = sa + kStripA;
                    mbar_expect_tx(&s.full[stage], stage_bytes);
                    if (A_MN) {
                        for (int j = 0; j < kTileCols / 64; ++j)
                            tma_load_3d(sa + j * (64 * kBK * 2), &p.tmA, &s.full[stage], col0 + 64 * j, kb * kBK, 0);
                    } else {
                        tma_load_3d(sa, &p.tmA, &s.full[stage], kb * kBK, col0, 0);
                    }
                    tma_load_3d(sb, &p.tmB, &s.full[stage], kb * kBK, row0, 0);
                    ++issued;
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (elect_one()) {
                const uint32_t idesc = idesc_bf16(kTileCols, p.tok, false, A_MN);
                constexpr uint32_t kALbo = A_MN ? 64 * kBK * 2 : 16, kAStep = A_MN ? (16 * 128) >> 4 : 32 >> 4;
                const uint64_t ad0 = desc_sw128(smem_u32(s.ring), kALbo, 1024);
                const uint64_t bd0 = desc_sw128(smem_u32(s.ring) + kStripA, 16, 1024);
                bool ok = true, ready = mbar_test_wait(&s.full[stage], phase);
                uint32_t d = tmem + uint32_t(kept) * acc_cols;
                for (int kb = first, left = per_part; kb < last; ++kb) {
                    if (!ready && !mbar_try_wait(&s.full[stage], phase) && !wait_l(p, s, &s.full[stage], phase, kLinSiteFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t off = (uint32_t(stage) * stage_bytes) >> 4;
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        mma_bf16(d, ad0 + off + uint64_t(kAStep * k), bd0 + off + uint64_t(2 * k), idesc, left < per_part || k ? 1u : 0u);
                    mma_commit(&s.empty[stage]);
                    if (--left == 0) {
                        left = per_part;
                        d += acc_cols;
                    }
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    ready = kb + 1 < last && mbar_test_wait(&s.full[stage], phase);
                }
                if (ok) mma_commit(s.acc);
            }
            __syncwarp();
        }
        good = wait_l(p, s, s.acc, uint32_t(round & 1), kLinSiteAcc);
        if (last == kb1) break;
        good = __syncthreads_and(good) != 0;   // all threads go on to the next round, or none does
        if (!good) break;
        tc_fence_after();
        for (int t0 = 0; t0 < nrows; t0 += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + uint32_t(t0), v);
            tmem_wait_ld_regs(v);
            add_parts(taddr + uint32_t(t0), acc_cols, used, v);
            tmem_st32(taddr + uint32_t(t0), v);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        next = until;
        first = last;
    }
    if (warp == 1 && elect_one()) {   // every MMA is done before the tensor memory is freed
        mma_commit(s.drain);
        drain_l(p, s.drain, 0);
    }
    __syncwarp();
    return good;
}

template <int MODE>
using StripParams = std::conditional_t<MODE == kLinPlain || MODE == kLinGateGrad, LinearStripParams, LinearStripMore>;

template <int LAYOUT, int MODE>
__global__ void __launch_bounds__(kThreadsL) cm_linear_strip_kernel(const __grid_constant__ StripParams<MODE> p) {
    constexpr bool B_MN = (LAYOUT & 1) != 0, A_MN = (LAYOUT & 2) != 0;
    extern __shared__ uint8_t smem_raw[];
    StripSmem s;
    s.ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bars[2 * kStripMaxStages + 2];
    __shared__ uint32_t slots[2];
    s.full = bars;
    s.empty = s.full + kStripMaxStages;
    s.acc = s.empty + kStripMaxStages;
    s.drain = s.acc + 1;
    s.tmem_slot = slots;
    s.abort = reinterpret_cast<volatile int *>(slots + 1);

    const int warp = int(threadIdx.x) >> 5;
    const uint32_t acc_cols = p.tok <= 32 ? 32u : p.tok <= 64 ? 64u : p.tok <= 128 ? 128u : 256u;
    // the loss's logits, forward and backward, are summed in parts, an accumulator each, as far as
    // half of the SM's tensor memory goes (multiply_parts)
    constexpr bool kStats = MODE == kLinStats, kParts = kStats || MODE == kLinSoftGrad;
    [[maybe_unused]] uint32_t acc_parts = 1;
    if constexpr (kParts)
        while (acc_parts * acc_cols < 256u && int(acc_parts) * p.splits * kStatSlices < p.kblocks) acc_parts *= 2;
    const uint32_t tmem_cols = acc_parts * acc_cols;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        mbar_init(s.acc, 1);
        mbar_init(s.drain, 1);
        *s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&p.tmA);
        prefetch_tmap(&p.tmB);
    }
    if (warp == 1) {
        tmem_alloc(s.tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s.tmem_slot;
    let_next_start();

    const int split = p.splits > 1 ? int(cluster_ctarank()) : 0;
    const int tile = int(blockIdx.x) / p.splits;
    const int ct = tile / p.row_tiles, rt = tile - ct * p.row_tiles;
    constexpr bool kGated = MODE == kLinGated;
    const int col0 = ct * (kGated ? kTileCols / 2 : kTileCols), row0 = rt * p.tok;
    const int kb0 = int(int64_t(p.kblocks) * split / p.splits), kb1 = int(int64_t(p.kblocks) * (split + 1) / p.splits);
    const uint32_t stage_bytes = uint32_t(kStripA + p.tok * kBK * 2);

    // The first slices of the column operand start on their way to L2 while the
    // previous kernel finishes.  Should that kernel still write them, L2 gets its
    // values all the same: the loads below, which come after it, read L2.
    if (warp == 0 && elect_one())
        for (int kb = kb0; kb < min(kb1, kb0 + p.stages); ++kb) {
            if constexpr (kGated) {   // 64 columns of each operand
                for (const CUtensorMap *m : {&p.tmA, &p.tmA2})
                    if (A_MN)
                        tma_prefetch_3d(m, col0, kb * kBK, 0);
                    else
                        tma_prefetch_3d(m, kb * kBK, col0, 0);
            } else if (A_MN) {
                for (int j = 0; j < kTileCols / 64; ++j) tma_prefetch_3d(&p.tmA, col0 + 64 * j, kb * kBK, 0);
            } else {
                tma_prefetch_3d(&p.tmA, kb * kBK, col0, 0);
            }
        }
    __syncwarp();
    wait_for_previous();

    int stage = 0, issued = 0;   // of the thread that loads, and of the one that multiplies
    uint32_t phase = 0;
    if (!kParts && warp == 0) {
        if (elect_one()) {
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_try_wait(&s.empty[stage], phase ^ 1u) && !wait_l(p, s, &s.empty[stage], phase ^ 1u, kLinSiteEmpty))
                    break;
                uint8_t *sa = s.ring + uint32_t(stage) * stage_bytes, *sb = sa + kStripA;
                mbar_expect_tx(&s.full[stage], stage_bytes);
                if constexpr (kGated) {
                    if (A_MN) {
                        tma_load_3d(sa, &p.tmA, &s.full[stage], col0, kb * kBK, 0);
                        tma_load_3d(sa + 64 * kBK * 2, &p.tmA2, &s.full[stage], col0, kb * kBK, 0);
                    } else {
                        tma_load_3d(sa, &p.tmA, &s.full[stage], kb * kBK, col0, 0);
                        tma_load_3d(sa + 64 * kBK * 2, &p.tmA2, &s.full[stage], kb * kBK, col0, 0);
                    }
                } else if (A_MN) {
                    for (int j = 0; j < kTileCols / 64; ++j)
                        tma_load_3d(sa + j * (64 * kBK * 2), &p.tmA, &s.full[stage], col0 + 64 * j, kb * kBK, 0);
                } else {
                    tma_load_3d(sa, &p.tmA, &s.full[stage], kb * kBK, col0, 0);
                }
                if (B_MN) {
                    for (int j = 0; j < p.tok / 64; ++j)
                        tma_load_3d(sb + j * (64 * kBK * 2), &p.tmB, &s.full[stage], row0 + 64 * j, kb * kBK, 0);
                } else {
                    tma_load_3d(sb, &p.tmB, &s.full[stage], kb * kBK, row0, 0);
                }
                ++issued;
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (!kParts && warp == 1) {
        if (elect_one()) {
            const uint32_t idesc = idesc_bf16(kTileCols, p.tok, B_MN, A_MN);
            constexpr uint32_t kALbo = A_MN ? 64 * kBK * 2 : 16, kBLbo = B_MN ? 64 * kBK * 2 : 16;
            constexpr uint32_t kAStep = A_MN ? (16 * 128) >> 4 : 32 >> 4, kBStep = B_MN ? (16 * 128) >> 4 : 32 >> 4;
            bool ok = true;
            const uint64_t ad0 = desc_sw128(smem_u32(s.ring), kALbo, 1024);
            const uint64_t bd0 = desc_sw128(smem_u32(s.ring) + kStripA, kBLbo, 1024);
            bool ready = mbar_test_wait(&s.full[0], 0);   // looked at ahead, so that its latency overlaps the issue
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!ready && !mbar_try_wait(&s.full[stage], phase) && !wait_l(p, s, &s.full[stage], phase, kLinSiteFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t off = (uint32_t(stage) * stage_bytes) >> 4;
                const uint64_t ad = ad0 + off, bd = bd0 + off;
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    mma_bf16(tmem, ad + uint64_t(kAStep * k), bd + uint64_t(kBStep * k), idesc, kb > kb0 || k ? 1u : 0u);
                mma_commit(&s.empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
                ready = kb + 1 < kb1 && mbar_test_wait(&s.full[stage], phase);
            }
            if (ok) mma_commit(s.acc);
            mma_commit(s.drain);
            drain_l(p, s.drain, 0);   // every MMA is done before the tensor memory is freed
        }
        __syncwarp();
    }
    bool good;
    [[maybe_unused]] int used = 1;
    if constexpr (kParts)
        good = multiply_parts<A_MN>(p, s, tmem, acc_cols, int(acc_parts), col0, row0, int(min(int64_t(p.tok), p.rows - row0)), kb0, kb1,
                                    used, stage, issued, phase);
    else
        good = wait_l(p, s, s.acc, 0, kLinSiteAcc);
    // The accumulator is complete once every load has landed.  If it was given up,
    // the loading thread waits for what it issued: no load may still write this
    // shared memory at exit.
    if (!good) {
        for (int i = 0; i < p.stages && i < issued; ++i) drain_l(p, &s.full[i], i < stage ? phase : phase ^ 1u);
    }
    __syncwarp();
    tc_fence_after();
    const int nrows = int(min(int64_t(p.tok), p.rows - row0));
    const int64_t col = int64_t(col0) + threadIdx.x;
    const uint32_t taddr = tmem + (uint32_t(warp * 32) << 16);
    const float bias = !kGated && col < p.cols ? lin::load_bias(p.e, col) : 0.0f;
    [[maybe_unused]] int count = 0;
    if constexpr (kParts) count = *p.count;
    if ((kGated || kStats) && p.splits == 1) {
        // gate and up columns, or those of a row's sum, lie in different threads' lanes:
        // they meet in the ring, whose loads have all been multiplied, 128 tokens at a time
        constexpr int kBlock = 128;
        static_assert(kBlock * kTileCols * 4 <= kStripShared, "a block of tokens fits in the ring");
        float *part = reinterpret_cast<float *>(s.ring);
        for (int b = 0; b < nrows; b += kBlock) {
            const int end = min(nrows - b, kBlock);
            for (int t0 = 0; t0 < end; t0 += 32) {
                uint32_t v[32];
                tmem_ld32(taddr + uint32_t(b + t0), v);
                tmem_wait_ld();
                if constexpr (kParts) add_parts(taddr + uint32_t(b + t0), acc_cols, used, v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (t0 + i < end) part[(t0 + i) * kTileCols + int(threadIdx.x)] = __uint_as_float(v[i]);
            }
            __syncthreads();
            if constexpr (kStats) {
                if (good) finish_stats(p.head, count, part, 1, 0, 1, end, int64_t(row0) + b, col0, p.cols);
            } else {
                if (good) finish_gated(p.e, part, 1, 0, 1, end, int64_t(row0) + b, col0, p.cols);
            }
            __syncthreads();
        }
    } else if (p.splits == 1) {
        for (int t0 = 0; t0 < nrows; t0 += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + uint32_t(t0), v);
            tmem_wait_ld();
            if constexpr (kParts) add_parts(taddr + uint32_t(t0), acc_cols, used, v);
            if (good && col < p.cols) {
#pragma unroll
                for (int b = 0; b < 32; b += kBatch)
                    if (t0 + b < nrows) {
                        float f[kBatch];
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) f[k] = __uint_as_float(v[b + k]);
                        if constexpr (MODE == kLinGateGrad)
                            finish_gate_grad(p.e, f, int64_t(row0) + t0 + b, 1, int64_t(row0) + nrows, col);
                        else if constexpr (MODE == kLinSoftGrad)
                            finish_softgrad(p.e, p.head, count, f, int64_t(row0) + t0 + b, 1, int64_t(row0) + nrows, col);
                        else
                            finish(p.e, f, bias, int64_t(row0) + t0 + b, 1, int64_t(row0) + nrows, col);
                    }
            }
        }
    } else {
        // all loads of the ring have landed and been multiplied: it now holds
        // the partial tile, [token][128]
        float *part = reinterpret_cast<float *>(s.ring);
        for (int t0 = 0; t0 < nrows; t0 += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + uint32_t(t0), v);
            tmem_wait_ld();
            if constexpr (kParts) add_parts(taddr + uint32_t(t0), acc_cols, used, v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (t0 + i < nrows) part[(t0 + i) * kTileCols + int(threadIdx.x)] = __uint_as_float(v[i]);
        }
        if (!good) *s.abort = 1;
        cluster_sync();
        if constexpr (kGated) {
            if (good) finish_gated(p.e, part, p.splits, split, p.splits, nrows, row0, col0, p.cols);
        } else if constexpr (kStats) {
            if (good) finish_stats(p.head, count, part, p.splits, split, p.splits, nrows, row0, col0, p.cols);
        } else if (col < p.cols && good)
            for (int t = split; t < nrows; t += p.splits * kBatch) {
                float f[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    f[k] = t + k * p.splits < nrows
                               ? cluster_sum(smem_u32(part + (t + k * p.splits) * kTileCols + int(threadIdx.x)), p.splits)
                               : 0.0f;
                if constexpr (MODE == kLinGateGrad)
                    finish_gate_grad(p.e, f, int64_t(row0) + t, p.splits, int64_t(row0) + nrows, col);
                else if constexpr (MODE == kLinSoftGrad)
                    finish_softgrad(p.e, p.head, count, f, int64_t(row0) + t, p.splits, int64_t(row0) + nrows, col);
                else
                    finish(p.e, f, bias, int64_t(row0) + t, p.splits, int64_t(row0) + nrows, col);
            }
        cluster_sync();   // the peers have read this CTA's partial tile
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, tmem_cols);
    }
}

using StripKernel = void (*)(LinearStripParams);
using StripMoreKernel = void (*)(LinearStripMore);

StripKernel strip_kernel(int layout, LinearMode mode) {
    if (mode == kLinGateGrad)
        return layout == 0   ? cm_linear_strip_kernel<0, kLinGateGrad>
               : layout == 2 ? cm_linear_strip_kernel<2, kLinGateGrad>
                             : nullptr;
    if (mode != kLinPlain) return nullptr;
    return layout == 0   ? cm_linear_strip_kernel<0, kLinPlain>
           : layout == 2 ? cm_linear_strip_kernel<2, kLinPlain>
           : layout == 3 ? cm_linear_strip_kernel<3, kLinPlain>
                         : nullptr;
}

StripMoreKernel strip_more_kernel(int layout, LinearMode mode) {
    const auto two = [&](StripMoreKernel k_major, StripMoreKernel mn_major) {
        return layout == 0 ? k_major : layout == 2 ? mn_major : nullptr;
    };
    switch (mode) {
        case kLinGated: return two(cm_linear_strip_kernel<0, kLinGated>, cm_linear_strip_kernel<2, kLinGated>);
        case kLinStats: return two(cm_linear_strip_kernel<0, kLinStats>, cm_linear_strip_kernel<2, kLinStats>);
        case kLinSoftGrad: return two(cm_linear_strip_kernel<0, kLinSoftGrad>, cm_linear_strip_kernel<2, kLinSoftGrad>);
        default: return nullptr;
    }
}

}  // namespace

int linear_strip_stages(int tok, int ring_bytes) {
    return std::min(kStripMaxStages, ring_bytes / (kStripA + tok * kBK * 2));
}

cudaError_t prepare_linear_strip(int sms, int *clusters) {
    const auto prepare = [](const void *fn) {
        return fn ? cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kStripAlone + 1024) : cudaSuccess;
    };
    for (LinearMode mode : {kLinPlain, kLinGated, kLinGateGrad, kLinStats, kLinSoftGrad})
        for (int layout : {0, 2, 3})
            for (const void *fn : {reinterpret_cast<const void *>(strip_kernel(layout, mode)),
                                   reinterpret_cast<const void *>(strip_more_kernel(layout, mode))}) {
                const cudaError_t e = prepare(fn);
                if (e != cudaSuccess) return e;
            }
    for (int i = 2; i <= kStripMostSplits; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(sms / i * i));
        cfg.blockDim = dim3(kThreadsL);
        cfg.dynamicSmemBytes = kStripAlone + 1024;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(i);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters[i], strip_kernel(0, kLinPlain), &cfg);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_linear_strip(const LinearStripMore &p, int layout, LinearMode mode, cudaStream_t stream) {
    const int64_t tile_cols = mode == kLinGated ? kTileCols / 2 : kTileCols;
    const int64_t grid = (p.cols + tile_cols - 1) / tile_cols * p.row_tiles * p.splits;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    // rounds of parts need a second accumulator
    if ((mode == kLinStats || mode == kLinSoftGrad) && p.tok > kStripRoundRows && (p.kblocks + p.splits - 1) / p.splits > kStatSlices)
        return cudaErrorInvalidValue;
    const size_t smem = size_t(p.ring_bytes) + 1024;
    if (const StripKernel fn = strip_kernel(layout, mode))
        return launch_after(fn, dim3(unsigned(grid)), kThreadsL, smem, unsigned(p.splits), stream, static_cast<const LinearStripParams &>(p));
    const StripMoreKernel fn = strip_more_kernel(layout, mode);
    if (!fn) return cudaErrorInvalidValue;
    return launch_after(fn, dim3(unsigned(grid)), kThreadsL, smem, unsigned(p.splits), stream, p);
}

}  // namespace cm
