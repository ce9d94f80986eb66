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

template <int LAYOUT>
__global__ void __launch_bounds__(kThreadsL) cm_linear_strip_kernel(const __grid_constant__ LinearStripParams p) {
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
    const uint32_t tmem_cols = p.tok <= 32 ? 32u : p.tok <= 64 ? 64u : p.tok <= 128 ? 128u : 256u;
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
    const int col0 = ct * kTileCols, row0 = rt * p.tok;
    const int kb0 = int(int64_t(p.kblocks) * split / p.splits), kb1 = int(int64_t(p.kblocks) * (split + 1) / p.splits);
    const uint32_t stage_bytes = uint32_t(kStripA + p.tok * kBK * 2);

    // The first slices of the column operand start on their way to L2 while the
    // previous kernel finishes.  Should that kernel still write them, L2 gets its
    // values all the same: the loads below, which come after it, read L2.
    if (warp == 0 && elect_one())
        for (int kb = kb0; kb < min(kb1, kb0 + p.stages); ++kb) {
            if (A_MN) {
                for (int j = 0; j < kTileCols / 64; ++j) tma_prefetch_3d(&p.tmA, col0 + 64 * j, kb * kBK, 0);
            } else {
                tma_prefetch_3d(&p.tmA, kb * kBK, col0, 0);
            }
        }
    __syncwarp();
    wait_for_previous();

    int stage = 0, issued = 0;   // of the thread that loads, and of the one that multiplies
    uint32_t phase = 0;
    if (warp == 0) {
        if (elect_one()) {
            for (int kb = kb0; kb < kb1; ++kb) {
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
    } else if (warp == 1) {
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
    const bool good = wait_l(p, s, s.acc, 0, kLinSiteAcc);
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
    const float bias = col < p.cols ? lin::load_bias(p.e, col) : 0.0f;
    if (p.splits == 1) {
        for (int t0 = 0; t0 < nrows; t0 += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + uint32_t(t0), v);
            tmem_wait_ld();
            if (good && col < p.cols) {
#pragma unroll
                for (int b = 0; b < 32; b += kBatch)
                    if (t0 + b < nrows) {
                        float f[kBatch];
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) f[k] = __uint_as_float(v[b + k]);
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
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (t0 + i < nrows) part[(t0 + i) * kTileCols + int(threadIdx.x)] = __uint_as_float(v[i]);
        }
        if (!good) *s.abort = 1;
        cluster_sync();
        if (col < p.cols && good)
            for (int t = split; t < nrows; t += p.splits * kBatch) {
                float f[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    f[k] = t + k * p.splits < nrows
                               ? cluster_sum(smem_u32(part + (t + k * p.splits) * kTileCols + int(threadIdx.x)), p.splits)
                               : 0.0f;
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

}  // namespace

int linear_strip_stages(int tok, int ring_bytes) {
    return std::min(kStripMaxStages, ring_bytes / (kStripA + tok * kBK * 2));
}

cudaError_t prepare_linear_strip(int sms, int *clusters) {
    void (*fns[3])(LinearStripParams) = {cm_linear_strip_kernel<0>, cm_linear_strip_kernel<2>, cm_linear_strip_kernel<3>};
    for (auto fn : fns) {
        cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kStripAlone + 1024);
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
        cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters[i], fns[0], &cfg);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_linear_strip(const LinearStripParams &p, int layout, cudaStream_t stream) {
    const int64_t col_tiles = (p.cols + kTileCols - 1) / kTileCols;
    const int64_t grid = col_tiles * p.row_tiles * p.splits;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    void (*fn)(LinearStripParams) = layout == 0   ? cm_linear_strip_kernel<0>
                                    : layout == 2 ? cm_linear_strip_kernel<2>
                                    : layout == 3 ? cm_linear_strip_kernel<3>
                                                  : nullptr;
    if (!fn) return cudaErrorInvalidValue;
    return launch_after(fn, dim3(unsigned(grid)), kThreadsL, size_t(p.ring_bytes) + 1024, unsigned(p.splits), stream, p);
}

}  // namespace cm
