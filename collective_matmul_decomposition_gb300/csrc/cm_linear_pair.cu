// cm_linear_pair.cu -- the linear layer's kernel for many rows: persistent
// 256 x 256 tiles on CTA pairs (tcgen05 .cta_group::2).
//
// D[row][col] = sum_k A[row][k] B[col][k].  CTA c of a pair stages rows
// 128c..128c+127 of the tile's A and columns 128c.. of its B; one MMA issued by
// the pair's leader multiplies the 256-row tile into both CTAs' tensor memory,
// so each CTA fetches half the operand bytes an MMA of its own tile would need.
// Two accumulators of 256 columns: the epilogue of a tile runs under the
// products of the next.  Cluster c takes tiles c, c + clusters, ...; the tiles
// run band by band of rows (32 MB of A, which then stay in L2) and column by
// column inside a band.
//
// Epilogue: a warp owns 32 rows x half the columns of the tile, in chunks of
// 128 bytes a row.  What the chunk needs besides the accumulator (residual,
// pre-activation, the old value) is fetched by TMA into a swizzled buffer while
// the products still run; a thread owns one row, replaces its part of the buffer
// by the result, and TMA writes the buffer out.  Global memory thus sees whole
// 128-byte rows, and ragged edges are the tensor map's business.
//
// Roles (384 threads): warp 0 loads, warp 1 MMAs (leader only), warps 4-11
// epilogue.  Every wait is bounded by p.timeout_ns, as in cm_linear_strip.cu.
#include <cuda_bf16.h>

#include <algorithm>

#include "cm_device.cuh"
#include "cm_kernel.cuh"
#include "cm_linear.cuh"
#include "cm_linear_epilogue.cuh"

namespace cm {
namespace {

using namespace dev;

constexpr int kTile = 256;              // rows of a pair's tile; columns: BN = 256 or 128
constexpr int kHalf = 128;              // rows staged by one CTA
constexpr int kLThreads = 384;
constexpr int kLEpiWarps = 8;
constexpr int kHalfBytes = kHalf * kBK * 2;      // 16 KB of A per stage
constexpr int kRingBytes = 160 * 1024;
constexpr int kEpiBuf = 32 * 128;                // 32 rows of 128 bytes
constexpr int kLSmem = kRingBytes + kLEpiWarps * 2 * kEpiBuf + 1024 /*barriers*/ + 1024 /*align*/;

template <int BN>
struct Tile {
    static constexpr int kB = BN / 2 * kBK * 2;                // bytes of B per stage and CTA
    static constexpr int kStages = BN == 256 ? 5 : 6;
    static_assert(kStages * (kHalfBytes + kB) <= kRingBytes, "the ring fits");
};

struct LSmem {
    uint8_t *a0, *b0, *epi;
    uint64_t *full, *empty, *tfull, *tempty, *drain, *ibar;
    uint32_t *tmem_slot;
    volatile int *abort;
};

__device__ __noinline__ void report_pair(LinearStatus *s, uint32_t site, int tile) {
    if (atomicCAS(&s->w[0], 0u, uint32_t(CM_ERR_TIMEOUT)) == 0u) {
        s->w[1] = uint32_t(tile);
        s->w[2] = blockIdx.x;
        s->w[3] = site;
        __threadfence();
    }
}

// Bounded wait; false once the bound has expired or the CTA is aborting.
__device__ bool wait_p(const LinearPairParams &p, const LSmem &s, uint64_t *bar, uint32_t parity, uint32_t site, int tile) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((it & 63u) == 0u) {
            if (*s.abort) return false;
            if (globaltimer() - t0 > p.timeout_ns) {
                report_pair(p.status, site, tile);
                *s.abort = 1;
                return false;
            }
        }
    }
}

__device__ void drain_p(const LinearPairParams &p, uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait_cluster(bar, parity))
        if (globaltimer() - t0 > p.timeout_ns) break;
}

__device__ __forceinline__ void tile_at(const LinearPairParams &p, int t, int &mt, int &nt) {
    const int per_band = p.band * p.ntiles;
    const int b = t / per_band;
    const int rows = min(p.band, p.mtiles - b * p.band);
    const int u = t - b * per_band;
    nt = u / rows;
    mt = b * p.band + (u - nt * rows);
}

template <int LAYOUT, int BN>
__device__ void load_tiles(const LinearPairParams &p, const LSmem &s, int rank) {
    constexpr bool B_MN = (LAYOUT & 1) != 0, A_MN = (LAYOUT & 2) != 0;
    constexpr int kStages = Tile<BN>::kStages, kB = Tile<BN>::kB;
    const uint32_t full_leader = mapa_shared(smem_u32(s.full), 0);
    const uint32_t a0 = smem_u32(s.a0), b0 = smem_u32(s.b0);
    const uint64_t tma = reinterpret_cast<uint64_t>(&p.tmA), tmb = reinterpret_cast<uint64_t>(&p.tmB);
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int t = int(blockIdx.x) >> 1; t < p.tiles && ok; t += int(gridDim.x) >> 1) {
        int mt, nt;
        tile_at(p, t, mt, nt);
        const int row0 = mt * kTile + rank * kHalf, col0 = nt * BN + rank * (BN / 2);
        for (int kb = 0; kb < p.kblocks; ++kb) {
            if (!mbar_try_wait(s.empty + stage, phase ^ 1u) &&
                !wait_p(p, s, s.empty + stage, phase ^ 1u, kLinSiteEmpty, t)) {
                ok = false;
                break;
            }
            const uint32_t bar = full_leader + 8u * uint32_t(stage);
            const uint32_t sa = a0 + uint32_t(stage) * kHalfBytes, sb = b0 + uint32_t(stage) * kB;
            const int k0 = kb * kBK;
            if (rank == 0) mbar_expect_tx(s.full + stage, 2u * (kHalfBytes + kB));
            if (A_MN) {
                tma_load_3d_pair_a(sa, tma, bar, row0, k0, 0);
                tma_load_3d_pair_a(sa + 64 * kBK * 2, tma, bar, row0 + 64, k0, 0);
            } else {
                tma_load_3d_pair_a(sa, tma, bar, k0, row0, 0);
            }
            if (B_MN) {
#pragma unroll
                for (int j = 0; j < BN / 128; ++j)
                    tma_load_3d_pair_a(sb + uint32_t(j * 64 * kBK * 2), tmb, bar, col0 + 64 * j, k0, 0);
            } else {
                tma_load_3d_pair_a(sb, tmb, bar, k0, col0, 0);
            }
            ++issued;
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    // the leader's barriers count both CTAs' loads: once they complete no load
    // is still writing this pair's shared memory
    if (rank == 0)
        for (int i = 0; i < kStages; ++i)
            if (uint32_t(i) < issued) drain_p(p, &s.full[i], i < stage ? phase : phase ^ 1u);
}

template <int LAYOUT, int BN>
__device__ void multiply_tiles(const LinearPairParams &p, const LSmem &s, uint32_t tmem) {
    constexpr bool B_MN = (LAYOUT & 1) != 0, A_MN = (LAYOUT & 2) != 0;
    constexpr int kStages = Tile<BN>::kStages, kB = Tile<BN>::kB;
    constexpr uint32_t kIdesc = idesc_bf16(kTile, BN, B_MN, A_MN);
    constexpr uint32_t kALbo = A_MN ? 64 * kBK * 2 : 16, kBLbo = B_MN ? 64 * kBK * 2 : 16;
    constexpr uint32_t kAStep = A_MN ? (16 * 128) >> 4 : 32 >> 4, kBStep = B_MN ? (16 * 128) >> 4 : 32 >> 4;
    const uint64_t ad0 = desc_sw128(smem_u32(s.a0), kALbo, 1024), bd0 = desc_sw128(smem_u32(s.b0), kBLbo, 1024);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = int(blockIdx.x) >> 1; t < p.tiles && ok; t += int(gridDim.x) >> 1) {
        if (!wait_p(p, s, &s.tempty[acc], acc_phase ^ 1u, kLinSiteTmem, t)) break;
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(acc * BN);
        bool ready = mbar_test_wait(s.full + stage, phase);   // looked at ahead, so that its latency overlaps the issue
        for (int kb = 0; kb < p.kblocks; ++kb) {
            if (!ready && !mbar_try_wait(s.full + stage, phase) && !wait_p(p, s, s.full + stage, phase, kLinSiteFull, t)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t ad = ad0 + uint64_t((uint32_t(stage) * kHalfBytes) >> 4);
            const uint64_t bd = bd0 + uint64_t((uint32_t(stage) * kB) >> 4);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
                mma_bf16_pair(d, ad + uint64_t(kAStep * k), bd + uint64_t(kBStep * k), kIdesc, (kb | k) != 0 ? 1u : 0u);
            mma_commit_pair_mc(s.empty + stage, uint16_t(3));
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
            ready = mbar_test_wait(s.full + stage, phase);
        }
        if (!ok) break;
        mma_commit_pair_mc(&s.tfull[acc], uint16_t(3));
        if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
        }
    }
    mma_commit_pair(s.drain);
    drain_p(p, s.drain, 0);
}

// 16-byte piece `c` of row `r` of a 128-byte-swizzled buffer
__device__ __forceinline__ uint4 *piece(uint8_t *buf, int r, int c) {
    return reinterpret_cast<uint4 *>(buf + r * 128 + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ void unpack8(const uint4 &w, float *f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float *f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// F32: y is fp32 (chunks of 32 columns), otherwise bf16 (64 columns).
template <bool F32, int BN>
__device__ void finish_tiles(const LinearPairParams &p, const LSmem &s, uint32_t tmem, int rank) {
    constexpr int kChunk = F32 ? 32 : 64, kCols = BN / 2;   // columns of a warp
    const LinearEpilogue &e = p.e;
    const int ew = int(threadIdx.x) / 32 - 4, lane = int(threadIdx.x) & 31;
    const int quad = ew & 3, half = ew >> 2;
    uint8_t *const buf0 = s.epi + ew * 2 * kEpiBuf, *const buf1 = buf0 + kEpiBuf;
    uint64_t *const ibar = &s.ibar[ew];
    const uint32_t tempty_leader = mapa_shared(smem_u32(&s.tempty[0]), 0);
    // inputs by TMA: buf0 the residual or the old value, buf1 the pre-activation.
    // With an fp32 y those are bf16 beside 4-byte chunks: read directly.
    const bool in0 = !F32 && (e.res || e.accumulate), in1 = !F32 && e.dact;
    const uint32_t in_bytes = uint32_t(in0 ? kEpiBuf : 0) + uint32_t(in1 ? kEpiBuf : 0);
    int acc = 0;
    uint32_t acc_phase = 0, in_phase = 0;
    bool pending = false;   // inputs asked for and not yet waited for
    bool ok = true;
    for (int t = int(blockIdx.x) >> 1; t < p.tiles && ok; t += int(gridDim.x) >> 1) {
        int mt, nt;
        tile_at(p, t, mt, nt);
        const int row0 = mt * kTile + rank * kHalf + quad * 32, cbase = nt * BN + half * kCols;
        const int nch = row0 < p.rows && cbase < p.cols ? min(kCols, int(min(p.cols - cbase, int64_t(kCols))) + kChunk - 1) / kChunk : 0;
        float bias[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = cbase + 32 * j + lane;
            bias[j] = c < p.cols ? lin::load_bias(e, c) : 0.0f;
        }
        auto ask = [&](int ch) {   // lane 0: the buffers are free, fetch the chunk's inputs
            bulk_wait_read<0>();
            if (in_bytes) {
                mbar_expect_tx(ibar, in_bytes);
                if (in0) tma_load_3d(buf0, &p.tmIn0, ibar, cbase + ch * kChunk, row0, 0);
                if (in1) tma_load_3d(buf1, &p.tmIn1, ibar, cbase + ch * kChunk, row0, 0);
            }
        };
        if (nch > 0 && in_bytes) {
            if (lane == 0) ask(0);
            pending = true;
        }
        ok = wait_p(p, s, &s.tfull[acc], acc_phase, kLinSiteAcc, t);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16) + uint32_t(acc * BN + half * kCols);
        for (int ch = 0; ch < nch; ++ch) {
            if (lane == 0 && !(ch == 0 && in_bytes)) ask(ch);
            __syncwarp();
            if (in_bytes) {
                pending = true;
                ok = wait_p(p, s, ibar, in_phase, kLinSiteFull, t);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                pending = false;
                in_phase ^= 1u;
            }
#pragma unroll
            for (int h = 0; h < kChunk / 32; ++h) {
                const int sub = ch * (kChunk / 32) + h;   // 32-column slice of the warp's columns
                uint32_t v[32];
                tmem_ld32(taddr + uint32_t(sub * 32), v);
                tmem_wait_ld();
                const float bsel = sub == 0 ? bias[0] : sub == 1 ? bias[1] : sub == 2 ? bias[2] : bias[3];
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
                if (e.bias) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] += __shfl_sync(0xffffffffu, bsel, i);
                }
                if constexpr (!F32) {
                    if (e.z) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) *piece(buf1, lane, h * 4 + j) = pack8(f + 8 * j);
                    }
                    if (e.dact) {
                        float z[32];
#pragma unroll
                        for (int j = 0; j < 4; ++j) unpack8(*piece(buf1, lane, h * 4 + j), z + 8 * j);
                        lin::mul_dact(f, z, e.act);
                    } else {
                        lin::apply_act(f, e.act);
                    }
                    if (in0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float r[8];
                            unpack8(*piece(buf0, lane, h * 4 + j), r);
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[8 * j + i] += r[i];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) *piece(buf0, lane, h * 4 + j) = pack8(f + 8 * j);
                } else {
                    const int64_t row = int64_t(row0) + lane;
                    const int col = cbase + ch * kChunk;
                    const bool live = row < p.rows;
                    auto at = [&](const void *m, int64_t ld, int i) {
                        return live && col + i < p.cols
                                   ? __bfloat162float(static_cast<const __nv_bfloat16 *>(m)[row * ld + col + i])
                                   : 0.0f;
                    };
                    if (e.z && live) {
                        __nv_bfloat16 *z = static_cast<__nv_bfloat16 *>(e.z) + row * e.ldz + col;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (col + i < p.cols) z[i] = __float2bfloat16_rn(f[i]);
                    }
                    if (e.dact) {
                        float z[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[i] = at(e.zin, e.ldzin, i);
                        lin::mul_dact(f, z, e.act);
                    } else {
                        lin::apply_act(f, e.act);
                    }
                    if (e.res) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] += at(e.res, e.ldr, i);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *piece(buf0, lane, j) = make_uint4(__float_as_uint(f[4 * j]), __float_as_uint(f[4 * j + 1]),
                                                           __float_as_uint(f[4 * j + 2]), __float_as_uint(f[4 * j + 3]));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (F32 && e.accumulate)
                    tma_reduce_add_3d(&p.tmY, buf0, cbase + ch * kChunk, row0, 0);
                else
                    tma_store_3d(&p.tmY, buf0, cbase + ch * kChunk, row0, 0);
                if (!F32 && e.z) tma_store_3d(&p.tmZ, buf1, cbase + ch * kChunk, row0, 0);
                bulk_commit();
            }
        }
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_leader + 8u * uint32_t(acc));
        if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
        }
    }
    if (lane == 0) {
        if (pending) drain_p(p, ibar, in_phase);   // leaving early: the inputs may still be landing
        bulk_wait<0>();
    }
    __syncwarp();
}

template <int LAYOUT, int BN>
__global__ void __launch_bounds__(kLThreads, 1) cm_linear_pair_kernel(const __grid_constant__ LinearPairParams p) {
    constexpr int kStages = Tile<BN>::kStages;
    extern __shared__ uint8_t smem_raw[];
    LSmem s;
    s.a0 = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    s.b0 = s.a0 + kStages * kHalfBytes;
    s.epi = s.a0 + kRingBytes;
    s.full = reinterpret_cast<uint64_t *>(s.epi + kLEpiWarps * 2 * kEpiBuf);
    s.empty = s.full + kStages;
    s.tfull = s.empty + kStages;
    s.tempty = s.tfull + 2;
    s.drain = s.tempty + 2;
    s.ibar = s.drain + 1;
    s.tmem_slot = reinterpret_cast<uint32_t *>(s.ibar + kLEpiWarps);
    s.abort = reinterpret_cast<volatile int *>(s.tmem_slot + 1);

    const int warp = int(threadIdx.x) >> 5;
    const int rank = int(cluster_ctarank());
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 2 * kLEpiWarps);
        }
        mbar_init(s.drain, 1);
        for (int i = 0; i < kLEpiWarps; ++i) mbar_init(&s.ibar[i], 1);
        *s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&p.tmA);
        prefetch_tmap(&p.tmB);
        prefetch_tmap(&p.tmY);
    }
    if (warp == 1) {
        tmem_alloc_pair(s.tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any cross-CTA arrival or load
    tc_fence_after();
    const uint32_t tmem = *s.tmem_slot;
    if (warp == 0) {
        if (elect_one()) load_tiles<LAYOUT, BN>(p, s, rank);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) multiply_tiles<LAYOUT, BN>(p, s, tmem);
        __syncwarp();
    } else if (warp >= 4) {
        if (p.e.y_f32)
            finish_tiles<true, BN>(p, s, tmem, rank);
        else
            finish_tiles<false, BN>(p, s, tmem, rank);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // no cross-CTA traffic is left when either CTA frees its tensor memory
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

cudaError_t pair_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, unsigned ctas, cudaStream_t stream) {
    cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kLThreads, 1, 1);
    cfg.dynamicSmemBytes = kLSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaSuccess;
}

}  // namespace

cudaError_t prepare_linear_pair(int device, int sms, int *max_clusters) {
    (void)device;
    void (*fns[6])(LinearPairParams) = {cm_linear_pair_kernel<0, 256>, cm_linear_pair_kernel<1, 256>,
                                        cm_linear_pair_kernel<3, 256>, cm_linear_pair_kernel<0, 128>,
                                        cm_linear_pair_kernel<1, 128>, cm_linear_pair_kernel<3, 128>};
    for (auto fn : fns) {
        cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kLSmem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    pair_config(cfg, attr, unsigned(sms / 2 * 2), nullptr);
    return cudaOccupancyMaxActiveClusters(max_clusters, cm_linear_pair_kernel<0, 256>, &cfg);
}

cudaError_t launch_linear_pair(const LinearPairParams &p, int layout, int clusters, cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    pair_config(cfg, attr, unsigned(2 * std::max(1, std::min(clusters, p.tiles))), stream);
    const bool wide = p.bn == 256;
    switch (layout) {
        case 0: return cudaLaunchKernelEx(&cfg, wide ? cm_linear_pair_kernel<0, 256> : cm_linear_pair_kernel<0, 128>, p);
        case 1: return cudaLaunchKernelEx(&cfg, wide ? cm_linear_pair_kernel<1, 256> : cm_linear_pair_kernel<1, 128>, p);
        case 3: return cudaLaunchKernelEx(&cfg, wide ? cm_linear_pair_kernel<3, 256> : cm_linear_pair_kernel<3, 128>, p);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace cm
