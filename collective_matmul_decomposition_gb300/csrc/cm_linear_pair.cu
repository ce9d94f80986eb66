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
// 128-byte rows, and what lies beyond the matrix is the tensor map's business.
//
// Bound by the tensor cores: 8192 x 8192 x 3584 takes 253.6 us, 1897 TFLOP/s, at
// full clock; 8192 x 8192 x 28672 with GELU and the pre-activation kept 2.29 to
// 2.39 ms, 1610 to 1680 TFLOP/s under the power cap.  With few K slices it is the
// epilogue: 2.5 us a wave of tiles, SiLU 1.4 more, GELU 2.6 (its tanh form 1.6);
// 8192 x 64 x 8192 takes 34.7, 54.8, 71.0 and 56.7 us.
//
// Calls with too few tiles for all SMs split the tiles' K slices: see
// cm_linear_split_kernel below.
//
// Roles (384 threads): warp 0 loads, warp 1 MMAs (leader only), warps 4-11
// epilogue.  Every wait is bounded by p.timeout_ns, as in cm_linear_strip.cu.
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
// Every barrier here hands over shared memory that TMA and the tensor cores
// write and read, or tensor memory: no wait has to order memory of the peer CTA.
__device__ bool wait_p(const LinearPairParams &p, const LSmem &s, uint64_t *bar, uint32_t parity, uint32_t site, int tile) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
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
    while (!mbar_try_wait(bar, parity))
        if (globaltimer() - t0 > p.timeout_ns) break;
}

__device__ __forceinline__ void tile_at(const LinearPairParams &p, int mtiles, int t, int &mt, int &nt) {
    const int per_band = p.band * p.ntiles;
    const int b = t / per_band;
    const int rows = min(p.band, mtiles - b * p.band);
    const int u = t - b * per_band;
    nt = u / rows;
    mt = b * p.band + (u - nt * rows);
}

// Modes whose products may end at the last slot (LinearLive), and the parameters of each.
template <int MODE>
constexpr bool kIsCounted = MODE == kLinStats || MODE == kLinSoftGrad || MODE == kLinCounted;
template <int MODE>
using PairParams = std::conditional_t<MODE == kLinPlain || MODE == kLinGateGrad, LinearPairParams, LinearPairMore>;

// The tiles and K slices of a CTA's pair: first, first + step, ... below
// `tiles`, each over slices kb0 .. kb1 - 1.  `leader` is the pair's even CTA.
struct Share {
    int first, step, kb0, kb1;
    uint32_t leader;
    // of the counted modes; the others have these from the parameters, at no register
    int tiles, mtiles;
    int64_t rows;
    const CUtensorMap *a, *b;   // the operands' maps
};
template <int MODE>
__device__ __forceinline__ int tiles_of(const LinearPairParams &p, const Share &w) {
    return kIsCounted<MODE> ? w.tiles : p.tiles;
}
template <int MODE>
__device__ __forceinline__ int mtiles_of(const LinearPairParams &p, const Share &w) {
    return kIsCounted<MODE> ? w.mtiles : p.mtiles;
}
template <int MODE>
__device__ __forceinline__ int64_t rows_of(const LinearPairParams &p, const Share &w) {
    return kIsCounted<MODE> ? w.rows : p.rows;
}
// of a persistent kernel's epilogue
template <int MODE>
__device__ __forceinline__ int first_of(const Share &w) {
    return kIsCounted<MODE> ? w.first : int(blockIdx.x) >> 1;
}
template <int MODE>
__device__ __forceinline__ int step_of(const Share &w) {
    return kIsCounted<MODE> ? w.step : int(gridDim.x) >> 1;
}

// Where a role stands in the ring of stages and in the two accumulators, from one
// share to the next.
struct Flow {
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    uint32_t issued = 0;      // of the loads
    uint32_t in_phase = 0;    // of the epilogue's inputs
    bool ok = true;           // no wait has expired
};

// A persistent kernel's share, cut down to the slots where they are counted.
template <int MODE>
__device__ __forceinline__ Share share_of(const PairParams<MODE> &p) {
    Share w = {int(blockIdx.x) >> 1, int(gridDim.x) >> 1, 0, p.kblocks, 0u, p.tiles, p.mtiles, p.rows, &p.tmA, &p.tmB};
    if constexpr (kIsCounted<MODE>) {
        if (!p.live.count) return w;
        const int n = *p.live.count;
        // where there is none, one slice or one row of tiles is computed all the same:
        // the slots behind the last are zeros
        if (p.live.of_k) {
            w.kb1 = max(1, min(p.kblocks, (n + kBK - 1) / kBK));
        } else {
            w.rows = n;
            if (p.live.skip) w.mtiles = max(1, (n + kTile - 1) / kTile);
            w.tiles = w.mtiles * p.ntiles;
        }
        if (n == p.live.whole && p.live.whole_is == 1) w.a = &p.tmWhole;
        if (n == p.live.whole && p.live.whole_is == 2) w.b = &p.tmWhole;
    }
    return w;
}

template <int LAYOUT, int BN, int MODE>
__device__ __forceinline__ void load_tiles(const PairParams<MODE> &p, const LSmem &s, const Share &w, int rank, Flow &flow) {
    constexpr bool B_MN = (LAYOUT & 1) != 0, A_MN = (LAYOUT & 2) != 0;
    constexpr int kStages = Tile<BN>::kStages, kB = Tile<BN>::kB;
    const uint32_t full_leader = mapa_shared(smem_u32(s.full), w.leader);
    const uint32_t a0 = smem_u32(s.a0), b0 = smem_u32(s.b0);
    uint64_t tma = reinterpret_cast<uint64_t>(&p.tmA), tmb = reinterpret_cast<uint64_t>(&p.tmB);
    if constexpr (kIsCounted<MODE>) tma = reinterpret_cast<uint64_t>(w.a), tmb = reinterpret_cast<uint64_t>(w.b);
    // gated: the pair's even CTA stages the gate's columns, the odd one the up projection's,
    // so that half of each CTA's accumulator columns belong to either
    if constexpr (MODE == kLinGated)
        if (rank) tmb = reinterpret_cast<uint64_t>(&p.tmB2);
    int stage = flow.stage;
    uint32_t phase = flow.phase, issued = flow.issued;
    bool ok = flow.ok;
    for (int t = w.first; t < tiles_of<MODE>(p, w) && ok; t += w.step) {
        int mt, nt;
        tile_at(p, mtiles_of<MODE>(p, w), t, mt, nt);
        const int row0 = mt * kTile + rank * kHalf, col0 = MODE == kLinGated ? nt * (BN / 2) : nt * BN + rank * (BN / 2);
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
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
    flow.stage = stage, flow.phase = phase, flow.issued = issued, flow.ok = ok;
}

// The leader's barriers count both CTAs' loads: once they complete no load
// is still writing this pair's shared memory.
template <int BN>
__device__ __forceinline__ void drain_loads(const LinearPairParams &p, const LSmem &s, int rank, const Flow &flow) {
    if (rank == 0)
        for (int i = 0; i < Tile<BN>::kStages; ++i)
            if (uint32_t(i) < flow.issued) drain_p(p, &s.full[i], i < flow.stage ? flow.phase : flow.phase ^ 1u);
}

template <int LAYOUT, int BN, int MODE>
__device__ __forceinline__ void multiply_tiles(const LinearPairParams &p, const LSmem &s, const Share &w, uint32_t tmem, Flow &flow) {
    constexpr bool B_MN = (LAYOUT & 1) != 0, A_MN = (LAYOUT & 2) != 0;
    constexpr int kStages = Tile<BN>::kStages, kB = Tile<BN>::kB;
    constexpr uint32_t kIdesc = idesc_bf16(kTile, BN, B_MN, A_MN);
    constexpr uint32_t kALbo = A_MN ? 64 * kBK * 2 : 16, kBLbo = B_MN ? 64 * kBK * 2 : 16;
    constexpr uint32_t kAStep = A_MN ? (16 * 128) >> 4 : 32 >> 4, kBStep = B_MN ? (16 * 128) >> 4 : 32 >> 4;
    const uint64_t ad0 = desc_sw128(smem_u32(s.a0), kALbo, 1024), bd0 = desc_sw128(smem_u32(s.b0), kBLbo, 1024);
    int stage = flow.stage, acc = flow.acc;
    uint32_t phase = flow.phase, acc_phase = flow.acc_phase;
    bool ok = flow.ok;
    const uint16_t both = uint16_t(3u << w.leader);   // the pair's CTAs
    constexpr bool kParts = MODE == kLinStats || MODE == kLinSoftGrad;   // an accumulator for each kStatSlices slices
    for (int t = w.first; t < tiles_of<MODE>(p, w) && ok; t += w.step) {
        if (!wait_p(p, s, &s.tempty[acc], acc_phase ^ 1u, kLinSiteTmem, t)) {
            ok = false;
            break;
        }
        tc_fence_after();
        uint32_t d = tmem + uint32_t(acc * BN);
        bool ready = mbar_test_wait(s.full + stage, phase);   // looked at ahead, so that its latency overlaps the issue
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
            if (kParts && kb > w.kb0 && (kb - w.kb0) % kStatSlices == 0) {
                mma_commit_pair_mc(&s.tfull[acc], both);
                acc ^= 1;
                acc_phase ^= acc == 0 ? 1u : 0u;
                if (!wait_p(p, s, &s.tempty[acc], acc_phase ^ 1u, kLinSiteTmem, t)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                d = tmem + uint32_t(acc * BN);
            }
            if (!ready && !mbar_try_wait(s.full + stage, phase) && !wait_p(p, s, s.full + stage, phase, kLinSiteFull, t)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t ad = ad0 + uint64_t((uint32_t(stage) * kHalfBytes) >> 4);
            const uint64_t bd = bd0 + uint64_t((uint32_t(stage) * kB) >> 4);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
                mma_bf16_pair(d, ad + uint64_t(kAStep * k), bd + uint64_t(kBStep * k), kIdesc,
                              (kParts ? (kb - w.kb0) % kStatSlices > 0 : kb > w.kb0) || k > 0 ? 1u : 0u);
            mma_commit_pair_mc(s.empty + stage, both);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
            ready = mbar_test_wait(s.full + stage, phase);
        }
        if (!ok) break;
        mma_commit_pair_mc(&s.tfull[acc], both);
        if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
        }
    }
    flow.stage = stage, flow.phase = phase, flow.acc = acc, flow.acc_phase = acc_phase, flow.ok = ok;
}

__device__ __forceinline__ void drain_products(const LinearPairParams &p, const LSmem &s) {
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

// The results of one row's columns col .. col + n - 1 (fewer than a 16-byte
// piece holds), the first of them at element `at` of the buffers' rows.
template <bool F32>
__device__ __noinline__ void store_rest(const LinearPairParams &p, uint8_t *buf0, uint8_t *buf1, int64_t row, int64_t col,
                                        int at, int n, int r) {
    if (row >= p.rows) return;
    if (F32) {
        const uint4 w = *piece(buf0, r, at >> 2);
        const float f[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
        float *y = static_cast<float *>(p.e.y) + row * p.e.ldy + col;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n) y[i] = p.e.accumulate ? y[i] + f[i] : f[i];
        return;
    }
    float f[8];
    unpack8(*piece(buf0, r, at >> 3), f);
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.e.y) + row * p.e.ldy + col;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) y[i] = __float2bfloat16_rn(f[i]);
    if (!p.e.z) return;
    unpack8(*piece(buf1, r, at >> 3), f);
    __nv_bfloat16 *z = static_cast<__nv_bfloat16 *>(p.e.z) + row * p.e.ldz + col;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) z[i] = __float2bfloat16_rn(f[i]);
}

// F32: y is fp32 (chunks of 32 columns), otherwise bf16 (64 columns).  MODE: kLinPlain, kLinGateGrad or kLinCounted.
template <bool F32, int BN, int MODE>
__device__ __forceinline__ void finish_tiles(const LinearPairParams &p, const LSmem &s, const Share &w, uint32_t tmem, int rank,
                                             Flow &flow) {
    constexpr int kChunk = F32 ? 32 : 64, kCols = BN / 2;   // columns of a warp
    const LinearEpilogue &e = p.e;
    const int ew = int(threadIdx.x) / 32 - 4, lane = int(threadIdx.x) & 31;
    const int quad = ew & 3, half = ew >> 2;
    uint8_t *const bufs = s.epi + ew * 2 * kEpiBuf;
    uint64_t *const ibar = &s.ibar[ew];
    const uint32_t tempty_leader = mapa_shared(smem_u32(&s.tempty[0]), 0);
    // inputs by TMA: the residual or the old value, and the pre-activation.
    // With an fp32 y those are bf16 beside 4-byte chunks: read directly.
    // The gate's gradients read both z and write one gradient over each.
    constexpr bool kGate = MODE == kLinGateGrad;
    // They pass through L2 once: they are not to push the operands out of it.
    [[maybe_unused]] uint64_t once = 0;
    if constexpr (kGate) once = policy_evict_first();
    const bool in0 = kGate || (!F32 && (e.res || e.accumulate)), in1 = kGate || (!F32 && e.dact);
    const uint32_t in_bytes = uint32_t(in0 ? kEpiBuf : 0) + uint32_t(in1 ? kEpiBuf : 0);
    // the second buffer holds the pre-activation if there is one; else chunks
    // take turns with the two, so that one is filled while the other is written out
    const bool two = !(in1 || (!F32 && e.z));
    uint8_t *buf0 = bufs, *const buf1 = bufs + kEpiBuf;
    // TMA writes whole 16-byte pieces: the maps written through end at the last
    // whole one of a row, and the threads write what is left of it
    constexpr int kPiece = F32 ? 4 : 8;
    const int rest = int(p.cols % kPiece);
    const int64_t whole = p.cols - rest;
    [[maybe_unused]] const float scale = MODE == kLinCounted && e.scale ? *e.scale : 1.0f;
    int acc = flow.acc;
    uint32_t acc_phase = flow.acc_phase, in_phase = flow.in_phase;
    bool pending = false;   // inputs asked for and not yet waited for
    bool ok = flow.ok;
    for (int t = first_of<MODE>(w); t < tiles_of<MODE>(p, w) && ok; t += step_of<MODE>(w)) {
        int mt, nt;
        tile_at(p, mtiles_of<MODE>(p, w), t, mt, nt);
        const int row0 = mt * kTile + rank * kHalf + quad * 32, cbase = nt * BN + half * kCols;
        const int nch = row0 < rows_of<MODE>(p, w) && cbase < p.cols ? min(kCols, int(min(p.cols - cbase, int64_t(kCols))) + kChunk - 1) / kChunk : 0;
        float bias[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = cbase + 32 * j + lane;
            bias[j] = c < p.cols ? lin::load_bias(e, c) : 0.0f;
        }
        auto ask = [&](int ch) {   // lane 0: wait for the chunk's buffer to be free, fetch its inputs
            if (two)
                bulk_wait_read<1>();
            else
                bulk_wait_read<0>();
            if (in_bytes) {
                mbar_expect_tx(ibar, in_bytes);
                if constexpr (kGate) {
                    tma_load_3d_hint(buf0, &p.tmIn0, ibar, cbase + ch * kChunk, row0, 0, once);
                    tma_load_3d_hint(buf1, &p.tmIn1, ibar, cbase + ch * kChunk, row0, 0, once);
                } else {
                    if (in0) tma_load_3d(buf0, &p.tmIn0, ibar, cbase + ch * kChunk, row0, 0);
                    if (in1) tma_load_3d(buf1, &p.tmIn1, ibar, cbase + ch * kChunk, row0, 0);
                }
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
        // the accumulator is in registers: the products of the next tile but one may start
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(tempty_leader + 8u * uint32_t(acc));
        };
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
            uint32_t raw[kChunk / 32][32];
#pragma unroll
            for (int h = 0; h < kChunk / 32; ++h) tmem_ld32(taddr + uint32_t(ch * kChunk + h * 32), raw[h]);
#pragma unroll
            for (int h = 0; h < kChunk / 32; ++h) {
                const int sub = ch * (kChunk / 32) + h;   // 32-column slice of the warp's columns
                uint32_t (&v)[32] = raw[h];
                tmem_wait_ld_regs(v);   // the first wait is for all loads of the chunk
                if (h == 0 && ch == nch - 1) release();
                const float bsel = sub == 0 ? bias[0] : sub == 1 ? bias[1] : sub == 2 ? bias[2] : bias[3];
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
                if constexpr (MODE == kLinCounted) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] *= scale;
                }
                if constexpr (kGate) {
                    float g[32], u[32];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        unpack8(*piece(buf1, lane, h * 4 + j), g + 8 * j);
                        unpack8(*piece(buf0, lane, h * 4 + j), u + 8 * j);
                    }
                    lin::gate_grad(f, g, u, e.act);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        *piece(buf1, lane, h * 4 + j) = pack8(g + 8 * j);
                        *piece(buf0, lane, h * 4 + j) = pack8(u + 8 * j);
                    }
                    continue;
                }
                // the columns' biases lie one to a lane (as fast as reading them
                // all from L1, and any address will do)
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
                    const bool live = row < rows_of<MODE>(p, w);
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
            const int c0 = cbase + ch * kChunk;
            if (rest && c0 + kChunk > whole)
                store_rest<F32>(p, buf0, buf1, int64_t(row0) + lane, whole, int(whole - c0), rest, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (c0 < whole) {
                    if constexpr (kGate)
                        tma_store_3d_hint(&p.tmY, buf0, c0, row0, 0, once);
                    else if (F32 && e.accumulate)
                        tma_reduce_add_3d(&p.tmY, buf0, c0, row0, 0);
                    else
                        tma_store_3d(&p.tmY, buf0, c0, row0, 0);
                    if constexpr (kGate)
                        tma_store_3d_hint(&p.tmZ, buf1, c0, row0, 0, once);
                    else if (!F32 && e.z)
                        tma_store_3d(&p.tmZ, buf1, c0, row0, 0);
                }
                bulk_commit();
            }
            if (two) buf0 = buf0 == bufs ? buf1 : bufs;
        }
        if (!ok) break;
        if (nch == 0) release();
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
    flow.acc = acc, flow.acc_phase = acc_phase, flow.in_phase = in_phase, flow.ok = ok;
}

// The columns behind a row's last whole 16-byte piece, n of them, from element `at` of the buffer's row.
__device__ __noinline__ void store_tail(uint8_t *buf, void *m, int64_t ld, int64_t row, int64_t col, int at, int n, int r) {
    float f[8];
    unpack8(*piece(buf, r, at >> 3), f);
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(m) + row * ld + col;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) y[i] = __float2bfloat16_rn(f[i]);
}

// The gated product: of a tile's 256 accumulator columns the first 128 are g, the
// others u of the same 128 columns.  A warp owns 32 rows x 64 of those.  Up to three
// matrices leave through its two buffers in turn (y, then z of both); each reads the
// accumulator again, which costs less than holding 128 columns in registers.
// Bound by the tensor cores where the products are long: 4096 x 8192 x 2 28672 with both z
// kept takes 2.26 to 2.34 ms, 1650 to 1700 TFLOP/s under the power cap, and no longer than
// a plain product of as many columns.  Below some 16 K slices a tile it is the epilogue:
// 4096 x 1024 x 2 4096 takes 37 us, 50 with both z kept (a plain product 43).
__device__ void finish_gated(const LinearPairMore &p, const LSmem &s, uint32_t tmem, int rank) {
    constexpr int BN = 256, kCols = 64;
    const LinearEpilogue &e = p.e;
    const int ew = int(threadIdx.x) / 32 - 4, lane = int(threadIdx.x) & 31;
    const int quad = ew & 3, half = ew >> 2;
    uint8_t *const bufs = s.epi + ew * 2 * kEpiBuf;
    uint8_t *buf = bufs;
    const uint32_t tempty_leader = mapa_shared(smem_u32(&s.tempty[0]), 0);
    const int rest = int(p.cols % 8);
    const int64_t whole = p.cols - rest;
    const int outs = e.z ? 3 : 1;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = int(blockIdx.x) >> 1; t < p.tiles; t += int(gridDim.x) >> 1) {
        int mt, nt;
        tile_at(p, p.mtiles, t, mt, nt);
        const int row0 = mt * kTile + rank * kHalf + quad * 32, c0 = nt * (BN / 2) + half * kCols;
        const bool live = row0 < p.rows && c0 < p.cols;
        float bg[2], bu[2];   // the columns' biases lie one to a lane
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 32 * h + lane;
            bg[h] = c < p.cols ? lin::load_bias(e.bias, e.bias_f32, c) : 0.0f;
            bu[h] = c < p.cols ? lin::load_bias(e.bias2, e.bias_f32, c) : 0.0f;
        }
        bool ok = wait_p(p, s, &s.tfull[acc], acc_phase, kLinSiteAcc, t);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16) + uint32_t(acc * BN + half * kCols);
        auto load = [&](int first, int h, float (&f)[32], const float (&b)[2]) {
            uint32_t v[32];
            tmem_ld32(taddr + uint32_t(first + 32 * h), v);
            tmem_wait_ld_regs(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
            if (e.bias) {
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] += __shfl_sync(0xffffffffu, h ? b[1] : b[0], i);
            }
        };
        for (int o = 0; live && o < outs; ++o) {
            if (lane == 0) bulk_wait_read<1>();   // the buffer's last store has been read out
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[32];
                if (o == 0) {
                    float u[32];
                    load(0, h, f, bg);
                    load(BN / 2, h, u, bu);
                    lin::apply_gate(f, u, e.act);
                } else if (o == 1) {
                    load(0, h, f, bg);
                } else {
                    load(BN / 2, h, f, bu);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) *piece(buf, lane, h * 4 + j) = pack8(f + 8 * j);
            }
            if (rest && c0 + kCols > whole && int64_t(row0) + lane < p.rows)
                store_tail(buf, o == 0 ? e.y : o == 1 ? e.z : e.z2, o == 0 ? e.ldy : e.ldz, int64_t(row0) + lane, whole,
                           int(whole - c0), rest, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (c0 < whole) tma_store_3d(o == 0 ? &p.tmY : o == 1 ? &p.tmZ : &p.tmZ2, buf, c0, row0, 0);
                bulk_commit();
            }
            buf = buf == bufs ? bufs + kEpiBuf : bufs;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty_leader + 8u * uint32_t(acc));
        if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
        }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
}

// A tile's logits, whose parts (kStatSlices) are added up in registers while the products
// go on: a thread owns one row and half of the tile's columns.  An accumulator is given
// back as soon as it is read.  False after an expired wait.
__device__ __forceinline__ bool add_up_parts(const LinearPairMore &p, const LSmem &s, const Share &w, uint32_t taddr0, uint32_t tempty_leader,
                                             bool live, int t, int &acc, uint32_t &acc_phase, float (&f)[8][16]) {
    const int parts = (w.kb1 - w.kb0 + kStatSlices - 1) / kStatSlices;
#pragma unroll
    for (int b = 0; b < 8; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) f[b][i] = 0.0f;
#pragma unroll 1
    for (int part = 0; part < parts; ++part) {
        const bool ok = wait_p(p, s, &s.tfull[acc], acc_phase, kLinSiteAcc, t);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc_fence_after();
        if (live) {
            const uint32_t taddr = taddr0 + uint32_t(acc * kTile);
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                uint32_t v[16];
                tmem_ld16(taddr + uint32_t(16 * b), v);
                tmem_wait_ld_regs(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) f[b][i] += __uint_as_float(v[i]);
            }
        }
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive_remote(tempty_leader + 8u * uint32_t(acc));
        acc ^= 1;
        acc_phase ^= acc == 0 ? 1u : 0u;
    }
    return true;
}

// The statistics of a softmax over the columns, without the logits: a thread reduces
// those of its row to the largest m and the sum of exp2(v log2(e) - m), all in fp32.
// What is not a column counts as -infinity.  A NaN stays one through the sum.
// It leaves 8 bytes for 128 logits and costs the products little: 8192 x 4096 x 131072
// takes 4.8 ms, 1830 TFLOP/s.  lse is off by 2.5e-7 of its value; with one
// accumulator a tile it was 8.6e-7 for 4096 terms and 1.5e-6 for 7040, in the same time.
__device__ void finish_stats(const LinearPairMore &p, const LSmem &s, const Share &w, uint32_t tmem, int rank) {
    constexpr int BN = 256, kCols = BN / 2, kBlocks = kCols / 16;
    const int ew = int(threadIdx.x) / 32 - 4, lane = int(threadIdx.x) & 31;
    const int quad = ew & 3, half = ew >> 2;
    const uint32_t tempty_leader = mapa_shared(smem_u32(&s.tempty[0]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = w.first; t < w.tiles; t += w.step) {
        int mt, nt;
        tile_at(p, w.mtiles, t, mt, nt);
        const int row0 = mt * kTile + rank * kHalf + quad * 32;
        const int64_t c0 = int64_t(nt) * BN + half * kCols;
        const bool live = row0 < w.rows && c0 < p.cols;   // the same in the whole warp
        float f[kBlocks][16];
        if (!add_up_parts(p, s, w, tmem + (uint32_t(quad * 32) << 16) + uint32_t(half * kCols), tempty_leader, live, t, acc, acc_phase, f)) break;
        const int row = row0 + lane;
        if (row >= w.rows) continue;
        if (!live) {   // no column is here
            p.head.stat[(int64_t(nt) * 2 + half) * p.head.stride + row] = make_float2(-INFINITY, 0.0f);
            continue;
        }
        // the target's place among these columns, if it is there
        const int64_t target = p.head.target[row], left = target - p.head.first - c0;
        if (target >= 0 && left >= 0 && left < kCols && c0 + left < p.cols) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (int(left) == 16 * b + i) p.head.picked[row] = f[b][i];
        }
        if (c0 + kCols > p.cols) {
            const int n = int(p.cols - c0);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) f[b][i] = 16 * b + i < n ? f[b][i] : -INFINITY;
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) top[i & 3] = fmaxf(top[i & 3], f[b][i]);
        const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * lin::kLog2e;
        const float base = m == -INFINITY ? 0.0f : m;   // no number: exp2(-inf - 0) is 0
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[i & 3] += lin::exp2_fast(fmaf(f[b][i], lin::kLog2e, -base));
        p.head.stat[(int64_t(nt) * 2 + half) * p.head.stride + row] = make_float2(m, (sum[0] + sum[1]) + (sum[2] + sum[3]));
    }
    __syncwarp();
}

// The same for tiles of one part, whose epilogue sets the pace: through the columns 32 at
// a time with the running maximum m and sum s,
//   m' = max(m, max v);  s' = s exp2(m - m') + sum exp2(v - m'),
// which needs half the registers and no copy of the columns.  65536 x 512 x 4096 takes
// 235 us, with the columns in registers 308; 8192 x 64 x 131072 374 and 407.
__device__ void finish_stats_few(const LinearPairMore &p, const LSmem &s, const Share &w, uint32_t tmem, int rank) {
    constexpr int BN = 256, kCols = BN / 2;
    const int ew = int(threadIdx.x) / 32 - 4, lane = int(threadIdx.x) & 31;
    const int quad = ew & 3, half = ew >> 2;
    const uint32_t tempty_leader = mapa_shared(smem_u32(&s.tempty[0]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = w.first; t < w.tiles; t += w.step) {
        int mt, nt;
        tile_at(p, w.mtiles, t, mt, nt);
        const int row0 = mt * kTile + rank * kHalf + quad * 32, row = row0 + lane;
        const int64_t c0 = int64_t(nt) * BN + half * kCols;
        // the target's place among the warp's columns; -1 if it is not there
        const int64_t target = row < w.rows ? p.head.target[row] : kNotHere, left = target - p.head.first - c0;
        const int at = target >= 0 && left >= 0 && left < kCols ? int(left) : -1;
        bool ok = wait_p(p, s, &s.tfull[acc], acc_phase, kLinSiteAcc, t);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16) + uint32_t(acc * BN + half * kCols);
        float m = -INFINITY, sum = 0.0f, picked = 0.0f;
        if (row0 < w.rows) {
#pragma unroll 1
            for (int c = 0; c < kCols && c0 + c < p.cols; c += 32) {
                uint32_t v[32];
                tmem_ld32(taddr + uint32_t(c), v);
                tmem_wait_ld_regs(v);
                float f[32];
                const int n = int(min(int64_t(32), p.cols - c0 - c));
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
                if (__any_sync(0xffffffffu, at >= c && at < c + 32)) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) picked = at == c + i ? f[i] : picked;
                }
                if (n < 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = i < n ? f[i] : -INFINITY;
                }
                float top = f[0];
#pragma unroll
                for (int i = 1; i < 32; ++i) top = fmaxf(top, f[i]);
                const float next = fmaxf(m, top * lin::kLog2e);
                const float base = next == -INFINITY ? 0.0f : next;   // no number yet: exp2(-inf - 0) is 0
                sum *= lin::exp2_fast(m - base);
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 32; ++i) part[i & 3] += lin::exp2_fast(fmaf(f[i], lin::kLog2e, -base));
                sum += (part[0] + part[1]) + (part[2] + part[3]);
                m = next;
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty_leader + 8u * uint32_t(acc));
        if (row < w.rows) {
            p.head.stat[(int64_t(nt) * 2 + half) * p.head.stride + row] = make_float2(m, sum);
            if (at >= 0 && c0 + at < p.cols) p.head.picked[row] = picked;
        }
        if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
        }
    }
    __syncwarp();
}

// The gradient of the logits, bf16: exp(D - lse) grad, less hit in the target's column.
// Rows behind the last slot are zeros up to the tile's end.  bf16 because two products
// read it; grad and hit are relative to the largest factor, so that what is rounded is a
// probability, not its product with a common factor (see cm_head_rows_kernel).
// PARTS: tiles of more than one part, whose logits then are the forward pass's, and
// near lse off by no more than lse is: the difference in the target's column is taken
// in fp32, and of a row that is sure of its target little is left.
// 2048 x 2048 x 32768 in two parts takes 147 to 149 us, as in one accumulator (146 to 149).
template <bool PARTS>
__device__ void finish_softgrad(const LinearPairMore &p, const LSmem &s, const Share &w, uint32_t tmem, int rank) {
    constexpr int BN = 256, kCols = BN / 2, kChunk = 64;
    const LinearEpilogue &e = p.e;
    const int ew = int(threadIdx.x) / 32 - 4, lane = int(threadIdx.x) & 31;
    const int quad = ew & 3, half = ew >> 2;
    uint8_t *const bufs = s.epi + ew * 2 * kEpiBuf;
    uint8_t *buf = bufs;
    const uint32_t tempty_leader = mapa_shared(smem_u32(&s.tempty[0]), 0);
    const int rest = int(p.cols % 8);
    const int64_t whole = p.cols - rest;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = w.first; t < w.tiles; t += w.step) {
        int mt, nt;
        tile_at(p, w.mtiles, t, mt, nt);
        const int row0 = mt * kTile + rank * kHalf + quad * 32, row = row0 + lane;
        const int cbase = nt * BN + half * kCols;
        const bool slot = row < w.rows;
        const float lse2 = slot ? p.head.lse2[row] : 0.0f, grad = slot ? p.head.grad[row] : 0.0f;
        const float hit = slot ? p.head.hit[row] : 0.0f;
        const int64_t target = slot ? p.head.target[row] : kNotHere, left = target - p.head.first - cbase;
        const int at = target >= 0 && left >= 0 && left < kCols ? int(left) : -1;
        const bool live = row0 < p.rows && cbase < p.cols;   // the same in the whole warp
        const uint32_t taddr0 = tmem + (uint32_t(quad * 32) << 16) + uint32_t(half * kCols);
        // 16 columns from c + 16 q on, as they lie in the buffer's rows
        auto finish16 = [&](int c, int q, const auto &v) {
            float g[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] = slot ? lin::exp2_fast(fmaf(v(i), lin::kLog2e, -lse2)) * grad : 0.0f;
            const int here = at - c - 16 * q;
            if (__any_sync(0xffffffffu, at >= 0 && here >= 0 && here < 16)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) g[i] -= at >= 0 && here == i ? hit : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) *piece(buf, lane, q * 2 + j) = pack8(g + 8 * j);
        };
        auto open_chunk = [&]() {
            if (lane == 0) bulk_wait_read<1>();   // the buffer's last store has been read out
            __syncwarp();
        };
        auto close_chunk = [&](int c) {
            const int c0 = cbase + c;
            if (rest && c0 + kChunk > whole && row < p.rows)
                store_tail(buf, e.y, e.ldy, row, whole, int(whole - c0), rest, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (c0 < whole) tma_store_3d(&p.tmY, buf, c0, row0, 0);
                bulk_commit();
            }
            buf = buf == bufs ? bufs + kEpiBuf : bufs;
        };
        if constexpr (PARTS) {
            float f[kCols / 16][16];
            if (!add_up_parts(p, s, w, taddr0, tempty_leader, live, t, acc, acc_phase, f)) break;
#pragma unroll
            for (int c = 0; c < kCols; c += kChunk) {
                if (!live || cbase + c >= p.cols) continue;
                open_chunk();
#pragma unroll
                for (int q = 0; q < 4; ++q) finish16(c, q, [&](int i) { return f[c / 16 + q][i]; });
                close_chunk(c);
            }
            continue;
        }
        bool ok = wait_p(p, s, &s.tfull[acc], acc_phase, kLinSiteAcc, t);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = taddr0 + uint32_t(acc * BN);
#pragma unroll 1
        for (int c = 0; live && c < kCols && cbase + c < p.cols; c += kChunk) {
            open_chunk();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[32];
                tmem_ld32(taddr + uint32_t(c + 32 * h), v);
                tmem_wait_ld_regs(v);
#pragma unroll
                for (int q = 0; q < 2; ++q) finish16(c, 2 * h + q, [&](int i) { return __uint_as_float(v[16 * q + i]); });
            }
            close_chunk(c);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty_leader + 8u * uint32_t(acc));
        if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
        }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
}

// Shared memory, barriers and tensor memory of a CTA.  Returns the accumulators' address.
template <int BN>
__device__ uint32_t open_pair(const LinearPairParams &p, LSmem &s, uint8_t *smem_raw) {
    constexpr int kStages = Tile<BN>::kStages;
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
    }
    if (threadIdx.x >> 5 == 1) {
        tmem_alloc_pair(s.tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the CTAs' barriers exist before any cross-CTA arrival or load
    tc_fence_after();
    let_next_start();
    wait_for_previous();
    return *s.tmem_slot;
}

// After an expired wait.  The leader's barriers count both CTAs' loads, but
// where the two gave up at different slices some complete no phase any more, and
// nothing tells when they have landed.  A load takes a few microseconds: the CTA,
// and with it its shared memory, stays for a millisecond after the last.
constexpr uint64_t kSettleNs = 1000000;
__device__ __noinline__ void settle() {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < kSettleNs) {
    }
}

__device__ void close_pair(const LSmem &s, uint32_t tmem) {
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // no cross-CTA traffic is left when a CTA frees its tensor memory
    tc_fence_after();
    // a slice that was not multiplied has kept both CTAs' accumulator waits from
    // ending, so both are aborting
    if (threadIdx.x == 0 && *s.abort) settle();
    if (threadIdx.x >> 5 == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

template <int LAYOUT, int BN, int MODE>
__global__ void __launch_bounds__(kLThreads, 1) cm_linear_pair_kernel(const __grid_constant__ PairParams<MODE> p) {
    extern __shared__ uint8_t smem_raw[];
    LSmem s;
    const uint32_t tmem = open_pair<BN>(p, s, smem_raw);
    const int warp = int(threadIdx.x) >> 5, rank = int(cluster_ctarank());
    const Share w = share_of<MODE>(p);
    if (warp == 0) {
        if (elect_one()) {
            Flow flow;
            load_tiles<LAYOUT, BN, MODE>(p, s, w, rank, flow);
            drain_loads<BN>(p, s, rank, flow);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            Flow flow;
            multiply_tiles<LAYOUT, BN, MODE>(p, s, w, tmem, flow);
            drain_products(p, s);
        }
        __syncwarp();
    } else if (warp >= 4) {
        [[maybe_unused]] Flow flow;
        if constexpr (MODE == kLinGated)
            finish_gated(p, s, tmem, rank);
        else if constexpr (MODE == kLinStats)
            if (w.kb1 - w.kb0 > kStatSlices)
                finish_stats(p, s, w, tmem, rank);
            else
                finish_stats_few(p, s, w, tmem, rank);
        else if constexpr (MODE == kLinSoftGrad)
            if (w.kb1 - w.kb0 > kStatSlices)
                finish_softgrad<true>(p, s, w, tmem, rank);
            else
                finish_softgrad<false>(p, s, w, tmem, rank);
        else if (MODE != kLinGateGrad && p.e.y_f32)
            finish_tiles<true, BN, MODE == kLinGateGrad ? kLinPlain : MODE>(p, s, w, tmem, rank, flow);
        else
            finish_tiles<false, BN, MODE>(p, s, w, tmem, rank, flow);
    }
    close_pair(s, tmem);
}

// ---- two products, one behind the other, in one launch ------------------------------
// Long tiles (of p0) leave pairs idle in their last round: with r tiles in it, all but r
// of them.  Those take q of the second product's shorter tiles each meanwhile, as
// many as a long one's K slices hold, and what is left of them goes round all pairs.
// The same tiles as in two launches, in fixed order.  Gradients of the loss, 1003 rows
// (653 of them counted), 4101 x 16381, dx and dw: 160 us in two launches.
struct TwoShares {
    Share w0, idle, rest;
};
__device__ __forceinline__ TwoShares two_shares(const LinearPairMore &p0, const LinearPairMore &p1) {
    constexpr int kLeast = 9;   // slices that the epilogue of a tile takes as long as
    TwoShares t;
    t.w0 = share_of<kLinCounted>(p0);
    t.idle = t.rest = share_of<kLinCounted>(p1);
    const int n = int(gridDim.x) >> 1, c = int(blockIdx.x) >> 1, r = t.w0.tiles % n;
    const int q = (t.w0.kb1 - t.w0.kb0) / max(t.rest.kb1 - t.rest.kb0, kLeast);
    const bool idle = r > 0 && c >= r;
    t.idle.step = 1;
    t.idle.first = idle ? int(min(int64_t(t.rest.tiles), int64_t(c - r) * q)) : 0;
    t.idle.tiles = idle ? int(min(int64_t(t.rest.tiles), int64_t(c - r + 1) * q)) : 0;
    const int given = r > 0 ? int(min(int64_t(t.rest.tiles), int64_t(n - r) * q)) : 0;
    t.rest.first = min(t.rest.tiles, given) + c;
    return t;
}

// L0: the first product's layout; the second's operands are both MN-major (3).
template <int L0>
__global__ void __launch_bounds__(kLThreads, 1) cm_linear_two_kernel(const __grid_constant__ LinearPairMore p0,
                                                                     const __grid_constant__ LinearPairMore p1) {
    extern __shared__ uint8_t smem_raw[];
    LSmem s;
    const uint32_t tmem = open_pair<256>(p0, s, smem_raw);
    const int warp = int(threadIdx.x) >> 5, rank = int(cluster_ctarank());
    const TwoShares t = two_shares(p0, p1);
    Flow flow;
    if (warp == 0) {
        if (elect_one()) {
            load_tiles<L0, 256, kLinCounted>(p0, s, t.w0, rank, flow);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) load_tiles<3, 256, kLinCounted>(p1, s, i ? t.rest : t.idle, rank, flow);
            drain_loads<256>(p0, s, rank, flow);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            multiply_tiles<L0, 256, kLinCounted>(p0, s, t.w0, tmem, flow);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) multiply_tiles<3, 256, kLinCounted>(p1, s, i ? t.rest : t.idle, tmem, flow);
            drain_products(p0, s);
        }
        __syncwarp();
    } else if (warp >= 4) {
        finish_tiles<true, 256, kLinCounted>(p0, s, t.w0, tmem, rank, flow);   // fp32 sums
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            if (p1.e.y_f32)
                finish_tiles<true, 256, kLinCounted>(p1, s, i ? t.rest : t.idle, tmem, rank, flow);
            else
                finish_tiles<false, 256, kLinCounted>(p1, s, i ? t.rest : t.idle, tmem, rank, flow);
        }
    }
    close_pair(s, tmem);
}

// ---- few tiles: K split over the pairs of a cluster ---------------------------------

// 16-byte piece (columns 4c .. 4c + 3) of row r of a partial tile of BN fp32
// columns; the pieces of a row are permuted within groups of eight, so that 32
// rows written at one column do not meet in one bank.
template <int BN>
__device__ __forceinline__ uint32_t partial_at(int r, int c) {
    return uint32_t(r * BN * 4 + ((c ^ (r & 7)) << 4));
}

// Four neighbouring elements of a row.
__device__ __forceinline__ void get4(const void *m, int64_t at, int n, float (&f)[4]) {
    const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(m) + at;
    if (n >= 4) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        f[0] = __uint_as_float(w.x << 16), f[1] = __uint_as_float(w.x & 0xffff0000u);
        f[2] = __uint_as_float(w.y << 16), f[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
    }
}
__device__ __forceinline__ void put4(void *m, int64_t at, int n, const float (&f)[4]) {
    __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(m) + at;
    if (n >= 4) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(f[i]);
    }
}

// The epilogue of columns col .. col + 3 (n of them inside) of four rows
// row, row + step, ... below `end`; loads of all rows before the first store.
__device__ __forceinline__ void finish4(const LinearEpilogue &e, float (&v)[4][4], const float (&bias)[4], int64_t row,
                                        int64_t step, int64_t end, int64_t col, int n) {
    float in[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] += bias[i];
    if (e.z) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (row + k * step < end) put4(e.z, (row + k * step) * e.ldz + col, n, v[k]);
    }
    auto read = [&](const void *m, int64_t ld) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (row + k * step < end) {
                get4(m, (row + k * step) * ld + col, n, in[k]);
            } else {
                in[k][0] = in[k][1] = in[k][2] = in[k][3] = 0.0f;
            }
    };
    auto add_in = [&]() {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] += in[k][i];
    };
    if (e.dact) {
        read(e.zin, e.ldzin);
#pragma unroll
        for (int k = 0; k < 4; ++k) lin::mul_dact(v[k], in[k], e.act);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) lin::apply_act(v[k], e.act);
    }
    if (e.res) {
        read(e.res, e.ldr);
        add_in();
    }
    if (!e.y_f32) {
        if (e.accumulate) {
            read(e.y, e.ldy);
            add_in();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (row + k * step < end) put4(e.y, (row + k * step) * e.ldy + col, n, v[k]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float *y = static_cast<float *>(e.y) + (row + k * step) * e.ldy + col;
        if (row + k * step >= end) continue;
        if (n >= 4) {
            if (e.accumulate) {
                const float4 o = *reinterpret_cast<const float4 *>(y);
                v[k][0] += o.x, v[k][1] += o.y, v[k][2] += o.z, v[k][3] += o.w;
            }
            *reinterpret_cast<float4 *>(y) = make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) y[i] = e.accumulate ? y[i] + v[k][i] : v[k][i];
        }
    }
}

// The same for the gate's gradients: v is the gradient of act(g) u.
__device__ __forceinline__ void finish4_gate_grad(const LinearEpilogue &e, float (&v)[4][4], int64_t row, int64_t step,
                                                  int64_t end, int64_t col, int n) {
    float g[4][4], u[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const bool live = row + k * step < end;
        get4(e.zin, (row + k * step) * e.ldzin + col, live ? n : 0, g[k]);
        get4(e.zin2, (row + k * step) * e.ldzin + col, live ? n : 0, u[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (row + k * step >= end) continue;
        lin::gate_grad(v[k], g[k], u[k], e.act);
        put4(e.z, (row + k * step) * e.ldz + col, n, g[k]);
        put4(e.y, (row + k * step) * e.ldy + col, n, u[k]);
    }
}

// A cluster of S pairs computes one tile, pair j the j-th part of its K slices.
// Each CTA leaves its 128 rows of the partial tile in its own shared memory as
// fp32 (the ring, whose loads have all been multiplied by then); after a
// cluster barrier pair j finishes the j-th part of the columns, adding the
// pairs' partial sums in their order.  No workspace, one launch, the same bits
// every time.  200 x 8192 x 3584 takes 19.9 us on four pairs a tile, 26.3 on two
// and 42.5 unsplit; the exchange and the summing cost 4 us (128 columns) to 6.5.
template <int LAYOUT, int BN, int S, int MODE>
__global__ void __launch_bounds__(kLThreads, 1) cm_linear_split_kernel(const __grid_constant__ PairParams<MODE> p) {
    extern __shared__ uint8_t smem_raw[];
    static_assert(kHalf * BN * 4 <= kRingBytes, "a partial tile fits in the ring");
    LSmem s;
    const uint32_t tmem = open_pair<BN>(p, s, smem_raw);
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    const int crank = int(cluster_ctarank()), rank = crank & 1, part = crank >> 1;
    const int tile = int(blockIdx.x) / (2 * S);
    const Share w = {tile, p.tiles, int(int64_t(p.kblocks) * part / S), int(int64_t(p.kblocks) * (part + 1) / S),
                     uint32_t(crank & ~1), p.tiles, p.mtiles, p.rows, &p.tmA, &p.tmB};
    int mt, nt;
    tile_at(p, p.mtiles, tile, mt, nt);
    const int row0 = mt * kTile + rank * kHalf;
    const int nrows = int(max(int64_t(0), min(int64_t(kHalf), p.rows - row0)));
    bool good = true;
    if (warp == 0) {
        if (elect_one()) {
            Flow flow;
            load_tiles<LAYOUT, BN, MODE>(p, s, w, rank, flow);
            drain_loads<BN>(p, s, rank, flow);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            Flow flow;
            multiply_tiles<LAYOUT, BN, MODE>(p, s, w, tmem, flow);
            drain_products(p, s);
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quad = warp & 3, half = (warp - 4) >> 2;
        good = wait_p(p, s, &s.tfull[0], 0, kLinSiteAcc, tile);
        good = __all_sync(0xffffffffu, good);
        tc_fence_after();
        const int r = quad * 32 + lane;
        if (good && quad * 32 < nrows) {
#pragma unroll 1
            for (int c0 = half * (BN / 2); c0 < (half + 1) * (BN / 2); c0 += 32) {
                uint32_t v[32];
                tmem_ld32(tmem + (uint32_t(quad * 32) << 16) + uint32_t(c0), v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4 *>(s.a0 + partial_at<BN>(r, c0 / 4 + j)) =
                        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
        }
        __syncwarp();
    }
    // after an expired wait the outputs are undefined; the barriers below are
    // reached all the same
    __syncthreads();
    cluster_sync();
    // gated: pair j finishes the j-th part of the gate's columns with the up projection's
    constexpr int kTileCols = MODE == kLinGated ? BN / 2 : BN;
    constexpr int kCols = kTileCols / S, kLanes = kCols / 4, kRows = kLThreads / kLanes;   // threads a row, rows at a time
    const int c = part * kCols + int(threadIdx.x) % kLanes * 4;
    const int64_t col = int64_t(nt) * kTileCols + c;
    const int n = int(max(int64_t(0), min(int64_t(4), p.cols - col)));
    if (n > 0) {
        float bias[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[i] = i < n ? lin::load_bias(p.e, col + i) : 0.0f;
        [[maybe_unused]] float bias2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bias2[i] = MODE == kLinGated && i < n ? lin::load_bias(p.e.bias2, p.e.bias_f32, col + i) : 0.0f;
        uint32_t base[S];
#pragma unroll
        for (int j = 0; j < S; ++j) base[j] = mapa_shared(smem_u32(s.a0), uint32_t(2 * j + rank));
        for (int r = int(threadIdx.x) / kLanes; r < nrows; r += 4 * kRows) {
            // the sum of row r + k kRows, columns at .. at + 3, over the pairs in their order
            auto sum = [&](int k, int at, float (&v)[4]) {
                float4 q[S];
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    q[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (r + k * kRows < nrows)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(q[j].x), "=f"(q[j].y), "=f"(q[j].z), "=f"(q[j].w)
                                     : "r"(base[j] + partial_at<BN>(r + k * kRows, at / 4))
                                     : "memory");
                }
                v[0] = q[0].x, v[1] = q[0].y, v[2] = q[0].z, v[3] = q[0].w;
#pragma unroll
                for (int j = 1; j < S; ++j) v[0] += q[j].x, v[1] += q[j].y, v[2] += q[j].z, v[3] += q[j].w;
            };
            float v[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) sum(k, c, v[k]);
            if constexpr (MODE == kLinGated) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float u[4];
                    sum(k, BN / 2 + c, u);
                    if (r + k * kRows >= nrows) continue;
                    const int64_t row = int64_t(row0) + r + k * kRows;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[k][i] += bias[i], u[i] += bias2[i];
                    if (p.e.z) {
                        put4(p.e.z, row * p.e.ldz + col, n, v[k]);
                        put4(p.e.z2, row * p.e.ldz + col, n, u);
                    }
                    lin::apply_gate(v[k], u, p.e.act);
                    put4(p.e.y, row * p.e.ldy + col, n, v[k]);
                }
            } else if constexpr (MODE == kLinGateGrad) {
                finish4_gate_grad(p.e, v, int64_t(row0) + r, kRows, int64_t(row0) + nrows, col, n);
            } else {
                finish4(p.e, v, bias, int64_t(row0) + r, kRows, int64_t(row0) + nrows, col, n);
            }
        }
    }
    close_pair(s, tmem);   // with its cluster barrier the peers have read this CTA's partial tile
}

cudaError_t pair_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, unsigned cluster, unsigned ctas,
                        cudaStream_t stream) {
    cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kLThreads, 1, 1);
    cfg.dynamicSmemBytes = kLSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaSuccess;
}

template <int MODE>
using PairKernel = void (*)(PairParams<MODE>);

// By operand layout (0, 1, 3), tile columns and pairs of a cluster; what a mode does
// not have is NULL.
template <int MODE, int LAYOUT>
PairKernel<MODE> pair_kernel_of(int bn, int splits) {
    constexpr bool kSplits = !kIsCounted<MODE>, kNarrow = MODE != kLinGated && MODE != kLinStats && MODE != kLinSoftGrad;
    if (bn == 256 && splits == 1) return cm_linear_pair_kernel<LAYOUT, 256, MODE>;
    if constexpr (kNarrow)
        if (bn == 128 && splits == 1) return cm_linear_pair_kernel<LAYOUT, 128, MODE>;
    if constexpr (kSplits) {
        if (bn == 256 && splits == 2) return cm_linear_split_kernel<LAYOUT, 256, 2, MODE>;
        if (bn == 256 && splits == 4) return cm_linear_split_kernel<LAYOUT, 256, 4, MODE>;
    }
    if constexpr (kSplits) {
        if (bn == 128 && splits == 2) return cm_linear_split_kernel<LAYOUT, 128, 2, MODE>;
        if (bn == 128 && splits == 4) return cm_linear_split_kernel<LAYOUT, 128, 4, MODE>;
    }
    return nullptr;
}
template <int MODE>
PairKernel<MODE> pair_kernel(int layout, int bn, int splits) {
    if (layout == 0) return pair_kernel_of<MODE, 0>(bn, splits);
    if (layout == 1) return pair_kernel_of<MODE, 1>(bn, splits);
    if constexpr (MODE == kLinPlain || MODE == kLinCounted)
        if (layout == 3) return pair_kernel_of<MODE, 3>(bn, splits);
    return nullptr;
}

template <int MODE>
cudaError_t prepare_pair() {
    for (int layout : {0, 1, 3})
        for (int bn : {256, 128})
            for (int splits : {1, 2, 4})
                if (const auto fn = pair_kernel<MODE>(layout, bn, splits)) {
                    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kLSmem);
                    if (e != cudaSuccess) return e;
                }
    return cudaSuccess;
}

template <int MODE>
cudaError_t launch_pair(const LinearPairMore &p, int layout, int splits, int clusters, cudaStream_t stream) {
    const auto fn = pair_kernel<MODE>(layout, p.bn, splits);
    if (!fn) return cudaErrorInvalidValue;
    // split: one cluster a tile; else persistent
    const int n = splits > 1 ? p.tiles : std::max(1, std::min(clusters, p.tiles));
    return launch_after(fn, dim3(unsigned(2 * splits * n)), kLThreads, size_t(kLSmem), unsigned(2 * splits), stream,
                        static_cast<const PairParams<MODE> &>(p));
}

}  // namespace

cudaError_t prepare_linear_pair(int sms, int *clusters) {
    cudaError_t e = cudaSuccess;
    for (auto prepare : {prepare_pair<kLinPlain>, prepare_pair<kLinGated>, prepare_pair<kLinGateGrad>, prepare_pair<kLinStats>,
                         prepare_pair<kLinSoftGrad>, prepare_pair<kLinCounted>})
        if ((e = prepare()) != cudaSuccess) return e;
    for (auto fn : {cm_linear_two_kernel<0>, cm_linear_two_kernel<1>})
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kLSmem)) != cudaSuccess) return e;
    for (int i = 0; i < 3; ++i) {
        const int splits = 1 << i;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[1];
        pair_config(cfg, attr, unsigned(2 * splits), unsigned(sms / (2 * splits) * (2 * splits)), nullptr);
        if ((e = cudaOccupancyMaxActiveClusters(&clusters[i], pair_kernel<kLinPlain>(0, 256, splits), &cfg)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_linear_pair(const LinearPairMore &p, int layout, LinearMode mode, int splits, int clusters,
                               cudaStream_t stream) {
    switch (mode) {
        case kLinPlain: return launch_pair<kLinPlain>(p, layout, splits, clusters, stream);
        case kLinGated: return launch_pair<kLinGated>(p, layout, splits, clusters, stream);
        case kLinGateGrad: return launch_pair<kLinGateGrad>(p, layout, splits, clusters, stream);
        case kLinStats: return launch_pair<kLinStats>(p, layout, splits, clusters, stream);
        case kLinSoftGrad: return launch_pair<kLinSoftGrad>(p, layout, splits, clusters, stream);
        case kLinCounted: return launch_pair<kLinCounted>(p, layout, splits, clusters, stream);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_linear_two(const LinearPairMore &p0, int layout0, const LinearPairMore &p1, int clusters, cudaStream_t stream) {
    const auto fn = layout0 == 0 ? cm_linear_two_kernel<0> : layout0 == 1 ? cm_linear_two_kernel<1> : nullptr;
    if (!fn || p0.bn != 256 || p1.bn != 256) return cudaErrorInvalidValue;
    return launch_after(fn, dim3(unsigned(2 * clusters)), kLThreads, size_t(kLSmem), 2u, stream, p0, p1);
}

}  // namespace cm
