// cm_embedding.cu -- embedding lookup and its gradient.
//
//   forward   y[t] = scale w[id[t] - first], zeros where the id is not one of the slice's
//   backward  dw[v] (+)= scale sum over the tokens t with id[t] = first + v of dy[t], t ascending
//
// Both are bound by memory: the rows read and written.  The gradient's tokens
// are sorted by (row, token) first, so that every row of dw is summed and written
// once, in one order, whatever the timing:
//   1. tiles of 1024 keys (row << 32 | token) are sorted in shared memory;
//   2. up to 32 sorted runs at a time become one: a key's place is its place in
//      its own run plus the number of smaller keys in each other run, found by
//      bisection; keys are all different, so no two meet.  Again while runs are left;
//   3. a warp takes an aligned piece of 16 sorted tokens and 256 columns, and writes
//      the sums of the rows whose tokens all lie in it.  A row that goes on beyond
//      the piece, or came from the one before, leaves its part in the workspace;
//   4. the parts of such a row are added in order by a warp, or where there are
//      many by the warps of a CTA, each neighbouring ones, then the warps' sums.
// Where dw is not added to, a launch of its own writes zeros to the absent rows.
#include <cuda_bf16.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cstdint>

#include "cm_internal.h"
#include "cm_launch.cuh"
#include "cm_vec.cuh"

namespace cm {
namespace {

using namespace vec;

constexpr int64_t kMaxExtent = int64_t(1) << 30;
constexpr int64_t kMostColumns = 65535 * 256;   // blocks of columns are counted by the grid's second extent
constexpr uint32_t kNoRow = 0xffffffffu;   // the row of a token that is not of the slice: sorted last

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

struct Ids {
    const void *p;
    int64_t first;
    int64_t rows;    // of the slice
    int bits;
};

// Row of the slice that token t looks up, or kNoRow.
__device__ __forceinline__ uint32_t row_of(const Ids &s, int64_t t) {
    const int64_t id = s.bits == 64 ? static_cast<const int64_t *>(s.p)[t] : int64_t(static_cast<const int32_t *>(s.p)[t]);
    return id >= s.first && id - s.first < s.rows ? uint32_t(id - s.first) : kNoRow;
}

__device__ __forceinline__ V8 scaled(const V8 &v, float a) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = mul(v.p[i], both(a));
    return r;
}
__device__ __forceinline__ void add_to(V8 &a, const V8 &b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a.p[i] = add(a.p[i], b.p[i]);
}

// Eight neighbouring elements at column c of a row of h: whole vectors (rows
// start on 16 bytes) or element by element.
template <bool VEC, typename T>
__device__ __forceinline__ V8 get8(const T *row, int c, int h) {
    if constexpr (VEC) {
        return load_row8(row, c, h);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < h ? to_f(row[c + i]) : 0.0f;
        return {{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
    }
}
template <bool VEC, typename T>
__device__ __forceinline__ void put8(T *row, int c, int h, const V8 &v) {
    if constexpr (VEC) {
        store_row8(row, c, h, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = parts(v.p[i]);
            if (c + 2 * i < h) from_f(row + c + 2 * i, p.x);
            if (c + 2 * i + 1 < h) from_f(row + c + 2 * i + 1, p.y);
        }
    }
}

// Eight neighbouring elements as they were loaded: of bf16 half the registers of the
// numbers, so that more warps fit on an SM.
template <typename T, bool VEC>
struct Raw8 {
    V8 v;
    __device__ __forceinline__ void load(const T *row, int c, int h) { v = get8<VEC>(row, c, h); }
    __device__ __forceinline__ V8 get() const { return v; }
};
template <>
struct Raw8<bf16, true> {
    uint4 w;
    __device__ __forceinline__ void load(const bf16 *row, int c, int h) {
        if (c + 8 <= h) {
            w = *reinterpret_cast<const uint4 *>(row + c);
            return;
        }
        const V8 v = load_row8(row, c, h);
        w = make_uint4(pack(v.p[0]), pack(v.p[1]), pack(v.p[2]), pack(v.p[3]));
    }
    __device__ __forceinline__ V8 get() const { return {{unpack(w.x), unpack(w.y), unpack(w.z), unpack(w.w)}}; }
};

// ---- lookup -------------------------------------------------------------------------
struct LookupParams {
    Ids ids;
    const void *w;
    void *y;
    int64_t ldw, ldy, tokens;
    int h, width;
    float scale;
};

constexpr int kLookThreads = 256, kLookBatch = 4;

// `width` (a power of two up to 256) neighbouring threads share a row, each with
// four of its vectors under way before its first store; rows of more than 1024
// vectors take several CTAs.  Bound by memory: 16384 tokens of 8192 elements take 62 us.
// (Counted through all rows' vectors, with a division each, 101; with half the CTAs an
// SM 78.)
template <typename W, typename Y, bool VEC>
__global__ void __launch_bounds__(kLookThreads, !VEC || sizeof(W) == 4 ? 4 : sizeof(Y) == 4 ? 6 : 8) cm_embedding_kernel(const LookupParams p) {
    let_next_start();
    wait_for_previous();
    const int lane = int(threadIdx.x) & (p.width - 1), rows = kLookThreads / p.width;
    const int64_t t = int64_t(blockIdx.x) * rows + int(threadIdx.x) / p.width;
    if (t >= p.tokens) return;
    const int c0 = (int(blockIdx.y) * kLookBatch * p.width + lane) * 8, step = p.width * 8;
    const uint32_t row = row_of(p.ids, t);
    const W *from = static_cast<const W *>(p.w) + int64_t(row == kNoRow ? 0 : row) * p.ldw;
    Y *to = static_cast<Y *>(p.y) + t * p.ldy;
    Raw8<W, VEC> v[kLookBatch];
#pragma unroll
    for (int k = 0; k < kLookBatch; ++k)
        if (row != kNoRow && c0 + k * step < p.h) v[k].load(from, c0 + k * step, p.h);
#pragma unroll
    for (int k = 0; k < kLookBatch; ++k)
        if (c0 + k * step < p.h) put8<VEC>(to, c0 + k * step, p.h, row != kNoRow ? scaled(v[k].get(), p.scale) : fill(0.0f));
}

// ---- tokens sorted by row -----------------------------------------------------------
constexpr int kSortTile = 1024, kMergeRuns = 32, kMergeThreads = 256;

__device__ __forceinline__ uint64_t lesser(uint64_t a, uint64_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint64_t greater(uint64_t a, uint64_t b) { return a < b ? b : a; }

// One key a thread, bitonic: partners less than a warp apart by shuffles, the
// others through shared memory.  Latency, 6 us for any number of tiles that run at once.
__global__ void __launch_bounds__(kSortTile) cm_embedding_sort_kernel(const Ids ids, int64_t tokens, uint64_t *keys, uint32_t *rows) {
    __shared__ uint64_t s[kSortTile];
    let_next_start();
    wait_for_previous();
    const int i = int(threadIdx.x);
    const int64_t t = int64_t(blockIdx.x) * kSortTile + i;
    uint64_t k = ~uint64_t(0);   // behind the last token: sorted behind everything, and not stored
    if (t < tokens) k = uint64_t(row_of(ids, t)) << 32 | uint64_t(t);
    for (int size = 2; size <= kSortTile; size *= 2)
        for (int d = size / 2; d; d /= 2) {
            uint64_t other;
            if (d >= 32) {
                __syncthreads();
                s[i] = k;
                __syncthreads();
                other = s[i ^ d];
            } else {
                other = __shfl_xor_sync(0xffffffffu, k, d);
            }
            const bool low = (i & d) == 0, up = (i & size) == 0;   // up: ascending (all of it in the last round)
            k = low == up ? lesser(k, other) : greater(k, other);
        }
    if (t < tokens) keys[t] = k, rows[t] = uint32_t(k >> 32);
}

// Groups of up to 32 sorted runs of `run` keys (a power of two) become one run each.
// Earlier runs hold earlier tokens: of equal rows theirs come first, so rows alone are
// compared.  Of each run 32 rows at equal distances lie in shared memory, where a
// bisection begins; in the first round the 32 rows that are left of a run are one line
// of cache.  A thread bisects eight runs at a time, whose loads do not wait for one
// another.  Latency: 10007 tokens take 9 us, 65536 in two rounds 45.
constexpr int kSamples = 32;
__global__ void __launch_bounds__(kMergeThreads) cm_embedding_merge_kernel(const uint64_t *in, const uint32_t *rows_in, uint64_t *out,
                                                                           uint32_t *rows_out, uint32_t tokens, uint32_t run) {
    __shared__ uint32_t sample[kMergeRuns * kSamples];
    let_next_start();
    wait_for_previous();
    // run is a multiple of a CTA's keys: they all lie in one run
    const uint32_t i0 = blockIdx.x * kMergeThreads, i = i0 + threadIdx.x;
    const uint32_t own = i0 / run % kMergeRuns, base = (i0 / run - own) * run, stride = run / kSamples;
    const int shift = __ffs(int(stride)) - 1;
    const uint32_t n = min(uint64_t(tokens - base), uint64_t(kMergeRuns) * run);   // keys of the group
    const uint32_t *const rows = rows_in + base;
#pragma unroll
    for (uint32_t j = threadIdx.x; j < kMergeRuns * kSamples; j += kMergeThreads) {
        const uint64_t at = uint64_t(j + 1) * stride - 1;
        sample[j] = at < n ? rows[at] : 0u;
    }
    __syncthreads();
    if (i >= tokens) return;
    const uint64_t k = in[i];
    const uint32_t row = uint32_t(k >> 32);
    uint32_t place = i - base - own * run;
    constexpr uint32_t kAtOnce = 8;
    for (uint32_t r0 = 0; r0 < kMergeRuns && uint64_t(r0) * run < n; r0 += kAtOnce) {
        uint32_t at[kAtOnce], left[kAtOnce];
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) {
            const uint64_t first = uint64_t(r0 + j) * run;
            at[j] = 0;
            left[j] = r0 + j == own || first >= n ? 0u : min(run, n - uint32_t(first));
        }
        uint32_t step = run;
        for (; step >= stride; step >>= 1)
#pragma unroll
            for (uint32_t j = 0; j < kAtOnce; ++j) {
                if (at[j] + step > left[j]) continue;
                const uint32_t other = sample[(r0 + j) * kSamples + ((at[j] + step) >> shift) - 1];
                if (other < row || (r0 + j < own && other == row)) at[j] += step;
            }
        for (; step; step >>= 1)
#pragma unroll
            for (uint32_t j = 0; j < kAtOnce; ++j) {
                if (at[j] + step > left[j]) continue;
                const uint32_t other = rows[(r0 + j) * run + at[j] + step - 1];
                if (other < row || (r0 + j < own && other == row)) at[j] += step;
            }
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) place += at[j];
    }
    out[base + place] = k;
    rows_out[base + place] = row;
}

// ---- sums of rows -------------------------------------------------------------------
struct SumParams {
    const uint64_t *keys;    // sorted
    const void *dy;
    void *dw;
    float *parts;            // [ceil(tokens / 16)][2][h, rounded up to 8]: of a row from the piece before, and into the next
    int64_t lddy, lddw, tokens, rows;
    int h;
    float scale;
    int accumulate;
    int64_t sum_ctas;
};

constexpr int kPiece = 16;                 // sorted tokens of a warp
constexpr int kAtOnce = 4;                 // rows under way at a time, and where dw is added to as many of its

__device__ __forceinline__ uint32_t row_at(const SumParams &p, int64_t i) { return uint32_t(p.keys[i] >> 32); }
__device__ __forceinline__ float *part_at(const SumParams &p, int64_t piece, int into_next, int c) {
    return p.parts + (piece * 2 + into_next) * ((p.h + 7) / 8 * 8) + c;
}

template <bool VEC, typename DW>
__device__ __forceinline__ V8 old_row(const SumParams &p, uint32_t row, int c) {
    return get8<VEC>(static_cast<const DW *>(p.dw) + int64_t(row) * p.lddw, c, p.h);
}
template <bool VEC, typename DW>
__device__ __forceinline__ void put_row(const SumParams &p, const V8 &acc, const V8 &old, uint32_t row, int c) {
    V8 v = scaled(acc, p.scale);
    if (p.accumulate) add_to(v, old);
    put8<VEC>(static_cast<DW *>(p.dw) + int64_t(row) * p.lddw, c, p.h, v);
}

// Rows of dw without a token: zeros.  A warp a row, which it looks up among the sorted
// tokens, 32 probes a round.  A launch of its own with little in it but stores, and CTAs
// that leave as soon as theirs are out, so that the SMs write one moving front:
// 131072 x 4096 fp32 in 270 to 285 us (a memset takes 277); with 32 rows a warp it was 359, with
// rows a persistent CTA's 320 to 500.
template <typename DW, bool VEC>
__global__ void __launch_bounds__(256) cm_embedding_zero_kernel(const SumParams p) {
    let_next_start();
    wait_for_previous();
    const int lane = int(threadIdx.x) & 31;
    const int64_t v = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (v >= p.rows) return;
    int64_t lo = 0, n = p.tokens;   // rows of tokens [.. lo) are smaller, of [lo + n ..) not
    while (n > 0) {
        const int64_t step = (n + 31) / 32, at = min(n, int64_t(lane + 1) * step) - 1;   // probes repeat at the end
        const uint32_t row = row_at(p, lo + at);
        if (__any_sync(0xffffffffu, row == v)) return;
        const int64_t right = min(n, __popc(__ballot_sync(0xffffffffu, row < v)) * step);
        lo += right;
        n = min(step - 1, n - right);
    }
    constexpr int kPer = 16 / int(sizeof(DW));
    const int whole = VEC ? p.h / kPer : 0;   // 16-byte pieces of a row
    DW *row = static_cast<DW *>(p.dw) + v * p.lddw;
#pragma unroll 8
    for (int i = lane; i < whole; i += 32) reinterpret_cast<uint4 *>(row)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int c = whole * kPer + lane; c < p.h; c += 32) from_f(row + c, 0.0f);
}

// A warp for each aligned piece of 16 sorted tokens and 256 columns; ADD: dw is added to.
// Four rows, and as many old ones of dw, are under way at a time.  Bound by memory for many
// tokens (16384 x 8192 into fp32, uniform: 108 us, 6 TB/s), by latency for few.
template <typename DY, typename DW, bool VEC, bool ADD>
__global__ void __launch_bounds__(256, ADD || sizeof(DY) == 4 || !VEC ? 2 : 4) cm_embedding_sum_kernel(const SumParams p) {
    let_next_start();
    wait_for_previous();
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    const int64_t blocks = (p.h + 255) / 256, unit = int64_t(blockIdx.x) * 8 + warp, piece = unit / blocks;
    const int c = int(unit - piece * blocks) * 256 + lane * 8;
    const int64_t i0 = piece * kPiece, i = i0 + lane;
    if (i0 >= p.tokens) return;
    // a lane holds one token: its row, and whether it is the row's first or last in the piece
    const uint64_t key = lane < kPiece && i < p.tokens ? p.keys[i] : ~uint64_t(0);
    const uint32_t row = uint32_t(key >> 32), token = uint32_t(key);
    const uint32_t before = __shfl_up_sync(0xffffffffu, row, 1), behind = __shfl_down_sync(0xffffffffu, row, 1);
    const uint32_t live = __ballot_sync(0xffffffffu, row != kNoRow);   // sorted: the first ones
    if (live == 0) return;
    const uint32_t first = __ballot_sync(0xffffffffu, lane == 0 || before != row);
    const uint32_t last = __ballot_sync(0xffffffffu, lane == kPiece - 1 || behind != row);
    const bool from_before = i0 > 0 && row_at(p, i0 - 1) == __shfl_sync(0xffffffffu, row, 0);
    const bool into_next = i0 + kPiece < p.tokens && row_at(p, i0 + kPiece) == __shfl_sync(0xffffffffu, row, kPiece - 1);
    const int n = __popc(live);
    // rows that go on in another piece: their parts go to the workspace
    const uint32_t apart = (from_before ? last & (0u - last) : 0u) | (into_next ? 1u << (kPiece - 1) : 0u);
    V8 acc = fill(0.0f);
#pragma unroll 1
    for (int j = 0; j < n; j += kAtOnce) {
        Raw8<DY, VEC> v[kAtOnce];
        [[maybe_unused]] V8 old[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const uint32_t t = __shfl_sync(0xffffffffu, token, j + k), r = __shfl_sync(0xffffffffu, row, j + k);
            if (j + k >= n || c >= p.h) continue;
            v[k].load(static_cast<const DY *>(p.dy) + int64_t(t) * p.lddy, c, p.h);
            if constexpr (ADD)
                if ((last & ~apart) >> (j + k) & 1) old[k] = old_row<VEC, DW>(p, r, c);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int at = j + k;
            const uint32_t r = __shfl_sync(0xffffffffu, row, at);
            if (at >= n || c >= p.h) continue;
            if (first >> at & 1) acc = fill(0.0f);
            add_to(acc, v[k].get());
            if (!(last >> at & 1)) continue;
            if (apart >> at & 1) {   // the piece's first row, where it came from before; else the last, which goes on
                store8(part_at(p, piece, from_before && (last & ((1u << at) - 1)) == 0 ? 0 : 1, c), acc);
                continue;
            }
            V8 sum = scaled(acc, p.scale);
            if constexpr (ADD) add_to(sum, old[k]);
            put8<VEC>(static_cast<DW *>(p.dw) + int64_t(r) * p.lddw, c, p.h, sum);
        }
    }
}

// The sum of parts k0 .. k1 - 1, in order, of the row that goes on from `piece` into
// the next: that piece's second part, and the first ones of the pieces behind.
__device__ __forceinline__ V8 add_parts(const SumParams &p, int64_t piece, int64_t k0, int64_t k1, int c) {
    constexpr int kParts = 4;
    V8 acc = fill(0.0f);
    for (int64_t k = k0; k < k1; k += kParts) {
        V8 v[kParts];
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            v[j] = fill(0.0f);
            if (k + j < k1) v[j] = load8(part_at(p, piece + k + j, k + j == 0, c));
        }
#pragma unroll
        for (int j = 0; j < kParts; ++j) add_to(acc, v[j]);
    }
    return acc;
}

// The rows that lie in several pieces.  A CTA looks at 16 pieces, a lane at each, for
// rows that begin there and go on; columns of 256.  A warp adds the parts of up to
// 32 pieces; longer rows are shared by the CTA's warps, each with a run of their parts.
// 16384 tokens by Zipf's law x 4096: 14 us.
constexpr int kJoinPieces = 16;
template <typename DW, bool VEC>
__global__ void __launch_bounds__(256, 3) cm_embedding_join_kernel(const SumParams p) {
    __shared__ V8 sums[8][32];
    let_next_start();
    wait_for_previous();
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31, c = int(blockIdx.y) * 256 + lane * 8;
    const int64_t piece0 = int64_t(blockIdx.x) * kJoinPieces, end = (piece0 + lane + 1) * kPiece;   // of the lane's piece
    uint32_t row = kNoRow;
    if (lane < kJoinPieces && end < p.tokens) {
        row = row_at(p, end);
        if (row_at(p, end - 1) != row) row = kNoRow;
        // began earlier
        if (end > kPiece && row_at(p, end - kPiece) == row && row_at(p, end - kPiece - 1) == row) row = kNoRow;
    }
    const uint32_t owners = __ballot_sync(0xffffffffu, row != kNoRow);   // the same in every warp
    uint32_t longer = 0;
    for (uint32_t left = owners, at = 0; left; left &= left - 1, ++at) {
        const int o = __ffs(left) - 1;
        const uint32_t r = __shfl_sync(0xffffffffu, row, o);
        const int64_t piece = piece0 + o, i = (piece + 2 + lane) * kPiece;
        // pieces behind the next that hold some of the row
        const uint32_t more = __ballot_sync(0xffffffffu, i < p.tokens && row_at(p, i) == r);
        if (more == 0xffffffffu) longer |= 1u << o;
        if (more == 0xffffffffu || int(at % 8) != warp || c >= p.h) continue;
        const V8 old = p.accumulate ? old_row<VEC, DW>(p, r, c) : fill(0.0f);
        put_row<VEC, DW>(p, add_parts(p, piece, 0, 2 + __popc(more), c), old, r, c);
    }
    for (; longer; longer &= longer - 1) {   // the same in every warp
        const int o = __ffs(longer) - 1;
        const uint32_t r = __shfl_sync(0xffffffffu, row, o);
        const int64_t piece = piece0 + o;
        int64_t n = 2;   // pieces that hold some of the row
        while (true) {
            const int64_t i = (piece + n + threadIdx.x) * kPiece;
            const int more = __syncthreads_count(i < p.tokens && row_at(p, i) == r);
            n += more;
            if (more < int(blockDim.x)) break;
        }
        if (c < p.h) sums[warp][lane] = add_parts(p, piece, n * warp / 8, n * (warp + 1) / 8, c);
        __syncthreads();
        if (warp == 0 && c < p.h) {
            V8 acc = sums[0][lane];
#pragma unroll
            for (int w = 1; w < 8; ++w) add_to(acc, sums[w][lane]);
            put_row<VEC, DW>(p, acc, p.accumulate ? old_row<VEC, DW>(p, r, c) : fill(0.0f), r, c);
        }
        __syncthreads();
    }
}

// ---- launches -----------------------------------------------------------------------
bool bad_dtype(cm_dtype t) { return t != CM_BF16 && t != CM_F32; }
bool misaligned(const void *p, cm_dtype t) { return (reinterpret_cast<uintptr_t>(p) & (t == CM_F32 ? 3u : 1u)) != 0; }
bool whole_vectors(const void *p, cm_dtype t, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % (t == CM_F32 ? 4 : 8) == 0;
}

cm_status check_rows(const void *p, cm_dtype t, int64_t ld, int64_t h) {
    if (!p) return CM_ERR_INVALID_ARG;
    if (ld < h || ld > kMaxExtent) return CM_ERR_SHAPE;
    return misaligned(p, t) ? CM_ERR_ALIGNMENT : CM_OK;
}

cm_status check_ids(const void *ids, int bits, int64_t first) {
    if (!ids || first < 0 || first > kMaxExtent) return CM_ERR_INVALID_ARG;
    return (reinterpret_cast<uintptr_t>(ids) & (bits == 64 ? 7u : 3u)) != 0 ? CM_ERR_ALIGNMENT : CM_OK;
}

cm_status check_extents(int64_t tokens, int64_t rows, int64_t h) {
    return tokens < 0 || rows <= 0 || h <= 0 || tokens > kMaxExtent || rows > kMaxExtent || h > kMaxExtent ? CM_ERR_SHAPE
                                                                                                          : CM_OK;
}

template <typename W, typename Y>
cudaError_t lookup(const LookupParams &p, bool vec, cudaStream_t stream) {
    const int rows = kLookThreads / p.width, per = kLookBatch * p.width * 8;
    const dim3 grid(unsigned((p.tokens + rows - 1) / rows), unsigned((p.h + per - 1) / per));
    return launch_after(vec ? cm_embedding_kernel<W, Y, true> : cm_embedding_kernel<W, Y, false>, grid, kLookThreads, 0, 1, stream, p);
}

// The workspace: keys and their rows twice, then the parts.
struct Space {
    uint64_t *keys[2];
    uint32_t *rows[2];
    float *parts;
    size_t bytes;
};
Space backward_space(void *ws, int64_t tokens, int64_t h) {
    Space s;
    uint8_t *const base = static_cast<uint8_t *>(ws);
    size_t used = 0;
    const auto take = [&](size_t bytes) {
        void *const at = base + used;
        used += (bytes + 255) / 256 * 256;
        return at;
    };
    for (auto &k : s.keys) k = static_cast<uint64_t *>(take(size_t(tokens) * 8));
    for (auto &r : s.rows) r = static_cast<uint32_t *>(take(size_t(tokens) * 4));
    // one piece has no neighbours
    s.parts = static_cast<float *>(take(tokens > kPiece ? size_t((tokens + kPiece - 1) / kPiece) * 2 * size_t((h + 7) / 8 * 8) * 4 : 256));
    s.bytes = used;
    return s;
}

// Sorted keys of all tokens, in either half of the workspace.
cudaError_t sort_tokens(const Ids &ids, int64_t tokens, const Space &s, const uint64_t **sorted, cudaStream_t stream) {
    cudaError_t e = launch_after(cm_embedding_sort_kernel, dim3(unsigned((tokens + kSortTile - 1) / kSortTile)), kSortTile, 0, 1,
                                 stream, ids, tokens, s.keys[0], s.rows[0]);
    int at = 0;
    for (int64_t run = kSortTile; run < tokens && e == cudaSuccess; run *= kMergeRuns, at ^= 1)
        e = launch_after(cm_embedding_merge_kernel, dim3(unsigned((tokens + kMergeThreads - 1) / kMergeThreads)), kMergeThreads,
                         0, 1, stream, static_cast<const uint64_t *>(s.keys[at]), static_cast<const uint32_t *>(s.rows[at]),
                         s.keys[at ^ 1], s.rows[at ^ 1], uint32_t(tokens), uint32_t(run));
    *sorted = s.keys[at];
    return e;
}

template <typename DY, typename DW, bool VEC>
cudaError_t sum_rows(const SumParams &p, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (!p.accumulate) e = launch_after(cm_embedding_zero_kernel<DW, VEC>, dim3(unsigned((p.rows + 7) / 8)), 256, 0, 1, stream, p);
    if (e == cudaSuccess)
        e = launch_after(p.accumulate ? cm_embedding_sum_kernel<DY, DW, VEC, true> : cm_embedding_sum_kernel<DY, DW, VEC, false>,
                         dim3(unsigned(p.sum_ctas)), 256, 0, 1, stream, p);
    if (e != cudaSuccess || p.tokens <= kPiece) return e;
    return launch_after(cm_embedding_join_kernel<DW, VEC>,
                        dim3(unsigned((p.tokens + kJoinPieces * kPiece - 1) / (kJoinPieces * kPiece)), unsigned((p.h + 255) / 256)), 256, 0, 1, stream, p);
}

template <typename DY, typename DW>
cudaError_t sum_rows(const SumParams &p, bool vec, cudaStream_t stream) {
    return vec ? sum_rows<DY, DW, true>(p, stream) : sum_rows<DY, DW, false>(p, stream);
}

}  // namespace
}  // namespace cm

using namespace cm;

#define CM_TRY(x)                        \
    do {                                 \
        const cm_status st_ = (x);       \
        if (st_ != CM_OK) return st_;    \
    } while (0)

extern "C" {

cm_status cm_embedding(const void *ids, int id_bits, int64_t first, const void *w, cm_dtype w_dtype, int64_t ldw, float scale,
                       void *y, cm_dtype y_dtype, int64_t ldy, int64_t tokens, int64_t n, int64_t h, cm_stream_t stream) {
    NvtxRange range("cm_embedding");
    if (bad_dtype(w_dtype) || bad_dtype(y_dtype) || (id_bits != 32 && id_bits != 64)) return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(tokens, n, h));
    if (tokens == 0) return CM_OK;
    CM_TRY(check_ids(ids, id_bits, first));
    CM_TRY(check_rows(w, w_dtype, ldw, h));
    CM_TRY(check_rows(y, y_dtype, ldy, h));
    if (h > kMostColumns) return CM_ERR_SHAPE;
    int width = 1;
    while (width < kLookThreads && width * kLookBatch * 8 < h) width *= 2;
    const LookupParams p = {{ids, first, n, id_bits}, w, y, ldw, ldy, tokens, int(h), width, scale};
    const bool vec = whole_vectors(w, w_dtype, ldw) && whole_vectors(y, y_dtype, ldy);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = w_dtype == CM_F32 ? y_dtype == CM_F32 ? lookup<float, float>(p, vec, s)
                                                                : lookup<float, bf16>(p, vec, s)
                          : y_dtype == CM_F32 ? lookup<bf16, float>(p, vec, s)
                                              : lookup<bf16, bf16>(p, vec, s);
    return e == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

size_t cm_embedding_backward_workspace_size(int64_t tokens, int64_t h) {
    return check_extents(tokens, 1, h) == CM_OK ? backward_space(nullptr, tokens, h).bytes : 0;
}

cm_status cm_embedding_backward(const void *dy, cm_dtype dy_dtype, int64_t lddy, const void *ids, int id_bits, int64_t first,
                                float scale, void *dw, cm_dtype dw_dtype, int64_t lddw, int accumulate, int64_t tokens,
                                int64_t n, int64_t h, void *ws, size_t ws_bytes, cm_stream_t stream_) {
    NvtxRange range("cm_embedding_backward");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (bad_dtype(dy_dtype) || bad_dtype(dw_dtype) || (id_bits != 32 && id_bits != 64)) return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(tokens, n, h));
    CM_TRY(check_rows(dw, dw_dtype, lddw, h));
    if (tokens == 0) {   // no token: the sums are zero
        const size_t es = dw_dtype == CM_F32 ? 4 : 2;
        return accumulate || cudaMemset2DAsync(dw, size_t(lddw) * es, 0, size_t(h) * es, size_t(n), stream) == cudaSuccess
                   ? CM_OK
                   : CM_ERR_CUDA;
    }
    CM_TRY(check_ids(ids, id_bits, first));
    CM_TRY(check_rows(dy, dy_dtype, lddy, h));
    const Space space = backward_space(ws, tokens, h);
    if (!ws || ws_bytes < space.bytes) return CM_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0) return CM_ERR_ALIGNMENT;
    const int64_t blocks = (h + 255) / 256;
    SumParams p = {};
    p.sum_ctas = ((tokens + kPiece - 1) / kPiece * blocks + 7) / 8;
    if (h > kMostColumns || p.sum_ctas > 0x7fffffff) return CM_ERR_SHAPE;
    if (sort_tokens({ids, first, n, id_bits}, tokens, space, &p.keys, stream) != cudaSuccess) return CM_ERR_CUDA;
    p.dy = dy;
    p.dw = dw;
    p.parts = space.parts;
    p.lddy = lddy;
    p.lddw = lddw;
    p.tokens = tokens;
    p.rows = n;
    p.h = int(h);
    p.scale = scale;
    p.accumulate = accumulate != 0;
    const bool vec = whole_vectors(dy, dy_dtype, lddy) && whole_vectors(dw, dw_dtype, lddw);
    const cudaError_t e = dy_dtype == CM_F32 ? dw_dtype == CM_F32 ? sum_rows<float, float>(p, vec, stream)
                                                                  : sum_rows<float, bf16>(p, vec, stream)
                          : dw_dtype == CM_F32 ? sum_rows<bf16, float>(p, vec, stream)
                                               : sum_rows<bf16, bf16>(p, vec, stream);
    return e == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

}  // extern "C"
