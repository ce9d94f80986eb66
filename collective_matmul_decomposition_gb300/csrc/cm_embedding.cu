// cm_embedding.cu -- embedding lookup and its gradient.
//
//   forward   y[t] = scale w[id[t] - first], zeros where the id is not one of the slice's
//   backward  dw[v] (+)= scale sum over the tokens t with id[t] = first + v of dy[t], t ascending
//
// Both are bound by memory: the rows read and written.  The gradient's tokens
// are sorted by (row, token) first, so that every row of dw is summed and written
// once, in one order, whatever the timing:
//   1. tiles of 1024 keys (row << 32 | token) are sorted in shared memory;
//   2. up to 64 sorted runs at a time become one: a key's place is its place in
//      its own run plus the number of smaller keys in each other run, found by
//      bisection; keys are all different, so no two meet.  Again while runs are left;
//   3. a token that occurs often would make one warp sum many rows: the aligned
//      pieces of 32 and 256 sorted tokens that lie in one row of dw are summed first
//      (a warp, or the eight warps of a CTA, each), into the workspace;
//   4. the first token of each row's run owns the row: its warps add up what the
//      pieces have left over and the pieces, in sorted order.  Where dw is not
//      added to, the other CTAs of the same launch write zeros to the absent rows.
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

// ---- lookup -------------------------------------------------------------------------
struct LookupParams {
    Ids ids;
    const void *w;
    void *y;
    int64_t ldw, ldy, tokens;
    int h;
    float scale;
};

constexpr int kLookThreads = 256, kLookBatch = 4;

// A CTA takes 1024 vectors of eight, counted through all tokens' rows, so that
// any row length fills it; a thread has four loads under way before its first store.
template <typename W, typename Y, bool VEC>
__global__ void __launch_bounds__(kLookThreads) cm_embedding_kernel(const LookupParams p) {
    let_next_start();
    wait_for_previous();
    const uint32_t per_row = uint32_t(p.h + 7) / 8;
    const int64_t v0 = int64_t(blockIdx.x) * (kLookThreads * kLookBatch);
    const int64_t t0 = v0 / per_row;
    const uint32_t off = uint32_t(v0 - t0 * per_row) + threadIdx.x;
    V8 v[kLookBatch];
#pragma unroll
    for (int k = 0; k < kLookBatch; ++k) {
        const uint32_t o = off + uint32_t(k * kLookThreads), r = o / per_row;
        const int64_t t = t0 + r;
        const int c = int(o - r * per_row) * 8;
        const uint32_t row = t < p.tokens ? row_of(p.ids, t) : kNoRow;
        v[k] = fill(0.0f);
        if (row != kNoRow) v[k] = scaled(get8<VEC>(static_cast<const W *>(p.w) + int64_t(row) * p.ldw, c, p.h), p.scale);
    }
#pragma unroll
    for (int k = 0; k < kLookBatch; ++k) {
        const uint32_t o = off + uint32_t(k * kLookThreads), r = o / per_row;
        const int64_t t = t0 + r;
        const int c = int(o - r * per_row) * 8;
        if (t < p.tokens) put8<VEC>(static_cast<Y *>(p.y) + t * p.ldy, c, p.h, v[k]);
    }
}

// ---- tokens sorted by row -----------------------------------------------------------
constexpr int kSortTile = 1024, kMergeRuns = 64, kMergeThreads = 256;

__device__ __forceinline__ uint64_t lesser(uint64_t a, uint64_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint64_t greater(uint64_t a, uint64_t b) { return a < b ? b : a; }

// One key a thread, bitonic: partners less than a warp apart by shuffles, the
// others through shared memory.
__global__ void __launch_bounds__(kSortTile) cm_embedding_sort_kernel(const Ids ids, int64_t tokens, uint64_t *keys) {
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
    if (t < tokens) keys[t] = k;
}

// Keys of in[0 .. n) that are smaller than k.
__device__ __forceinline__ uint32_t smaller(const uint64_t *in, uint32_t n, uint64_t k) {
    uint32_t lo = 0;
    while (n > 0) {
        const uint32_t half = n >> 1;
        const bool right = in[lo + half] < k;
        lo = right ? lo + half + 1 : lo;
        n = right ? n - half - 1 : half;
    }
    return lo;
}

// Groups of up to kMergeRuns sorted runs of `run` keys become one run each.
__global__ void __launch_bounds__(kMergeThreads) cm_embedding_merge_kernel(const uint64_t *in, uint64_t *out, int64_t tokens,
                                                                           int64_t run) {
    let_next_start();
    wait_for_previous();
    const int64_t i = int64_t(blockIdx.x) * kMergeThreads + threadIdx.x;
    if (i >= tokens) return;
    const int64_t own = i / run, group = own / kMergeRuns * kMergeRuns, base = group * run;
    const uint64_t k = in[i];
    int64_t place = i - own * run;
    const int runs = int(min(int64_t(kMergeRuns), (tokens - base + run - 1) / run));
#pragma unroll 4
    for (int r = 0; r < runs; ++r) {
        const int64_t b = base + r * run;
        if (group + r != own) place += smaller(in + b, uint32_t(min(run, tokens - b)), k);
    }
    out[base + place] = k;
}

// ---- sums of rows -------------------------------------------------------------------
struct SumParams {
    const uint64_t *keys;    // sorted
    const void *dy;
    void *dw;
    float *pieces;           // [ceil(tokens / 32)][h, rounded up to 8]: sums of aligned pieces, NULL where none are made
    int64_t lddy, lddw, tokens, rows;
    int h;
    float scale;
    int accumulate;
    int64_t sum_ctas;        // CTAs that sum; those behind them write zeros
};

constexpr int kPiece = 32, kWhole = 256;   // sorted tokens of a warp's piece, and of a CTA's
constexpr int kAtOnce = 8;                 // rows under way at a time

__device__ __forceinline__ uint32_t row_at(const SumParams &p, int64_t i) { return uint32_t(p.keys[i] >> 32); }
// The aligned piece of n sorted tokens at i lies in one row of dw.
__device__ __forceinline__ bool one_row(const SumParams &p, int64_t i, int n, uint32_t row) {
    return i % n == 0 && i + n <= p.tokens && row_at(p, i + n - 1) == row;
}

__device__ __forceinline__ float *piece_at(const SumParams &p, int64_t i, int c) {
    return p.pieces + (i / kPiece) * ((p.h + 7) / 8 * 8) + c;
}

// Sum over sorted tokens i .. i + n - 1 of column c .. c + 7, in order.
template <bool VEC, typename DY>
__device__ __forceinline__ void add_tokens(const SumParams &p, V8 &acc, int64_t i, int n, int c) {
    for (int j = 0; j < n; j += kAtOnce) {
        V8 v[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            v[k] = fill(0.0f);
            if (j + k < n)
                v[k] = get8<VEC>(static_cast<const DY *>(p.dy) + int64_t(uint32_t(p.keys[i + j + k])) * p.lddy, c, p.h);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (j + k < n) add_to(acc, v[k]);
    }
}

// grid: aligned pieces of 256 sorted tokens x column blocks of 256.  A warp sums 32
// tokens; where all 256 lie in one row, the eight sums are added in order.
template <typename DY, bool VEC>
__global__ void __launch_bounds__(256) cm_embedding_pieces_kernel(const SumParams p) {
    __shared__ V8 part[8][32];
    let_next_start();
    wait_for_previous();
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    const int64_t i0 = int64_t(blockIdx.x) * kWhole, i = i0 + warp * kPiece;
    const int c = int(blockIdx.y) * 256 + lane * 8;
    const uint32_t row0 = row_at(p, i0);
    const bool whole = row0 != kNoRow && one_row(p, i0, kWhole, row0);   // the same in every thread
    const uint32_t row = i < p.tokens ? row_at(p, i) : kNoRow;
    if (c < p.h && row != kNoRow && (whole || one_row(p, i, kPiece, row))) {
        V8 acc = fill(0.0f);
        add_tokens<VEC, DY>(p, acc, i, kPiece, c);
        if (whole)
            part[warp][lane] = acc;
        else
            store8(piece_at(p, i, c), acc);
    }
    if (!whole) return;
    __syncthreads();
    if (warp == 0 && c < p.h) {
        V8 acc = part[0][lane];
#pragma unroll
        for (int w = 1; w < 8; ++w) add_to(acc, part[w][lane]);
        store8(piece_at(p, i0, c), acc);
    }
}

// Rows of dw without a token, 64 to a CTA: zeros.
constexpr int kZeroRows = 64;
template <typename DW, bool VEC>
__device__ void zero_absent(const SumParams &p, int64_t v0) {
    __shared__ unsigned long long seen;
    __shared__ int64_t bounds[2];
    const int n = int(min(int64_t(kZeroRows), p.rows - v0));
    if (threadIdx.x == 0) seen = 0;
    if (threadIdx.x < 2) {   // first sorted token of row v0, and of the row behind the last
        const uint64_t k = uint64_t(v0 + (threadIdx.x ? n : 0)) << 32;
        bounds[threadIdx.x] = smaller(p.keys, uint32_t(p.tokens), k);
    }
    __syncthreads();
    for (int64_t i = bounds[0] + threadIdx.x; i < bounds[1]; i += blockDim.x)
        if (i == bounds[0] || row_at(p, i) != row_at(p, i - 1)) atomicOr(&seen, 1ull << (row_at(p, i) - v0));
    __syncthreads();
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    const V8 zero = fill(0.0f);
    for (int r = warp; r < n; r += int(blockDim.x) >> 5) {
        if (seen >> r & 1) continue;
        DW *row = static_cast<DW *>(p.dw) + (v0 + r) * p.lddw;
        for (int c = lane * 8; c < p.h; c += 256) put8<VEC>(row, c, p.h, zero);
    }
}

// A warp for each sorted token and 256 columns; those of a row's first token sum the row.
template <typename DY, typename DW, bool VEC>
__global__ void __launch_bounds__(256) cm_embedding_sum_kernel(const SumParams p) {
    let_next_start();
    wait_for_previous();
    if (int64_t(blockIdx.x) >= p.sum_ctas) {
        zero_absent<DW, VEC>(p, (int64_t(blockIdx.x) - p.sum_ctas) * kZeroRows);
        return;
    }
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    const int64_t blocks = (p.h + 255) / 256, unit = int64_t(blockIdx.x) * 8 + warp;
    int64_t i = unit / blocks;
    const int c = int(unit - i * blocks) * 256 + lane * 8;
    if (i >= p.tokens) return;
    const uint32_t row = row_at(p, i);
    if (row == kNoRow || (i > 0 && row_at(p, i - 1) == row)) return;
    V8 acc = fill(0.0f);
    while (true) {   // the same way in all lanes
        // up to 32 tokens of the row, as far as the next aligned piece
        const int64_t at = i + lane;
        const bool mine = at < p.tokens && row_at(p, at) == row;
        const uint32_t live = __ballot_sync(0xffffffffu, mine);
        int n = live == 0xffffffffu ? 32 : __ffs(~live) - 1;   // sorted: the row's tokens come first
        if (n == 0) break;
        if (p.pieces && i % kPiece == 0 && n == kPiece) {
            const bool whole = one_row(p, i, kWhole, row);
            if (c < p.h) add_to(acc, load8(piece_at(p, i, c)));
            i += whole ? kWhole : kPiece;
            continue;
        }
        if (p.pieces) n = min(n, kPiece - int(i % kPiece));
        if (c < p.h) add_tokens<VEC, DY>(p, acc, i, n, c);
        i += n;
    }
    if (c >= p.h) return;
    DW *out = static_cast<DW *>(p.dw) + int64_t(row) * p.lddw;
    acc = scaled(acc, p.scale);
    if (p.accumulate) add_to(acc, get8<VEC>(out, c, p.h));
    put8<VEC>(out, c, p.h, acc);
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
cudaError_t lookup(const LookupParams &p, bool vec, int64_t ctas, cudaStream_t stream) {
    return launch_after(vec ? cm_embedding_kernel<W, Y, true> : cm_embedding_kernel<W, Y, false>, dim3(unsigned(ctas)),
                        kLookThreads, 0, 1, stream, p);
}

// The workspace: keys twice, then the pieces' sums.
size_t key_bytes(int64_t tokens) { return (size_t(tokens) * sizeof(uint64_t) + 255) / 256 * 256; }
bool has_pieces(int64_t tokens) { return tokens >= 2 * kPiece; }
size_t backward_workspace(int64_t tokens, int64_t h) {
    const size_t pieces = has_pieces(tokens) ? size_t((tokens + kPiece - 1) / kPiece) * size_t((h + 7) / 8 * 8) * sizeof(float) : 0;
    return 2 * key_bytes(tokens) + pieces + 256;
}

// Sorted keys of all tokens; in either half of the workspace.
cudaError_t sort_tokens(const Ids &ids, int64_t tokens, uint64_t *a, uint64_t *b, const uint64_t **sorted, cudaStream_t stream) {
    cudaError_t e = launch_after(cm_embedding_sort_kernel, dim3(unsigned((tokens + kSortTile - 1) / kSortTile)), kSortTile, 0, 1,
                                 stream, ids, tokens, a);
    for (int64_t run = kSortTile; run < tokens && e == cudaSuccess; run *= kMergeRuns) {
        e = launch_after(cm_embedding_merge_kernel, dim3(unsigned((tokens + kMergeThreads - 1) / kMergeThreads)), kMergeThreads,
                         0, 1, stream, static_cast<const uint64_t *>(a), b, tokens, run);
        std::swap(a, b);
    }
    *sorted = a;
    return e;
}

template <typename DY, typename DW, bool VEC>
cudaError_t sum_rows(const SumParams &p, cudaStream_t stream) {
    if (p.pieces) {
        const cudaError_t e = launch_after(cm_embedding_pieces_kernel<DY, VEC>,
                                           dim3(unsigned((p.tokens + kWhole - 1) / kWhole), unsigned((p.h + 255) / 256)), 256, 0, 1,
                                           stream, p);
        if (e != cudaSuccess) return e;
    }
    const int64_t zeros = p.accumulate ? 0 : (p.rows + kZeroRows - 1) / kZeroRows;
    return launch_after(cm_embedding_sum_kernel<DY, DW, VEC>, dim3(unsigned(p.sum_ctas + zeros)), 256, 0, 1, stream, p);
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
    const int64_t per_cta = kLookThreads * kLookBatch, ctas = (tokens * ((h + 7) / 8) + per_cta - 1) / per_cta;
    if (ctas > 0x7fffffff) return CM_ERR_SHAPE;
    const LookupParams p = {{ids, first, n, id_bits}, w, y, ldw, ldy, tokens, int(h), scale};
    const bool vec = whole_vectors(w, w_dtype, ldw) && whole_vectors(y, y_dtype, ldy);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = w_dtype == CM_F32 ? y_dtype == CM_F32 ? lookup<float, float>(p, vec, ctas, s)
                                                                : lookup<float, bf16>(p, vec, ctas, s)
                          : y_dtype == CM_F32 ? lookup<bf16, float>(p, vec, ctas, s)
                                              : lookup<bf16, bf16>(p, vec, ctas, s);
    return e == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

size_t cm_embedding_backward_workspace_size(int64_t tokens, int64_t h) {
    return check_extents(tokens, 1, h) == CM_OK ? backward_workspace(tokens, h) : 0;
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
    if (!ws || ws_bytes < backward_workspace(tokens, h)) return CM_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0) return CM_ERR_ALIGNMENT;
    const int64_t blocks = (h + 255) / 256;
    SumParams p = {};
    p.sum_ctas = (tokens * blocks + 7) / 8;
    if (blocks > 65535 || p.sum_ctas + n / kZeroRows + 1 > 0x7fffffff) return CM_ERR_SHAPE;
    uint8_t *base = static_cast<uint8_t *>(ws);
    if (sort_tokens({ids, first, n, id_bits}, tokens, reinterpret_cast<uint64_t *>(base),
                    reinterpret_cast<uint64_t *>(base + key_bytes(tokens)), &p.keys, stream) != cudaSuccess)
        return CM_ERR_CUDA;
    p.dy = dy;
    p.dw = dw;
    p.pieces = has_pieces(tokens) ? reinterpret_cast<float *>(base + 2 * key_bytes(tokens)) : nullptr;
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
