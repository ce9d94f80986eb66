// cm_linear_api.cu -- the C ABI of the linear layer: argument checks, tensor
// maps, the choice of kernel and tile, and the launches.
#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <mutex>

#include "cm_internal.h"
#include "cm_kernel.cuh"
#include "cm_linear.cuh"

namespace cm {
namespace {

__device__ LinearStatus g_linear_status;

// The longest wait is for a tile's products: a second, and a microsecond a slice (they take
// 0.28: dw of the loss of 2^28 rows has 2^22 slices a tile, 1.2 s).
uint64_t linear_timeout_ns(int kblocks) { return 1000000000ull + 1000ull * uint64_t(kblocks); }
constexpr int64_t kMaxExtent = int64_t(1) << 30;

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// Row-major bf16 (or fp32) [rows][cols] with row stride ld, in boxes of 128
// bytes x box_rows, 128-byte swizzle; elements outside are read as zeros and
// not written.
bool map_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows, bool f32 = false) {
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), 1};
    const cuuint64_t row_bytes = cuuint64_t(ld) * (f32 ? 4 : 2);
    // the third extent is 1: its stride is never used and only has to be valid
    cuuint64_t strides[2] = {row_bytes, row_bytes};
    cuuint32_t box[3] = {f32 ? 32u : 64u, cuuint32_t(box_rows), 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A matrix that 32-row boxes are stored to: up to the last whole 16-byte piece
// of its rows, because stores are clipped in such pieces (a map needs one at
// least; where there is none nothing is stored through it).
bool map_written(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, bool f32) {
    const int64_t piece = f32 ? 4 : 8;
    return map_rows(m, base, rows, std::max(piece, cols / piece * piece), ld, 32, f32);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool misaligned(const void *p, cm_dtype t) { return (reinterpret_cast<uintptr_t>(p) & (t == CM_F32 ? 3u : 1u)) != 0; }
bool bad_dtype(cm_dtype t) { return t != CM_BF16 && t != CM_F32; }

// A matrix the kernels read with TMA or write in 16-byte pieces.
cm_status check_matrix(const void *p, int64_t ld, int64_t cols) {
    if (!p) return CM_ERR_INVALID_ARG;
    if (ld < cols || ld > kMaxExtent) return CM_ERR_SHAPE;
    if (ld % 8 != 0 || !aligned16(p)) return CM_ERR_ALIGNMENT;
    return CM_OK;
}

cm_status check_extents(int64_t M, int64_t K, int64_t n) {
    return M < 0 || K <= 0 || n <= 0 || M > kMaxExtent || K > kMaxExtent || n > kMaxExtent ? CM_ERR_SHAPE : CM_OK;
}

struct Device {
    int id = 0, sms = 0;
    int clusters[3] = {0, 0, 0};                    // of 1, 2 and 4 pairs
    int strip_clusters[kStripMostSplits + 1] = {};  // of so many strip CTAs, one CTA an SM
    LinearStatus *status = nullptr;
};

cm_status device(Device *d) {
    if (cudaGetDevice(&d->id) != cudaSuccess) return CM_ERR_CUDA;
    static std::mutex mu;
    static Device cached[64];
    if (d->id < 0 || d->id >= 64) return CM_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(mu);
    Device &c = cached[d->id];
    if (!c.status) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d->id) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, d->id) != cudaSuccess ||
            cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, d->id) != cudaSuccess)
            return CM_ERR_CUDA;
        if (major != 10 || minor != 3) return CM_ERR_UNSUPPORTED;
        if (prepare_linear_strip(c.sms, c.strip_clusters) != cudaSuccess) return CM_ERR_CUDA;
        if (prepare_linear_pair(c.sms, c.clusters) != cudaSuccess) return CM_ERR_CUDA;
        if (c.clusters[0] < 1) return CM_ERR_UNSUPPORTED;
        void *sp = nullptr;
        if (cudaGetSymbolAddress(&sp, g_linear_status) != cudaSuccess) return CM_ERR_CUDA;
        c.status = static_cast<LinearStatus *>(sp);
        c.id = d->id;
    }
    *d = c;
    return CM_OK;
}

// One operand: `rows` x `k` where k is the contracted extent; K-major when
// the contracted extent is contiguous.
struct Operand {
    const void *p;
    int64_t ld;
    bool mn_major;
};

bool map_operand(CUtensorMap *m, const Operand &o, int64_t rows, int64_t k, int tile_rows) {
    return o.mn_major ? map_rows(m, o.p, k, rows, o.ld, 64) : map_rows(m, o.p, rows, k, o.ld, tile_rows);
}

constexpr int64_t kBandBytes = int64_t(32) << 20;   // of the row operand, kept in L2 while a band runs

// How a product is run: pair (256 x bn tiles on CTA pairs, K split over 1, 2
// or 4 pairs) or strip (128 columns x tok rows, K split over up to 8 CTAs).
struct Choice {
    bool pair = false;
    int bn = 256;
    int tok = 16, splits = 1, ring_bytes = 0;
};

// The choice with the least estimated time.  The estimates' constants were
// fitted to 110 forward calls (up to 1000 rows, K and columns from 256 to 28672)
// with [n][K] weights from HBM, bf16 outputs and nothing else in the epilogue, on
// one GB300, in us: 89 calls at random and 21 picked, 11 of them for sizes that
// this library runs elsewhere or that lie at a border below, ten for having been
// chosen badly before.  The choices take 2 % longer than the best of each call on
// average, the worst 1.2 times as long (33 rows, K 1048, cols 2864: 8.2 for 6.7).
// Other layouts, the gradients and fp32 outputs use the same constants, which
// were not fitted to them; the bytes of outputs, residuals and pre-activations
// are not in the estimate.
//   pair: a K slice of 64 takes a wave of tiles 0.32 (256 columns) or 0.21
//     (128), but no wave is shorter than its epilogue, 2.9 or 2.0; a launch
//     takes 3.8 beyond that, summing over a cluster's pairs 2.6 or 1.6.
//   strip: a launch takes 3.4, and 0.04 a row of the tile; split, 3.7 and 0.063.
//     A slice takes 0.125.
//   Between, HBM and L2 (every tile its own copy of the rows) are given 8.5 and
//   22 TB/s, since of what is not the longest a part shows as well.
// Measured on both sides of where the choice changes (best strip / best pair):
//   rows 45,  K 8190, cols 3579:  14.6 / 17.1     rows 100, K 8192,  cols 3584: 18.9 / 19.0
//   rows 200, K 8192, cols 3584:  24.9 / 19.6     rows 256, K 12288, cols 4608: 37.4 / 29.5
//   rows 100, K 1024, cols 2048:   7.0 / 6.5      rows 512, K 4096,  cols 4096: 22.9 / 17.7
//   rows 272, K 4480, cols 14832: 40.3 / 46.8     rows 434, K 5552,  cols 11856: 73 / 59 (not looked at above 384)
// between pair tiles (256 columns / 128 / 128 on two pairs a tile):
//   rows 2048, K 12288, cols 4608:  129 / 161 / -     rows 1024, K 8192, cols 1024:  40.1 / 23.1 / 16.8
// and between strips (one tile of rows / more, shorter ones):
//   rows 64, K 4096, cols 2048:  10.6 / 9.1 (two)     rows 33, K 2048, cols 28672:  22.8 / 29.0 (three)
// A gated product is estimated as one of the columns of both its operands.
// What a product's kernels have: all of the above; of the gated ones no unsplit pair
// tiles of 128 columns (their epilogue needs 64 columns a warp of either operand); of the
// loss's logits unsplit pair tiles of 256 columns, and strips (choose_logits); of the
// counted ones unsplit pair tiles.
enum class Has { all, gated, logits, counted };
Choice choose(const Device &d, int64_t rows, int64_t cols, int64_t k, bool row_mn, Has has = Has::all) {
    Choice best;
    double least = 1e30;
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t slices = up(k, kBK);
    const double from_hbm = double(cols) * double(k) * 2.0 / 8.5e6;
    // pair tiles waste what they have beyond `rows`: not worth a look below 33
    for (int bn = 256; bn >= (has == Has::logits ? 256 : 128) && (rows > 32 || has == Has::counted); bn /= 2) {
        const int64_t tiles = up(rows, 256) * up(cols, bn);
        for (int i = 0; i < 3; ++i) {
            const int splits = 1 << i;
            if (i > 0 && (has == Has::logits || has == Has::counted || tiles > d.clusters[i] || slices < 2 * splits)) break;
            if (i == 0 && bn == 128 && has == Has::gated) continue;
            const double wave = std::max(double(up(slices, splits)) * (bn == 256 ? 0.32 : 0.21), bn == 256 ? 2.9 : 2.0);
            const double run = double(up(tiles, d.clusters[i])) * wave;
            const double t = 3.8 + (i == 0 ? 0.0 : bn == 256 ? 2.6 : 1.6) + std::max(run, from_hbm) +
                             0.22 * std::min(run, from_hbm);
            if (t < least) {
                least = t;
                best.pair = true;
                best.bn = bn;
                best.splits = splits;
            }
        }
    }
    for (int64_t parts = 1; parts <= 4 && rows <= 384 && has != Has::counted; ++parts) {
        const int64_t unit = row_mn ? 64 : 16, tok = up(up(rows, parts), unit) * unit;
        if (tok > 256) continue;
        const int64_t tiles = up(rows, tok) * up(cols, 128);
        const double from_l2 = double(tiles) * double(128 + tok) * double(k) * 2.0 / 22e6;
        // unsplit, or split as far as all tiles' clusters run at once, two CTAs
        // an SM (9 rows, K 3728, cols 5504: 43 tiles of seven CTAs each take
        // 16.3 us, of six 10.4).  Partial tiles of up to 208 rows fit two to an SM,
        // but the constants were fitted with splits of 128 rows at most: with splits
        // up to 208, 21 of 400 random calls of 129 to 384 rows went otherwise, 12 of
        // them faster (by up to 23 %) and five slower (by up to 38 %)
        int64_t most = tok > 128 ? 1 : std::min<int64_t>(kStripMostSplits, slices);
        while (most > 1 && tiles > 2 * d.strip_clusters[most]) --most;
        for (int64_t splits = 1; splits <= most; splits += std::max<int64_t>(1, most - 1)) {
            const double run = 0.125 * double(up(slices, splits)) * double(up(tiles * splits, d.sms));
            const double longest = std::max({from_hbm, from_l2, run});
            const double second = std::max(std::min(from_hbm, from_l2), std::min(std::max(from_hbm, from_l2), run));
            double t = (splits > 1 ? 3.7 + 0.063 * double(tok) : 3.4 + 0.04 * double(tok)) + longest + 0.5 * second;
            if (has == Has::logits && rows > 32) {   // see choose_logits
                if (splits == 1) continue;
                t *= 1.6;
            }
            if (t >= least) continue;
            least = t;
            best.pair = false;
            best.tok = int(tok);
            best.splits = int(splits);
            // a CTA has an SM to itself where there are SMs enough; clusters
            // of such CTAs only pack where half of them are
            best.ring_bytes = tiles * splits <= (splits == 1 ? d.sms : d.sms / 2) ? kStripAlone : kStripShared;
        }
    }
    return best;
}

// What a product is beyond a plain one.
struct Kind {
    LinearMode mode = kLinPlain;
    const Operand *a2 = nullptr;      // gated: the second column operand
    LinearLive live = {};             // of the slots' rows
    const Operand *whole = nullptr;   // what tmWhole maps
    LinearHead head = {};
};

cm_status pair_params(LinearPairMore &p, const Device &d, const Choice &c, const Kind &kind, const Operand &a, const Operand &b,
                      int64_t rows, int64_t cols, int64_t k, const LinearEpilogue &e) {
    const LinearMode mode = kind.mode;
    p.e = e;
    p.live = kind.live;
    p.head = kind.head;
    p.rows = rows;
    p.cols = cols;
    p.bn = c.bn;
    p.kblocks = int((k + kBK - 1) / kBK);
    p.mtiles = int((rows + 255) / 256);
    const int tile_cols = mode == kLinGated ? c.bn / 2 : c.bn;
    p.ntiles = int((cols + tile_cols - 1) / tile_cols);
    if (int64_t(p.mtiles) * p.ntiles > 0x7fffffff) return CM_ERR_SHAPE;
    p.tiles = p.mtiles * p.ntiles;
    p.band = int(std::max<int64_t>(1, std::min<int64_t>(p.mtiles, kBandBytes / (int64_t(p.kblocks) * 256 * kBK * 2))));
    // An fp32 weight gradient of few slices is bound by its stores: the tiles that run together
    // take whole rows of it, one front in memory (28672 x 4096, 256 rows: 94 -> 83 us, 512 rows
    // 121 -> 110, 1024 rows 176 -> 167; in bf16 no difference, other products are up to 5 % slower)
    if (a.mn_major && b.mn_major && e.y_f32 && p.kblocks <= 16)
        p.band = std::min(p.band, (d.clusters[0] + p.ntiles - 1) / p.ntiles);
    p.status = d.status;
    p.timeout_ns = linear_timeout_ns(p.kblocks);
    if (!map_operand(&p.tmA, b, rows, k, 128) || !map_operand(&p.tmB, a, cols, k, c.bn / 2) ||
        (kind.a2 && !map_operand(&p.tmB2, *kind.a2, cols, k, c.bn / 2)) ||
        (e.y && !map_written(&p.tmY, e.y, rows, cols, e.ldy, e.y_f32 != 0)))
        return CM_ERR_CUDA;
    // the row operand is A of a tile here (1), the column operand B (2)
    if (kind.whole && !(kind.live.whole_is == 1 ? map_operand(&p.tmWhole, *kind.whole, rows, k, 128)
                                                : map_operand(&p.tmWhole, *kind.whole, cols, k, c.bn / 2)))
        return CM_ERR_CUDA;
    if (mode == kLinGateGrad) {
        if (!map_written(&p.tmZ, e.z, rows, cols, e.ldz, false) || !map_rows(&p.tmIn0, e.zin2, rows, cols, e.ldzin, 32) ||
            !map_rows(&p.tmIn1, e.zin, rows, cols, e.ldzin, 32))
            return CM_ERR_CUDA;
    } else if (mode == kLinGated) {
        if (e.z && (!map_written(&p.tmZ, e.z, rows, cols, e.ldz, false) || !map_written(&p.tmZ2, e.z2, rows, cols, e.ldz, false)))
            return CM_ERR_CUDA;
    } else if ((mode == kLinPlain || mode == kLinCounted) && !e.y_f32) {
        if (e.z && !map_written(&p.tmZ, e.z, rows, cols, e.ldz, false)) return CM_ERR_CUDA;
        if (e.accumulate && !map_rows(&p.tmIn0, e.y, rows, cols, e.ldy, 32)) return CM_ERR_CUDA;
        if (e.res && !map_rows(&p.tmIn0, e.res, rows, cols, e.ldr, 32)) return CM_ERR_CUDA;
        if (e.dact && !map_rows(&p.tmIn1, e.zin, rows, cols, e.ldzin, 32)) return CM_ERR_CUDA;
    }
    return CM_OK;
}

cm_status product_pair(const Device &d, const Choice &c, const Kind &kind, const Operand &a, const Operand &b, int64_t rows,
                       int64_t cols, int64_t k, const LinearEpilogue &e, cudaStream_t stream) {
    LinearPairMore p;
    const cm_status st = pair_params(p, d, c, kind, a, b, rows, cols, k, e);
    if (st != CM_OK) return st;
    const LinearMode mode = kind.mode;
    const int layout = (a.mn_major ? 1 : 0) | (b.mn_major ? 2 : 0);
    return launch_linear_pair(p, layout, mode, c.splits, d.clusters[0], stream) == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

cm_status product_strip(const Device &d, const Choice &c, const Kind &kind, const Operand &a, const Operand &b, int64_t rows,
                        int64_t cols, int64_t k, const LinearEpilogue &e, cudaStream_t stream) {
    const bool gated = kind.mode == kLinGated;
    LinearStripMore p;
    p.e = e;
    p.rows = rows;
    p.cols = cols;
    p.kblocks = int((k + kBK - 1) / kBK);
    p.tok = c.tok;
    p.row_tiles = int((rows + c.tok - 1) / c.tok);
    p.splits = c.splits;
    p.ring_bytes = c.ring_bytes;
    p.stages = linear_strip_stages(c.tok, c.ring_bytes);
    p.head = kind.head;
    p.count = kind.live.count;
    p.status = d.status;
    p.timeout_ns = linear_timeout_ns(p.kblocks);
    if (!map_operand(&p.tmA, a, cols, k, gated ? 64 : 128) || (gated && !map_operand(&p.tmA2, *kind.a2, cols, k, 64)) ||
        !map_operand(&p.tmB, b, rows, k, c.tok))
        return CM_ERR_CUDA;
    const int layout = (b.mn_major ? 1 : 0) | (a.mn_major ? 2 : 0);
    return launch_linear_strip(p, layout, kind.mode, stream) == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

// D [rows][cols] = B [rows][k] A [cols][k]^T with the epilogue e, of all rows.
cm_status product(const Device &d, const Operand &a, const Operand &b, int64_t rows, int64_t cols, int64_t k,
                  const LinearEpilogue &e, cudaStream_t stream, const Kind &kind = {}) {
    const bool gated = kind.mode == kLinGated;
    const Choice c = choose(d, rows, gated ? 2 * cols : cols, k, b.mn_major, gated ? Has::gated : Has::all);
    return c.pair ? product_pair(d, c, kind, a, b, rows, cols, k, e, stream) : product_strip(d, c, kind, a, b, rows, cols, k, e, stream);
}

// Logits: unsplit strips up to 32 rows; above that strips that are split, over a slice of a
// few thousand columns, where choose() gives them less than pair tiles.  They take 1.6 times
// the estimate, which knows of no softmax.  Loss, and its dx alone, by strips / pair tiles,
// us in a graph with cold caches:
//   unsplit: 1 row, 4096 x 131072:   177 / 320, 329 / 394     16 rows, 4096 x 131072: 185 / 194, 339 / 351
//            33 rows, 4096 x 32768:  74 / 74, 119 / 122       100 rows, 4096 x 32768: 82 / 75, 136 / 133
//            48 rows, 1024 x 131072: 87 / 74, 154 / 139       80 rows, 512 x 131072:  78 / 47, 127 / 93
//            64 rows, 8192 x 131072: 366 / 362, 673 / 678
//   split:   64 rows, 4096 x 4000:   30 / 36, 43 / 56         200 rows, 4096 x 4000:  41 / 36, 58 / 56
//            160 rows, 8192 x 4000:  52 / 56, 75 / 90         256 rows, 8192 x 4000:  61 / 56, 83 / 91
// Above 256 rows pair tiles always: 300 rows, 8192 x 4000: 67 / 59, 101 / 89.
Choice choose_logits(const Device &d, int64_t rows, int64_t cols, int64_t k) {
    Choice c;
    c.pair = true;
    return rows <= 256 ? choose(d, rows, cols, k, false, Has::logits) : c;
}

// ---- the loss over a vocabulary -----------------------------------------------------
// Pieces of a workspace, one behind the other, each on 256 bytes.
struct Carve {
    uint8_t *base;
    size_t used = 0;
    explicit Carve(void *p) : base(static_cast<uint8_t *>(p)) {}
    template <typename T>
    T *take(size_t n) {
        T *const at = reinterpret_cast<T *>(base + used);
        used += (n * sizeof(T) + 255) / 256 * 256;
        return at;
    }
};

// Whole 128-byte lines: the rows of a box that a product loads then do not straddle them.
int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }

// The groups that many rows are counted in.
HeadGroup *head_groups(Carve &c, int64_t M) { return M > kHeadRowsOnce ? c.take<HeadGroup>(kHeadGroups) : nullptr; }

struct LossSpace {
    int32_t *count, *row_of, *target;
    HeadGroup *groups;
    float *picked;
    uint16_t *xs;
    float2 *stat;
};
LossSpace loss_space(Carve &c, int64_t M, int64_t K, int64_t n) {
    LossSpace s;
    s.count = c.take<int32_t>(1);
    s.row_of = c.take<int32_t>(size_t(M));
    s.target = c.take<int32_t>(size_t(M));
    s.picked = c.take<float>(size_t(M));
    s.xs = c.take<uint16_t>(size_t(M) * size_t(up64(K)));
    s.stat = c.take<float2>(size_t((n + 255) / 256 * 2) * size_t(M));
    s.groups = head_groups(c, M);
    return s;
}

// Columns of the vocabulary whose logits' gradients are there at a time: the
// workspace holds them in bf16, 256 MB of them or 2048 columns.
constexpr int64_t kLossGradBytes = int64_t(256) << 20;
int64_t loss_grad_columns(int64_t M, int64_t n) {
    const int64_t most = std::max<int64_t>(2048, kLossGradBytes / (2 * M) / 256 * 256);
    if (n <= most) return n;
    const int64_t chunks = (n + most - 1) / most;
    return ((n + chunks - 1) / chunks + 255) / 256 * 256;
}

struct LossGradSpace {
    int32_t *count, *slot_of, *target;
    HeadGroup *groups;
    float *scale, *lse2, *grad, *hit, *sum;
    uint16_t *xs, *p;
    int64_t columns, ldp, lds;
};
LossGradSpace loss_grad_space(Carve &c, int64_t M, int64_t K, int64_t n) {
    LossGradSpace s;
    s.columns = loss_grad_columns(M, n);
    s.ldp = up64(s.columns);
    s.lds = up64(K);
    s.count = c.take<int32_t>(1);
    s.scale = c.take<float>(1);
    s.slot_of = c.take<int32_t>(size_t(M));
    s.target = c.take<int32_t>(size_t(M));
    s.lse2 = c.take<float>(size_t(M));
    s.grad = c.take<float>(size_t(M));
    s.hit = c.take<float>(size_t(M));
    s.xs = c.take<uint16_t>(size_t(M) * size_t(s.lds));
    s.p = c.take<uint16_t>(size_t(M) * size_t(s.ldp));
    s.sum = c.take<float>(size_t(M) * size_t(s.lds));
    s.groups = head_groups(c, M);
    return s;
}

cm_status check_head(const void *x, int64_t ldx, const void *w, int64_t ldw, cm_wlayout wlayout, const void *targets,
                     int target_bits, int64_t first, int64_t vocab, int64_t M, int64_t K, int64_t n) {
    // tiles are counted in 31 bits (of 128 columns, where a product takes those): found out
    // before the first launch of several
    const int64_t m = (M + 127) / 128, k = (K + 127) / 128, v = (n + 127) / 128;
    if (m * v > 0x7fffffff || m * k > 0x7fffffff || k * v > 0x7fffffff) return CM_ERR_SHAPE;
    if (!targets || first < 0 || first > kMaxExtent || vocab < first + n || vocab > 2 * kMaxExtent) return CM_ERR_INVALID_ARG;
    const cm_status st = check_matrix(x, ldx, K);
    if (st != CM_OK) return st;
    const cm_status sw = check_matrix(w, ldw, wlayout == CM_W_NK ? K : n);
    if (sw != CM_OK) return sw;
    return (reinterpret_cast<uintptr_t>(targets) & (target_bits == 64 ? 7u : 3u)) != 0 ? CM_ERR_ALIGNMENT : CM_OK;
}

size_t wgrad_workspace(int64_t M, int64_t n) {
    return std::max<size_t>(256, size_t(colsum_chunks(M, n)) * size_t(n) * sizeof(float));
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

cm_status cm_linear(const void *x, int64_t ldx, const void *w, int64_t ldw, cm_wlayout wlayout, const void *bias,
                    cm_dtype bias_dtype, cm_act act, const void *residual, int64_t ldr, void *preact, int64_t ldz,
                    void *y, cm_dtype y_dtype, int64_t ldy, int64_t M, int64_t K, int64_t n, cm_stream_t stream) {
    NvtxRange range("cm_linear");
    if (bad_dtype(y_dtype) || (bias && bad_dtype(bias_dtype)) || (wlayout != CM_W_KN && wlayout != CM_W_NK) ||
        act < CM_ACT_NONE || act > CM_ACT_SILU)
        return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(M, K, n));
    if (M == 0) return CM_OK;
    CM_TRY(check_matrix(x, ldx, K));
    CM_TRY(check_matrix(w, ldw, wlayout == CM_W_NK ? K : n));
    CM_TRY(check_matrix(y, ldy, n));
    if (residual) CM_TRY(check_matrix(residual, ldr, n));
    if (preact) CM_TRY(check_matrix(preact, ldz, n));
    if (misaligned(bias, bias_dtype)) return CM_ERR_ALIGNMENT;
    Device d;
    CM_TRY(device(&d));
    LinearEpilogue e = {};
    e.y = y;
    e.ldy = ldy;
    e.y_f32 = y_dtype == CM_F32;
    e.bias = bias;
    e.bias_f32 = bias_dtype == CM_F32;
    e.act = act;
    e.res = residual;
    e.ldr = ldr;
    e.z = preact;
    e.ldz = ldz;
    return product(d, {w, ldw, wlayout == CM_W_KN}, {x, ldx, false}, M, n, K, e, reinterpret_cast<cudaStream_t>(stream));
}

cm_status cm_linear_dgrad(const void *dy, int64_t lddy, const void *w, int64_t ldw, cm_wlayout wlayout,
                          const void *preact, int64_t ldz, cm_act act, const void *residual, int64_t ldr, void *dx,
                          cm_dtype dx_dtype, int64_t lddx, int64_t M, int64_t K, int64_t n, cm_stream_t stream) {
    NvtxRange range("cm_linear_dgrad");
    if (bad_dtype(dx_dtype) || (wlayout != CM_W_KN && wlayout != CM_W_NK) || act < CM_ACT_NONE || act > CM_ACT_SILU ||
        (act != CM_ACT_NONE && !preact))
        return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(M, K, n));
    if (M == 0) return CM_OK;
    CM_TRY(check_matrix(dy, lddy, n));
    CM_TRY(check_matrix(w, ldw, wlayout == CM_W_NK ? K : n));
    CM_TRY(check_matrix(dx, lddx, K));
    if (residual) CM_TRY(check_matrix(residual, ldr, K));
    if (act != CM_ACT_NONE) CM_TRY(check_matrix(preact, ldz, K));
    Device d;
    CM_TRY(device(&d));
    LinearEpilogue e = {};
    e.y = dx;
    e.ldy = lddx;
    e.y_f32 = dx_dtype == CM_F32;
    e.act = act;
    e.dact = act != CM_ACT_NONE;
    e.zin = preact;
    e.ldzin = ldz;
    e.res = residual;
    e.ldr = ldr;
    // W stored [n][K]: its K columns are contiguous, the contracted n is not
    return product(d, {w, ldw, wlayout == CM_W_NK}, {dy, lddy, false}, M, K, n, e, reinterpret_cast<cudaStream_t>(stream));
}

cm_status cm_linear_gated(const void *x, int64_t ldx, const void *w_gate, const void *w_up, int64_t ldw, cm_wlayout wlayout,
                          const void *bias_gate, const void *bias_up, cm_dtype bias_dtype, cm_act act, void *z_gate,
                          void *z_up, int64_t ldz, void *y, int64_t ldy, int64_t M, int64_t K, int64_t n,
                          cm_stream_t stream) {
    NvtxRange range("cm_linear_gated");
    if ((bias_gate && bad_dtype(bias_dtype)) || (wlayout != CM_W_KN && wlayout != CM_W_NK) || act < CM_ACT_NONE ||
        act > CM_ACT_SILU || !bias_gate != !bias_up || !z_gate != !z_up)
        return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(M, K, n));
    if (n > kMaxExtent / 2) return CM_ERR_SHAPE;
    if (M == 0) return CM_OK;
    CM_TRY(check_matrix(x, ldx, K));
    for (const void *w : {w_gate, w_up}) CM_TRY(check_matrix(w, ldw, wlayout == CM_W_NK ? K : n));
    CM_TRY(check_matrix(y, ldy, n));
    if (z_gate)
        for (const void *z : {z_gate, z_up}) CM_TRY(check_matrix(z, ldz, n));
    if (misaligned(bias_gate, bias_dtype) || misaligned(bias_up, bias_dtype)) return CM_ERR_ALIGNMENT;
    Device d;
    CM_TRY(device(&d));
    LinearEpilogue e = {};
    e.y = y;
    e.ldy = ldy;
    e.bias = bias_gate;
    e.bias2 = bias_up;
    e.bias_f32 = bias_dtype == CM_F32;
    e.act = act;
    e.z = z_gate;
    e.z2 = z_up;
    e.ldz = ldz;
    const Operand gate = {w_gate, ldw, wlayout == CM_W_KN}, up = {w_up, ldw, wlayout == CM_W_KN};
    Kind kind;
    kind.mode = kLinGated;
    kind.a2 = &up;
    return product(d, gate, {x, ldx, false}, M, n, K, e, reinterpret_cast<cudaStream_t>(stream), kind);
}

cm_status cm_linear_gated_dgrad(const void *dy, int64_t lddy, const void *w, int64_t ldw, cm_wlayout wlayout,
                                const void *z_gate, const void *z_up, int64_t ldz, cm_act act, void *dz_gate, void *dz_up,
                                int64_t lddz, int64_t M, int64_t K, int64_t n, cm_stream_t stream) {
    NvtxRange range("cm_linear_gated_dgrad");
    if ((wlayout != CM_W_KN && wlayout != CM_W_NK) || act < CM_ACT_NONE || act > CM_ACT_SILU) return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(M, K, n));
    if (M == 0) return CM_OK;
    CM_TRY(check_matrix(dy, lddy, n));
    CM_TRY(check_matrix(w, ldw, wlayout == CM_W_NK ? K : n));
    for (const void *z : {z_gate, z_up}) CM_TRY(check_matrix(z, ldz, K));
    for (const void *z : {dz_gate, dz_up}) CM_TRY(check_matrix(z, lddz, K));
    Device d;
    CM_TRY(device(&d));
    LinearEpilogue e = {};
    e.y = dz_up;
    e.ldy = lddz;
    e.z = dz_gate;
    e.ldz = lddz;
    e.act = act;
    e.zin = z_gate;
    e.zin2 = z_up;
    e.ldzin = ldz;
    Kind kind;
    kind.mode = kLinGateGrad;
    return product(d, {w, ldw, wlayout == CM_W_NK}, {dy, lddy, false}, M, K, n, e, reinterpret_cast<cudaStream_t>(stream), kind);
}

size_t cm_linear_wgrad_workspace_size(int64_t M, int64_t K, int64_t n) {
    if (check_extents(M, K, n) != CM_OK) return 0;
    return wgrad_workspace(M, n);
}

cm_status cm_linear_wgrad(const void *x, int64_t ldx, const void *dy, int64_t lddy, void *dw, cm_dtype dw_dtype,
                          int64_t lddw, cm_wlayout wlayout, void *db, cm_dtype db_dtype, int accumulate, int64_t M,
                          int64_t K, int64_t n, void *ws, size_t ws_bytes, cm_stream_t stream_) {
    NvtxRange range("cm_linear_wgrad");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (bad_dtype(dw_dtype) || (db && bad_dtype(db_dtype)) || (wlayout != CM_W_KN && wlayout != CM_W_NK))
        return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(M, K, n));
    const bool nk = wlayout == CM_W_NK;
    CM_TRY(check_matrix(dw, lddw, nk ? K : n));
    if (M > 0) {
        CM_TRY(check_matrix(x, ldx, K));
        CM_TRY(check_matrix(dy, lddy, n));
    }
    if (db && (!ws || ws_bytes < wgrad_workspace(M, n))) return CM_ERR_WORKSPACE;
    if (db && (!aligned16(ws) || misaligned(db, db_dtype))) return CM_ERR_ALIGNMENT;
    Device d;
    CM_TRY(device(&d));
    if (M == 0) {   // the sum over no rows
        if (accumulate) return CM_OK;
        const size_t es = dw_dtype == CM_F32 ? 4 : 2;
        if (cudaMemset2DAsync(dw, size_t(lddw) * es, 0, size_t(nk ? K : n) * es, size_t(nk ? n : K), stream) !=
            cudaSuccess)
            return CM_ERR_CUDA;
        if (db && cudaMemsetAsync(db, 0, size_t(n) * (db_dtype == CM_F32 ? 4 : 2), stream) != cudaSuccess)
            return CM_ERR_CUDA;
        return CM_OK;
    }
    if (db && launch_colsum(dy, lddy, M, n, static_cast<float *>(ws), db, db_dtype == CM_F32, accumulate != 0,
                            stream) != cudaSuccess)
        return CM_ERR_CUDA;
    LinearEpilogue e = {};
    e.y = dw;
    e.ldy = lddw;
    e.y_f32 = dw_dtype == CM_F32;
    e.accumulate = accumulate != 0;
    const Operand ox = {x, ldx, true}, ody = {dy, lddy, true};
    return nk ? product(d, ox, ody, n, K, M, e, stream) : product(d, ody, ox, K, n, M, e, stream);
}

size_t cm_linear_cross_entropy_workspace_size(int64_t M, int64_t K, int64_t n) {
    if (check_extents(M, K, n) != CM_OK) return 0;
    Carve c(nullptr);
    loss_space(c, M, K, n);
    return c.used;
}

cm_status cm_linear_cross_entropy(const void *x, int64_t ldx, const void *w, int64_t ldw, cm_wlayout wlayout,
                                  const void *targets, int target_bits, int64_t first, int64_t vocab, float *loss, float *lse,
                                  float *picked, int64_t M, int64_t K, int64_t n, void *ws, size_t ws_bytes,
                                  cm_stream_t stream_) {
    NvtxRange range("cm_linear_cross_entropy");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if ((wlayout != CM_W_KN && wlayout != CM_W_NK) || (target_bits != 32 && target_bits != 64)) return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(M, K, n));
    if (M == 0) return CM_OK;
    CM_TRY(check_head(x, ldx, w, ldw, wlayout, targets, target_bits, first, vocab, M, K, n));
    if (!ws || ws_bytes < cm_linear_cross_entropy_workspace_size(M, K, n)) return CM_ERR_WORKSPACE;
    if (!aligned16(ws) || misaligned(loss, CM_F32) || misaligned(lse, CM_F32) || misaligned(picked, CM_F32)) return CM_ERR_ALIGNMENT;
    Device d;
    CM_TRY(device(&d));
    Carve carve(ws);
    const LossSpace s = loss_space(carve, M, K, n);
    HeadRows r = {};
    r.targets = targets;
    r.target_bits = target_bits;
    r.first = first;
    r.n = n;
    r.vocab = vocab;
    r.rows = M;
    r.K = K;
    r.x = x;
    r.ldx = ldx;
    r.xs = s.xs;
    r.ldxs = up64(K);
    r.count = s.count;
    r.row_of = s.row_of;
    r.target = s.target;
    r.picked = s.picked;
    r.loss = loss;
    r.lse_out = lse;
    r.picked_out = picked;
    r.groups = s.groups;
    const Choice c = choose_logits(d, M, n, K);
    r.always = !c.pair;
    if (launch_head_rows(r, stream) != cudaSuccess) return CM_ERR_CUDA;
    const Operand rows = {s.xs, up64(K), false}, all = {x, ldx, false};
    Kind kind;
    kind.mode = kLinStats;
    kind.live = {s.count, 1, 0, 1, M};
    kind.whole = &all;
    kind.head.target = s.target;
    kind.head.stat = s.stat;
    kind.head.picked = s.picked;
    kind.head.stride = M;
    const Operand weights = {w, ldw, wlayout == CM_W_KN};
    CM_TRY(c.pair ? product_pair(d, c, kind, weights, rows, M, n, K, {}, stream)
                  : product_strip(d, c, kind, weights, rows, M, n, K, {}, stream));
    const HeadJoin j = {s.stat, c.pair ? (n + 255) / 256 * 2 : (n + 127) / 128, M, s.count, s.row_of, s.target, s.picked, loss, lse, picked};
    return launch_head_join(j, stream) == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

size_t cm_linear_cross_entropy_backward_workspace_size(int64_t M, int64_t K, int64_t n) {
    if (check_extents(M, K, n) != CM_OK) return 0;
    if (M == 0) return 256;
    Carve c(nullptr);
    loss_grad_space(c, M, K, n);
    return c.used;
}

cm_status cm_linear_cross_entropy_backward(const void *x, int64_t ldx, const void *w, int64_t ldw, cm_wlayout wlayout,
                                           const void *targets, int target_bits, int64_t first, int64_t vocab,
                                           const float *lse, const float *dloss, const float *dlse, void *dx,
                                           cm_dtype dx_dtype, int64_t lddx, void *dw, cm_dtype dw_dtype, int64_t lddw,
                                           int accumulate, int64_t M, int64_t K, int64_t n, void *ws, size_t ws_bytes,
                                           cm_stream_t stream_) {
    NvtxRange range("cm_linear_cross_entropy_backward");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if ((wlayout != CM_W_KN && wlayout != CM_W_NK) || (target_bits != 32 && target_bits != 64) || (dx && bad_dtype(dx_dtype)) ||
        (dw && bad_dtype(dw_dtype)))
        return CM_ERR_INVALID_ARG;
    CM_TRY(check_extents(M, K, n));
    const bool nk = wlayout == CM_W_NK;
    if (dw) CM_TRY(check_matrix(dw, lddw, nk ? K : n));
    if (M == 0) {   // the sum over no rows
        const size_t es = dw_dtype == CM_F32 ? 4 : 2;
        if (dw && !accumulate && cudaMemset2DAsync(dw, size_t(lddw) * es, 0, size_t(nk ? K : n) * es, size_t(nk ? n : K), stream) != cudaSuccess)
            return CM_ERR_CUDA;
        return CM_OK;
    }
    if (!lse || !dloss) return CM_ERR_INVALID_ARG;
    CM_TRY(check_head(x, ldx, w, ldw, wlayout, targets, target_bits, first, vocab, M, K, n));
    if (dx) CM_TRY(check_matrix(dx, lddx, K));
    if (!ws || ws_bytes < cm_linear_cross_entropy_backward_workspace_size(M, K, n)) return CM_ERR_WORKSPACE;
    if (!aligned16(ws) || misaligned(lse, CM_F32) || misaligned(dloss, CM_F32) || misaligned(dlse, CM_F32)) return CM_ERR_ALIGNMENT;
    if (!dx && !dw) return CM_OK;
    Device d;
    CM_TRY(device(&d));
    Carve carve(ws);
    const LossGradSpace s = loss_grad_space(carve, M, K, n);
    // a chunk's logits and the two products behind them; tiles that are split, and strips, take all rows.
    // dw's are not split: its extents are the weights', and its epilogue scales
    const Choice cp = choose_logits(d, M, s.columns, K), cx = choose(d, M, K, s.columns, false);
    const Choice cw = choose(d, nk ? s.columns : K, nk ? K : s.columns, M, true, Has::counted);
    const bool counted = cp.pair && (!dx || (cx.pair && cx.splits == 1));
    HeadRows r = {};
    r.targets = targets;
    r.target_bits = target_bits;
    r.first = first;
    r.n = n;
    r.vocab = vocab;
    r.rows = M;
    r.K = K;
    r.x = x;
    r.ldx = ldx;
    r.xs = s.xs;
    r.ldxs = s.lds;
    r.always = !counted;
    r.count = s.count;
    r.slot_of = s.slot_of;
    r.target = s.target;
    r.lse = lse;
    r.dloss = dloss;
    r.dlse = dlse;
    r.lse2 = s.lse2;
    r.grad = s.grad;
    r.hit = s.hit;
    r.scale = s.scale;
    r.groups = s.groups;
    if (launch_head_rows(r, stream) != cudaSuccess) return CM_ERR_CUDA;
    const Operand rows = {s.xs, s.lds, false}, rows_t = {s.xs, s.lds, true}, all = {x, ldx, false}, all_t = {x, ldx, true};
    for (int64_t c0 = 0; c0 < n; c0 += s.columns) {
        const int64_t cols = std::min(s.columns, n - c0);
        const void *const wc = static_cast<const uint16_t *>(w) + (nk ? c0 * ldw : c0);
        Kind kind;
        kind.mode = kLinSoftGrad;
        kind.live = {s.count, counted ? 1 : 0, 0, counted ? 1 : 0, M};
        kind.whole = counted ? &all : nullptr;
        kind.head.target = s.target;
        kind.head.lse2 = s.lse2;
        kind.head.grad = s.grad;
        kind.head.hit = s.hit;
        kind.head.first = c0;
        LinearEpilogue e = {};
        e.y = s.p;
        e.ldy = s.ldp;
        const Operand weights = {wc, ldw, !nk};
        CM_TRY(cp.pair ? product_pair(d, cp, kind, weights, rows, M, cols, K, e, stream)
                       : product_strip(d, cp, kind, weights, rows, M, cols, K, e, stream));
        // dx's part of the chunk, added up in fp32, and the chunk's rows (columns) of dw
        LinearEpilogue ex = {}, ew = {};
        ex.y = s.sum;
        ex.ldy = s.lds;
        ex.y_f32 = 1;
        ex.accumulate = c0 > 0;
        ew.y = static_cast<uint8_t *>(dw) + (nk ? c0 * lddw : c0) * (dw_dtype == CM_F32 ? 4 : 2);
        ew.ldy = lddw;
        ew.y_f32 = dw_dtype == CM_F32;
        ew.accumulate = accumulate != 0;
        ew.scale = s.scale;
        const Operand ax = {wc, ldw, nk}, bx = {s.p, s.ldp, false}, pt = {s.p, s.ldp, true};
        const Operand &aw = nk ? rows_t : pt, &bw = nk ? pt : rows_t;
        const int64_t dr = nk ? cols : K, dc = nk ? K : cols;
        Kind kx, kw;
        kw.mode = kLinCounted;
        if (counted) {
            kx.mode = kLinCounted;
            kx.live = {s.count, 1, 0, 0, M};
            kw.live = {s.count, 0, 1, nk ? 2 : 1, M};
            kw.whole = &all_t;
        }
        if (dx && dw && counted && cx.bn == 256 && cw.bn == 256) {
            LinearPairMore px, pw;
            CM_TRY(pair_params(px, d, cx, kx, ax, bx, M, K, cols, ex));
            CM_TRY(pair_params(pw, d, cw, kw, aw, bw, dr, dc, M, ew));
            if (launch_linear_two(px, nk ? 1 : 0, pw, d.clusters[0], stream) != cudaSuccess) return CM_ERR_CUDA;
            continue;
        }
        if (dx) CM_TRY(counted ? product_pair(d, cx, kx, ax, bx, M, K, cols, ex, stream) : product(d, ax, bx, M, K, cols, ex, stream));
        if (dw) CM_TRY(product_pair(d, cw, kw, aw, bw, dr, dc, M, ew, stream));
    }
    if (!dx) return CM_OK;
    const HeadScatter g = {s.sum, s.lds, s.slot_of, s.scale, dx, dx_dtype == CM_F32, lddx, M, K};
    return launch_head_scatter(g, stream) == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

cm_status cm_linear_choose(int64_t rows, int64_t cols, int64_t k, int transposed, cm_linear_tile *tile) {
    if (!tile) return CM_ERR_INVALID_ARG;
    if (rows == 0) return CM_ERR_SHAPE;
    CM_TRY(check_extents(rows, k, cols));
    Device d;
    CM_TRY(device(&d));
    const Choice c = choose(d, rows, cols, k, transposed != 0);
    tile->pair = c.pair ? 1 : 0;
    tile->rows = c.pair ? 256 : c.tok;
    tile->cols = c.pair ? c.bn : 128;
    tile->splits = c.splits;
    tile->ctas_per_sm = !c.pair && c.ring_bytes == kStripShared ? 2 : 1;
    return CM_OK;
}

cm_status cm_linear_check_status(cm_stream_t stream_, int32_t info[4]) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    Device d;
    CM_TRY(device(&d));
    LinearStatus s = {};
    if (cudaMemcpyAsync(&s, d.status, sizeof(s), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return CM_ERR_CUDA;
    if (s.w[0] != 0 && (cudaMemsetAsync(d.status, 0, sizeof(s), stream) != cudaSuccess ||
                        cudaStreamSynchronize(stream) != cudaSuccess))
        return CM_ERR_CUDA;
    if (info)
        for (int i = 0; i < 4; ++i) info[i] = int32_t(s.w[i]);
    return static_cast<cm_status>(s.w[0]);
}

}  // extern "C"
