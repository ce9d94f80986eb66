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

constexpr uint64_t kLinearTimeoutNs = 1000000000ull;
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
// A gated product is estimated as one of the columns of both its operands; its
// pair tiles have 256 of them (`wide`).
Choice choose(const Device &d, int64_t rows, int64_t cols, int64_t k, bool row_mn, bool wide = false) {
    Choice best;
    double least = 1e30;
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t slices = up(k, kBK);
    const double from_hbm = double(cols) * double(k) * 2.0 / 8.5e6;
    // pair tiles waste what they have beyond `rows`: not worth a look below 33
    for (int bn = 256; bn >= (wide ? 256 : 128) && rows > 32; bn /= 2) {
        const int64_t tiles = up(rows, 256) * up(cols, bn);
        for (int i = 0; i < 3; ++i) {
            const int splits = 1 << i;
            if (i > 0 && (tiles > d.clusters[i] || slices < 2 * splits)) break;
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
    for (int64_t parts = 1; parts <= 4 && rows <= 384; ++parts) {
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
            const double t = (splits > 1 ? 3.7 + 0.063 * double(tok) : 3.4 + 0.04 * double(tok)) + longest + 0.5 * second;
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

// a2: the second column operand of a gated product, else NULL.
cm_status product_pair(const Device &d, const Choice &c, LinearMode mode, const Operand &a, const Operand *a2, const Operand &b,
                       int64_t rows, int64_t cols, int64_t k, const LinearEpilogue &e, cudaStream_t stream) {
    LinearPairParams p;
    p.e = e;
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
    p.status = d.status;
    p.timeout_ns = kLinearTimeoutNs;
    if (!map_operand(&p.tmA, b, rows, k, 128) || !map_operand(&p.tmB, a, cols, k, c.bn / 2) ||
        (a2 && !map_operand(&p.tmB2, *a2, cols, k, c.bn / 2)) || !map_written(&p.tmY, e.y, rows, cols, e.ldy, e.y_f32 != 0))
        return CM_ERR_CUDA;
    if (mode == kLinGateGrad) {
        if (!map_written(&p.tmZ, e.z, rows, cols, e.ldz, false) || !map_rows(&p.tmIn0, e.zin2, rows, cols, e.ldzin, 32) ||
            !map_rows(&p.tmIn1, e.zin, rows, cols, e.ldzin, 32))
            return CM_ERR_CUDA;
    } else if (mode == kLinGated) {
        if (e.z && (!map_written(&p.tmZ, e.z, rows, cols, e.ldz, false) || !map_written(&p.tmZ2, e.z2, rows, cols, e.ldz, false)))
            return CM_ERR_CUDA;
    } else if (!e.y_f32) {
        if (e.z && !map_written(&p.tmZ, e.z, rows, cols, e.ldz, false)) return CM_ERR_CUDA;
        if (e.accumulate && !map_rows(&p.tmIn0, e.y, rows, cols, e.ldy, 32)) return CM_ERR_CUDA;
        if (e.res && !map_rows(&p.tmIn0, e.res, rows, cols, e.ldr, 32)) return CM_ERR_CUDA;
        if (e.dact && !map_rows(&p.tmIn1, e.zin, rows, cols, e.ldzin, 32)) return CM_ERR_CUDA;
    }
    const int layout = (a.mn_major ? 1 : 0) | (b.mn_major ? 2 : 0);
    return launch_linear_pair(p, layout, mode, c.splits, d.clusters[0], stream) == cudaSuccess ? CM_OK : CM_ERR_CUDA;
}

// D [rows][cols] = B [rows][k] A [cols][k]^T with the epilogue e; a2: see product_pair().
cm_status product(const Device &d, const Operand &a, const Operand &b, int64_t rows, int64_t cols, int64_t k,
                  const LinearEpilogue &e, cudaStream_t stream, LinearMode mode = kLinPlain, const Operand *a2 = nullptr) {
    const bool gated = mode == kLinGated;
    const Choice c = choose(d, rows, gated ? 2 * cols : cols, k, b.mn_major, gated);
    if (c.pair) return product_pair(d, c, mode, a, a2, b, rows, cols, k, e, stream);
    LinearStripParams p;
    p.e = e;
    p.rows = rows;
    p.cols = cols;
    p.kblocks = int((k + kBK - 1) / kBK);
    p.tok = c.tok;
    p.row_tiles = int((rows + c.tok - 1) / c.tok);
    p.splits = c.splits;
    p.ring_bytes = c.ring_bytes;
    p.stages = linear_strip_stages(c.tok, c.ring_bytes);
    p.status = d.status;
    p.timeout_ns = kLinearTimeoutNs;
    if (!map_operand(&p.tmA, a, cols, k, gated ? 64 : 128) || (gated && !map_operand(&p.tmA2, *a2, cols, k, 64)) ||
        !map_operand(&p.tmB, b, rows, k, c.tok))
        return CM_ERR_CUDA;
    const int layout = (b.mn_major ? 1 : 0) | (a.mn_major ? 2 : 0);
    return launch_linear_strip(p, layout, mode, stream) == cudaSuccess ? CM_OK : CM_ERR_CUDA;
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
    return product(d, gate, {x, ldx, false}, M, n, K, e, reinterpret_cast<cudaStream_t>(stream), kLinGated, &up);
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
    return product(d, {w, ldw, wlayout == CM_W_NK}, {dy, lddy, false}, M, K, n, e, reinterpret_cast<cudaStream_t>(stream),
                   kLinGateGrad);
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
