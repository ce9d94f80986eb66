// cm_linear.cuh -- parameters and launch entries of the linear layer's kernels:
// one matrix product whose epilogue adds the bias, applies the activation (or
// multiplies by its derivative) and adds the residual.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cm.h"

namespace cm {

// The matrix product's result D[row][col] passes, in fp32 and in this order:
//   + bias[col];  z = bf16(.) if `z`;  act(.) or, if `dact`, * act'(zin[row][col]);
//   + res[row][col];  + y[row][col] if `accumulate`;  one rounding to y's type.
struct LinearEpilogue {
    void *y;
    const void *bias;
    const void *res;    // bf16
    const void *zin;    // bf16
    void *z;            // bf16
    int64_t ldy, ldr, ldzin, ldz;
    int y_f32, bias_f32;
    int act;            // cm_act
    int dact;
    int accumulate;
};

// Device status of the linear kernels: {code, tile, CTA, site} of the first
// bounded wait that expired since it was last read.
struct LinearStatus {
    uint32_t w[4];
};

enum LinearSite : uint32_t {
    kLinSiteEmpty = 32,
    kLinSiteFull = 33,
    kLinSiteAcc = 34,
    kLinSiteTmem = 35,
};

// One output tile is 128 columns x tok rows: the columns (weights) take the
// 128 rows of the tensor core's tile, so that a call with few rows (tokens)
// still fills it, and the k-slices of a tile can be split over a cluster.
struct LinearStripParams {
    CUtensorMap tmA;    // column operand: [n][K] (K-major) or [K][n]
    CUtensorMap tmB;    // row operand: [rows][K] (K-major) or [K][rows]
    LinearEpilogue e;
    int64_t rows, cols;
    int kblocks;        // 64-wide K slices
    int tok;            // rows of a tile: a multiple of 16 up to 256 (of 64 if the row operand is MN-major)
    int row_tiles;
    int splits;         // CTAs of a cluster that share a tile's K slices
    int ring_bytes;     // shared memory for `stages` slices, and for a split tile's partial sums
    int stages;
    LinearStatus *status;
    uint64_t timeout_ns;
};

// layout: bit 0 = row operand MN-major, bit 1 = column operand MN-major.
constexpr int kStripAlone = 216 * 1024, kStripShared = 108 * 1024;   // ring bytes of a CTA alone on its SM, of one of two
// clusters[i]: clusters of i CTAs (2 to kStripMostSplits) that run together, one CTA an SM.
constexpr int kStripMostSplits = 8;
cudaError_t prepare_linear_strip(int sms, int *clusters);
cudaError_t launch_linear_strip(const LinearStripParams &p, int layout, cudaStream_t stream);
int linear_strip_stages(int tok, int ring_bytes);

// Tiles of 256 rows x bn columns on CTA pairs.  A is the row operand here, B the
// column operand.
struct LinearPairParams {
    CUtensorMap tmA, tmB;
    CUtensorMap tmY;          // bf16: 64 x 32 boxes, fp32: 32 x 32
    CUtensorMap tmZ;          // pre-activation kept (bf16 y only), 64 x 32
    CUtensorMap tmIn0, tmIn1; // residual (or y, to be added to) and pre-activation read; bf16 y only
    LinearEpilogue e;
    int64_t rows, cols;
    int kblocks, mtiles, ntiles, tiles;
    int bn;                   // columns of a tile: 256 or 128
    int band;                 // row tiles that run through all columns together
    LinearStatus *status;
    uint64_t timeout_ns;
};

// layout: bit 0 = B MN-major, bit 1 = A MN-major.  splits: 1 (persistent, on
// `clusters` pairs), or 2 or 4 pairs a cluster that share a tile's K slices,
// one cluster a tile.  clusters[i]: clusters of 2^i pairs that run together.
cudaError_t prepare_linear_pair(int sms, int *clusters);
cudaError_t launch_linear_pair(const LinearPairParams &p, int layout, int splits, int clusters, cudaStream_t stream);

// Column sums out[c] (+)= sum_r x[r][c] of a bf16 matrix (cm_norm.cu): partial
// sums per row chunk in `partial`, then their sum in chunk order.
int64_t colsum_chunks(int64_t rows, int64_t cols);
cudaError_t launch_colsum(const void *x, int64_t ldx, int64_t rows, int64_t cols, float *partial, void *out,
                          bool out_f32, bool accumulate, cudaStream_t stream);

}  // namespace cm
