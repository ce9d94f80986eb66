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
    // of the gated kernels (LinearMode): the up projection's bias, and its z read or written
    const void *bias2;
    const void *zin2;   // bf16
    void *z2;           // bf16
    const float *scale; // kLinCounted; on the device, NULL for 1
};

// What a kernel's epilogue computes.
//   kLinPlain  LinearEpilogue's chain.
//   kLinGated  two products of the same rows, g with the first column operand and u
//              with the second: g += bias, u += bias2; z = bf16(g), z2 = bf16(u) if
//              kept; y = act(g) u.
//   kLinGateGrad  D is the gradient of such a y: z = D zin2 act'(zin), y = D act(zin)
//              (zin = g, zin2 = u as they were kept; y is u's gradient, z is g's).
//   kLinStats  D are logits: of each row and each half of a tile's columns the largest
//              and the sum of exp(. - largest), and the target's logit (LinearHead).
//   kLinSoftGrad  y = exp(D - lse) grad, less hit where the column is the target.
//   kLinCounted  kLinPlain with D times `scale` first, of rows that are counted on the
//              device (LinearLive).  A mode of its own: the two checks cost a plain
//              weight gradient of few slices a tile 0.6 us of 7.6.
enum LinearMode { kLinPlain = 0, kLinGated = 1, kLinGateGrad = 2, kLinStats = 3, kLinSoftGrad = 4, kLinCounted = 5 };

// The loss over a vocabulary, by slots: the rows that have a target, in order.
struct LinearHead {
    const int32_t *target;   // column of the weights' slice, or kNotHere, kNoToken
    const float *lse2;       // lse log2(e)
    const float *grad, *hit;
    float2 *stat;            // [part][stride]: {largest, sum} of 128 columns
    float *picked;           // the target's logit, where it lies in the slice
    int64_t stride;          // slots there may be
    int64_t first;           // column of the slice that the product's first one is
};
// The tensor cores cut a sum off at each step of 16 terms, by which long sums fall
// short: by 5e-6 of a logit of 4096 terms.  The loss's logits are therefore summed in
// parts of this many slices of 64 terms, whose fp32 results are added with rounding,
// and in the same parts again for their gradient exp(z - lse): lse holds what z does.
constexpr int kStatSlices = 16;
constexpr int32_t kNotHere = -1, kNoToken = -2;   // of another slice; beyond the vocabulary

// A product of the slots' rows: how many there are is known on the device only.
struct LinearLive {
    const int32_t *count;    // NULL: all rows
    int skip;                // tiles of rows behind the last slot are left out (else they are computed as zeros)
    int of_k;                // it limits the contracted extent, not the rows
    int whole_is;            // where every row is a slot, tmWhole stands for tmA (1) or tmB (2)
    int64_t whole;           // rows there are
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

// And of the modes that need more (kernel parameters are copied at each launch).
struct LinearStripMore : LinearStripParams {
    CUtensorMap tmA2;       // gated: the second column operand; a tile then has 64 columns of each
    LinearHead head;        // of the head's modes: 128 columns a part
    const int32_t *count;   // slots there are
};

// layout: bit 0 = row operand MN-major, bit 1 = column operand MN-major.  The other modes take 0 and 2; there is no kLinCounted.
constexpr int kStripAlone = 216 * 1024, kStripShared = 108 * 1024;   // ring bytes of a CTA alone on its SM, of one of two
// clusters[i]: clusters of i CTAs (2 to kStripMostSplits) that run together, one CTA an SM.
constexpr int kStripMostSplits = 8;
constexpr int kStripRoundRows = 128;   // tiles of up to so many rows have two accumulators: parts of a sum in any number
cudaError_t prepare_linear_strip(int sms, int *clusters);
cudaError_t launch_linear_strip(const LinearStripMore &p, int layout, LinearMode mode, cudaStream_t stream);
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

// And of the modes that need more.
struct LinearPairMore : LinearPairParams {
    CUtensorMap tmB2, tmZ2;   // gated: the second column operand, and its z kept
    CUtensorMap tmWhole;      // see LinearLive
    LinearLive live;          // of the head's modes and kLinCounted
    LinearHead head;
};

// layout: bit 0 = B MN-major, bit 1 = A MN-major; the gated modes take 0 and 1, and
// kLinGated, half of whose columns are of each operand, unsplit tiles of 256; the head's modes have
// 0 and 1, tiles of 256 columns and no splits; kLinCounted has no splits.  splits: 1 (persistent, on
// `clusters` pairs), or 2 or 4 pairs a cluster that share a tile's K slices,
// one cluster a tile.  clusters[i]: clusters of 2^i pairs that run together.
cudaError_t prepare_linear_pair(int sms, int *clusters);
cudaError_t launch_linear_pair(const LinearPairMore &p, int layout, LinearMode mode, int splits, int clusters,
                               cudaStream_t stream);

// Two products (kLinCounted) of 256-column tiles in one launch, the first of layout 0 or 1 with
// an fp32 y, the second of layout 3.
cudaError_t launch_linear_two(const LinearPairMore &p0, int layout0, const LinearPairMore &p1, int clusters, cudaStream_t stream);

// Column sums out[c] (+)= sum_r x[r][c] of a bf16 matrix (cm_norm.cu): partial
// sums per row chunk in `partial`, then their sum in chunk order.
int64_t colsum_chunks(int64_t rows, int64_t cols);
cudaError_t launch_colsum(const void *x, int64_t ldx, int64_t rows, int64_t cols, float *partial, void *out,
                          bool out_f32, bool accumulate, cudaStream_t stream);

// Rows that have a target, gathered (cm_head.cu).  Slot j is the j-th of them.  More than
// kHeadRowsOnce rows are counted in up to kHeadGroups groups by a launch of their own.
constexpr int64_t kHeadRowsOnce = 32768;
constexpr int kHeadGroups = 1024;
struct HeadGroup {
    int32_t count;   // rows with a target
    float top;       // the largest finite |dloss|, |dloss + dlse| of them
};
struct HeadRows {
    const void *targets;
    int target_bits;
    int64_t first, n, vocab;     // the slice's ids, and how many there are in all
    int64_t rows, K;
    const void *x;               // bf16 [rows][ldx]
    int64_t ldx;
    void *xs;                    // the slots' rows, [rows][ldxs]; zeros behind the last up to a multiple of 64, or all
    int64_t ldxs;
    int always;                  // gather where every row is a slot too, and write zeros to all rows behind
    int32_t *count;
    int32_t *row_of;             // by slot (forward), NULL
    int32_t *slot_of;            // by row (backward), -1 for none; NULL
    int32_t *target;             // by slot
    float *picked;               // by slot, zeroed (forward)
    float *loss, *lse_out, *picked_out;   // by row, zeros for rows without a target (forward); may be NULL
    const float *lse, *dloss, *dlse;      // by row (backward); dlse may be NULL
    float *lse2, *grad, *hit, *scale;     // by slot, and one (backward)
    HeadGroup *groups;                    // kHeadGroups where rows > kHeadRowsOnce
};
cudaError_t launch_head_rows(const HeadRows &p, cudaStream_t stream);

struct HeadJoin {
    const float2 *stat;          // [parts][stride]
    int64_t parts, stride;
    const int32_t *count, *row_of, *target;
    const float *picked;
    float *loss, *lse, *picked_out;
};
cudaError_t launch_head_join(const HeadJoin &p, cudaStream_t stream);

// dx[row] = scale sum[slot_of[row]], zeros for rows without a slot.
struct HeadScatter {
    const float *sum;            // [slot][ld], ld a multiple of 8
    int64_t ld;
    const int32_t *slot_of;
    const float *scale;
    void *dx;
    int dx_f32;
    int64_t lddx, rows, K;
};
cudaError_t launch_head_scatter(const HeadScatter &p, cudaStream_t stream);

}  // namespace cm
