// fp8.h -- argument blocks and kernel tables of the 8-bit path: rows or
// blocks rounded to 8-bit floating point with a scale for every 128 columns
// (fp8_rows.cuh), shared by the kernels and the host code that launches them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsk {

constexpr int kFp8Group = 128;             // columns that share a scale
constexpr int kFp8Window = 16384;          // most columns a row kernel holds

// Rows: the norm (of x, or of the stored sum x + r) or x alone, rounded to 8
// bits with a scale for each 128 columns of a row.
struct Fp8RowsParams {
    const void *x;     // [M,H]
    const void *r;     // [M,H] residual input, or unused
    const void *w;     // [H], or unused without the norm
    void *q;           // [M,H] one byte an element
    float *scale;      // [M,G]
    void *h;           // [M,H] residual sum out, or unused
    float *rstd;       // [M] or nullptr
    int64_t M;
    int H;
    int G;             // groups in a row: ceil(H / 128)
    float eps;
    int e5m2;          // format of q: 0 e4m3, 1 e5m2
    int64_t ldx, ldr, ldq, ldh;   // row strides (elements; bytes for q)
};

// Blocks of 128 x 128: one scale each.
struct Fp8BlocksParams {
    const void *x;     // [M,H]
    void *q;           // [M,H]
    float *scale;      // [ceil(M / 128), G]
    int64_t M;
    int H;
    int G;
    int e5m2;
    int64_t ldx, ldq;
};

// One shape of the row kernel.
struct Fp8RowKernel {
    const void *fn;
    int E;               // elements a pack
    int V;               // packs a lane
    int lanes;           // lanes a row (rows share a warp); 0: a whole CTA a row
    int max_threads;
    int64_t max_cols() const { return (int64_t)E * V * (lanes ? lanes : max_threads); }
};

// The shapes of one element type, for x alone, the norm, and the norm of
// x + r: 32-byte packs with rows that share a warp [0..3], with a CTA a row
// for few rows [4], for many rows, narrow [5] and wide [6]; 16-byte packs
// [7]; loose packs, rows that share a warp [8], [9], a CTA a row [10].
// Blocks: 32-byte, 16-byte, loose packs.
constexpr int kFp8SubShapes = 4, kFp8RowShapes = 11;
struct Fp8RowSet {
    Fp8RowKernel k[3][kFp8RowShapes];
    const void *blocks[3];
    int blocks_E[3];
};
extern const Fp8RowSet fp8_rows_bf16, fp8_rows_f16, fp8_rows_f32;

} // namespace rmsk
