// heads.h -- argument blocks and kernel tables of the operators on attention
// heads (rotation, cache, attention), shared by the kernels and the host code
// that launches them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsk {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 256;             // RMSNORM_ROPE_MAX_D
constexpr int kKv4Tile = 16;               // tokens stored together
constexpr int kKv4Group = 16;              // values that share a scale

// Heads as rows: row (t, h) of `heads` heads starts at x + t xt + h xh
// (elements).
struct RopeRows {
    const void *x;
    int64_t xt, xh;
    const void *w;             // [D], or nullptr: no norm
    void *y;
    int64_t yt, yh;
    int heads;
    int chunks;                // pieces of HC heads
};

// Where a rotation comes from: angle of pair i = position * freq[i].
struct RopeTurn {
    const void *pos;           // [T] int32 or int64
    const double *freq;        // [rot / 2]
    int rot;                   // columns that turn; 0: none
    int pos64;
    int adjacent;              // pairs (2i, 2i + 1); else (i, i + rot / 2)
    float amp;
};

// A paged cache behind k and v (part[1], part[2]).
struct RopeCache {
    const void *slots;         // [T] int32 or int64
    int slot64;
    int bits4;                 // 4-bit tiles at part[1].y; else rows of the dtype
    int64_t page_size, limit;  // limit: slots of the cache
    int64_t kpage, vpage;      // page strides (elements; bytes of the whole for 4 bits)
    const float *kscale, *vscale;   // [heads] or nullptr: 1
};

struct RopeParams {
    RopeRows part[3];          // q, k, v
    RopeTurn turn;
    RopeCache cache;
    float *rstd;               // [T, q heads + k heads] or nullptr
    int64_t T;
    int D;
    int shift;                 // log2 of the lanes a row
    int HC;                    // heads a piece
    float eps;
};

struct RopeGradRows {
    const void *dy;
    int64_t yt, yh;
    const void *x;
    int64_t xt, xh;
    const void *w;
    void *dx;
    int64_t dt, dh;
    float *dw;
    int heads;
    int chunks;
};

struct RopeGradParams {
    RopeGradRows part[2];
    RopeTurn turn;
    const float *rstd;         // [T, q heads + k heads] or nullptr
    float *partial;            // [CTAs, D]
    int64_t T;
    int D;
    int shift;
    int HC;
    int ctas_q;                // CTAs that work on part[0]; the others on part[1]
    float eps;
};

// The kernels of one element type: packs of 16 bytes, of half of it (16-bit
// types), of one element; [1]: adjacent pairs. E: elements a pack.
struct RopeKernel {
    int E;
    const void *fwd[2], *append[2], *bwd[2];
};
struct RopeSet {
    int n;
    RopeKernel k[3];
};
extern const RopeSet rope_bf16, rope_f16, rope_f32;
extern const void *const rope_dw_kernel;

// 4-bit cache rows out as 8-bit rows (kv4_read).
struct Kv4ReadParams {
    const uint8_t *cache;
    const void *slots;
    int slot64;
    int heads, D;
    int64_t page_size, limit, n;
    uint8_t *k, *ks, *v, *vs;
};
extern const void *const kv4_read_kernel;

} // namespace rmsk
