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

// A paged cache behind k and v: rows at part[1].y and part[2].y, or 4-bit tiles
// at part[1].y.
struct RopeCache {
    const void *slots;         // [T] int32 or int64
    int slot64;
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
    float eps, inv_d;          // 1 / D
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
    float eps, inv_d;
};

// The kernels of one element type: packs of 16 bytes, of half of it (16-bit
// types), of one element. fwd[form][adjacent pairs]: the forward, the append
// of rows, the append in 4 bits; with their shared memory. E: elements a pack.
struct RopeKernel {
    int E;
    const void *fwd[3][2];
    int fwd_smem[3];
    const void *bwd[2];
    int bwd_smem;
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

// Attention over a 4-bit cache (kv4_attend.cuh).
struct Kv4Params {
    const void *q;             // rows (t, h) at q + t qt + h qh (elements)
    int64_t qt, qh;
    void *out;
    int64_t ot, oh;
    float *lse;                // [T, heads] or nullptr
    const uint8_t *cache;
    int64_t pages;
    int tpp;                   // tiles a page
    const float *kscale, *vscale;
    const int *table;          // [B, blocks], rows table_ld apart
    int64_t table_ld;
    int blocks;
    const int *lens;           // [B]
    const int *starts;         // [B + 1] first rows of the sequences, or nullptr: one each
    int B, T, Hk, G;           // G query heads to a key head
    float scale;
    int vec;                   // q and out rows start at 16 bytes
    float *ws;                 // partial results, two a warp
    int cluster;               // CTAs that share a segment; 0: the list
    uint32_t extra_tx, wait_limit_us;
    unsigned int *timeouts;
};

constexpr int kKv4Cluster = 8;             // most CTAs to a segment
constexpr int kKv4Warps = 8;
constexpr int kKv4Slot = 32;               // tokens a stage
// Shared memory of a CTA: the warps' rings, then their mbarriers.
__host__ __device__ constexpr int kv4_stages(int D) { return D == 128 ? 3 : 6; }
__host__ __device__ constexpr int kv4_slot_bytes(int D) { return kKv4Slot / kKv4Tile * 18 * D; }
__host__ __device__ constexpr int kv4_smem(int D)
{
    return kKv4Warps * kv4_stages(D) * (kv4_slot_bytes(D) + 8);
}
// CTAs of a grid to an SM: the ring and the registers allow two of 8 rows.
__host__ __device__ constexpr int kv4_ctas_per_sm(int NT) { return NT == 1 ? 2 : 1; }
// Floats of one partial result: NT * 8 rows of D sums, then their maxima and
// denominators.
__host__ __device__ constexpr int kv4_partial(int D, int NT) { return 8 * NT * (D + 2); }

// [dtype: bf16, fp16][D: 64, 128][NT - 1]; heads of 64 in tiles of 8 rows only.
struct Kv4Kernels {
    const void *attend[2][2][2], *combine[2][2][2];
};
extern const Kv4Kernels kv4_kernels;

// Pieces of prompts (kv4_prompt.cuh): [dtype][D], and their shared memory [D].
struct Kv4PromptKernels {
    const void *fn[2][2];
    int smem[2];
    int rows;                  // of a CTA
    int threads;
};
extern const Kv4PromptKernels kv4_prompt_kernels;

} // namespace rmsk
