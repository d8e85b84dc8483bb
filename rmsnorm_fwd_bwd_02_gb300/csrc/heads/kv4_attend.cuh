// kv4_attend.cuh -- attention over a paged cache held in 4 bits, for one or a
// few query tokens of each sequence:
//     o_i = sum_j p_ij v_j,  p_i = softmax_j(scale q_i k_j),  j < len - n + i + 1
// for the i-th of a sequence's n query tokens, with G query heads to each key
// head.
//
// Mathematics. A cached value is code * scale * g: an e2m1 code (one fraction
// bit) times an e4m3 scale (three) has at most five significant bits and lies
// within 2^-10 and 2688, so it is exact in fp16: the products run on fp16
// MMAs with fp32 sums without any rounding of the cache. q goes to fp16 with
// its row scaled by a power of two that brings the largest element to 2^14:
// bf16's eight bits are kept for elements down to 2^-29 of the largest. The
// heads' g and that power go into the softmax's scale.
// Softmax in one pass, in powers of two: the warp holds a reference m for
// each row and adds p = 2^(x - m + 8). m moves only when some x passes m + 7,
// which one vote a stage finds: after a row's first stages that is rare, and
// p stays below 2^15. The denominators add p in fp32; the second product takes
// it rounded to fp16, within 2^-11 of itself down to 2^-22 of the row's maximum. For
// bf16 outputs that is an eighth of the output's own half step (a row's error
// against 64 bits 1.673e-3, 1.661e-3 with that step alone); for fp16 ones it
// would be all of it, so they take what the rounding lost as a second half
// (2.08e-4, which is the output's step alone).
//
// Layout. The cache's rows are the MMAs' M, the query rows (up to 8 NT of one
// key head: G heads times the tokens) their N, since G is small: S^T = K Q^T
// and O^T = V^T P^T with m16n8k16. Both operands of the cache come straight
// from its bytes, because neither the order of the features inside a product
// over them nor that of a product's rows matters:
//  - K: lane (r, c) = (lane / 4, lane % 4) holds of tokens r and r + 8 the
//    features [c D / 4, (c + 1) D / 4): 16 (8) code bytes side by side. Step s
//    of the product takes bytes 2s and 2s + 1; a byte is a register's pair.
//  - V: lane (r, c) holds of tokens 2c, 2c + 1, 2c + 8, 2c + 9 the features
//    [r D / 8, (r + 1) D / 8). Its registers want pairs of tokens of one
//    feature: the nibbles of two tokens' words are interleaved (four logical
//    operations for 16 values) before they are widened, and the pair is
//    multiplied by the pair of the tokens' scales. m-tile t has the features
//    r D / 8 + 2t (row r) and + 2t + 1 (row r + 8).
//  - P: S^T's accumulators hold pairs of query rows of a token; the second
//    product wants pairs of tokens of a row: a transposition of 8 x 8
//    (movmatrix) for each.
// Bytes move once: each warp has a ring of stages of 32 tokens, filled by bulk
// copies (a tile of 16 tokens of one head is 18 D contiguous bytes) that one
// lane issues as soon as the warp has emptied a stage; no barrier between
// warps.
//
// Split. The work of a call is a list of stages of 32 tokens of segments
// (sequence, key head, tile of query rows), with a few more entries a segment
// for what it costs besides. Every warp computes from the lengths, which
// only the device knows, its equal run of the list, so lengths may differ at
// will and a captured call replays with others. A warp that has the whole of
// a segment writes its output. A CTA whose eight runs lie in one segment joins
// their sums in shared memory; what is still a part of a segment goes to the
// workspace, and kv4_combine joins a segment's parts in their order. Where the
// segments are few and short enough to run at once, each gets a cluster of
// CTAs instead, which joins its sums through distributed shared memory: one
// launch, no workspace.
//
// What bounds it. 16 tokens of a key head are 18 D bytes and, at D = 128, 280
// warp instructions, of which 64 widen codes and 64 multiply by scales: four
// warps a scheduler (what the registers allow) issue in 61 % of the cycles.
// Measured (GB300): 4 sequences of some 116000 tokens, 40 heads on 8, 104 us, 5.3
// TB/s of the cache; 64 of 1 to 8192, 32 heads on 8, 70 us; one of 4001 8.6 us.
// Runs of warps, not of CTAs: with units of 256 tokens for whole CTAs, joined
// after each segment, the 64 sequences took 114 us; with twice the CTAs, so that
// late ones even out, 80.
#pragma once

#include "../split.cuh"
#include "../stream.cuh"
#include "rope.cuh"

namespace rmsk {

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// The four bytes of w as four pairs of fp16.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 scales as fp16.
__device__ __forceinline__ uint32_t scales2(uint16_t s)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(s));
    return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// ------------------------------------------------------------ work list
// What a segment costs besides its stages (q, the ring's first copies, the
// output), in stages: 64 sequences of 1 to 8192 take 74.8 us with 1, 71.8 with
// 2, 71.1 with 3, 70.1 with 5; 16 x 5 tokens over 500 to 3000 15.8, 14.8, 14.9
// and 15.3.
constexpr int kKv4Extra = 3;

struct Kv4Seq {
    int q0, n;           // first row, rows
    int len;             // tokens in the cache
    int tiles;           // of 8 NT query rows
    int stages;          // of 32 tokens
    __device__ __forceinline__ int cost() const { return stages + kKv4Extra; }
    __device__ __forceinline__ uint32_t total(int Hk) const { return (uint32_t)tiles * Hk * cost(); }
};

// Sequence b as far as its lengths are sound: rows within [0, T), tokens
// within what the table reaches.
template <int NT>
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4Params &p, int b)
{
    Kv4Seq s;
    const int reach = p.blocks * p.tpp * kKv4Tile;             // below 2^31
    s.len = max(0, min(__ldg(p.lens + b), reach));
    if (p.starts != nullptr) {
        s.q0 = min(max(__ldg(p.starts + b), 0), p.T);
        s.n = max(min(__ldg(p.starts + b + 1), p.T) - s.q0, 0);
    } else {
        s.q0 = b;
        s.n = 1;
    }
    s.tiles = (s.n * p.G + 8 * NT - 1) / (8 * NT);             // T heads is below 2^31
    s.stages = (s.len + kKv4Slot - 1) / kKv4Slot;
    return s;
}

// Sums of entries stop at 2^31 - 1. Sound starts stay below (the host sees to
// it); rows that several sequences claim, of starts that run back and forth,
// could pass 2^32 and come to segments that are none. Such a list is not worked on.
constexpr uint32_t kKv4TooMany = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t kv4_add(uint32_t a, uint32_t b) { return min(a + b, kKv4TooMany); }

// Where in the list (of fewer than 2^31 entries) the sequences begin: the sums
// of 32 sequences at a time, the last such run of them in the lanes.
struct Kv4List {
    int base;            // first sequence in the lanes
    uint32_t mine, sum;   // this lane's entries, and all up to and with it
    uint32_t before;      // entries before `base`
    uint32_t total;       // of the whole call

    template <int NT>
    __device__ __forceinline__ void load(const Kv4Params &p, int from)
    {
        const int b = from + (threadIdx.x & 31);
        base = from;
        mine = b < p.B ? kv4_seq<NT>(p, b).total(p.Hk) : 0;
        sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if ((threadIdx.x & 31) >= o)
                sum = kv4_add(sum, t);
        }
    }
    __device__ __forceinline__ uint32_t all() const { return __shfl_sync(0xFFFFFFFFu, sum, 31); }
    template <int NT> __device__ __forceinline__ void init(const Kv4Params &p)
    {
        before = total = 0;
        for (int from = 32; from < p.B; from += 32) {
            load<NT>(p, from);
            total = kv4_add(total, all());
        }
        load<NT>(p, 0);
        total = kv4_add(total, all());
    }
    // The sequence that holds entry u < total, and the entries before it.
    template <int NT>
    __device__ __forceinline__ int find(const Kv4Params &p, uint32_t u, uint32_t &first)
    {
        if (u < before) {
            before = 0;
            load<NT>(p, 0);
        }
        for (;;) {
            const unsigned at = __ballot_sync(0xFFFFFFFFu, before + sum > u);
            if (at) {
                const int l = __ffs(at) - 1;
                first = before + __shfl_sync(0xFFFFFFFFu, sum - mine, l);
                return base + l;
            }
            before += all();
            load<NT>(p, base + 32);
            if (base >= p.B)
                return -1;                                      // lengths that change under the call
        }
    }
};

// The sequence of segment `id` of the call (a sequence's segments side by
// side), and the segment within it; -1: there is none.
template <int NT>
__device__ __forceinline__ int kv4_segment_of(const Kv4Params &p, uint32_t id, uint32_t &seg)
{
    const int lane = threadIdx.x & 31;
    uint32_t before = 0;
    for (int base = 0; base < p.B; base += 32) {
        const uint32_t n = base + lane < p.B ? (uint32_t)kv4_seq<NT>(p, base + lane).tiles * p.Hk : 0;
        uint32_t sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o)
                sum += t;
        }
        const unsigned at = __ballot_sync(0xFFFFFFFFu, before + sum > id);
        if (at) {
            const int l = __ffs(at) - 1;
            seg = id - before - __shfl_sync(0xFFFFFFFFu, sum - n, l);
            return base + l;
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    return -1;
}

// A segment in the list: its first entries stand for what it costs besides, its
// stages follow.
struct Kv4Segment {
    int h, tile;
    uint32_t at;          // entry of its first stage
};

__device__ __forceinline__ Kv4Segment kv4_segment(const Kv4Seq &s, uint32_t first, uint32_t u)
{
    const uint32_t seg = (u - first) / (uint32_t)s.cost();
    Kv4Segment g;
    g.h = (int)(seg / (uint32_t)s.tiles);
    g.tile = (int)seg - g.h * s.tiles;
    g.at = first + seg * s.cost() + kKv4Extra;
    return g;
}

// Four features of a row of the output.
template <typename T>
__device__ __forceinline__ void kv4_store(const Kv4Params &p, int t, int h, int d, float4 v)
{
    char *o = static_cast<char *>(p.out) + (t * p.ot + h * p.oh + d) * (int64_t)sizeof(T);
    const uint32_t a = Half16<T>::narrow2(v.x, v.y), b = Half16<T>::narrow2(v.z, v.w);
    if (p.vec) {
        asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(o), "r"(a), "r"(b) : "memory");
    } else {
        st_row_b16(o, (uint16_t)a);
        st_row_b16(o + 2, (uint16_t)(a >> 16));
        st_row_b16(o + 4, (uint16_t)b);
        st_row_b16(o + 6, (uint16_t)(b >> 16));
    }
}

constexpr float kKv4Least = -INFINITY;

__device__ __forceinline__ float exp2_of(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log sum exp of a row from its reference m, which 2^base stands for, and
// denominator.
__device__ __forceinline__ float kv4_lse(float m, float l, float base = 8.f)
{
    return l > 0.f ? (m - base + log2f(l)) * 0.69314718055994531f : (l != l ? l : kKv4Least);
}

// What the rows of one tile of a segment share, in each lane.
template <typename T, int D, int NT>
struct Kv4Query {
    uint32_t b[NT][D / 16][2];     // q as the MMAs' B
    float2 mul[NT];                // scores to powers of two (not negative), for the lane's two rows of a tile of 8
    int lim[NT][2];                // tokens that they see
    int most, least;               // of all rows of the tile: most seen, and fewest of the real ones

    __device__ __forceinline__ void load(const Kv4Params &p, const Kv4Seq &s, int h, int tile)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
        const float base = p.scale * 1.4426950408889634f * (p.kscale ? __ldg(p.kscale + h) : 1.f);
        most = 0;
        least = INT32_MAX;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = tile * 8 * NT + nt * 8 + r;
            const bool real = row < s.n * p.G;
            const int i = real ? row / p.G : 0, hq = h * p.G + (real ? row - i * p.G : 0);
            const char *q = static_cast<const char *>(p.q) +
                            ((int64_t)(s.q0 + i) * p.qt + hq * p.qh + c * (D / 4)) * (int64_t)sizeof(T);
            uint32_t w[D / 8];
#pragma unroll
            for (int j = 0; j < D / 8; j += 4) {
                if (!real) {
                    w[j] = w[j + 1] = w[j + 2] = w[j + 3] = 0;
                } else if (p.vec) {
                    const uint4 v = ld_row_v4(q + j * 4);
                    w[j] = v.x; w[j + 1] = v.y; w[j + 2] = v.z; w[j + 3] = v.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[j + e] = (uint32_t)ld_row_b16(q + (j + e) * 4) |
                                   (uint32_t)ld_row_b16(q + (j + e) * 4 + 2) << 16;
                }
            }
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                const float2 v = Half16<T>::wide2(w[j]);
                m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            const int e = max((int)(__float_as_uint(m) >> 23) - 127, -100);
            // the factor's sign goes into q: the largest score is then the largest power
            const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - e) << 23), base);
            const float mine = fabsf(base) * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                const float2 v = Half16<T>::wide2(w[j]);
                b[nt][j >> 1][j & 1] = Half16<f16>::narrow2(v.x * up, v.y * up);
            }
            const int see = real ? max(0, s.len - s.n + i + 1) : 0;
            if (real) {
                most = max(most, see);
                least = min(least, see);
            }
            mul[nt].x = __shfl_sync(0xFFFFFFFFu, mine, 8 * c);
            mul[nt].y = __shfl_sync(0xFFFFFFFFu, mine, 8 * c + 4);
            lim[nt][0] = __shfl_sync(0xFFFFFFFFu, see, 8 * c);
            lim[nt][1] = __shfl_sync(0xFFFFFFFFu, see, 8 * c + 4);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
            least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
        }
    }
};

// The parts of a segment in the workspace: of each warp two at most, the first
// of its run and the last; a CTA that joined its warps' sums uses its first.
__device__ __forceinline__ int64_t kv4_part(uint32_t warp, bool later) { return 2 * (int64_t)warp + (later ? 1 : 0); }

// A part that a wait which ran out has kept from being made: references of NaN,
// which no part has otherwise. kv4_combine leaves its rows unwritten.
template <int D, int NT>
__device__ __forceinline__ void kv4_mark_lost(const Kv4Params &p, uint32_t warp, bool later)
{
    const int lane = threadIdx.x & 31;
    if (lane < 8 * NT)
        p.ws[kv4_part(warp, later) * kv4_partial(D, NT) + 8 * NT * D + lane] = __int_as_float(0x7FFFFFFF);
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32, kv4_ctas_per_sm(NT)) kv4_attend(Kv4Params p)
{
    constexpr int kTile = kv4_tile_bytes(D), kSlot = kv4_slot_bytes(D), R = kv4_stages(D), W = D / 8;
    constexpr int kRow = D + 4;                                // floats of a merged row (bank offset)
    constexpr bool kLow = std::is_same<T, f16>::value;         // p in two halves (see below)
    static_assert(8 * NT * kRow * 4 <= R * kSlot, "a warp's sums fit in its ring");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sm_m[kKv4Warps][8 * NT], sm_l[kKv4Warps][8 * NT];
    __shared__ int sm_bad;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    uint8_t *const ring = smem + warp * R * kSlot;
    const uint32_t ring_s = smem_addr(ring), bars = smem_addr(smem) + kKv4Warps * R * kSlot + warp * R * 8;
    if (lane == 0) {
        for (int i = 0; i < R; ++i)
            mbar_init(bars + 8 * i, 1);
        mbar_init_fence();
    }
    if (threadIdx.x == 0)
        sm_bad = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    // The list, or a segment for each cluster of CTAs, whose warps have equal
    // runs of its stages (its own list: an entry besides, then the stages).
    Kv4List list = {};
    uint32_t cta0 = 0, cta1 = 0, run0, run1, first = 0;
    const uint32_t gw = blockIdx.x * kKv4Warps + warp;
    int seq;
    Kv4Seq s;
    Kv4Segment g;
    bool joined = true;
    if (p.cluster) {
        uint32_t seg;
        seq = kv4_segment_of<NT>(p, blockIdx.x / p.cluster, seg);
        if (seq < 0)
            return;                                             // for the whole cluster
        s = kv4_seq<NT>(p, seq);
        g.h = (int)(seg / (uint32_t)s.tiles);
        g.tile = (int)seg - g.h * s.tiles;
        g.at = 1;
        const uint32_t n = (uint32_t)p.cluster * kKv4Warps, each = ((uint32_t)s.stages + n - 1) / n;
        run0 = 1 + min((blockIdx.x % p.cluster * kKv4Warps + warp) * each, (uint32_t)s.stages);
        run1 = min(run0 + each, 1 + (uint32_t)s.stages);
    } else {
        list.init<NT>(p);
        if (list.total == kKv4TooMany)
            return;                                             // for the whole grid
        const uint32_t warps = gridDim.x * kKv4Warps, C = (list.total + warps - 1) / warps;
        // (unsigned sums below 2^31 + 2^15 each)
        cta0 = min(blockIdx.x * kKv4Warps * C, list.total);
        cta1 = min(cta0 + kKv4Warps * C, list.total);
        if (cta0 >= cta1)
            return;                                             // for the whole CTA
        run0 = min(gw * C, list.total);
        run1 = min(run0 + C, list.total);
        seq = list.find<NT>(p, cta0, first);
        if (seq < 0)
            return;
        s = kv4_seq<NT>(p, seq);
        // whether the CTA's runs lie in one segment
        g = kv4_segment(s, first, cta0);
        joined = cta1 <= g.at + s.stages;
    }
    const unsigned long long limit = wait_limit_ns(p.wait_limit_us);
    uint32_t st_fill = 0, st_use = 0, phase = 0;                // stages of the ring; a phase bit for each
    bool ok = true;

    Kv4Query<T, D, NT> q;
    float o[NT][D / 16][4], l[NT][2], m[NT][2];
    float2 less[NT];                                            // 8 - m, 0 before there is one
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        m[nt][0] = m[nt][1] = kKv4Least;

    for (uint32_t u = run0; u < run1 && ok;) {
        if (p.cluster == 0) {
            if (u >= first + s.total(p.Hk)) {
                seq = list.find<NT>(p, u, first);
                if (seq < 0)
                    break;
                s = kv4_seq<NT>(p, seq);
            }
            g = kv4_segment(s, first, u);
        }
        if ((unsigned)g.h >= (unsigned)p.Hk)
            break;                                              // lengths that change under the call
        const int from = u > g.at ? (int)(u - g.at) : 0;        // this run's stages
        const int to = run1 > g.at ? min(s.stages, (int)(run1 - g.at)) : 0;
        u = g.at + s.stages;                                    // the next segment
        if (from >= to && s.stages > 0)
            continue;                                           // its first entries alone
        // pages of the stages ahead
        const int *row = p.table + seq * p.table_ld;
        const int t0 = 2 * from;
        int blk = t0 / p.tpp, tin = t0 - blk * p.tpp;
        const int lastblk = min(p.blocks, (2 * to + p.tpp - 1) / p.tpp);
        auto page_of = [&](int b) {
            const int v = b < lastblk ? __ldg(row + b) : -1;
            return v < p.pages ? v : -1;
        };
        int p0 = page_of(blk), p1 = page_of(blk + 1);
        q.load(p, s, g.h, g.tile);
        const int seen = min(to, (q.most + kKv4Slot - 1) / kKv4Slot);
        const int count = max(0, seen - from);
        const int last = (q.most + kKv4Tile - 1) / kKv4Tile;    // tiles that hold seen tokens
        const uint8_t *head = p.cache + (int64_t)g.h * p.tpp * kTile;
        const uint32_t page_bytes = (uint32_t)p.Hk * p.tpp * kTile;      // below 2^31
        uint32_t there = 0;                                     // two bits a stage of the ring: its tiles are there
        auto next_tile = [&]() {
            if (++tin == p.tpp) {
                tin = 0;
                p0 = p1;
                ++blk;
                p1 = page_of(blk + 1);
            }
        };
        const bool pairs = (p.tpp & 1) == 0;                    // a stage's two tiles lie side by side in a page
        auto fill = [&](int i) {
            if (i >= count)
                return;
            const uint32_t dst = ring_s + st_fill * kSlot, bar = bars + 8 * st_fill;
            const bool second = t0 + 2 * i + 1 < last;
            const int pa = p0;
            const uint8_t *src = head + (uint64_t)(uint32_t)pa * (uint32_t)page_bytes + (uint32_t)tin * kTile;
            uint32_t bits;
            if (pairs) {
                bits = pa >= 0 ? (second ? 3u : 1u) : 0u;
                if (lane == 0) {
                    const uint32_t bytes = bits == 0 ? 0u : (second ? 2u * kTile : (uint32_t)kTile);
                    mbar_expect_tx(bar, bytes + p.extra_tx);
                    if (bits)
                        bulk_g2s(dst, src, bytes, bar);
                }
                tin += 2;
                if (tin == p.tpp) {
                    tin = 0;
                    p0 = p1;
                    ++blk;
                    p1 = page_of(blk + 1);
                }
            } else {
                next_tile();
                const int pb = second ? p0 : -1;
                bits = (pa >= 0 ? 1u : 0u) | (pb >= 0 ? 2u : 0u);
                if (lane == 0) {
                    mbar_expect_tx(bar, ((pa >= 0) + (pb >= 0)) * kTile + p.extra_tx);
                    if (pa >= 0)
                        bulk_g2s(dst, src, kTile, bar);
                    if (pb >= 0)
                        bulk_g2s(dst + kTile, head + (uint64_t)(uint32_t)pb * (uint32_t)page_bytes + (uint32_t)tin * kTile,
                                 kTile, bar);
                }
                next_tile();
            }
            there = (there & ~(3u << (2 * st_fill))) | bits << (2 * st_fill);
            st_fill = st_fill + 1 == R ? 0 : st_fill + 1;
        };
#pragma unroll
        for (int i = 0; i < R; ++i)
            fill(i);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kKv4Least;
            l[nt][0] = l[nt][1] = 0.f;
            less[nt] = make_float2(0.f, 0.f);
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
                o[nt][t][0] = o[nt][t][1] = o[nt][t][2] = o[nt][t][3] = 0.f;
        }

        for (int i = 0; i < count; ++i) {
            const uint8_t *at = ring + st_use * kSlot;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bars + 8 * st_use, (phase >> st_use) & 1u, limit));
            if (!ok) {
                // a copy never came: wait, with a limit again, for the others in flight
                for (int n = i + 1; n < min(i + R, count); ++n) {
                    st_use = st_use + 1 == R ? 0 : st_use + 1;
                    (void)mbar_wait_bounded(bars + 8 * st_use, (phase >> st_use) & 1u, limit);
                }
                __syncwarp();
                break;
            }
            phase ^= 1u << st_use;
            const int tok = (from + i) * kKv4Slot;
            const uint32_t here = there >> (2 * st_use) & 3u;
            const bool whole = tok + kKv4Slot <= q.least && here == 3u;
            float x[NT][2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // S^T of 16 tokens
                uint32_t k0[D / 32], k1[D / 32], s0[D / 64], s1[D / 64];
                const uint8_t *ka = at + j * kTile + r * (D / 2) + c * (D / 8), *kb = ka + 8 * (D / 2);
                const uint8_t *sa = at + j * kTile + kv4_kscale(D) + r * (D / 16) + c * (D / 64),
                              *sb = sa + 8 * (D / 16);
                if constexpr (D == 128) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(ka), b = *reinterpret_cast<const uint4 *>(kb);
                    k0[0] = a.x; k0[1] = a.y; k0[2] = a.z; k0[3] = a.w;
                    k1[0] = b.x; k1[1] = b.y; k1[2] = b.z; k1[3] = b.w;
                    const uint32_t u0 = scales2(*reinterpret_cast<const uint16_t *>(sa)),
                                   u1 = scales2(*reinterpret_cast<const uint16_t *>(sb));
                    s0[0] = __byte_perm(u0, u0, 0x1010); s0[1] = __byte_perm(u0, u0, 0x3232);
                    s1[0] = __byte_perm(u1, u1, 0x1010); s1[1] = __byte_perm(u1, u1, 0x3232);
                } else {
                    const uint2 a = *reinterpret_cast<const uint2 *>(ka), b = *reinterpret_cast<const uint2 *>(kb);
                    k0[0] = a.x; k0[1] = a.y;
                    k1[0] = b.x; k1[1] = b.y;
                    s0[0] = scales2((uint16_t)(*sa * 0x0101u));
                    s1[0] = scales2((uint16_t)(*sb * 0x0101u));
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[nt][j][e] = 0.f;
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {              // a word: two steps of the product
                    uint32_t a0[4], a1[4];
                    widen4(k0[w], a0);
                    widen4(k1[w], a1);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t f0 = s0[w >> 1], f1 = s1[w >> 1];
                        const uint32_t a[4] = {hmul2(a0[2 * t], f0), hmul2(a1[2 * t], f1),
                                               hmul2(a0[2 * t + 1], f0), hmul2(a1[2 * t + 1], f1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(x[nt][j], a, q.b[nt][2 * w + t][0], q.b[nt][2 * w + t][1]);
                    }
                }
            }
            // powers of two less the reference, which p = 2^8 stands for
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float2 y = __ffma2_rn(make_float2(x[nt][j][e], x[nt][j][e + 1]), q.mul[nt], less[nt]);
                        x[nt][j][e] = y.x;
                        x[nt][j][e + 1] = y.y;
                    }
            if (!whole) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (tok + j * 16 + r + (e & 2) * 4 >= q.lim[nt][e & 1] || !(here & (1u << j)))
                                x[nt][j][e] = kKv4Least;
            }
            // a new reference where a score has left the old one's range
            float top = kKv4Least;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    top = fmaxf(top, fmaxf(x[nt][0][e], x[nt][1][e]));
            bool far = top > 15.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)                     // a row without one: its first scores
                far |= m[nt][0] == kKv4Least || m[nt][1] == kKv4Least;
            if (__any_sync(0xFFFFFFFFu, far)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float n = fmaxf(fmaxf(x[nt][0][e], x[nt][0][e + 2]), fmaxf(x[nt][1][e], x[nt][1][e + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            n = fmaxf(n, __shfl_xor_sync(0xFFFFFFFFu, n, d));
                        // the scores are relative to what was taken off
                        const float off = e ? less[nt].y : less[nt].x, was = m[nt][e], now = fmaxf(was, n - off);
                        const float f = now == kKv4Least ? 1.f : exp2_of(was - now);
                        const float take = now == kKv4Least ? off : 8.f - now, by = take - off;
                        m[nt][e] = now;
                        (e ? less[nt].y : less[nt].x) = take;
                        l[nt][e] *= f;
#pragma unroll
                        for (int t = 0; t < D / 16; ++t) {
                            o[nt][t][e] *= f;
                            o[nt][t][e + 2] *= f;
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            x[nt][j][e] += by;
                            x[nt][j][e + 2] += by;
                        }
                    }
                }
            }
            // p, transposed for the second product; for fp16 outputs in two
            // halves, with which the weights are good to 2^-22.
            uint32_t pb[NT][2][2], pl[kLow ? NT : 1][2][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x0 = exp2_of(x[nt][j][2 * e]), x1 = exp2_of(x[nt][j][2 * e + 1]);
                        const float2 sum = __fadd2_rn(make_float2(l[nt][0], l[nt][1]), make_float2(x0, x1));
                        l[nt][0] = sum.x;
                        l[nt][1] = sum.y;
                        const uint32_t hi = Half16<f16>::narrow2(x0, x1);
                        pb[nt][j][e] = movmatrix(hi);
                        if constexpr (kLow) {
                            const float2 w = Half16<f16>::wide2(hi);
                            pl[nt][j][e] = movmatrix(Half16<f16>::narrow2(x0 - w.x, x1 - w.y));
                        }
                    }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // O^T of 16 tokens
                uint32_t v[4][D / 64];
                const uint8_t *base = at + j * kTile + kv4_v(D);
                const uint8_t *sc;
                if constexpr (D == 128) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(base + r * 128 + c * 16),
                                b = *reinterpret_cast<const uint4 *>(base + r * 128 + c * 16 + 64);
                    v[0][0] = a.x; v[0][1] = a.y; v[1][0] = a.z; v[1][1] = a.w;
                    v[2][0] = b.x; v[2][1] = b.y; v[3][0] = b.z; v[3][1] = b.w;
                    sc = at + j * kTile + kv4_vscale(D) + r * 16 + 2 * c;
                } else {
                    const uint8_t *a = base + (r >> 1) * 128 + c * 16 + (r & 1) * 4;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e][0] = *reinterpret_cast<const uint32_t *>(a + (e & 1) * 8 + (e & 2) * 32);
                    sc = at + j * kTile + kv4_vscale(D) + (r >> 1) * 16 + 2 * c;
                }
                uint32_t f0 = scales2(*reinterpret_cast<const uint16_t *>(sc));
                uint32_t f1 = scales2(*reinterpret_cast<const uint16_t *>(sc + 8));
                if (!whole) {
                    // tokens that are not there count as zeros, whatever bytes lie in their place
                    const int k = tok + j * 16 + 2 * c;
                    const bool in = here & (1u << j);
                    f0 = (in && k < s.len ? f0 & 0xFFFFu : 0u) | (in && k + 1 < s.len ? f0 & 0xFFFF0000u : 0u);
                    f1 = (in && k + 8 < s.len ? f1 & 0xFFFFu : 0u) | (in && k + 9 < s.len ? f1 & 0xFFFF0000u : 0u);
                }
#pragma unroll
                for (int w = 0; w < D / 64; ++w) {
                    uint32_t e0[4], e1[4], e2[4], e3[4];        // even and odd features, tokens 2c.. and 2c + 8..
                    widen4((v[0][w] & 0x0F0F0F0Fu) | ((v[1][w] << 4) & 0xF0F0F0F0u), e0);
                    widen4(((v[0][w] >> 4) & 0x0F0F0F0Fu) | (v[1][w] & 0xF0F0F0F0u), e1);
                    widen4((v[2][w] & 0x0F0F0F0Fu) | ((v[3][w] << 4) & 0xF0F0F0F0u), e2);
                    widen4(((v[2][w] >> 4) & 0x0F0F0F0Fu) | (v[3][w] & 0xF0F0F0F0u), e3);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t a[4] = {hmul2(e0[t], f0), hmul2(e1[t], f0), hmul2(e2[t], f1),
                                               hmul2(e3[t], f1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(o[nt][4 * w + t], a, pb[nt][j][0], pb[nt][j][1]);
                            if constexpr (kLow)
                                mma_f16(o[nt][4 * w + t], a, pl[nt][j][0], pl[nt][j][1]);
                        }
                    }
                }
            }
            // the stage is read: refill it
            fence_proxy_async_smem();
            __syncwarp();
            st_use = st_use + 1 == R ? 0 : st_use + 1;
            fill(i + R);
        }
        if (!ok)
            break;
        // a row's terms lie in the eight lanes of its column
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], d);
        // a row of NaN alone never had a reference; its sums are to be joined all the same
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (l[nt][e] != l[nt][e] && m[nt][e] == kKv4Least)
                    m[nt][e] = 0.f;
        if (joined)
            break;
        // the row's D / 8 features of this lane: to the output, or to the workspace as a part
        const bool all = from == 0 && to == s.stages;
        const float gv = p.vscale ? __ldg(p.vscale + g.h) : 1.f;
        float *part = p.ws + kv4_part(gw, g.at - kKv4Extra > run0) * kv4_partial(D, NT);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = nt * 8 + 2 * c + e, qrow = g.tile * 8 * NT + n;
                if (all && qrow >= s.n * p.G)
                    continue;
                const int i = qrow / p.G, hq = g.h * p.G + qrow - i * p.G;
                const float f = all ? (l[nt][e] > 0.f || l[nt][e] != l[nt][e] ? gv / l[nt][e] : 0.f) : 1.f;
#pragma unroll
                for (int t = 0; t < D / 16; t += 2) {
                    const float4 v = make_float4(o[nt][t][e] * f, o[nt][t][e + 2] * f, o[nt][t + 1][e] * f,
                                                 o[nt][t + 1][e + 2] * f);
                    if (all)
                        kv4_store<T>(p, s.q0 + i, hq, r * W + 2 * t, v);
                    else
                        *reinterpret_cast<float4 *>(part + n * D + r * W + 2 * t) = v;
                }
                if (r == 0 && all && p.lse != nullptr)
                    p.lse[(int64_t)(s.q0 + i) * p.Hk * p.G + hq] = kv4_lse(m[nt][e], l[nt][e]);
                if (r == 0 && !all) {
                    part[8 * NT * D + n] = m[nt][e];
                    part[8 * NT * (D + 1) + n] = l[nt][e];
                }
            }
    }
    if (!ok && lane == 0) {
        atomicAdd(p.timeouts, 1u);
        sm_bad = 1;
    }
    if (!joined) {
        if (!ok)                                                // the parts that this run still owed
            for (int later = g.at - kKv4Extra > run0; later < 2; ++later)
                kv4_mark_lost<D, NT>(p, gw, later);
        return;
    }

    // join the warps' sums in their rings, which are empty now
    float *sums = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = nt * 8 + 2 * c + e;
            if (r == 0) {
                sm_m[warp][n] = m[nt][e];
                sm_l[warp][n] = l[nt][e];
            }
            float *d = sums + n * kRow + r * W;
            if (m[nt][e] != kKv4Least)
#pragma unroll
                for (int t = 0; t < D / 16; t += 2)
                    *reinterpret_cast<float4 *>(d + 2 * t) =
                        make_float4(o[nt][t][e], o[nt][t][e + 2], o[nt][t + 1][e], o[nt][t + 1][e + 2]);
        }
    __syncthreads();
    const bool several = p.cluster > 1;
    if (sm_bad && !several) {
        if (p.cluster == 0 && warp == 0)
            kv4_mark_lost<D, NT>(p, gw, false);
        return;
    }
    if (p.cluster == 0)
        g = kv4_segment(s, first, cta0);
    const bool all = p.cluster > 0 || (cta0 <= g.at && cta1 == g.at + s.stages);
    const float gv = p.vscale ? __ldg(p.vscale + g.h) : 1.f;
    float *part = p.ws + kv4_part(blockIdx.x * kKv4Warps, false) * kv4_partial(D, NT);
    auto write = [&](int n, int d, float4 a, float mm, float ll) {
        const int qrow = g.tile * 8 * NT + n;
        if (qrow >= s.n * p.G)
            return;
        const int i = qrow / p.G, hq = g.h * p.G + qrow - i * p.G;
        const float f = ll > 0.f || ll != ll ? gv / ll : 0.f;
        kv4_store<T>(p, s.q0 + i, hq, d, make_float4(a.x * f, a.y * f, a.z * f, a.w * f));
        if (d == 0 && p.lse != nullptr)
            p.lse[(int64_t)(s.q0 + i) * p.Hk * p.G + hq] = kv4_lse(mm, ll);
    };
    constexpr int kItems = 8 * NT * (D / 4), kThreads = kKv4Warps * 32, kEach = (kItems + kThreads - 1) / kThreads;
    float4 a[kEach];
    float mm[kEach], ll[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int k = threadIdx.x + i * kThreads, n = k / (D / 4), d = (k - n * (D / 4)) * 4;
        mm[i] = kKv4Least;
        ll[i] = 0.f;
        a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k >= kItems)
            continue;
#pragma unroll
        for (int w = 0; w < kKv4Warps; ++w)
            mm[i] = fmaxf(mm[i], sm_m[w][n]);
#pragma unroll
        for (int w = 0; w < kKv4Warps; ++w) {
            if (sm_m[w][n] == kKv4Least)
                continue;
            const float f = exp2_of(sm_m[w][n] - mm[i]);
            const float4 v = *reinterpret_cast<const float4 *>(
                reinterpret_cast<const float *>(smem + w * R * kSlot) + n * kRow + d);
            ll[i] = fmaf(f, sm_l[w][n], ll[i]);
            a[i].x = fmaf(f, v.x, a[i].x); a[i].y = fmaf(f, v.y, a[i].y);
            a[i].z = fmaf(f, v.z, a[i].z); a[i].w = fmaf(f, v.w, a[i].w);
        }
        if (several)
            continue;
        if (all) {
            write(n, d, a[i], mm[i], ll[i]);
        } else {
            *reinterpret_cast<float4 *>(part + n * D + d) = a[i];
            if (d == 0) {
                part[8 * NT * D + n] = mm[i];
                part[8 * NT * (D + 1) + n] = ll[i];
            }
        }
    }
    if (!several)
        return;

    // join the cluster's sums: each CTA leaves its own where the first warp's
    // were and adds up its share of the rows' features, in rank order, out of
    // its peers' shared memory
    __syncthreads();
    float *mine = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int k = threadIdx.x + i * kThreads, n = k / (D / 4), d = (k - n * (D / 4)) * 4;
        if (k < kItems) {
            *reinterpret_cast<float4 *>(mine + n * kRow + d) = a[i];
            if (d == 0) {
                sm_m[0][n] = mm[i];
                sm_l[0][n] = ll[i];
            }
        }
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    const int share = kItems / p.cluster;
    const uint32_t rank = blockIdx.x % p.cluster;
    for (int i = threadIdx.x; i < share; i += kThreads) {
        const int k = rank * share + i, n = k / (D / 4), d = (k - n * (D / 4)) * 4;
        float pm[kKv4Cluster], pll[kKv4Cluster], top = kKv4Least, sum = 0.f;
        float4 v[kKv4Cluster], out = make_float4(0.f, 0.f, 0.f, 0.f);
        uint32_t failed = 0;
#pragma unroll
        for (int r2 = 0; r2 < kKv4Cluster; ++r2) {
            pm[r2] = kKv4Least;
            if (r2 < p.cluster) {
                const uint32_t at = cluster_map(smem_addr(mine + n * kRow + d), r2);
                pm[r2] = ld_cluster_f32(&sm_m[0][n], r2);
                pll[r2] = ld_cluster_f32(&sm_l[0][n], r2);
                asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(v[r2].x), "=f"(v[r2].y), "=f"(v[r2].z), "=f"(v[r2].w)
                             : "r"(at)
                             : "memory");
                uint32_t f;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(f) : "r"(cluster_map(smem_addr(&sm_bad), r2)) : "memory");
                failed |= f;
            }
        }
#pragma unroll
        for (int r2 = 0; r2 < kKv4Cluster; ++r2)
            top = fmaxf(top, pm[r2]);
#pragma unroll
        for (int r2 = 0; r2 < kKv4Cluster; ++r2) {
            if (pm[r2] == kKv4Least)
                continue;
            const float f = exp2_of(pm[r2] - top);
            sum = fmaf(f, pll[r2], sum);
            out.x = fmaf(f, v[r2].x, out.x); out.y = fmaf(f, v[r2].y, out.y);
            out.z = fmaf(f, v[r2].z, out.z); out.w = fmaf(f, v[r2].w, out.w);
        }
        if (!failed)
            write(n, d, out, top, sum);
    }
    // no CTA leaves while a peer may still read from it
    cluster_arrive_release();
    cluster_wait_acquire();
}

// Joins the parts of the segments that several warps or CTAs worked on, in the
// order of the list. CTA x: segment x of the call (a sequence's segments side
// by side); `ctas` is the grid of kv4_attend.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(256) kv4_combine(Kv4Params p, int ctas)
{
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    // the sequence of this segment, and the entries before it
    uint32_t segs = 0, entries = 0, seg = 0, first = 0;
    bool found = false;
    Kv4Seq s = {};
    for (int base = 0; base < p.B; base += 32) {
        const Kv4Seq t = base + lane < p.B ? kv4_seq<NT>(p, base + lane) : Kv4Seq{};
        const uint32_t n = (uint32_t)t.tiles * p.Hk, v = base + lane < p.B ? t.total(p.Hk) : 0;
        uint32_t sn = n, sv = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xFFFFFFFFu, sn, o), b = __shfl_up_sync(0xFFFFFFFFu, sv, o);
            if (lane >= o) {
                sn = kv4_add(sn, a);
                sv = kv4_add(sv, b);
            }
        }
        const unsigned at = __ballot_sync(0xFFFFFFFFu, segs + sn > blockIdx.x);
        if (at && !found) {
            found = true;
            const int l = __ffs(at) - 1;
            seg = blockIdx.x - (segs + __shfl_sync(0xFFFFFFFFu, sn - n, l));
            first = entries + __shfl_sync(0xFFFFFFFFu, sv - v, l);
            s.q0 = __shfl_sync(0xFFFFFFFFu, t.q0, l);
            s.n = __shfl_sync(0xFFFFFFFFu, t.n, l);
            s.tiles = __shfl_sync(0xFFFFFFFFu, t.tiles, l);
            s.stages = __shfl_sync(0xFFFFFFFFu, t.stages, l);
        }
        segs = kv4_add(segs, __shfl_sync(0xFFFFFFFFu, sn, 31));
        entries = kv4_add(entries, __shfl_sync(0xFFFFFFFFu, sv, 31));
    }
    if (!found || s.stages == 0 || entries == kKv4TooMany)
        return;
    const uint32_t warps = ctas * kKv4Warps, C = (entries + warps - 1) / warps;
    const uint32_t start = first + seg * s.cost(), end = start + s.cost();
    const uint32_t w0 = (start + kKv4Extra) / C, w1 = (end - 1) / C;      // the warps that have stages of it
    if (w0 == w1)
        return;                                                 // one warp had all of it
    const uint32_t c0 = w0 / kKv4Warps, c1 = w1 / kKv4Warps;
    // CTAs whose runs all lie in the segment have one part; only the first and
    // the last may have others
    auto inside = [&](uint32_t cta) {
        return cta * kKv4Warps * C >= start && min((cta + 1) * kKv4Warps * C, entries) <= end;
    };
    const bool in0 = inside(c0), in1 = inside(c1);
    if (c0 == c1 && in0)
        return;                                                 // one CTA had all of it
    const int n0 = in0 ? 1 : (int)(min(w1, c0 * kKv4Warps + kKv4Warps - 1) - w0 + 1);
    const int n1 = c0 == c1 ? 0 : (in1 ? 1 : (int)(w1 - c1 * kKv4Warps + 1));
    const int parts = n0 + n1 + (c0 == c1 ? 0 : (int)(c1 - c0 - 1));
    auto part_at = [&](int i) {
        uint32_t w;
        if (i < n0)
            w = in0 ? c0 * kKv4Warps : w0 + i;
        else if (i < parts - n1)
            w = (c0 + 1 + i - n0) * kKv4Warps;
        else
            w = c1 * kKv4Warps + (i - (parts - n1));
        return p.ws + kv4_part(w, w * C < start) * kv4_partial(D, NT);
    };
    const int h = (int)seg / s.tiles, tile = (int)seg - h * s.tiles;
    const float gv = p.vscale ? __ldg(p.vscale + h) : 1.f;
    for (int k = threadIdx.x; k < 8 * NT * (D / 4); k += 256) {
        const int n = k / (D / 4), d = (k - n * (D / 4)) * 4, qrow = tile * 8 * NT + n;
        if (qrow >= s.n * p.G)
            continue;
        float mm = kKv4Least, ll = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        bool lost = false;
        for (int i = 0; i < parts; i += 8) {
            float m[8], l[8];
            float4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float *part = part_at(min(i + j, parts - 1));
                m[j] = i + j < parts ? __ldcg(part + 8 * NT * D + n) : kKv4Least;
                l[j] = __ldcg(part + 8 * NT * (D + 1) + n);
                v[j] = __ldcg(reinterpret_cast<const float4 *>(part + n * D + d));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                lost |= m[j] != m[j];
                if (m[j] == kKv4Least)
                    continue;
                const float up = fmaxf(mm, m[j]);
                const float f0 = mm == kKv4Least ? 0.f : exp2_of(mm - up), f1 = exp2_of(m[j] - up);
                mm = up;
                ll = ll * f0 + l[j] * f1;
                a.x = a.x * f0 + v[j].x * f1; a.y = a.y * f0 + v[j].y * f1;
                a.z = a.z * f0 + v[j].z * f1; a.w = a.w * f0 + v[j].w * f1;
            }
        }
        if (lost)
            continue;
        const int i = qrow / p.G, hq = h * p.G + qrow - i * p.G;
        const float f = ll > 0.f || ll != ll ? gv / ll : 0.f;
        kv4_store<T>(p, s.q0 + i, hq, d, make_float4(a.x * f, a.y * f, a.z * f, a.w * f));
        if (d == 0 && p.lse != nullptr)
            p.lse[(int64_t)(s.q0 + i) * p.Hk * p.G + hq] = kv4_lse(mm, ll);
    }
}

} // namespace rmsk
