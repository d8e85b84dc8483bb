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
// it rounded to fp16, 2^-12 relative down to 2^-22 of the row's maximum: its
// output has 16 bits too.
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
// Split. The work of a call is a list of units of 256 tokens (one stage for
// each of the eight warps) of segments (sequence, key head, tile of query
// rows). Every CTA computes from the lengths, which only the device knows,
// an equal run of consecutive units. A CTA that has the whole of a segment
// writes its output; of the first and the last it may have a part, which goes
// to the workspace, and kv4_combine joins the parts of a segment in order.
// Lengths may thus differ at will, and a captured call replays with others.
#pragma once

#include "../stream.cuh"
#include "rope.cuh"

namespace rmsk {

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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

__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint16_t lds16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds8(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

// ------------------------------------------------------------ work list
struct Kv4Seq {
    int q0, n;           // first row, rows
    int len;             // tokens in the cache
    int tiles;           // of 8 NT query rows
    int units;           // of a tile of a head: at least one, which writes the zeros of empty rows
    __device__ __forceinline__ int64_t total(int Hk) const { return (int64_t)tiles * Hk * units; }
};

// Sequence b as far as its lengths are sound: rows within [0, T), tokens
// within what the table reaches.
template <int NT>
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4Params &p, int b)
{
    Kv4Seq s;
    if (p.starts != nullptr) {
        s.q0 = min(max(__ldg(p.starts + b), 0), p.T);
        s.n = max(min(__ldg(p.starts + b + 1), p.T) - s.q0, 0);
    } else {
        s.q0 = b;
        s.n = 1;
    }
    const int64_t reach = (int64_t)p.blocks * p.tpp * kKv4Tile;
    s.len = (int)max((int64_t)0, min((int64_t)__ldg(p.lens + b), reach));
    s.tiles = (int)(((int64_t)s.n * p.G + 8 * NT - 1) / (8 * NT));
    s.units = max(1, (s.len + kKv4Unit - 1) / kKv4Unit);
    return s;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Units of the whole call; every warp finds the same.
template <int NT>
__device__ __forceinline__ int64_t kv4_units(const Kv4Params &p, int to)
{
    int64_t v = 0;
    for (int b = threadIdx.x & 31; b < to; b += 32)
        v += kv4_seq<NT>(p, b).total(p.Hk);
    return warp_sum64(v);
}

// The sequence that holds unit u, and the units before it.
template <int NT>
__device__ __forceinline__ void kv4_find(const Kv4Params &p, int64_t u, int &seq, int64_t &before)
{
    const int lane = threadIdx.x & 31;
    before = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int64_t v = base + lane < p.B ? kv4_seq<NT>(p, base + lane).total(p.Hk) : 0;
        int64_t sum = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o)
                sum += t;
        }
        const unsigned at = __ballot_sync(0xFFFFFFFFu, before + sum > u);
        if (at) {
            const int l = __ffs(at) - 1;
            seq = base + l;
            before += __shfl_sync(0xFFFFFFFFu, sum - v, l);
            return;
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    seq = p.B;
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

// What the rows of one tile of a segment share, in each lane.
template <typename T, int D, int NT>
struct Kv4Query {
    uint32_t b[NT][D / 16][2];     // q as the MMAs' B
    float mul[NT][2];              // scores to powers of two, for the lane's two rows of a tile of 8
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
            const int64_t row = (int64_t)tile * 8 * NT + nt * 8 + r;
            const bool real = row < (int64_t)s.n * p.G;
            const int i = real ? (int)(row / p.G) : 0, hq = h * p.G + (real ? (int)(row - (int64_t)i * p.G) : 0);
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
            const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            const float mine = base * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
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
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mul[nt][j] = __shfl_sync(0xFFFFFFFFu, mine, 4 * (2 * c + j));
                lim[nt][j] = __shfl_sync(0xFFFFFFFFu, see, 4 * (2 * c + j));
            }
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
            least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
        }
    }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32, NT == 1 ? 2 : 1) kv4_attend(Kv4Params p)
{
    constexpr int kTile = kv4_tile_bytes(D), kSlot = kv4_slot_bytes(D), R = kv4_stages(D);
    constexpr int kRow = D + 4;                                // floats of a merged row (bank offset)
    static_assert(8 * NT * kRow * 4 <= R * kSlot, "a warp's sums fit in its ring");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sm_m[kKv4Warps][8 * NT], sm_l[kKv4Warps][8 * NT];
    __shared__ int sm_bad;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * R * kSlot;
    const uint32_t bars = smem_addr(smem) + kKv4Warps * R * kSlot + warp * R * 8;
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

    const int64_t total = kv4_units<NT>(p, p.B);
    const int64_t C = (total + gridDim.x - 1) / gridDim.x;
    int64_t u = (int64_t)blockIdx.x * C;
    const int64_t u_end = min(u + C, total);
    if (u >= u_end)
        return;
    int seq;
    int64_t before;
    kv4_find<NT>(p, u, seq, before);
    const int64_t u_first = u;
    const unsigned long long limit = wait_limit_ns(p.wait_limit_us);
    uint32_t used = 0;                                          // stages filled and emptied so far
    bool ok = true;

    while (u < u_end && seq < p.B) {
        const Kv4Seq s = kv4_seq<NT>(p, seq);
        const int64_t mine = s.total(p.Hk);
        if (u >= before + mine) {
            before += mine;
            ++seq;
            continue;
        }
        const int64_t within = u - before;
        const int seg = (int)(within / s.units), unit = (int)(within - (int64_t)seg * s.units);
        const int h = seg / s.tiles, tile = seg - h * s.tiles;
        const int units = (int)min((int64_t)(s.units - unit), u_end - u);
        Kv4Query<T, D, NT> q;
        q.load(p, s, h, tile);
        // the stages of this run that some row sees, every eighth one this warp's
        const int from = unit * kKv4Warps + warp;
        const int stages = min((unit + units) * kKv4Warps, (q.most + kKv4Slot - 1) / kKv4Slot);
        const int count = stages > from ? (stages - from + kKv4Warps - 1) / kKv4Warps : 0;
        const int *row = p.table + seq * p.table_ld;
        const uint8_t *head = p.cache + (int64_t)h * p.tpp * kTile;
        const int64_t page_bytes = (int64_t)p.Hk * p.tpp * kTile;
        const int last = (q.most + kKv4Tile - 1) / kKv4Tile;    // tiles that hold seen tokens

        // a stage's two tiles: their pages (-1: none)
        auto pages = [&](int i, int (&pg)[2]) {
            const int t0 = (from + i * kKv4Warps) * 2;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                pg[j] = -1;
                if (i < count && t0 + j < last) {
                    const int v = __ldg(row + (t0 + j) / p.tpp);
                    pg[j] = v >= 0 && v < p.pages ? v : -1;
                }
            }
        };
        auto fill = [&](int i, const int (&pg)[2]) {
            if (i >= count || lane != 0)
                return;
            const int t0 = (from + i * kKv4Warps) * 2;
            const uint32_t st = (used + i) % R, bar = bars + 8 * st;
            mbar_expect_tx(bar, ((pg[0] >= 0) + (pg[1] >= 0)) * kTile + p.extra_tx);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (pg[j] >= 0)
                    bulk_g2s(ring + st * kSlot + j * kTile,
                             head + pg[j] * page_bytes + (int64_t)((t0 + j) % p.tpp) * kTile, kTile, bar);
        };
        // which tiles of the stages in flight are there: two bits each, the oldest lowest
        uint32_t there = 0;
        int pg[2];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            pages(i, pg);
            there |= ((pg[0] >= 0 ? 1u : 0u) | (pg[1] >= 0 ? 2u : 0u)) << (2 * i);
            fill(i, pg);
        }
        pages(R, pg);                                           // fetched ahead of their use

        float o[NT][D / 16][4] = {}, l[NT][2] = {}, m[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            m[nt][0] = m[nt][1] = kKv4Least;

        for (int i = 0; i < count; ++i) {
            const uint32_t st = (used + i) % R, at = ring + st * kSlot;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bars + 8 * st, ((used + i) / R) & 1, limit));
            if (!ok) {
                // a copy never came: wait, with a limit again, for the others in flight
                for (int n = i + 1; n < min(i + R, count); ++n)
                    (void)mbar_wait_bounded(bars + 8 * ((used + n) % R), ((used + n) / R) & 1, limit);
                __syncwarp();
                break;
            }
            const int tok = (from + i * kKv4Warps) * kKv4Slot;
            const bool whole = tok + kKv4Slot <= q.least && (there & 3u) == 3u;
            float x[NT][2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // S^T of 16 tokens
                uint32_t k0[D / 32], k1[D / 32], s0[D / 64], s1[D / 64];
                const uint32_t ka = at + j * kTile + r * (D / 2) + c * (D / 8), kb = ka + 8 * (D / 2);
                const uint32_t sa = at + j * kTile + kv4_kscale(D) + r * (D / 16) + c * (D / 64),
                               sb = sa + 8 * (D / 16);
                if constexpr (D == 128) {
                    const uint4 a = lds128(ka), b = lds128(kb);
                    k0[0] = a.x; k0[1] = a.y; k0[2] = a.z; k0[3] = a.w;
                    k1[0] = b.x; k1[1] = b.y; k1[2] = b.z; k1[3] = b.w;
                    const uint32_t u0 = scales2(lds16(sa)), u1 = scales2(lds16(sb));
                    s0[0] = __byte_perm(u0, u0, 0x1010); s0[1] = __byte_perm(u0, u0, 0x3232);
                    s1[0] = __byte_perm(u1, u1, 0x1010); s1[1] = __byte_perm(u1, u1, 0x3232);
                } else {
                    const uint2 a = lds64(ka), b = lds64(kb);
                    k0[0] = a.x; k0[1] = a.y;
                    k1[0] = b.x; k1[1] = b.y;
                    const uint32_t v0 = lds8(sa), v1 = lds8(sb);
                    s0[0] = scales2((uint16_t)(v0 * 0x0101u));
                    s1[0] = scales2((uint16_t)(v1 * 0x0101u));
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
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[nt][j][e] *= q.mul[nt][e & 1];
                        if (!whole && (tok + j * 16 + r + (e & 2) * 4 >= q.lim[nt][e & 1] || !(there & (1u << j))))
                            x[nt][j][e] = kKv4Least;
                    }
            }
            // a new reference where a score has left the old one's range
            bool far = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    far |= fmaxf(x[nt][0][e], x[nt][1][e]) > m[nt][e & 1] + 7.f;
            if (__any_sync(0xFFFFFFFFu, far)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float n = fmaxf(fmaxf(x[nt][0][e], x[nt][0][e + 2]), fmaxf(x[nt][1][e], x[nt][1][e + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            n = fmaxf(n, __shfl_xor_sync(0xFFFFFFFFu, n, d));
                        n = fmaxf(n, m[nt][e]);
                        const float f = n == kKv4Least ? 1.f : exp2_of(m[nt][e] - n);
                        m[nt][e] = n;
                        l[nt][e] *= f;
#pragma unroll
                        for (int t = 0; t < D / 16; ++t) {
                            o[nt][t][e] *= f;
                            o[nt][t][e + 2] *= f;
                        }
                    }
            }
            uint32_t pb[NT][2][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float b0 = m[nt][0] == kKv4Least ? 0.f : m[nt][0] - 8.f;
                const float b1 = m[nt][1] == kKv4Least ? 0.f : m[nt][1] - 8.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float p0 = exp2_of(x[nt][j][0] - b0), p1 = exp2_of(x[nt][j][1] - b1);
                    const float p2 = exp2_of(x[nt][j][2] - b0), p3 = exp2_of(x[nt][j][3] - b1);
                    l[nt][0] += p0 + p2;
                    l[nt][1] += p1 + p3;
                    pb[nt][j][0] = movmatrix(Half16<f16>::narrow2(p0, p1));
                    pb[nt][j][1] = movmatrix(Half16<f16>::narrow2(p2, p3));
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // O^T of 16 tokens
                constexpr int W = D / 64;                       // words of a token's features
                uint32_t v[4][W];
                const uint32_t base = at + j * kTile + kv4_v(D);
                uint32_t f0, f1;
                if constexpr (D == 128) {
                    const uint4 a = lds128(base + r * 128 + c * 16), b = lds128(base + r * 128 + c * 16 + 64);
                    v[0][0] = a.x; v[0][1] = a.y; v[1][0] = a.z; v[1][1] = a.w;
                    v[2][0] = b.x; v[2][1] = b.y; v[3][0] = b.z; v[3][1] = b.w;
                    const uint32_t sc = at + j * kTile + kv4_vscale(D) + r * 16 + 2 * c;
                    f0 = scales2(lds16(sc));
                    f1 = scales2(lds16(sc + 8));
                } else {
                    const uint32_t a = base + (r >> 1) * 128 + c * 16 + (r & 1) * 4;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t t;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(t) : "r"(a + (e & 1) * 8 + (e & 2) * 32));
                        v[e][0] = t;
                    }
                    const uint32_t sc = at + j * kTile + kv4_vscale(D) + (r >> 1) * 16 + 2 * c;
                    f0 = scales2(lds16(sc));
                    f1 = scales2(lds16(sc + 8));
                }
                if (!whole) {
                    // tokens that are not there count as zeros, whatever bytes lie in their place
                    const int t0 = tok + j * 16 + 2 * c;
                    const bool in = there & (1u << j);
                    f0 = (in && t0 < s.len ? f0 & 0xFFFFu : 0u) | (in && t0 + 1 < s.len ? f0 & 0xFFFF0000u : 0u);
                    f1 = (in && t0 + 8 < s.len ? f1 & 0xFFFFu : 0u) |
                         (in && t0 + 9 < s.len ? f1 & 0xFFFF0000u : 0u);
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
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
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(o[nt][4 * w + t], a, pb[nt][j][0], pb[nt][j][1]);
                    }
                }
            }
            // the stage is read: refill it
            fence_proxy_async_smem();
            __syncwarp();
            there >>= 2;
            there |= ((pg[0] >= 0 ? 1u : 0u) | (pg[1] >= 0 ? 2u : 0u)) << (2 * (R - 1));
            fill(i + R, pg);
            pages(i + R + 1, pg);
        }
        used += count;
        // a row's terms lie in the eight lanes of its column
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], d);

        // join the warps' sums in their rings, which are empty now
        float *sums = reinterpret_cast<float *>(smem + warp * R * kSlot);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = nt * 8 + 2 * c + e;
                if (r == 0) {
                    sm_m[warp][n] = m[nt][e];
                    sm_l[warp][n] = l[nt][e];
                }
                float *d = sums + n * kRow + r * (D / 8);
#pragma unroll
                for (int t = 0; t < D / 16; t += 2)
                    *reinterpret_cast<float4 *>(d + 2 * t) =
                        make_float4(o[nt][t][e], o[nt][t][e + 2], o[nt][t + 1][e], o[nt][t + 1][e + 2]);
            }
        if (!ok)
            sm_bad = 1;
        __syncthreads();
        const bool all = unit == 0 && units == s.units;
        const float gv = p.vscale ? __ldg(p.vscale + h) : 1.f;
        float *part = p.ws + (2 * (int64_t)blockIdx.x + (u - unit > u_first ? 1 : 0)) * kv4_partial(D, NT);
        for (int k = threadIdx.x; k < 8 * NT * (D / 4); k += kKv4Warps * 32) {
            const int n = k / (D / 4), d = (k - n * (D / 4)) * 4;
            float mm = kKv4Least, ll = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kKv4Warps; ++w)
                mm = fmaxf(mm, sm_m[w][n]);
#pragma unroll
            for (int w = 0; w < kKv4Warps; ++w) {
                const float f = sm_m[w][n] == kKv4Least ? 0.f : exp2_of(sm_m[w][n] - mm);
                const float4 v = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(smem + w * R * kSlot) + n * kRow + d);
                if (f != 0.f) {
                    ll = fmaf(f, sm_l[w][n], ll);
                    a.x = fmaf(f, v.x, a.x); a.y = fmaf(f, v.y, a.y);
                    a.z = fmaf(f, v.z, a.z); a.w = fmaf(f, v.w, a.w);
                }
            }
            const int64_t qrow = (int64_t)tile * 8 * NT + n;
            if (!all) {
                *reinterpret_cast<float4 *>(part + n * D + d) = a;
                if (d == 0) {
                    part[8 * NT * D + n] = mm;
                    part[8 * NT * (D + 1) + n] = ll;
                }
            } else if (qrow < (int64_t)s.n * p.G && !sm_bad) {
                const int i = (int)(qrow / p.G), hq = h * p.G + (int)(qrow - (int64_t)i * p.G);
                const float f = ll > 0.f || ll != ll ? gv / ll : 0.f;
                kv4_store<T>(p, s.q0 + i, hq, d, make_float4(a.x * f, a.y * f, a.z * f, a.w * f));
                if (d == 0 && p.lse != nullptr)
                    p.lse[(int64_t)(s.q0 + i) * p.Hk * p.G + hq] =
                        ll > 0.f ? (mm - 8.f + log2f(ll)) * 0.69314718055994531f : (ll != ll ? ll : kKv4Least);
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (sm_bad) {
            if (threadIdx.x == 0)
                atomicAdd(p.timeouts, 1u);
            break;
        }
        u += units;
    }
}

// Joins the parts of the segments that several CTAs worked on, in the order of
// the CTAs. CTA x: segment x of the call (a sequence's segments side by side);
// `ctas` is the grid of kv4_attend.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(256) kv4_combine(Kv4Params p, int ctas)
{
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    // the sequence of this segment, and the units before the segment
    int64_t segs = 0, units = 0, seg = -1, u0 = 0, total = 0;
    Kv4Seq s = {};
    for (int base = 0; base < p.B; base += 32) {
        const Kv4Seq t = base + lane < p.B ? kv4_seq<NT>(p, base + lane) : Kv4Seq{};
        const int64_t n = (int64_t)t.tiles * p.Hk, v = n * t.units;
        int64_t sn = n, sv = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xFFFFFFFFu, sn, o), b = __shfl_up_sync(0xFFFFFFFFu, sv, o);
            if (lane >= o) {
                sn += a;
                sv += b;
            }
        }
        const unsigned at = __ballot_sync(0xFFFFFFFFu, segs + sn > blockIdx.x);
        if (at && seg < 0) {
            const int l = __ffs(at) - 1;
            seg = blockIdx.x - (segs + __shfl_sync(0xFFFFFFFFu, sn - n, l));
            u0 = units + __shfl_sync(0xFFFFFFFFu, sv - v, l);
            s.q0 = __shfl_sync(0xFFFFFFFFu, t.q0, l);
            s.n = __shfl_sync(0xFFFFFFFFu, t.n, l);
            s.tiles = __shfl_sync(0xFFFFFFFFu, t.tiles, l);
            s.units = __shfl_sync(0xFFFFFFFFu, t.units, l);
        }
        segs += __shfl_sync(0xFFFFFFFFu, sn, 31);
        units += __shfl_sync(0xFFFFFFFFu, sv, 31);
    }
    total = units;
    if (seg < 0)
        return;
    u0 += seg * s.units;
    const int64_t C = (total + ctas - 1) / ctas;
    const int first = (int)(u0 / C), last = (int)((u0 + s.units - 1) / C);
    if (first == last)
        return;                                                 // one CTA had all of it
    const int h = (int)seg / s.tiles, tile = (int)seg - h * s.tiles;
    const float gv = p.vscale ? __ldg(p.vscale + h) : 1.f;
    for (int k = threadIdx.x; k < 8 * NT * (D / 4); k += 256) {
        const int n = k / (D / 4), d = (k - n * (D / 4)) * 4;
        const int64_t qrow = (int64_t)tile * 8 * NT + n;
        if (qrow >= (int64_t)s.n * p.G)
            continue;
        float mm = kKv4Least, ll = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = first; i <= last; ++i) {
            const float *part = p.ws + (2 * (int64_t)i + ((int64_t)i * C >= u0 ? 0 : 1)) * kv4_partial(D, NT);
            const float m = __ldcg(part + 8 * NT * D + n), l = __ldcg(part + 8 * NT * (D + 1) + n);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + n * D + d));
            if (m == kKv4Least)
                continue;
            const float up = fmaxf(mm, m), f0 = mm == kKv4Least ? 0.f : exp2_of(mm - up), f1 = exp2_of(m - up);
            mm = up;
            ll = ll * f0 + l * f1;
            a.x = a.x * f0 + v.x * f1; a.y = a.y * f0 + v.y * f1;
            a.z = a.z * f0 + v.z * f1; a.w = a.w * f0 + v.w * f1;
        }
        const int i = (int)(qrow / p.G), hq = h * p.G + (int)(qrow - (int64_t)i * p.G);
        const float f = ll > 0.f || ll != ll ? gv / ll : 0.f;
        kv4_store<T>(p, s.q0 + i, hq, d, make_float4(a.x * f, a.y * f, a.z * f, a.w * f));
        if (d == 0 && p.lse != nullptr)
            p.lse[(int64_t)(s.q0 + i) * p.Hk * p.G + hq] =
                ll > 0.f ? (mm - 8.f + log2f(ll)) * 0.69314718055994531f : (ll != ll ? ll : kKv4Least);
    }
}

} // namespace rmsk
