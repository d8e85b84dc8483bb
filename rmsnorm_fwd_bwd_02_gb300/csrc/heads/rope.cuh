// rope.cuh -- heads turned by their positions, after the heads' RMSNorm where
// there is one (QK-norm): forward, on the way into a paged cache, backward.
//
// Mathematics. A head's row x of D features is z = x, or z = x r w with
// r = 1 / sqrt(mean x^2 + eps); of its first `rot` columns pair i, (a, b) =
// (z_i, z_{i + rot/2}) or (z_{2i}, z_{2i+1}), becomes
//     (s (a cos t - b sin t), s (b cos t + a sin t)),   t = position * freq_i,
// with an amplitude s; the other columns stay. The backward turns dy back
// (g = the transposed map) and goes on as the norm's: c = mean(w g x),
// dx = r (w g - x r^2 c), dw = sum over tokens and heads of g x r.
//
// Angles. A float product position * freq has lost the angle's fraction at
// far positions (2^-24 of 10^5 radians is 0.006), and 64-bit floating point
// is slow on this GPU. Here freq / 2 pi becomes once, per thread, a 64-bit
// fixed-point fraction of a turn; position * fraction modulo 2^64 is then
// plain integer arithmetic in which whole turns drop out by themselves: three
// integer multiply-adds give the top 32 bits for any 64-bit position. Their
// top two bits, rounded, are the quadrant; the rest is an angle of at most
// pi / 4, for which the Taylor polynomials (to x^9 and x^10, within 3e-9)
// give sine and cosine. No table of positions is kept or read.
//
// Layout. Packs of 16 bytes; a lane holds the two packs of a row whose
// elements pair up (i and i + rot/2, or neighbours), so a row takes D / 16
// lanes (16-bit types) and no data crosses lanes but the norm's sum. A group
// of lanes takes a piece of HC heads of one token and computes the sines once
// for it. One pass, every row read and written once. Rows come through each
// lane's own ring of asynchronous copies: loads into registers, of four rows at
// a time, had too little in flight (32768 x 40 x 128 bf16 with the norm 137 us,
// through the ring 117), and a map of the piece (weights times sines) halves
// what a row then takes (107 us: 92 % of the copy bandwidth; with three CTAs an
// SM in fewer registers 189). The backward reads two rows for one written and
// keeps dw besides: 16384 x 40 x 128 in 95 us, 78 %, bound by its 400
// instructions a row and lane as much as by DRAM. One token of 16 heads: 2.3 us.
#pragma once

#include "../common.cuh"
#include "heads.h"

namespace rmsk {

// 16-bit formats, 8-byte packs (heads whose halves are no multiple of 16 bytes).
template <typename T> struct Pack<T, 4, typename Half16<T>::Tag> {
    using C = Half16<T>;
    uint2 u;
    static constexpr int E = 4;
    __device__ __forceinline__ static Pack load(const void *base, int64_t idx)
    {
        Pack p;
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                     : "=r"(p.u.x), "=r"(p.u.y)
                     : "l"(static_cast<const uint2 *>(base) + idx));
        return p;
    }
    __device__ __forceinline__ static Pack load_cached(const void *base, int64_t idx)
    {
        Pack p; p.u = __ldg(static_cast<const uint2 *>(base) + idx); return p;
    }
    __device__ __forceinline__ void store(void *base, int64_t idx) const
    {
        asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(static_cast<uint2 *>(base) + idx),
                     "r"(u.x), "r"(u.y)
                     : "memory");
    }
    __device__ __forceinline__ void widen(Vals<4> &f) const
    {
        f.v[0] = C::wide2(u.x);
        f.v[1] = C::wide2(u.y);
    }
    __device__ __forceinline__ static Pack narrow(const Vals<4> &f)
    {
        Pack p;
        p.u.x = C::narrow2(f.v[0].x, f.v[0].y); p.u.y = C::narrow2(f.v[1].x, f.v[1].y);
        return p;
    }
    __device__ __forceinline__ static Pack zero() { Pack p; p.u = make_uint2(0, 0); return p; }
};

__device__ __forceinline__ int64_t ld_index(const void *p, int64_t i, int wide)
{
    return wide ? __ldg(static_cast<const long long *>(p) + i)
                : (int64_t)__ldg(static_cast<const int *>(p) + i);
}

// freq (radians a position) as a fraction of a turn, 2^64 to the turn, rounded to
// the nearest, whole turns dropped: its 53 bits times 2^130 / (2 pi), a constant of
// 128 bits, shifted by its exponent. The constant is within half a unit, so the
// fraction within 1/2 + |freq| 2^-67 units of 2^-64 (with 64 bits of it, 2^-3 |freq|).
// In integers: 64-bit floating point is slow here (one token of 16 heads took
// 5.0 us with it, 3.6 without).
__device__ __forceinline__ uint64_t turn_fraction(double freq)
{
    const uint64_t bits = (uint64_t)__double_as_longlong(freq);
    const int e = (int)(bits >> 52) & 0x7FF;
    const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
    const uint64_t k1 = 11743562013128004905ull, k0 = 18169587780923219393ull;   // 2^130 / (2 pi)
    const uint64_t w0 = m * k0, lo = m * k1, w1 = lo + __umul64hi(m, k0);
    const uint64_t w2 = __umul64hi(m, k1) + (w1 < lo ? 1 : 0);
    auto word = [&](int i) { return i == 0 ? w0 : (i == 1 ? w1 : (i == 2 ? w2 : 0)); };
    const int right = 1141 - e;                          // of the product's three words
    uint64_t t = 0;
    if (right > 0) {
        const int i = right >> 6, by = right & 63, last = right - 1;
        t = by ? word(i) >> by | word(i + 1) << (64 - by) : word(i);
        t += word(last >> 6) >> (last & 63) & 1;
    } else if (right > -64) {
        t = w0 << -right;
    }
    if (e == 0)
        t = 0;                                           // zero and what is no normal number
    return bits >> 63 ? 0 - t : t;
}

// sine and cosine of 2 pi * fraction * pos
__device__ __forceinline__ void sincos_turn(uint64_t fraction, int64_t pos, float &s, float &c)
{
    const uint32_t fl = (uint32_t)fraction, fh = (uint32_t)(fraction >> 32);
    const uint32_t pl = (uint32_t)pos, ph = (uint32_t)((uint64_t)pos >> 32);
    const uint32_t t = __umulhi(fl, pl) + fh * pl + fl * ph;
    const uint32_t quad = (t + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(t - (quad << 30)) * 1.46291807926715968e-9f;   // 2 pi / 2^32
    const float x2 = x * x;
    float ps = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
    ps = fmaf(x2, ps, 1.f / 120.f);
    ps = fmaf(x2, ps, -1.f / 6.f);
    ps = fmaf(x2 * x, ps, x);
    float pc = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    pc = fmaf(x2, pc, -1.f / 720.f);
    pc = fmaf(x2, pc, 1.f / 24.f);
    pc = fmaf(x2, pc, -0.5f);
    pc = fmaf(x2, pc, 1.f);
    const bool swap = quad & 1u;
    s = swap ? pc : ps;
    c = swap ? ps : pc;
    if (quad & 2u)
        s = -s;
    if ((quad + 1u) & 2u)
        c = -c;
}

// The packs that a lane holds of a row, and how many of its pairs turn. Slot
// v of a lane is pair of packs number lane + v L.
struct RopeSlot {
    int a, b;            // pack indices; the row has `np`
    int turns;           // of its E pairs the first `turns` turn
};

template <int E, bool ADJ>
__device__ __forceinline__ RopeSlot rope_slot(int pair, int rot, int adjacent)
{
    const int half = rot / (2 * E);
    const int n = rot / 2 - pair * E;
    RopeSlot s;
    s.turns = n < 0 ? 0 : (n > E ? E : n);
    // past the turning pairs the packs follow in order (2 pair, 2 pair + 1)
    const bool halves = !ADJ && !(E == 1 && adjacent) && pair < half;
    s.a = halves ? pair : 2 * pair;
    s.b = halves ? pair + half : 2 * pair + 1;
    return s;
}

// Sum over the 2^shift lanes of a group; all lanes of the warp take part. Eight
// lanes (heads of 128 in 16 bits) have their own code, without branches.
__device__ __forceinline__ float lanes_sum(float v, int shift)
{
    if (shift == 3)
        return group_allreduce<8>(v);
#pragma unroll
    for (int i = 4; i >= 0; --i)
        if (shift > i)                                   // the same for all lanes
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 1 << i);
    return v;
}

__device__ __forceinline__ float swapped(float v) { return v; }
__device__ __forceinline__ float2 swapped(float2 v) { return make_float2(v.y, v.x); }

// The map of a slot's two packs, the weight before the rotation:
//   halves:   a' = a m[0] + b n[0],  b' = b m[1] + a n[1]
//   adjacent: a' = a m[0] + swapped(a) n[0], and b' likewise (pairs lie within
//   the two-element words)
// with m = w cos and n = -+ w sin, made once for a token and a part, so that a
// head takes two operations an element. Elements that do not turn have m = w.
template <int E, bool ADJ>
struct RopeMap {
    using F = typename Vals<E>::F;
    static constexpr int N = Vals<E>::N;
    F m[2][N], n[2][N];

    __device__ __forceinline__ void make(const float (&cs)[E], const float (&sn)[E], const Vals<E> &wa,
                                         const Vals<E> &wb, int turns)
    {
        if constexpr (ADJ) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float2 w = e < E / 2 ? wa.v[e] : wb.v[e - E / 2];
                const bool on = e < turns;
                m[e / (E / 2)][e % (E / 2)] = on ? make_float2(w.x * cs[e], w.y * cs[e]) : w;
                n[e / (E / 2)][e % (E / 2)] = make_float2(-w.y * sn[e], w.x * sn[e]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                F c, s;
                if constexpr (E == 1) {
                    c = cs[0];
                    s = sn[0];
                } else {
                    c = make_float2(cs[2 * i], cs[2 * i + 1]);
                    s = make_float2(sn[2 * i], sn[2 * i + 1]);
                }
                const F none = splat<F>(0.f);
                m[0][i] = turns ? vmul(wa.v[i], c) : wa.v[i];
                m[1][i] = turns ? vmul(wb.v[i], c) : wb.v[i];
                n[0][i] = vfma(vmul(wb.v[i], s), splat<F>(-1.f), none);
                n[1][i] = vmul(wa.v[i], s);
            }
        }
    }
    __device__ __forceinline__ void apply(Vals<E> &a, Vals<E> &b, int turns) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const F x = a.v[i], y = b.v[i];
            a.v[i] = vmul(x, m[0][i]);
            b.v[i] = vmul(y, m[1][i]);
            if constexpr (ADJ) {
                // what does not turn is not touched by its neighbour, an infinity for instance
                if (i < turns)
                    a.v[i] = vfma(swapped(x), n[0][i], a.v[i]);
                if (i + E / 2 < turns)
                    b.v[i] = vfma(swapped(y), n[1][i], b.v[i]);
            } else if (turns) {
                a.v[i] = vfma(y, n[0][i], a.v[i]);
                b.v[i] = vfma(x, n[1][i], b.v[i]);
            }
        }
    }
};

template <int E>
__device__ __forceinline__ Vals<E> rope_ones()
{
    Vals<E> r;
#pragma unroll
    for (int i = 0; i < Vals<E>::N; ++i)
        r.v[i] = splat<typename Vals<E>::F>(1.f);
    return r;
}

// The frequencies' fractions, one copy a CTA (a lane's own would take it
// sixteen registers).
__device__ __forceinline__ void rope_fractions(const RopeTurn &t, uint64_t *f)
{
    for (int i = threadIdx.x; i < t.rot / 2; i += kRopeThreads)
        f[i] = turn_fraction(__ldg(t.freq + i));
    __syncthreads();
}

// cs and sn of the slot's pairs; sign: 1 to turn, -1 to turn back.
template <int E>
__device__ __forceinline__ void rope_angles(const uint64_t *f, int pair, int turns, int64_t pos, float amp,
                                            float sign, float (&cs)[E], float (&sn)[E])
{
#pragma unroll
    for (int e = 0; e < E; ++e) {
        sincos_turn(e < turns ? f[pair * E + e] : 0, pos, sn[e], cs[e]);
        sn[e] *= amp * sign;
        cs[e] *= amp;
    }
}

// ------------------------------------------------------------ 4-bit rows
// 16 values of a group as eight bytes of e2m1 codes (the even one in a byte's
// low half) and one e4m3 scale (fp32 g: the head's own): the scale is
// max / (6 g) rounded once, between 2^-9 and 448; a code is the quotient
// x / (scale g) in fp32 rounded to nearest even, at most 6. A NaN counts for
// nothing in the maximum and is stored as the largest code.
__device__ __forceinline__ uint2 quant4(const float (&x)[16], float g, uint8_t &scale)
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        m = fmaxf(m, fabsf(x[i]));
    const float t = fminf(fmaxf(__fdiv_rn(m, 6.f * g), 0.001953125f), 448.f);
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(t));
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(s8));
    const float d = Half16<f16>::wide1((uint16_t)h2) * g;
    scale = (uint8_t)s8;
    // Quotients by Markstein's theorem: with r the rounded reciprocal of d and q
    // the rounded x r, q + r (x - q d) in two fused steps is x / d rounded once.
    // (A division each takes several times as long; many values of 16 bits lie
    // right between two codes, so a mere product with r would not do.) Infinities
    // keep q; scales far from one take the divisions.
    const float r = __frcp_rn(d);
    const bool plain = !(d > 1e-18f && d < 1e18f);      // (the residual keeps its bits)
    const float2 r2 = make_float2(r, r), nd = make_float2(-d, -d);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t b;
        const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
        const float2 q = __fmul2_rn(v, r2), e = __ffma2_rn(q, nd, v);
        float2 y = __ffma2_rn(e, r2, q);
        if (plain) {
            y.x = __fdiv_rn(v.x, d);
            y.y = __fdiv_rn(v.y, d);
        }
        const float lo = y.x == y.x ? y.x : q.x, hi = y.y == y.y ? y.y : q.y;
        asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
            : "=r"(b)
            : "f"(hi), "f"(lo));
        w[i >> 2] |= b << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

// Byte offsets in a tile of 16 tokens of one head (18 D bytes): the keys'
// codes [16][D / 2] and scales [16][D / 16], the values' codes [D / 16][16][8]
// and scales [D / 16][16].
__host__ __device__ constexpr int kv4_tile_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int kv4_kscale(int D) { return 8 * D; }
__host__ __device__ constexpr int kv4_v(int D) { return 9 * D; }
__host__ __device__ constexpr int kv4_vscale(int D) { return 17 * D; }

// ------------------------------------------------------------- the pipeline
// Rows on their way: a lane copies its packs of the next batches of heads into
// slots of its own in shared memory (asynchronous copies of 16 or 8 bytes) and
// reads them back when their group of copies is done; no other lane looks at
// them, so nothing is synchronised, and what is in flight takes no registers.
// Single elements (E = 1) are loaded where they are used.
constexpr int kRopeDepth = 3;                          // batches in the ring
template <int E> __host__ __device__ constexpr int rope_fwd_heads(int form)
{
    return E == 1 ? 1 : (form == 2 ? 2 : 4);           // heads a batch; 4-bit rows want room beside the ring
}
template <int E> __host__ __device__ constexpr int rope_bwd_heads() { return E == 1 ? 1 : 2; }
constexpr int kRopeFractions = kRopeMaxD / 2 * 8;      // bytes of the frequencies' fractions
constexpr int kRopeStage = 640;                        // floats of a warp's staged rows (append in 4 bits)
template <int E>
__host__ __device__ constexpr int rope_fwd_smem(int form, size_t es)
{
    return kRopeFractions + (E == 1 ? 0 : kRopeDepth * rope_fwd_heads<E>(form) * 2 * E * (int)es * kRopeThreads) +
           (form == 2 ? kRopeThreads / 32 * kRopeStage * 4 : 0);
}
template <int E>
__host__ __device__ constexpr int rope_bwd_smem(size_t es)
{
    const int ring = E == 1 ? 0 : kRopeDepth * rope_bwd_heads<E>() * 4 * E * (int)es * kRopeThreads;
    const int sums = kRopeThreads * 2 * E * (E == 1 ? 4 : 1) * 4;
    return kRopeFractions + (ring > sums ? ring : sums);
}

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The ring of one lane: slot i of batch b at base + ((b % depth) N + i) of the
// CTA's lanes' packs.
template <typename T, int E, int N>
struct RopeRing {
    static constexpr int kBytes = E * (int)sizeof(T);
    uint8_t *base;
    __device__ __forceinline__ uint8_t *at(int stage, int i) const
    {
        return base + (stage * N + i) * (kRopeThreads * kBytes);
    }
    __device__ __forceinline__ void fetch(int stage, int i, const void *row, int pack) const
    {
        copy_async<kBytes>((uint32_t)__cvta_generic_to_shared(at(stage, i)),
                           static_cast<const char *>(row) + pack * kBytes);
    }
    __device__ __forceinline__ Pack<T, E> get(int stage, int i) const
    {
        Pack<T, E> p;
        p.u = *reinterpret_cast<const decltype(p.u) *>(at(stage, i));
        return p;
    }
};

// The order of a call's pieces: those of `first` (every token's), then those of
// `then`, so that the rows a warp works on at a time are of one kind; a step
// leads from one into the other. T is below 2^31, and so is a step.
struct RopeOrder {
    uint32_t T;
    int first, then;             // pieces a token
    uint32_t dt0, dt1;           // a step in tokens, and the pieces left over
    int dc0, dc1;
    __device__ __forceinline__ RopeOrder(uint32_t T, int first, int then, uint32_t step)
        : T(T), first(first), then(then), dt0(first ? step / first : 0), dt1(then ? step / then : 0),
          dc0(first ? step - dt0 * first : 0), dc1(then ? step - dt1 * then : 0)
    {
    }
};

// Where a group of lanes is: token t, piece c of its heads (of the first kind's
// or of the second's), head hc of the piece. Done at t >= T.
struct RopeCursor {
    uint32_t t;
    int c, hc, second;
    __device__ __forceinline__ void cross(const RopeOrder &o, uint32_t over)
    {
        second = 1;
        t = o.then ? over / o.then : o.T;
        c = o.then ? over - t * o.then : 0;
    }
    __device__ __forceinline__ void start(const RopeOrder &o, uint32_t i)
    {
        hc = second = 0;
        t = o.first ? i / o.first : 0;
        c = o.first ? i - t * o.first : 0;
        if (t >= o.T || o.first == 0)
            cross(o, i - o.T * o.first);
    }
    __device__ __forceinline__ void next(const RopeOrder &o, int U, int HC)
    {
        hc += U;
        if (hc < HC)
            return;
        hc = 0;
        const int n = second ? o.then : o.first;
        t = min(t + (second ? o.dt1 : o.dt0), 0x80000000u);
        c += second ? o.dc1 : o.dc0;
        if (c >= n) {
            c -= n;
            ++t;
        }
        if (!second && t >= o.T)
            cross(o, (t - o.T) * o.first + c);
    }
};

// Rows of a warp in shared memory as fp32, a group of 16 in 20 words (reads
// of whole groups then meet no bank twice); lane g of a row's lanes rounds
// group g and writes it to its tile.
__device__ __forceinline__ void store_tile4(const float *stage, int D, int lane, uint8_t *tile, int t,
                                            bool is_v, float g)
{
    const int G = D / kKv4Group;
    if (lane >= G)
        return;
    float x[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(stage + lane * 20 + 4 * i);
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
    }
    uint8_t s;
    const uint2 c = quant4(x, g, s);
    uint8_t *codes = is_v ? tile + kv4_v(D) + lane * 128 + t * 8 : tile + t * (D / 2) + lane * 8;
    uint8_t *scale = is_v ? tile + kv4_vscale(D) + lane * 16 + t : tile + kv4_kscale(D) + t * G + lane;
    *reinterpret_cast<uint2 *>(codes) = c;
    *scale = s;
}

// FORM 0: the forward; 1: the append, rows of the dtype; 2: the append, 4 bits.
template <typename T, int E, bool ADJ, int FORM>
__global__ void __launch_bounds__(kRopeThreads, 2) rms_rope_fwd(RopeParams p)
{
    constexpr bool APP = FORM > 0;
    constexpr int V = E == 1 ? 4 : 1, U = rope_fwd_heads<E>(FORM);
    using P = Pack<T, E>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *fractions = reinterpret_cast<uint64_t *>(smem);
    // the fractions first, the staged rows, then the ring
    float *stage_all = reinterpret_cast<float *>(smem + kRopeFractions);
    const RopeRing<T, E, 2 * U> ring = {smem + kRopeFractions + (FORM == 2 ? kRopeThreads / 32 * kRopeStage * 4 : 0) +
                                        threadIdx.x * (E * sizeof(T))};

    const int L = 1 << p.shift, lane = threadIdx.x & (L - 1), np = p.D / E;
    RopeSlot slot[V];
    int pair[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        pair[v] = lane + v * L;
        slot[v] = rope_slot<E, ADJ>(pair[v], p.turn.rot, p.turn.adjacent);
    }
    griddep_wait();
    griddep_launch_dependents();

    // in 4 bits q's pieces before k's and v's, which take several times as long
    constexpr bool kApart = FORM == 2;
    const int kv = p.part[1].chunks + (APP ? p.part[2].chunks : 0);
    const RopeOrder order((uint32_t)p.T, p.part[0].chunks + (kApart ? 0 : kv), kApart ? kv : 0,
                          gridDim.x * (kRopeThreads >> p.shift));
    RopeCursor cur, ahead;
    cur.start(order, (blockIdx.x * kRopeThreads + threadIdx.x) >> p.shift);
    ahead = cur;

    // which heads a piece has, and its number among theirs
    auto part_of = [&](const RopeCursor &at, int &ci) {
        ci = at.c;
        if (kApart ? !at.second : ci < p.part[0].chunks)
            return 0;
        if (!kApart)
            ci -= p.part[0].chunks;
        if (!APP || ci < p.part[1].chunks)
            return 1;
        ci -= p.part[1].chunks;
        return 2;
    };
    auto fetch = [&](int stage) {
        if constexpr (E > 1) {
            if (ahead.t < order.T) {
                int ci;
                const RopeRows &r = p.part[part_of(ahead, ci)];
                const int h0 = ci * p.HC + ahead.hc, h1 = min(r.heads, ci * p.HC + p.HC);
                const char *x = static_cast<const char *>(r.x) + ((int64_t)ahead.t * r.xt + h0 * r.xh) * (int64_t)sizeof(T);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h0 + u < h1) {
                        if (slot[0].a < np)
                            ring.fetch(stage, 2 * u, x, slot[0].a);
                        if (slot[0].b < np)
                            ring.fetch(stage, 2 * u + 1, x, slot[0].b);
                    }
                    x += r.xh * (int64_t)sizeof(T);
                }
            }
            ahead.next(order, U, p.HC);
            copies_commit();
        }
    };
#pragma unroll
    for (int i = 0; i < kRopeDepth - 1; ++i)
        fetch(i);
    rope_fractions(p.turn, fractions);

    const bool any_norm = p.part[0].w != nullptr || p.part[1].w != nullptr;
    RopeMap<E, ADJ> map[V];
    int64_t page = 0, within = 0;
    bool kept = true, mapped = false, norm = false;
    int stage = 0, part = 0, ci = 0;
    // the lanes of a warp stay together in the sums' shuffles: done when all are
    while (__any_sync(0xFFFFFFFFu, cur.t < order.T)) {
        fetch(stage == 0 ? kRopeDepth - 1 : stage - 1);
        const bool live = cur.t < order.T;
        if (cur.hc == 0) {
            // a new piece: its part, its token's rotation and its row of the cache
            part = part_of(cur, ci);
            const RopeRows &r = p.part[part];
            norm = r.w != nullptr && live;
            mapped = live && (norm || (p.turn.rot > 0 && part < 2));
            if (mapped) {
                const bool turn = p.turn.rot > 0;
                const int64_t pos = turn ? ld_index(p.turn.pos, cur.t, p.turn.pos64) : 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    Vals<E> wa = rope_ones<E>(), wb = rope_ones<E>();
                    if (norm) {
                        if (slot[v].a < np)
                            P::load_cached(r.w, slot[v].a).widen(wa);
                        if (slot[v].b < np)
                            P::load_cached(r.w, slot[v].b).widen(wb);
                    }
                    float cs[E], sn[E];
                    rope_angles<E>(fractions, pair[v], slot[v].turns, pos, p.turn.amp, 1.f, cs, sn);
                    map[v].make(cs, sn, wa, wb, slot[v].turns);
                }
            }
            if (APP) {
                kept = true;
                if (part > 0 && live) {
                    const int64_t s = ld_index(p.cache.slots, cur.t, p.cache.slot64);
                    kept = s >= 0 && s < p.cache.limit;
                    page = kept ? s / p.cache.page_size : 0;
                    within = kept ? s - page * p.cache.page_size : 0;
                }
            }
        }
        const RopeRows &r = p.part[part];
        const int h0 = ci * p.HC + cur.hc, h1 = live ? min(r.heads, ci * p.HC + p.HC) : 0;
        char *yr = static_cast<char *>(r.y);
        if (!APP || part == 0)
            yr += ((int64_t)cur.t * r.yt + h0 * r.yh) * (int64_t)sizeof(T);
        else
            yr += (page * (part == 1 ? p.cache.kpage : p.cache.vpage) + within * r.yt + h0 * r.yh) *
                  (int64_t)sizeof(T);
        if constexpr (E > 1)
            copies_wait<kRopeDepth - 1>();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (cur.hc + u >= p.HC)
                break;                       // the same for all lanes
            const int h = h0 + u;
            const bool on = h < h1 && kept;
            P xa[V], xb[V];
            if constexpr (E > 1) {
                xa[0] = on && slot[0].a < np ? ring.get(stage, 2 * u) : P::zero();
                xb[0] = on && slot[0].b < np ? ring.get(stage, 2 * u + 1) : P::zero();
            } else {
                const char *x = static_cast<const char *>(r.x) + ((int64_t)cur.t * r.xt + h * r.xh) * (int64_t)sizeof(T);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    xa[v] = on && slot[v].a < np ? P::load(x, slot[v].a) : P::zero();
                    xb[v] = on && slot[v].b < np ? P::load(x, slot[v].b) : P::zero();
                }
            }
            Vals<E> a[V], b[V];
            using F = typename Vals<E>::F;
            F ss = splat<F>(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                xa[v].widen(a[v]);
                xb[v].widen(b[v]);
            }
            if (any_norm) {                                              // the same for all lanes
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < Vals<E>::N; ++i)
                        ss = vfma(b[v].v[i], b[v].v[i], vfma(a[v].v[i], a[v].v[i], ss));
                const float rs = rsqrtf(fmaf(lanes_sum(hsum(ss), p.shift), p.inv_d, p.eps));
                if (norm) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int i = 0; i < Vals<E>::N; ++i) {
                            a[v].v[i] = vmul(a[v].v[i], splat<F>(rs));
                            b[v].v[i] = vmul(b[v].v[i], splat<F>(rs));
                        }
                    if (on && lane == 0 && p.rstd != nullptr && part < 2)
                        p.rstd[(int64_t)cur.t * (p.part[0].heads + p.part[1].heads) + (part ? p.part[0].heads : 0) + h] =
                            rs;
                }
            }
            if (mapped)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    map[v].apply(a[v], b[v], slot[v].turns);
            if constexpr (FORM == 2) {
                // k and v go through shared memory, a group a lane
                float *st = stage_all + (threadIdx.x >> 5) * kRopeStage +
                            ((threadIdx.x & 31) >> p.shift) * (p.D / kKv4Group) * 20;
                __syncwarp();
                if (on && part > 0) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const int ia = slot[v].a * E + e, ib = slot[v].b * E + e;
                            if (ia < p.D)
                                st[(ia >> 4) * 20 + (ia & 15)] = a[v].get(e);
                            if (ib < p.D)
                                st[(ib >> 4) * 20 + (ib & 15)] = b[v].get(e);
                        }
                }
                __syncwarp();
                if (on && part > 0) {
                    const float *gs = part == 1 ? p.cache.kscale : p.cache.vscale;
                    uint8_t *tile = static_cast<uint8_t *>(p.part[1].y) + page * p.cache.kpage +
                                    (h * (p.cache.page_size / kKv4Tile) + within / kKv4Tile) *
                                        kv4_tile_bytes(p.D);
                    store_tile4(st, p.D, lane, tile, (int)(within % kKv4Tile), part == 2,
                                gs ? __ldg(gs + h) : 1.f);
                }
            }
            if (on && (FORM != 2 || part == 0)) {
                char *y = yr + u * r.yh * (int64_t)sizeof(T);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (slot[v].a < np)
                        P::narrow(a[v]).store(y, slot[v].a);
                    if (slot[v].b < np)
                        P::narrow(b[v]).store(y, slot[v].b);
                }
            }
        }
        stage = stage + 1 == kRopeDepth ? 0 : stage + 1;
        cur.next(order, U, p.HC);
    }
}

// The backward. A CTA works on the q heads or on the k heads alone, so that it
// has one dw; its partial row is summed over its groups in a fixed order and
// added up by rope_dw_reduce.
template <typename T, int E, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, 2) rms_rope_bwd(RopeGradParams p)
{
    constexpr int V = E == 1 ? 4 : 1, U = rope_bwd_heads<E>();
    using P = Pack<T, E>;
    using F = typename Vals<E>::F;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *fractions = reinterpret_cast<uint64_t *>(smem);
    const RopeRing<T, E, 4 * U> ring = {smem + kRopeFractions + threadIdx.x * (E * sizeof(T))};

    const int part = blockIdx.x >= p.ctas_q ? 1 : 0;
    const RopeGradRows &r = p.part[part];
    const uint32_t ctas = part ? gridDim.x - p.ctas_q : p.ctas_q;
    const int cta = part ? (int)blockIdx.x - p.ctas_q : (int)blockIdx.x;
    const int heads_all = p.part[0].heads + p.part[1].heads, head0 = part ? p.part[0].heads : 0;
    const int L = 1 << p.shift, lane = threadIdx.x & (L - 1), np = p.D / E;
    const bool norm = r.w != nullptr;                          // the same for the CTA
    RopeSlot slot[V];
    int pair[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        pair[v] = lane + v * L;
        slot[v] = rope_slot<E, ADJ>(pair[v], p.turn.rot, p.turn.adjacent);
    }
    griddep_wait();
    griddep_launch_dependents();

    const RopeOrder order((uint32_t)p.T, r.chunks, 0, ctas * (kRopeThreads >> p.shift));
    RopeCursor cur, ahead;
    cur.start(order, (cta * kRopeThreads + threadIdx.x) >> p.shift);
    ahead = cur;
    auto fetch = [&](int stage) {
        if constexpr (E > 1) {
            if (ahead.t < order.T) {
                const int h0 = ahead.c * p.HC + ahead.hc, h1 = min(r.heads, ahead.c * p.HC + p.HC);
                const char *y = static_cast<const char *>(r.dy) + ((int64_t)ahead.t * r.yt + h0 * r.yh) * (int64_t)sizeof(T);
                const char *x = static_cast<const char *>(r.x) + ((int64_t)ahead.t * r.xt + h0 * r.xh) * (int64_t)sizeof(T);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h0 + u < h1) {
                        if (slot[0].a < np) {
                            ring.fetch(stage, 4 * u, y, slot[0].a);
                            if (norm)
                                ring.fetch(stage, 4 * u + 2, x, slot[0].a);
                        }
                        if (slot[0].b < np) {
                            ring.fetch(stage, 4 * u + 1, y, slot[0].b);
                            if (norm)
                                ring.fetch(stage, 4 * u + 3, x, slot[0].b);
                        }
                    }
                    y += r.yh * (int64_t)sizeof(T);
                    x += r.xh * (int64_t)sizeof(T);
                }
            }
            ahead.next(order, U, p.HC);
            copies_commit();
        }
    };
#pragma unroll
    for (int i = 0; i < kRopeDepth - 1; ++i)
        fetch(i);
    rope_fractions(p.turn, fractions);
    Vals<E> wa[V], wb[V], da[V], db[V];
    RopeMap<E, ADJ> map[V];
    const Vals<E> one = rope_ones<E>();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        {
            const float none[E] = {};
            map[v].make(none, none, one, one, 0);        // a group without a row turns zeros
        }
        (norm && slot[v].a < np ? P::load_cached(r.w, slot[v].a) : P::zero()).widen(wa[v]);
        (norm && slot[v].b < np ? P::load_cached(r.w, slot[v].b) : P::zero()).widen(wb[v]);
        da[v] = Vals<E>::zero();
        db[v] = Vals<E>::zero();
    }

    int stage = 0;
    // the lanes of a warp stay together in the sums' shuffles: done when all are
    while (__any_sync(0xFFFFFFFFu, cur.t < order.T)) {
        fetch(stage == 0 ? kRopeDepth - 1 : stage - 1);
        const bool live = cur.t < order.T;
        const int h0 = cur.c * p.HC + cur.hc, h1 = live ? min(r.heads, cur.c * p.HC + p.HC) : 0;
        if (cur.hc == 0 && p.turn.rot > 0 && live) {
            const int64_t pos = ld_index(p.turn.pos, cur.t, p.turn.pos64);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float cs[E], sn[E];
                rope_angles<E>(fractions, pair[v], slot[v].turns, pos, p.turn.amp, -1.f, cs, sn);
                map[v].make(cs, sn, one, one, slot[v].turns);
            }
        }
        float rsv[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            rsv[u] = h0 + u < h1 && norm && p.rstd != nullptr
                         ? __ldg(p.rstd + (int64_t)cur.t * heads_all + head0 + h0 + u) : 0.f;
        if constexpr (E > 1)
            copies_wait<kRopeDepth - 1>();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (cur.hc + u >= p.HC)
                break;
            const int h = h0 + u;
            const bool on = h < h1;
            Vals<E> a[V], b[V], fa[V], fb[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                P ya = P::zero(), yb = P::zero(), xa = P::zero(), xb = P::zero();
                if constexpr (E > 1) {
                    if (on && slot[0].a < np) {
                        ya = ring.get(stage, 4 * u);
                        if (norm)
                            xa = ring.get(stage, 4 * u + 2);
                    }
                    if (on && slot[0].b < np) {
                        yb = ring.get(stage, 4 * u + 1);
                        if (norm)
                            xb = ring.get(stage, 4 * u + 3);
                    }
                } else if (on) {
                    const char *y = static_cast<const char *>(r.dy) + ((int64_t)cur.t * r.yt + h * r.yh) * (int64_t)sizeof(T);
                    const char *x = static_cast<const char *>(r.x) + ((int64_t)cur.t * r.xt + h * r.xh) * (int64_t)sizeof(T);
                    if (slot[v].a < np) {
                        ya = P::load(y, slot[v].a);
                        if (norm)
                            xa = P::load(x, slot[v].a);
                    }
                    if (slot[v].b < np) {
                        yb = P::load(y, slot[v].b);
                        if (norm)
                            xb = P::load(x, slot[v].b);
                    }
                }
                ya.widen(a[v]);
                yb.widen(b[v]);
                xa.widen(fa[v]);
                xb.widen(fb[v]);
                if (p.turn.rot > 0)
                    map[v].apply(a[v], b[v], slot[v].turns);
            }
            if (norm) {
                F ss = splat<F>(0.f), sc = splat<F>(0.f);
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < Vals<E>::N; ++i) {
                        sc = vfma(vmul(a[v].v[i], fa[v].v[i]), wa[v].v[i], sc);
                        sc = vfma(vmul(b[v].v[i], fb[v].v[i]), wb[v].v[i], sc);
                        if (p.rstd == nullptr)
                            ss = vfma(fb[v].v[i], fb[v].v[i], vfma(fa[v].v[i], fa[v].v[i], ss));
                    }
                float rs = rsv[u];
                if (p.rstd == nullptr)
                    rs = rsqrtf(fmaf(lanes_sum(hsum(ss), p.shift), p.inv_d, p.eps));
                if (!on)
                    rs = 0.f;                            // no row: nothing to add
                // (rstd c first: rstd cubed alone leaves fp32's range for rows of 1e-13 or 1e15)
                const float k = -(rs * (lanes_sum(hsum(sc), p.shift) * p.inv_d)) * rs * rs;
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < Vals<E>::N; ++i) {
                        a[v].v[i] = vmul(a[v].v[i], splat<F>(rs));
                        b[v].v[i] = vmul(b[v].v[i], splat<F>(rs));
                        da[v].v[i] = vfma(a[v].v[i], fa[v].v[i], da[v].v[i]);
                        db[v].v[i] = vfma(b[v].v[i], fb[v].v[i], db[v].v[i]);
                        a[v].v[i] = vfma(a[v].v[i], wa[v].v[i], vmul(fa[v].v[i], splat<F>(k)));
                        b[v].v[i] = vfma(b[v].v[i], wb[v].v[i], vmul(fb[v].v[i], splat<F>(k)));
                    }
            }
            if (on) {
                char *d = static_cast<char *>(r.dx) + ((int64_t)cur.t * r.dt + h * r.dh) * (int64_t)sizeof(T);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (slot[v].a < np)
                        P::narrow(a[v]).store(d, slot[v].a);
                    if (slot[v].b < np)
                        P::narrow(b[v]).store(d, slot[v].b);
                }
            }
        }
        stage = stage + 1 == kRopeDepth ? 0 : stage + 1;
        cur.next(order, U, p.HC);
    }
    if (!norm)
        return;
    // the ring is empty: its place holds the groups' sums
    float *sums = reinterpret_cast<float *>(smem + kRopeFractions);
    if constexpr (E > 1)
        copies_wait<0>();
    __syncthreads();
    const int grp = threadIdx.x >> p.shift, groups = kRopeThreads >> p.shift;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (slot[v].a < np)
                sums[grp * p.D + slot[v].a * E + e] = da[v].get(e);
            if (slot[v].b < np)
                sums[grp * p.D + slot[v].b * E + e] = db[v].get(e);
        }
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kRopeThreads) {
        float s = 0.f;
        for (int g = 0; g < groups; ++g)
            s += sums[g * p.D + d];
        p.partial[(int64_t)blockIdx.x * p.D + d] = s;
    }
}

} // namespace rmsk
