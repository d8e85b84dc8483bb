// fp8_rows.cuh -- rows rounded to 8-bit floating point with one fp32 scale
// for every 128 columns: of the RMSNorm's output, of the norm of a residual
// sum, or of a matrix as it is; and the same for blocks of 128 x 128.
//
// Mathematics. For a row v (x, or h = round(x + r)) of H features
//   y_j = v_j rstd w_j,   rstd = 1 / sqrt(mean(v^2) + eps)       (fp32)
// and for each group g of 128 columns, with F the format's largest finite
// value (448 for e4m3, 57344 for e5m2),
//   a_g = max |y_j| over the group,  s_g = max(a_g, 2^-100) / F,
//   q_j = y_j / s_g rounded to nearest even.
// y is not rounded to the input's type on the way: the 8-bit rounding (2^-4
// of the value in e4m3) is the only one, where the norm followed by a
// quantisation would add one of 2^-9 (bf16) whose ties it would inherit. The
// floor on a_g keeps s_g and its reciprocal normal fp32 numbers; below it
// values flush towards zero. A group that holds a NaN or an infinity has no
// scale: its scale and all of its q are NaN, so that what is computed from
// it shows it.
// s_g is that quotient, rounded once. q_j is formed as y_j (1 / s_g) with an
// approximate reciprocal (1 ulp, 2^-23 of it at most) and a product rounded in
// fp32 (2^-24): together within 2^-22 of the quotient, which can turn one that
// lies so near the middle between two 8-bit values to the other neighbour, and
// nothing else. (A division rounded in fp32 does the same within 2^-24: of
// rows of bf16 values, whose quotients meet such middles often, 1.3 in 1000
// elements come out otherwise than from the exact quotient, and 1.1 here.)
//
// What bounds it: DRAM. The plain norm reads 2 bytes and writes 1 an element
// (bf16), with the residual it reads 4 and writes 3; the arithmetic is some
// 6 operations an element against the 16 that an SM has time for.
//
// Layout: that of the row kernels (rows.cuh). Lane l of a row's L lanes owns
// the packs l, l + L, ...; a row stays in registers from load to store, so x
// is read once. 32-byte packs put 16 (16-bit types) or 8 (fp32) elements in a
// lane, so a group of 128 columns is 8 or 16 neighbouring lanes and its
// maximum takes 3 or 4 shuffles; the q of a lane is one 16- or 8-byte store.
// Rows that may start at any address ("loose" packs, 16 bytes) are read as
// the four-byte words that hold them, and h is written so, shifted into place
// in registers.
//
// What it took (GB300, bf16, dispatch as in fp8_api.cu): the reduction, the
// group maxima and the conversion form one chain per row, so a CTA that
// loads a row only when it has stored the one before leaves DRAM idle.
// Asking for the next row before working on this one (AHEAD) takes the norm
// at 32768 x 4096 from 71 to 62.5 us (two packs a lane, w read again from L1
// for each row instead of held: 80 registers, six CTAs an SM). With the
// residual there are twice the loads in flight for the same chain and the
// registers are worth more as occupancy: 88 us without AHEAD at 16384 x 5120,
// 100 with it.
#pragma once

#include <cuda_fp8.h>

#include "../common.cuh"
#include "fp8.h"

namespace rmsk {

constexpr int kFp8ModeQuant = 0, kFp8ModeNorm = 1, kFp8ModeResidual = 2;

constexpr float kFp8AmaxMin = 0x1p-100f;

// max(a, |b|) that keeps a NaN of either
__device__ __forceinline__ float amax_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// The scale of a group whose largest magnitude is `amax`, and the factor
// that takes its values to 8 bits. Both NaN when amax is not finite.
struct Fp8Scale {
    float s, inv;
    __device__ __forceinline__ Fp8Scale(float amax, int e5m2)
    {
        // m / F, correctly rounded. Both F are 448 times a power of two, and the
        // quotient by the constant 448 is the product with its rounded
        // reciprocal c, corrected once by its remainder (N. Brisebarre, J.-M.
        // Muller, S. K. Raina, "Accelerating correctly rounded floating-point
        // division when the divisor is known in advance", IEEE Trans. Computers
        // 53, 2004; right for each of the 2^23 significands, and from 2^-100 on
        // no step underflows). It takes 0.2 % over widths of 128 to 16384 (1.8 at
        // most) beside a plain product with c; a general division takes the norm
        // at 262144 x 896 from 114 to 124 us.
        constexpr float c = 1.f / 448.f;
        const float m = fmaxf(amax, kFp8AmaxMin), t = m * c;
        s = __fmaf_rn(__fmaf_rn(-448.f, t, m), c, t) * (e5m2 ? 0x1p-7f : 1.f);
        if (!(amax < __int_as_float(0x7f800000)))
            s = __int_as_float(0x7fffffff);
        // s is a normal number with a normal reciprocal (or NaN)
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    }
};

// Two values to 8 bits, the lower address in the low byte; magnitudes past
// the largest (by the rounding of `inv` alone) become the largest.
__device__ __forceinline__ uint32_t fp8_pair(float lo, float hi, int e5m2)
{
    const float2 v = make_float2(lo, hi);
    return e5m2 ? __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E5M2)
                : __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

// A 16-byte pack of a row that may start at any address ("loose"), as the
// four-byte words that hold it: five where elements of two bytes may start
// inside a word, read through L1, where the lanes of a warp share the lines.
// No word without a byte of the row is touched. (Aligned 16-byte words, the
// neighbour's by shuffles, take a load where this takes five, but some 25
// instructions more to put the bytes in their places: the norm at 8590 x 5597,
// 46 us, took some 18 us longer.)
template <typename T> struct LooseRaw {
    static constexpr int E = 16 / (int)sizeof(T), NW = sizeof(T) == 2 ? 5 : 4;
    uint32_t w[NW];
    __device__ __forceinline__ static LooseRaw zero()
    {
        LooseRaw r;
#pragma unroll
        for (int i = 0; i < NW; ++i)
            r.w[i] = 0;
        return r;
    }
    // The words of pack vi of a row of H elements, zero where they hold none.
    __device__ __forceinline__ static LooseRaw load(const void *row, int vi, int H)
    {
        const char *p = static_cast<const char *>(row) + (int64_t)vi * 16;
        const int m = (int)((uintptr_t)row & 3), n = (H - vi * E) * (int)sizeof(T) + m;
        LooseRaw r = zero();
#pragma unroll
        for (int i = 0; i < NW; ++i)
            if (4 * i < n && (i < 4 || m != 0))
                asm volatile("ld.global.b32 %0, [%1];" : "=r"(r.w[i]) : "l"(p - m + 4 * i));
        return r;
    }
    // The pack, zero past the row's end.
    __device__ __forceinline__ uint4 pack(const void *row, int vi, int H) const
    {
        uint32_t o[4];
        if constexpr (sizeof(T) == 2) {
            const uint32_t sh = ((uint32_t)(uintptr_t)row & 2u) * 8u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = __funnelshift_r(w[i], w[i + 1], sh);
            const int n = H - vi * E;
            if (n < E) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = n <= 2 * i ? 0u : n == 2 * i + 1 ? o[i] & 0xFFFFu : o[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = w[i];
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
};

// Pack vi of a row that may start at any address, written as four-byte words.
// Where elements of two bytes start inside a word, the first word is the end
// of the pack before (the lane before has it) and the beginning of this one;
// the first lane of a warp (or of a row's lanes) then writes its half alone,
// the last also its pack's last element. Every lane of the warp takes part;
// ok: the row exists.
template <typename T>
__device__ __forceinline__ void store_loose(void *row, int vi, int H, uint4 u, bool ok, bool first,
                                            bool last)
{
    char *p = static_cast<char *>(row) + (int64_t)vi * 16;
    if constexpr (sizeof(T) == 4) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (ok && vi * 4 + i < H)
                st_row_b32(p + 4 * i, w[i]);
    } else {
        const uint32_t before = __shfl_up_sync(0xFFFFFFFFu, u.w, 1);
        const int n = ok ? H - vi * 8 : -1;         // elements of the row from here on
        const uint32_t odd = (uint32_t)(uintptr_t)row & 2u;
        const uint32_t w[5] = {before, u.x, u.y, u.z, u.w};
        // word i holds elements 2 i - 1 and 2 i of the pack (odd) or 2 i and
        // 2 i + 1
        const uint32_t sh = odd ? 16u : 0u;
        const int in = n + (odd ? 1 : 0);           // whole word i: 2 i + 2 <= in
        p -= odd;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = odd ? __funnelshift_r(w[i], w[i + 1], sh) : w[i + 1];
            if (2 * i + 2 <= in && !(i == 0 && odd && first))
                st_row_b32(p + 4 * i, v);
            else if (2 * i + 1 == in && !(i == 0 && odd && (first || n <= 0)))
                st_row_b16(p + 4 * i, (uint16_t)(v & 0xFFFFu));     // the row's last element
        }
        if (odd && n >= 1 && first)
            st_row_b16(p + 2, (uint16_t)(u.x & 0xFFFFu));
        if (odd && n >= 8 && (last || n == 8))
            st_row_b16(p + 16, (uint16_t)(u.w >> 16));
    }
}

// What a load leaves in registers; the load of pack vi of the row that is
// `row` rows of `ld` elements from base, and its pack.
template <typename T, int E, bool LOOSE>
using Fp8Raw = typename std::conditional<LOOSE, LooseRaw<T>, Pack<T, E>>::type;

template <typename T, int E, bool LOOSE>
__device__ __forceinline__ Fp8Raw<T, E, LOOSE> fp8_load(const void *base, int64_t row, uint32_t ld,
                                                        int vi, int H)
{
    if constexpr (LOOSE)
        return LooseRaw<T>::load(static_cast<const T *>(base) + row * ld, vi, H);
    else
        return vi * E < H ? Pack<T, E>::load(base, row * (ld / E) + vi) : Pack<T, E>::zero();
}

template <typename T, int E, bool LOOSE>
__device__ __forceinline__ Pack<T, E> fp8_pack(const Fp8Raw<T, E, LOOSE> &r, const void *base,
                                               int64_t row, uint32_t ld, int vi, int H)
{
    if constexpr (LOOSE) {
        Pack<T, E> p;
        p.u = r.pack(static_cast<const T *>(base) + row * ld, vi, H);
        return p;
    } else {
        return r;
    }
}

// The E values of pack vi of a row, times inv, as bytes at qrow + vi E. With
// LOOSE those past H are left out, and the bytes go out as one word only
// where they may (`whole`: the row starts at a multiple of E bytes).
template <int E, bool LOOSE>
__device__ __forceinline__ void fp8_store(char *qrow, int vi, int H, bool whole, const Vals<E> &y,
                                          float inv, int e5m2)
{
    char *q = qrow + (int64_t)vi * E;
    uint32_t u[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        const float2 a = vmul(y.v[2 * i], splat<float2>(inv));
        const float2 b = vmul(y.v[2 * i + 1], splat<float2>(inv));
        u[i] = fp8_pair(a.x, a.y, e5m2) | (fp8_pair(b.x, b.y, e5m2) << 16);
    }
    if (LOOSE && !(whole && vi * E + E <= H)) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (vi * E + i < H)
                asm volatile("st.global.b8 [%0], %1;" ::"l"(q + i),
                             "r"((u[i / 4] >> (8 * (i % 4))) & 0xFFu)
                             : "memory");
    } else if constexpr (E == 16) {
        st_row_v4(q, make_uint4(u[0], u[1], u[2], u[3]));
    } else if constexpr (E == 8) {
        asm volatile("st.global.v2.b32 [%0], {%1,%2};" ::"l"(q), "r"(u[0]), "r"(u[1]) : "memory");
    } else {
        st_row_b32(q, u[0]);
    }
}

// Largest magnitude of a pack's values, a NaN kept; two values a step (the
// sm_100 family's maximum takes three operands).
template <int E>
__device__ __forceinline__ float pack_amax(const Vals<E> &y)
{
    float a = 0.f;
#pragma unroll
    for (int e = 0; e < E / 2; ++e)
        asm("max.NaN.f32 %0, %1, %2, %3;"
            : "=f"(a)
            : "f"(a), "f"(fabsf(y.v[e].x)), "f"(fabsf(y.v[e].y)));
    return a;
}

// The maximum over groups of N neighbouring lanes.
template <int N>
__device__ __forceinline__ float lanes_amax(float a)
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1)
        a = amax_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    return a;
}

// E: elements a pack; V: packs a lane; LR: lanes a row when several rows
// share a warp, or 0: the whole CTA (whole warps, as many as the host picks)
// takes a row; AHEAD: the next row's loads are issued before this one is
// worked on; HOLD: w stays in registers; LOOSE: as above. Grid: persistent.
template <typename T, int E, int V, int LR, int MAXT, int MINB, int MODE, bool AHEAD, bool HOLD,
          bool LOOSE>
__global__ void __launch_bounds__(MAXT, MINB)
rms_fp8_rows(const Fp8RowsParams prm)
{
    Fp8RowsParams p = prm;
    if constexpr (MODE == kFp8ModeQuant) {
        // rows wider than a CTA holds: a window of columns to a block in y
        // (the groups do not depend on one another)
        const int c0 = (int)blockIdx.y * kFp8Window;
        p.x = static_cast<const T *>(p.x) + c0;
        p.q = static_cast<char *>(p.q) + c0;
        p.scale += c0 / kFp8Group;
        p.H = min(p.H - c0, kFp8Window);
    }
    using P = Pack<T, E>;
    using R = Fp8Raw<T, E, LOOSE>;
    using X = Vals<E>;
    constexpr bool NORM = MODE != kFp8ModeQuant, RES = MODE == kFp8ModeResidual;
    constexpr bool TREE = RES && !LOOSE, FOURS = !TREE && MAXT > 160;
    constexpr int LG = kFp8Group / E;               // lanes in one group of columns
    static_assert(LG <= 32 && (LR == 0 || LR % LG == 0), "lanes of a group");
    static_assert(!LOOSE || E * sizeof(T) == 16, "loose packs are 16 bytes");
    __shared__ __align__(16) float red[2][32];

    const int L = LR ? LR : (int)blockDim.x;
    const int lane = LR ? (int)threadIdx.x % LR : (int)threadIdx.x;
    const int sub = LR ? (int)threadIdx.x / LR : 0;
    const int S = LR ? (int)blockDim.x / LR : 1;    // rows of the CTA at a time
    const int NV = (p.H + E - 1) / E;               // packs a row (E divides H unless LOOSE)
    const float fH = (float)p.H;
    const uint32_t ldx = (uint32_t)p.ldx, ldr = (uint32_t)p.ldr, ldh = (uint32_t)p.ldh;
    const bool whole = LOOSE && ((uintptr_t)p.q % E == 0) && p.ldq % E == 0;

    auto load = [&](const void *base, uint32_t ld, int64_t row, R (&to)[V]) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int vi = lane + k * L;
            to[k] = row < p.M ? fp8_load<T, E, LOOSE>(base, row, ld, vi, p.H) : R::zero();
        }
    };
    const bool first = lane % (LR ? LR : 32) == 0, last = lane % (LR ? LR : 32) == (LR ? LR : 32) - 1;
    auto pack = [&](const R &r, const void *base, uint32_t ld, int64_t row, int k) {
        return fp8_pack<T, E, LOOSE>(r, base, row, ld, lane + k * L, p.H);
    };
    auto load_w = [&](int vi) {
        if (vi >= NV)
            return P::zero();
        if constexpr (LOOSE) {
            P w;
            w.u = LooseRaw<T>::load(p.w, vi, p.H).pack(p.w, vi, p.H);
            return w;
        } else {
            return P::load_cached(p.w, vi);
        }
    };

    if constexpr (NORM && LR == 0 && FOURS) {       // the sums that no warp writes
        if (threadIdx.x < 32)
            red[0][threadIdx.x] = red[1][threadIdx.x] = 0.f;
        __syncthreads();
    }
    griddep_wait();
    constexpr bool kHold = NORM && HOLD;
    P wv[kHold ? V : 1];
    if constexpr (kHold) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            wv[k] = load_w(lane + k * L);
    }

    const int64_t ntiles = (p.M + S - 1) / S;
    int buf = 0;
    R xn[AHEAD ? V : 1], rn[AHEAD && RES ? V : 1];
    if constexpr (AHEAD) {
        const int64_t row = (int64_t)blockIdx.x * S + sub;
        load(p.x, ldx, row, xn);
        if constexpr (RES)
            load(p.r, ldr, row, rn);
    }
    for (int64_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
        const int64_t row = t * S + sub;
        P xv[V];
        R rv[RES ? V : 1];
        if constexpr (AHEAD) {
            // this row was asked for a tile ago; now the next one
#pragma unroll
            for (int k = 0; k < V; ++k) {
                xv[k] = pack(xn[k], p.x, ldx, row, k);
                if constexpr (RES)
                    rv[k] = rn[k];
            }
            const int64_t next = row + (int64_t)gridDim.x * S;
            load(p.x, ldx, next, xn);
            if constexpr (RES)
                load(p.r, ldr, next, rn);
        } else {
            R xr[V];
            load(p.x, ldx, row, xr);
            if constexpr (RES)
                load(p.r, ldr, row, rv);
#pragma unroll
            for (int k = 0; k < V; ++k)
                xv[k] = pack(xr[k], p.x, ldx, row, k);
        }
        if constexpr (RES) {
            // the stored h is what the norm sees
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int vi = lane + k * L;
                X a, b;
                xv[k].widen(a);
                pack(rv[k], p.r, ldr, row, k).widen(b);
#pragma unroll
                for (int i = 0; i < X::N; ++i)
                    a.v[i] = vadd(a.v[i], b.v[i]);
                xv[k] = P::narrow(a);
                if constexpr (LOOSE)
                    store_loose<T>(static_cast<T *>(p.h) + row * ldh, vi, p.H, xv[k].u, row < p.M,
                                   first, last);
                else if (row < p.M && vi < NV)
                    xv[k].store(p.h, row * (ldh / E) + vi);
            }
        }

        float rs = 1.f;
        if constexpr (NORM) {
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                X a;
                xv[k].widen(a);
#pragma unroll
                for (int i = 0; i < X::N; ++i)
                    acc = vfma(a.v[i], a.v[i], acc);
            }
            float ss = group_allreduce<LR ? LR : 32>(hsum(acc));
            if constexpr (LR == 0) {                // the warps' sums, in a fixed order
                const int warp = threadIdx.x / 32, nw = blockDim.x / 32;
                if (nw > 1) {
                    if ((threadIdx.x & 31) == 0)
                        red[buf][warp] = ss;
                    __syncthreads();
                    // By a tree in every warp for whole packs with a residual,
                    // where few warps are there to hide the latency of a chain
                    // (32768 x 4096 bf16 146 us, 153 by the chain); else by a
                    // chain, over the sums of four warps where there may be
                    // many (8590 x 5597 46 us, 48 without the fours, 51 by the
                    // tree; at 32768 x 4096, four warps, 62 without, 64 with).
                    if constexpr (TREE) {
                        const int q = threadIdx.x & 31;
                        ss = group_allreduce<32>(q < nw ? red[buf][q] : 0.f);
                    } else if constexpr (FOURS) {
                        ss = 0.f;
#pragma unroll 1
                        for (int q = 0; q < nw; q += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(&red[buf][q]);
                            ss += (f.x + f.y) + (f.z + f.w);
                        }
                    } else {
                        ss = 0.f;
                        for (int q = 0; q < nw; ++q)
                            ss += red[buf][q];
                    }
                    buf ^= 1;                       // read again only after the next barrier
                }
            }
            rs = rsqrtf(ss / fH + p.eps);
            if (p.rstd != nullptr && lane == 0 && row < p.M)
                p.rstd[row] = rs;
        }

#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int vi = lane + k * L;
            X y;
            xv[k].widen(y);
            if constexpr (NORM) {
                X w;
                if constexpr (kHold)
                    wv[k].widen(w);
                else
                    load_w(vi).widen(w);
#pragma unroll
                for (int i = 0; i < X::N; ++i)
                    y.v[i] = vmul(vmul(y.v[i], splat<float2>(rs)), w.v[i]);
            }
            if constexpr (NORM && LOOSE) {
                // columns past H do not count: with rs not finite their zeros
                // would be NaN
                if (vi * E + E > p.H) {
#pragma unroll
                    for (int i = 0; i < X::N; ++i) {
                        if (vi * E + 2 * i >= p.H)
                            y.v[i].x = 0.f;
                        if (vi * E + 2 * i + 1 >= p.H)
                            y.v[i].y = 0.f;
                    }
                }
            }
            float a = pack_amax<E>(y);
            if (NORM && vi >= NV)                   // nor do whole packs past H
                a = 0.f;
            a = lanes_amax<LG>(a);
            if (row < p.M && vi < NV) {
                const Fp8Scale sc(a, p.e5m2);
                if (lane % LG == 0)
                    p.scale[row * p.G + vi / LG] = sc.s;
                fp8_store<E, LOOSE>(static_cast<char *>(p.q) + row * p.ldq, vi, p.H, whole, y, sc.inv,
                                    p.e5m2);
            }
        }
    }
    griddep_launch_dependents();
}

// One CTA of 256 threads to a block of 128 x 128; grid (G, ceil(M / 128)). A
// thread holds 64 elements: a row of the block is LG lanes, so a pass of the
// CTA takes 256 / LG rows and all passes' loads are in flight at once. Bound
// by DRAM, with three CTAs an SM (80 registers a thread): 44.5 us, all of the
// copy bandwidth, at 24576 x 4096 bf16, where two take 51 us and four, which
// spill, 48. Loose fp32 packs need more registers: two CTAs (76 us at
// 25921 x 3195, where three take 98 and one, with all the registers that the
// compiler then uses, 118).
constexpr int kFp8BlockThreads = 256;

template <typename T, int E, bool LOOSE>
__global__ void __launch_bounds__(kFp8BlockThreads, LOOSE && sizeof(T) == 4 ? 2 : 3)
rms_fp8_blocks(const Fp8BlocksParams p)
{
    using P = Pack<T, E>;
    using R = Fp8Raw<T, E, LOOSE>;
    using X = Vals<E>;
    constexpr int LG = kFp8Group / E;
    constexpr int ROWS = kFp8BlockThreads / LG;     // rows a pass
    constexpr int NP = kFp8Group / ROWS;            // passes
    __shared__ float red[kFp8BlockThreads / 32];

    const int lane = threadIdx.x % LG, sub = threadIdx.x / LG;
    const int NV = (p.H + E - 1) / E;
    const uint32_t ldx = (uint32_t)p.ldx;
    const int vi = (int)blockIdx.x * LG + lane;
    const bool whole = LOOSE && ((uintptr_t)p.q % E == 0) && p.ldq % E == 0;

    griddep_wait();
    for (int64_t rb = blockIdx.y; rb * kFp8Group < p.M; rb += gridDim.y) {
        const int64_t row0 = rb * kFp8Group + sub;
        R xv[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int64_t row = row0 + i * ROWS;
            xv[i] = row < p.M ? fp8_load<T, E, LOOSE>(p.x, row, ldx, vi, p.H) : R::zero();
        }
        float a = 0.f;
        P xp[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int64_t row = row0 + i * ROWS;
            xp[i] = fp8_pack<T, E, LOOSE>(xv[i], p.x, row, ldx, vi, p.H);
            X y;
            xp[i].widen(y);
            a = amax_nan(a, pack_amax<E>(y));
        }
        a = lanes_amax<32>(a);
        if ((threadIdx.x & 31) == 0)
            red[threadIdx.x / 32] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kFp8BlockThreads / 32; ++w)
            a = amax_nan(a, red[w]);
        __syncthreads();                            // read before the next block's
        const Fp8Scale sc(a, p.e5m2);
        if (threadIdx.x == 0)
            p.scale[rb * p.G + blockIdx.x] = sc.s;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int64_t row = row0 + i * ROWS;
            X y;
            xp[i].widen(y);
            if (row < p.M && vi < NV)
                fp8_store<E, LOOSE>(static_cast<char *>(p.q) + row * p.ldq, vi, p.H, whole, y, sc.inv,
                                    p.e5m2);
        }
    }
    griddep_launch_dependents();
}

#define RMSK_FP8_ROWS(T, MODE, E, V, LR, MAXT, MINB, AHEAD, HOLD, LOOSE)                      \
    {(const void *)&rms_fp8_rows<T, E, V, LR, MAXT, MINB, MODE, AHEAD, HOLD, LOOSE>, E, V, LR, MAXT}

} // namespace rmsk
