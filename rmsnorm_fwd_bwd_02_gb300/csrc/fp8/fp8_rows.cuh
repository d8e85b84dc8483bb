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
// q_j is formed as y_j (1 / s_g): the reciprocal and the product are each
// rounded once in fp32 (2^-24), which can turn a quotient within 2^-22 of the
// middle between two 8-bit values to the other neighbour, and nothing else.
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
// Single elements (rows that start at any address) are dealt so that a group
// is four elements of each lane of one warp.
#pragma once

#include <cuda_fp8.h>

#include "../common.cuh"
#include "fp8.h"

namespace rmsk {

constexpr int kFp8ModeQuant = 0, kFp8ModeNorm = 1, kFp8ModeResidual = 2;

constexpr float kFp8AmaxMin = 0x1p-100f;

__device__ __forceinline__ float fp8_largest(int e5m2) { return e5m2 ? 57344.f : 448.f; }

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
        const float big = fp8_largest(e5m2);
        s = fmaxf(amax, kFp8AmaxMin) / big;
        if (!(amax < __int_as_float(0x7f800000)))
            s = __int_as_float(0x7fffffff);
        inv = 1.f / s;
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

// The E values of one pack, times inv, as E bytes at q.
template <int E>
__device__ __forceinline__ void fp8_store(void *q, const Vals<E> &y, float inv, int e5m2)
{
    if constexpr (E == 1) {
        const uint32_t b = fp8_pair(y.v[0] * inv, 0.f, e5m2);
        asm volatile("st.global.b8 [%0], %1;" ::"l"(q), "r"(b & 0xFFu) : "memory");
    } else {
        uint32_t u[E / 4];
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const float2 a = vmul(y.v[2 * i], splat<float2>(inv));
            const float2 b = vmul(y.v[2 * i + 1], splat<float2>(inv));
            u[i] = fp8_pair(a.x, a.y, e5m2) | (fp8_pair(b.x, b.y, e5m2) << 16);
        }
        if constexpr (E == 16)
            st_row_v4(q, make_uint4(u[0], u[1], u[2], u[3]));
        else if constexpr (E == 8)
            asm volatile("st.global.v2.b32 [%0], {%1,%2};" ::"l"(q), "r"(u[0]), "r"(u[1])
                         : "memory");
        else
            st_row_b32(q, u[0]);
    }
}

// Largest magnitude of a pack's values, a NaN kept.
template <int E>
__device__ __forceinline__ float pack_amax(const Vals<E> &y, float a)
{
#pragma unroll
    for (int e = 0; e < E; ++e)
        a = amax_nan(a, y.get(e));
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

// E: elements a pack; V: packs a lane; NG: rows a group of lanes takes at a
// time; LR: lanes a row when several rows share a warp, or 0: the whole CTA
// (whole warps, as many as the host picks) takes a row. Grid: persistent.
template <typename T, int E, int V, int NG, int LR, int MAXT, int MINB, int MODE>
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
    using X = Vals<E>;
    using F = typename X::F;
    constexpr bool NORM = MODE != kFp8ModeQuant, RES = MODE == kFp8ModeResidual;
    constexpr int KG = E == 1 ? 4 : 1;              // a lane's packs in one group of columns
    constexpr int LG = E == 1 ? 32 : kFp8Group / E; // lanes in one group of columns
    static_assert(V % KG == 0 && (LR == 0 || (LR % LG == 0 && E > 1)), "groups are whole lanes");
    __shared__ float red[2][32 * NG];

    const int L = LR ? LR : (int)blockDim.x;
    const int lane = LR ? (int)threadIdx.x % LR : (int)threadIdx.x;
    const int sub = LR ? (int)threadIdx.x / LR : 0;
    const int S = LR ? (int)blockDim.x / LR : 1;    // groups of lanes in the CTA
    const int NV = p.H / E;                         // packs a row (E divides H)
    const float fH = (float)p.H;
    const uint32_t sx = (uint32_t)p.ldx / E, sr = (uint32_t)p.ldr / E, sh = (uint32_t)p.ldh / E;
    auto index = [&](int k) {
        if constexpr (E == 1)
            return ((k >> 2) * L + (lane & ~31)) * 4 + (k & 3) * 32 + (lane & 31);
        else
            return lane + k * L;
    };

    griddep_wait();
    P wv[NORM && E > 1 ? V : 1];
    if constexpr (NORM && E > 1) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            wv[k] = index(k) < NV ? P::load_cached(p.w, index(k)) : P::zero();
    }

    const int64_t tile = (int64_t)S * NG;
    const int64_t ntiles = (p.M + tile - 1) / tile;
    int buf = 0;
    for (int64_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
        const int64_t row0 = t * tile + (int64_t)sub * NG;
        P xv[NG][V];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int vi = index(k);
                xv[g][k] = row0 + g < p.M && vi < NV ? P::load(p.x, (row0 + g) * sx + vi) : P::zero();
            }
        if constexpr (RES) {
            P rv[NG][V];
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int vi = index(k);
                    rv[g][k] =
                        row0 + g < p.M && vi < NV ? P::load(p.r, (row0 + g) * sr + vi) : P::zero();
                }
            // the stored h is what the norm sees
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int vi = index(k);
                    X a, b;
                    xv[g][k].widen(a);
                    rv[g][k].widen(b);
#pragma unroll
                    for (int i = 0; i < X::N; ++i)
                        a.v[i] = vadd(a.v[i], b.v[i]);
                    xv[g][k] = P::narrow(a);
                    if (row0 + g < p.M && vi < NV)
                        xv[g][k].store(p.h, (row0 + g) * sh + vi);
                }
        }

        float rs[NG];
        if constexpr (NORM) {
            float ss[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                F acc = splat<F>(0.f);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    X a;
                    xv[g][k].widen(a);
#pragma unroll
                    for (int i = 0; i < X::N; ++i)
                        acc = vfma(a.v[i], a.v[i], acc);
                }
                ss[g] = group_allreduce<LR ? LR : 32>(hsum(acc));
            }
            if constexpr (LR == 0) {                // the warps' sums, added in warp order
                const int warp = threadIdx.x / 32, nw = blockDim.x / 32;
                if (nw > 1) {
                    if ((threadIdx.x & 31) == 0) {
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            red[buf][warp * NG + g] = ss[g];
                    }
                    __syncthreads();
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        ss[g] = 0.f;
                        for (int q = 0; q < nw; ++q)
                            ss[g] += red[buf][q * NG + g];
                    }
                    buf ^= 1;                       // read again only after the next barrier
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                rs[g] = rsqrtf(ss[g] / fH + p.eps);
                if (p.rstd != nullptr && lane == 0 && row0 + g < p.M)
                    p.rstd[row0 + g] = rs[g];
            }
        }

#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int64_t row = row0 + g;
#pragma unroll
            for (int k0 = 0; k0 < V; k0 += KG) {
                X y[KG];
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < KG; ++j) {
                    xv[g][k0 + j].widen(y[j]);
                    if constexpr (NORM) {
                        X w;
                        if constexpr (E > 1)
                            wv[k0 + j].widen(w);
                        else if (index(k0 + j) < NV)
                            P::load_cached(p.w, index(k0 + j)).widen(w);
                        else
                            w = X::zero();
#pragma unroll
                        for (int i = 0; i < X::N; ++i)
                            y[j].v[i] = vmul(vmul(y[j].v[i], splat<F>(rs[g])), w.v[i]);
                    }
                    // columns past H do not count (a row of infinities times
                    // the padding's zero would)
                    if (index(k0 + j) < NV)
                        a = pack_amax<E>(y[j], a);
                }
                a = lanes_amax<LG>(a);
                const int v0 = index(k0);
                if (row < p.M && v0 < NV) {
                    const Fp8Scale sc(a, p.e5m2);
                    if (lane % LG == 0)
                        p.scale[row * p.G + (E == 1 ? v0 / kFp8Group : v0 / LG)] = sc.s;
                    char *qr = static_cast<char *>(p.q) + row * p.ldq;
#pragma unroll
                    for (int j = 0; j < KG; ++j)
                        if (index(k0 + j) < NV)
                            fp8_store<E>(qr + (int64_t)index(k0 + j) * E, y[j], sc.inv, p.e5m2);
                }
            }
        }
    }
    griddep_launch_dependents();
}

// One CTA of 256 threads to a block of 128 x 128; grid (G, ceil(M / 128)). A
// thread holds 64 elements: a row of the block is LG lanes, so a pass of the
// CTA takes 256 / LG rows and all passes' loads are in flight at once.
constexpr int kFp8BlockThreads = 256;

template <typename T, int E>
__global__ void __launch_bounds__(kFp8BlockThreads)
rms_fp8_blocks(const Fp8BlocksParams p)
{
    using P = Pack<T, E>;
    using X = Vals<E>;
    constexpr int KG = E == 1 ? 4 : 1;
    constexpr int LG = E == 1 ? 32 : kFp8Group / E;
    constexpr int ROWS = kFp8BlockThreads / LG;     // rows a pass
    constexpr int NP = kFp8Group / ROWS;            // passes
    __shared__ float red[kFp8BlockThreads / 32];

    const int lane = threadIdx.x % LG, sub = threadIdx.x / LG;
    const int NV = p.H / E;
    const uint32_t sx = (uint32_t)p.ldx / E;
    const int v0 = (int)blockIdx.x * (kFp8Group / E);
    auto index = [&](int j) { return v0 + lane + j * 32; };

    griddep_wait();
    for (int64_t rb = blockIdx.y; rb * kFp8Group < p.M; rb += gridDim.y) {
        const int64_t row0 = rb * kFp8Group + sub;
        P xv[NP][KG];
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < KG; ++j) {
                const int64_t row = row0 + i * ROWS;
                xv[i][j] = row < p.M && index(j) < NV ? P::load(p.x, row * sx + index(j)) : P::zero();
            }
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < KG; ++j) {
                X y;
                xv[i][j].widen(y);
                a = pack_amax<E>(y, a);
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
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < KG; ++j) {
                const int64_t row = row0 + i * ROWS;
                X y;
                xv[i][j].widen(y);
                if (row < p.M && index(j) < NV)
                    fp8_store<E>(static_cast<char *>(p.q) + row * p.ldq + (int64_t)index(j) * E, y,
                                 sc.inv, p.e5m2);
            }
    }
    griddep_launch_dependents();
}

// fn of one shape for the three modes
#define RMSK_FP8_ROWS(T, E, V, NG, LR, MAXT, MINB)                                          \
    {{(const void *)&rms_fp8_rows<T, E, V, NG, LR, MAXT, MINB, kFp8ModeQuant>,              \
      (const void *)&rms_fp8_rows<T, E, V, NG, LR, MAXT, MINB, kFp8ModeNorm>,               \
      (const void *)&rms_fp8_rows<T, E, V, NG, LR, MAXT, MINB, kFp8ModeResidual>},          \
     E, V, NG, LR, MAXT}

} // namespace rmsk
