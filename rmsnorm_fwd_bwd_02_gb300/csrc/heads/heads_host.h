// heads_host.h -- argument checks and launches that the entry points on
// attention heads share on the host.
#pragma once

#include <algorithm>

#include "../host.h"
#include "heads.h"

namespace rmsk {

// Whether rows of D elements at n[i] steps of ld[i] in each of three
// directions lie apart from each other and end within 2^60 elements.
inline bool rows_apart(const int64_t (&n)[3], const int64_t (&ld)[3], int64_t D)
{
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return ld[a] < ld[b]; });
    __int128 need = D;
    for (int i : order)
        if (n[i] > 1) {
            if (ld[i] < need)
                return false;
            need += (__int128)(n[i] - 1) * ld[i];
        }
    return need <= ((__int128)1 << 60);
}

// The same for inputs, which may overlap themselves (strides of 0).
inline bool rows_within(const int64_t (&n)[3], const int64_t (&ld)[3], int64_t D)
{
    __int128 need = D;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1) {
            if (ld[i] < 0)
                return false;
            need += (__int128)(n[i] - 1) * ld[i];
        }
    return need <= ((__int128)1 << 60);
}

// Heads [T, heads, D] as the bytes they touch: rows of tokens where a token's
// heads lie together, rows of heads where a head's tokens do, else all between
// the first and the last.
inline Span heads_span(const void *p, int64_t T, int64_t heads, int64_t D, int64_t xt, int64_t xh, size_t es)
{
    const int64_t e = (int64_t)es;
    if (p == nullptr || T < 1 || heads < 1)
        return {nullptr, 0, 0, 0};
    if (T == 1)
        return {p, 1, ((heads - 1) * xh + D) * e, ((heads - 1) * xh + D) * e};
    if (heads == 1 || xt >= (heads - 1) * xh + D)
        return {p, T, (heads == 1 ? D : (heads - 1) * xh + D) * e, xt * e};
    if (xh >= (T - 1) * xt + D)
        return {p, heads, ((T - 1) * xt + D) * e, xh * e};
    const int64_t all = ((T - 1) * xt + (heads - 1) * xh + D) * e;
    return {p, 1, all, all};
}

// Whether rows of heads in y may go with those in x: the same rows exactly, or no
// byte in common. The spans do not say which of their directions the tokens are:
// of as many tokens as heads, a buffer and its transpose have equal ones.
inline bool heads_same_or_disjoint(Span y, int64_t yt, int64_t yh, Span x, int64_t xt, int64_t xh, int64_t T,
                                   int64_t heads)
{
    const bool rows = y.p == x.p && (T <= 1 || yt == xt) && (heads <= 1 || yh == xh);
    return rows || !overlap(y, x);
}

inline bool dtype_ok(int dtype)
{
    return dtype == RMSNORM_F32 || dtype == RMSNORM_BF16 || dtype == RMSNORM_F16;
}

inline bool index_bits_ok(int bits) { return bits == 32 || bits == 64; }

// A launch that may begin while the kernel before it ends, of clusters of
// `cluster` CTAs.
inline cudaError_t launch_pdl(const void *fn, dim3 grid, int threads, size_t smem, cudaStream_t s, void **args,
                              int cluster = 1)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

} // namespace rmsk
