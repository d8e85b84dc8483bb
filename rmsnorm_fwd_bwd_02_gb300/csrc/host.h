// host.h -- what the library's entry points share on the host: the state
// behind rmsnorm_last_cuda_error / rmsnorm_last_path and the test hooks,
// argument checks, device properties and the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <map>
#include <mutex>
#include <tuple>

#include "rmsnorm.h"
#include "context.h"

namespace rmsk {

inline thread_local int t_last_cuda_error = 0;
inline thread_local int t_last_path = 0;
// Test hook for the kernels' bounded waits (see rmsnorm.h).
inline std::atomic<unsigned> g_test_extra_tx{0}, g_test_wait_us{0};

inline int cuda_fail(cudaError_t e)
{
    t_last_cuda_error = (int)e;
    return RMSNORM_ERR_CUDA;
}

inline size_t elem_size(int dtype) { return dtype == RMSNORM_F32 ? 4 : 2; }

inline bool aligned(const void *p, size_t a) { return p == nullptr || (uintptr_t)p % a == 0; }

// A tensor argument as the bytes it touches: `rows` rows of `row_bytes`
// bytes whose starts are `ld_bytes` apart (a flat buffer is one row).
struct Span {
    const void *p;
    int64_t rows, row_bytes, ld_bytes;
    bool empty() const { return p == nullptr || rows <= 0 || row_bytes <= 0; }
    uintptr_t begin() const { return (uintptr_t)p; }
    uintptr_t end() const { return (uintptr_t)p + (rows - 1) * ld_bytes + row_bytes; }
};

inline Span flat(const void *p, size_t n) { return {p, 1, (int64_t)n, (int64_t)n}; }

inline Span rows_span(const void *p, int64_t M, int64_t H, int64_t ld, size_t es)
{
    return {p, M, H * (int64_t)es, ld * (int64_t)es};
}

// Whether two arguments may share a byte. Exact for disjoint address
// ranges and for row windows of one stride that never meet (the rows of b
// fall, modulo the stride, after the end of a's rows and before the next
// row of a starts); any other pair whose ranges intersect counts as
// overlapping.
inline bool overlap(Span a, Span b)
{
    if (a.empty() || b.empty())
        return false;
    if (!(a.begin() < b.end() && b.begin() < a.end()))
        return false;
    if (a.ld_bytes == b.ld_bytes && a.ld_bytes > 0) {
        const int64_t ld = a.ld_bytes;
        const int64_t d = (int64_t)(b.begin() - a.begin());
        const int64_t s = ((d % ld) + ld) % ld;   // b's row offset within a's row frame
        if (s >= a.row_bytes && s + b.row_bytes <= ld)
            return false;
    }
    return true;
}

inline bool same(Span a, Span b)
{
    return a.p == b.p && a.rows == b.rows && a.row_bytes == b.row_bytes &&
           (a.rows == 1 || a.ld_bytes == b.ld_bytes);
}

// Allowed: the same tensor exactly (same start, shape and stride), or no
// shared byte at all.
inline bool same_or_disjoint(Span a, Span b) { return same(a, b) || !overlap(a, b); }

inline int check_common(int64_t M, int64_t H, float eps, int dtype)
{
    if (dtype != RMSNORM_F32 && dtype != RMSNORM_BF16 && dtype != RMSNORM_F16)
        return RMSNORM_ERR_BAD_DTYPE;
    if (M < 0 || H < 1)
        return RMSNORM_ERR_BAD_SHAPE;
    if (H > RMSNORM_MAX_H)
        return RMSNORM_ERR_UNSUPPORTED;
    if (M > INT64_MAX / 8 / H)
        return RMSNORM_ERR_BAD_SHAPE;
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return RMSNORM_ERR_BAD_EPS;
    return RMSNORM_OK;
}

// A row stride is at least H and below 2^31 (the row kernels hold strides in
// 32 bits), and the tensor's last byte stays far below 2^63 (so every byte
// offset the kernels form fits an int64).
inline bool stride_ok(int64_t ld, int64_t M, int64_t H)
{
    if (ld < H || ld > INT32_MAX)
        return false;
    return M <= 1 || ld <= (INT64_MAX / 8 - H) / (M - 1);
}

// Row strides (elements) whose byte size is a multiple of `a`.
inline bool strides_multiple(size_t a, size_t es, std::initializer_list<int64_t> lds)
{
    for (int64_t ld : lds)
        if ((ld * (int64_t)es) % (int64_t)a != 0)
            return false;
    return true;
}

// ------------------------------------------------------- device properties
inline int current_device(int *dev)
{
    cudaError_t e = cudaGetDevice(dev);
    return e == cudaSuccess ? RMSNORM_OK : cuda_fail(e);
}

inline int sm_count(int dev, int *sms)
{
    cudaError_t e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return e == cudaSuccess ? RMSNORM_OK : cuda_fail(e);
}

// Resident CTAs per SM for a kernel launched with `smem` bytes of dynamic
// shared memory, cached per (kernel, device, smem). A kernel that needs more
// than the default 48 KB is opted in to the device's maximum (not to this
// size: a later call with more shared memory must still launch).
// Entries hold for the context they were made in (context.h).
inline int blocks_per_sm(const void *fn, int threads, int dev, int *out, int smem = 0)
{
    static std::mutex mu;
    static std::map<std::tuple<const void *, int, int, unsigned long long>, int> cache;
    const unsigned long long ctx = current_context_id();
    if (ctx != 0) {
        std::lock_guard<std::mutex> g(mu);
        auto it = cache.find(std::make_tuple(fn, dev, smem, ctx));
        if (it != cache.end()) {
            *out = it->second;
            return RMSNORM_OK;
        }
    }
    int n = 0;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) {
        // the device's per-CTA maximum less the kernel's static shared memory
        int most = 0;
        cudaFuncAttributes fa;
        e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (e == cudaSuccess)
            e = cudaFuncGetAttributes(&fa, fn);
        if (e == cudaSuccess) {
            most -= (int)fa.sharedSizeBytes;
            if (smem > most)
                return cuda_fail(cudaErrorInvalidValue);
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        }
    }
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem);
    if (e != cudaSuccess)
        return cuda_fail(e);
    if (n < 1)
        return cuda_fail(cudaErrorInvalidConfiguration);
    // the context the attribute was set in (the calls above create the
    // primary context if none was current)
    const unsigned long long made_in = current_context_id();
    if (made_in != 0) {
        std::lock_guard<std::mutex> g(mu);
        cache[std::make_tuple(fn, dev, smem, made_in)] = n;
    }
    *out = n;
    return RMSNORM_OK;
}

// Clusters of `cs` CTAs of `fn` that can be resident at once on device
// `dev` (a cluster must fit within one GPC, so fewer CTAs than SMs x
// blocks_per_sm may run together).
inline int max_active_clusters(const void *fn, int threads, int smem, int cs, int dev, int *out)
{
    static std::mutex mu;
    static std::map<std::tuple<const void *, int, int, int, unsigned long long>, int> cache;
    const unsigned long long ctx = current_context_id();
    if (ctx != 0) {
        std::lock_guard<std::mutex> g(mu);
        auto it = cache.find(std::make_tuple(fn, dev, smem, cs, ctx));
        if (it != cache.end()) {
            *out = it->second;
            return RMSNORM_OK;
        }
    }
    int bps;
    int st = blocks_per_sm(fn, threads, dev, &bps, smem);     // sets the smem limit
    if (st)
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cs);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = (unsigned)cs;
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
    if (e != cudaSuccess)
        return cuda_fail(e);
    if (n < 1)
        return cuda_fail(cudaErrorInvalidConfiguration);
    const unsigned long long made_in = current_context_id();
    if (made_in != 0) {
        std::lock_guard<std::mutex> g(mu);
        cache[std::make_tuple(fn, dev, smem, cs, made_in)] = n;
    }
    *out = n;
    return RMSNORM_OK;
}

// ------------------------------------------------------------ tensor maps
// cuTensorMapEncodeTiled, from the driver through the runtime's entry-point
// query (the library does not link the driver library itself); nullptr if
// the driver does not offer it.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

} // namespace rmsk
