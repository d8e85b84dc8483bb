// fp8_api.cu -- the 8-bit entry points of include/rmsnorm.h: host-side
// argument checks, kernel choice and launches. No allocation, no
// synchronisation, no host copies; everything is enqueued on the caller's
// stream.
#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

#include "../host.h"
#include "../registry.h"
#include "fp8.h"
#include "fp8_gemm.cuh"
#include "fp8_gemm_pair.cuh"
#include "fp8_registry.h"

using namespace rmsk;

namespace {

constexpr uint32_t kFp8MaxSmem = 227 * 1024, kFp8HalfSmem = 113 * 1024;
constexpr int kPathFp8Rows = 9, kPathFp8Blocks = 10, kPathFp8Gemm = 11,
              kPathFp8Pair = 12;

// Test hook: the product's kernel (see rmsnorm.h).
std::atomic<int> g_test_gemm_fp8{0};

bool fp8_type(int t) { return t == RMSNORM_E4M3 || t == RMSNORM_E5M2; }

const Fp8RowSet &fp8_set(int dtype)
{
    return dtype == RMSNORM_BF16 ? fp8_rows_bf16
                                 : (dtype == RMSNORM_F16 ? fp8_rows_f16 : fp8_rows_f32);
}

// The width of pack that the alignment of every row allows: 0 for `E0`
// elements, 1 for `E1` (es bytes an element, one in q; w and 32-byte packs
// are also read 16 bytes at a time), else 2, elements one at a time.
int pack_width(int E0, int E1, size_t es, int64_t H, const void *x, int64_t ldx, const void *r,
               int64_t ldr, const void *w, const void *q, int64_t ldq, const void *h, int64_t ldh)
{
    const int widths[2] = {E0, E1};
    for (int i = 0; i < 2; ++i) {
        const size_t E = (size_t)widths[i], a = E * es;
        if (H % widths[i] == 0 && aligned(x, a) && aligned(r, a) && aligned(h, a) &&
            aligned(w, 16) && aligned(q, E) && strides_multiple(a, es, {ldx, ldr, ldh}) &&
            strides_multiple(E, 1, {ldq}))
            return i;
    }
    return 2;
}

cudaError_t launch1(const void *fn, dim3 grid, int threads, cudaStream_t s, void *arg)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void *args[1] = {arg};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Resident CTAs per SM of a row kernel, whose CTAs are as wide as the rows
// need (so blocks_per_sm, which keeps one figure a kernel, is not enough).
int row_blocks_per_sm(const void *fn, int threads, int dev, int *out)
{
    static std::mutex mu;
    static std::map<std::tuple<const void *, int, int, unsigned long long>, int> cache;
    const auto key = std::make_tuple(fn, threads, dev, current_context_id());
    const bool known = std::get<3>(key) != 0;
    if (known) {
        std::lock_guard<std::mutex> g(mu);
        auto it = cache.find(key);
        if (it != cache.end()) {
            *out = it->second;
            return RMSNORM_OK;
        }
    }
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, 0);
    if (e != cudaSuccess)
        return cuda_fail(e);
    if (n < 1)
        return cuda_fail(cudaErrorInvalidConfiguration);
    if (known) {
        std::lock_guard<std::mutex> g(mu);
        cache[key] = n;
    }
    *out = n;
    return RMSNORM_OK;
}

// Shape of a row kernel (fp8_rows.cuh) for M rows of H columns: rows that
// share a warp where they are short enough; a lane a pack while the rows do
// not fill the SMs (latency); else more packs a lane. Measured (GB300, bf16,
// the norm): at 524288 x 128 eight lanes a row take 35 us, sixteen 66, a warp
// 126; at 262144 x 896 a warp a row takes 115 us, a CTA of one with two packs a
// lane 112, of two with one pack 147; at 32768 x 4096 two packs a lane take
// 62.5 us, one 90, and at 300 rows one takes 2.0, two 2.3. Wider rows take two
// packs a lane in 64 registers: at 12160 x 11008 72 us (four packs a lane 76,
// three 70), at 16264 x 8192 63 (64 and 71), at 8056 x 16384 66 (65.5 and 72).
const Fp8RowKernel &pick_fp8_rows(const Fp8RowKernel *k, int width, int64_t M, int64_t H, int sms)
{
    if (width > 0) {
        // short rows share warps in loose packs, whose width is 16 bytes too
        for (int i = 8; i < 10; ++i)
            if (H <= k[i].max_cols())
                return k[i];
        return k[width == 1 ? 7 : 10];
    }
    const bool few = M <= 2 * (int64_t)sms;
    for (int i = 0; i < kFp8SubShapes - (few ? 1 : 0); ++i)
        if (H <= k[i].max_cols())
            return k[i];
    if (few)
        return k[4];
    return H <= k[5].max_cols() ? k[5] : k[6];
}

int rows_impl(const Fp8RowsParams &prm, int mode, int dtype, cudaStream_t stream)
{
    Fp8RowsParams p = prm;
    const Fp8RowSet &set = fp8_set(dtype);
    int dev, sms, bps, st;
    if ((st = current_device(&dev)) || (st = sm_count(dev, &sms)))
        return st;
    const Fp8RowKernel *shapes = set.k[mode];
    const int width = pack_width(shapes[0].E, shapes[7].E, elem_size(dtype), p.H, p.x, p.ldx, p.r,
                                 p.ldr, p.w, p.q, p.ldq, p.h, p.ldh);
    const int64_t Hw = std::min<int64_t>(p.H, kFp8Window);      // widest window of columns
    const int windows = (int)((p.H + kFp8Window - 1) / kFp8Window);
    const Fp8RowKernel &k = pick_fp8_rows(shapes, width, p.M * windows, Hw, sms);
    int threads = k.max_threads;
    int64_t tile = 1;
    if (k.lanes) {
        tile = threads / k.lanes;
    } else {
        const int64_t lanes = ((Hw + k.E - 1) / k.E + k.V - 1) / k.V;
        threads = (int)((lanes + 31) / 32 * 32);
    }
    if ((st = row_blocks_per_sm(k.fn, threads, dev, &bps)))
        return st;
    const int64_t tiles = (p.M + tile - 1) / tile;
    const int64_t cap = std::max<int64_t>((int64_t)bps * sms / windows, 1);
    const cudaError_t e = launch1(k.fn, dim3((unsigned)std::min(tiles, cap), (unsigned)windows),
                                  threads, stream, &p);
    if (e != cudaSuccess)
        return cuda_fail(e);
    t_last_path = kPathFp8Rows;
    return RMSNORM_OK;
}

int blocks_impl(const Fp8RowsParams &r, int dtype, cudaStream_t stream)
{
    Fp8BlocksParams p = {r.x, r.q, r.scale, r.M, r.H, r.G, r.e5m2, r.ldx, r.ldq};
    const Fp8RowSet &set = fp8_set(dtype);
    const int width = pack_width(set.blocks_E[0], set.blocks_E[1], elem_size(dtype), p.H, p.x, p.ldx,
                                 nullptr, 0, nullptr, p.q, p.ldq, nullptr, 0);
    const int64_t rb = (p.M + kFp8Group - 1) / kFp8Group;
    const cudaError_t e =
        launch1(set.blocks[width], dim3((unsigned)p.G, (unsigned)std::min<int64_t>(rb, 65535)),
                256, stream, &p);
    if (e != cudaSuccess)
        return cuda_fail(e);
    t_last_path = kPathFp8Blocks;
    return RMSNORM_OK;
}

// ------------------------------------------------------------- the product
struct Fp8GemmArgs {
    const void *a, *b;
    const float *sa, *sb;
    void *out;
    int64_t lda, ldb, ldo, M, N, K;
    int at, bt, dtype, static_w;
    int G() const { return (int)((K + kFp8Group - 1) / kFp8Group); }
};

// A [rows][cols] tensor of `es`-byte elements (row stride ld elements) in
// boxes of box_rows x box_cols; reads past the end are zero, stores left out.
int fp8_map(CUtensorMap *map, const void *base, size_t es, int64_t rows, int64_t cols, int64_t ld,
            int box_rows, int box_cols, CUtensorMapSwizzle swizzle)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr)
        return RMSNORM_ERR_UNSUPPORTED;
    const CUtensorMapDataType type = es == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : es == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                               : CU_TENSOR_MAP_DATA_TYPE_UINT32;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * es};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    if (encode(map, type, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cuda_fail(cudaErrorInvalidValue);
    return RMSNORM_OK;
}

// An operand of the product: boxes of one group of columns, 128-byte swizzle.
int fp8_operand_map(CUtensorMap *map, const void *base, int64_t rows, int64_t K, int64_t ld,
                    int box_rows)
{
    return fp8_map(map, base, 1, rows, K, ld, box_rows, kFp8Group, CU_TENSOR_MAP_SWIZZLE_128B);
}

int launch_gemm(const void *fn, int64_t ctas, int threads, size_t smem, int cluster,
                cudaStream_t stream, void **args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    return e == cudaSuccess ? RMSNORM_OK : cuda_fail(e);
}

// Whether the paired kernel was compiled to the registers that its split
// among the warps draws on (with fewer its wider warps would wait for ever).
int pair_registers(const void *fn, int dtype)
{
    static std::atomic<int> checked[3];
    if (checked[dtype].load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, fn);
        if (e != cudaSuccess)
            return cuda_fail(e);
        if (fa.numRegs < kPairRegs)
            return cuda_fail(cudaErrorInvalidConfiguration);
        checked[dtype].store(1, std::memory_order_relaxed);
    }
    return RMSNORM_OK;
}

// Pairs of CTAs on tiles of 256 x 256 (fp8_gemm_pair.cuh).
int pair_impl(const Fp8GemmArgs &g, int dev, int64_t tiles_m, int64_t tiles_n, cudaStream_t stream)
{
    const void *fn = fp8_pair_kernels.fn[g.dtype];
    int pairs, st;
    if ((st = pair_registers(fn, g.dtype)) ||
        (st = max_active_clusters(fn, kPairThreads, (int)kPairSmem, 2, dev, &pairs)))
        return st;
    const size_t es = elem_size(g.dtype);
    const bool vec = aligned(g.out, 16) && g.ldo * (int64_t)es % 16 == 0;
    CUtensorMap mapA, mapB, mapO = {};
    unsigned int *tmo = stream_timeout_counter(dev);
    if (tmo == nullptr)
        return cuda_fail(cudaErrorInvalidSymbol);
    if ((st = fp8_operand_map(&mapA, g.a, g.M, g.K, g.lda, 128)) ||
        (st = fp8_operand_map(&mapB, g.b, g.N, g.K, g.ldb, 128)) ||
        (vec && (st = fp8_map(&mapO, g.out, es, g.M, g.N, g.ldo, 32, (int)(kPairRowBytes / es),
                              CU_TENSOR_MAP_SWIZZLE_64B))))
        return st;
    Fp8PairParams p = {g.sa, g.sb, g.out, g.ldo, (int)g.M, (int)g.N, g.G(), (int)tiles_m,
                       (int)tiles_n,
                       umma_idesc_f8((uint32_t)g.at, (uint32_t)g.bt, kPairTile, kPairTile),
                       g.static_w, vec ? (g.N * (int64_t)es % 16 == 0 ? 2 : 1) : 0,
                       g_test_extra_tx.load(std::memory_order_relaxed),
                       g_test_wait_us.load(std::memory_order_relaxed)};
    void *args[5] = {&p, &mapA, &mapB, &mapO, &tmo};
    if ((st = launch_gemm(fn, 2 * std::min<int64_t>(pairs, tiles_m * tiles_n), kPairThreads, kPairSmem,
                          2, stream, args)))
        return st;
    t_last_path = kPathFp8Pair;
    return RMSNORM_OK;
}

constexpr int kPairLongK = 32;          // groups of a long K (see gemm_impl)

int gemm_impl(const Fp8GemmArgs &g, cudaStream_t stream)
{
    static const int kBN[4] = {16, 32, 64, 128};
    const int64_t M = g.M, N = g.N;
    const int G = g.G();
    int dev, sms, bps, st;
    if ((st = current_device(&dev)) || (st = sm_count(dev, &sms)))
        return st;
    // Pairs of CTAs where tiles of 128 x 128 would not all run at once, two to
    // an SM, or, with a long K, one to an SM (two share its tensor cores), and
    // a pair's tile of 256 rows is not half empty. Measured (GB300, weights from
    // DRAM, tile kernel / pairs): one tile an SM, 256 x 6144 x 4096 15.1 / 20.1
    // us, 1024 x 1024 x 4096 10.9 / 19.4; two, 1024 x 2560 at K = 384 6.0 / 8.2,
    // 2048 11.8 / 14.1, 5120 22.5 / 23.5, 1024 x 4096 at 768 7.8 / 10.3, 5120
    // 24.8 / 24.0; more, 4096 x 1280 x 2048 20.4 / 21.9, 2048 x 24576 x 4096
    // 210 / 161; one row of tiles, 128 x 24576 x 4096 23 / 37.
    const int64_t tm = (M + kPairTile - 1) / kPairTile, tn = (N + kPairTile - 1) / kPairTile;
    const int64_t t128 = ((M + 127) / 128) * ((N + 127) / 128);
    const int ov = g_test_gemm_fp8.load(std::memory_order_relaxed);
    const bool fits = tm * tn * G < INT32_MAX;
    const int64_t at_once = (G < kPairLongK ? 2 : 1) * (int64_t)sms;
    if (fits && (ov == kPathFp8Pair || (ov != kPathFp8Gemm && M > 128 && t128 > at_once)))
        return pair_impl(g, dev, tm, tn, stream);
    // the narrowest column operand that holds the tokens, whose scales must
    // fit in shared memory; else tokens in tiles of 128 rows
    int v = 0;
    Fp8GemmLayout L;
    int KS = 0;
    int64_t tiles_r = 0, tiles_c = 0;
    for (;; ++v) {
        const bool swap = v < 3;
        const int BN = kBN[v];
        if (swap && M > BN)
            continue;
        tiles_r = ((swap ? N : M) + kFp8TileR - 1) / kFp8TileR;
        tiles_c = ((swap ? M : N) + BN - 1) / BN;
        // Clusters with which the whole grid runs at once (a few late ones
        // cost as much as all the others: 64 x 6144 x 4096 with three CTAs a
        // cluster, of which 46 run at once, 17 us, with two 10), with a ring
        // of up to six stages. Of those the one for which a CTA's groups and
        // the exchange with its peers take least (in units of 10 ns, fitted
        // to 896 -> 2048, 4096 -> 1024 and 1024 -> 1024 features at 8 to 200
        // rows: 64 x 2048 x 896 takes 4.9 us with four CTAs, 5.8 with three,
        // 6.2 with one, 5.1 with six). The runtime's count of clusters is
        // that of one CTA an SM.
        static const int kGroup[4] = {25, 25, 27, 40}, kPeer[4] = {12, 15, 12, 40};
        KS = 0;
        int least = INT32_MAX;
        for (int ks = std::min(kFp8MaxCluster, G); ks >= 1; --ks) {
            const int ng = (G + ks - 1) / ks;
            Fp8GemmLayout l;
            for (int stages = std::min(ng, 6);; --stages) {
                l = fp8_gemm_layout(BN, swap, stages, ng, ks);
                if (l.total <= kFp8MaxSmem || stages <= 3)
                    break;
            }
            const int64_t cost = (int64_t)ng * kGroup[v] + (ks > 1 ? ks * kPeer[v] : 0);
            if (l.total > kFp8MaxSmem || cost >= least)
                continue;
            const void *fn = fp8_gemm_kernels.fn[v][g.dtype];
            int n;
            if ((st = blocks_per_sm(fn, fp8_gemm_threads(BN), dev, &bps, (int)l.total)) ||
                (st = max_active_clusters(fn, fp8_gemm_threads(BN), (int)l.total, ks, dev, &n)))
                return st;
            if (tiles_r * tiles_c <= (int64_t)n * bps) {
                KS = ks;
                L = l;
                least = (int)cost;
            }
        }
        if (KS < 1) {
            // more tiles than run at once: a tile a CTA, two CTAs an SM (one
            // starts while the other ends) with the ring that this leaves
            KS = 1;
            int stages = std::min(G, 6);
            do
                L = fp8_gemm_layout(BN, swap, stages, G, 1);
            while (L.total > kFp8HalfSmem && --stages >= 3);
            if (stages < 3)
                L = fp8_gemm_layout(BN, swap, std::min(G, 3), G, 1);
        }
        if (!swap || L.total <= kFp8MaxSmem)
            break;
    }
    const bool swap = v < 3;
    const int BN = kBN[v];
    const int64_t ctas = tiles_r * tiles_c * KS;
    CUtensorMap mapA, mapB;
    unsigned int *tmo = stream_timeout_counter(dev);
    if (tmo == nullptr)
        return cuda_fail(cudaErrorInvalidSymbol);
    if ((st = fp8_operand_map(&mapA, g.a, M, g.K, g.lda, swap ? BN : kFp8TileR)) ||
        (st = fp8_operand_map(&mapB, g.b, N, g.K, g.ldb, swap ? kFp8TileR : BN)))
        return st;
    const void *fn = fp8_gemm_kernels.fn[v][g.dtype];
    const size_t es = elem_size(g.dtype);
    Fp8GemmParams p = {g.sa, g.sb, g.out, g.ldo, (int)M, (int)N, G, KS, (int)tiles_r,
                       swap ? umma_idesc_f8((uint32_t)g.bt, (uint32_t)g.at, kFp8TileR, BN)
                            : umma_idesc_f8((uint32_t)g.at, (uint32_t)g.bt, kFp8TileR, BN),
                       g.static_w, aligned(g.out, 4 * es) && g.ldo % 4 == 0 ? 1 : 0,
                       g_test_extra_tx.load(std::memory_order_relaxed),
                       g_test_wait_us.load(std::memory_order_relaxed), L};
    void *args[4] = {&p, swap ? &mapB : &mapA, swap ? &mapA : &mapB, &tmo};
    if ((st = blocks_per_sm(fn, fp8_gemm_threads(BN), dev, &bps, (int)L.total)) ||
        (st = launch_gemm(fn, ctas, fp8_gemm_threads(BN), L.total, KS, stream, args)))
        return st;
    t_last_path = kPathFp8Gemm;
    return RMSNORM_OK;
}

// Checks and the launch that rmsnorm_fwd_fp8 and the row form of
// rmsnorm_quant_fp8 share. w null: x alone.
int rows_checked(const void *x, int64_t ldx, const void *r, int64_t ldr, const void *w, bool norm,
                 void *q, int64_t ldq, float *scale, void *h, int64_t ldh, float *rstd, int64_t M,
                 int64_t H, float eps, int dtype, int qtype, int block_rows, cudaStream_t stream)
{
    const bool res = r != nullptr || h != nullptr;
    if (!stride_ok(ldx, M, H) || !stride_ok(ldq, M, H) ||
        (res && (!stride_ok(ldr, M, H) || !stride_ok(ldh, M, H))))
        return RMSNORM_ERR_BAD_STRIDE;
    if (M == 0)
        return RMSNORM_OK;
    if (!x || (norm && !w) || !q || !scale || (res && (!r || !h)))
        return RMSNORM_ERR_NULLPTR;
    const size_t es = elem_size(dtype);
    if (!aligned(x, es) || !aligned(r, es) || !aligned(w, es) || !aligned(h, es) ||
        !aligned(scale, 4) || !aligned(rstd, 4))
        return RMSNORM_ERR_MISALIGNED;
    if (!res)
        ldr = ldh = H;
    const int64_t G = (H + kFp8Group - 1) / kFp8Group;
    const int64_t srows = block_rows == 1 ? M : (M + kFp8Group - 1) / kFp8Group;
    const Span sx = rows_span(x, M, H, ldx, es), sr = rows_span(r, M, H, ldr, es),
               sw = flat(w, (size_t)H * es), sq = rows_span(q, M, H, ldq, 1),
               ss = flat(scale, (size_t)(srows * G) * 4), sh = rows_span(h, M, H, ldh, es),
               st = flat(rstd, (size_t)M * 4);
    for (Span o : {sq, ss, st})
        for (Span i : {sx, sr, sw, sh})
            if (overlap(o, i))
                return RMSNORM_ERR_ALIAS;
    if (overlap(sq, ss) || overlap(sq, st) || overlap(ss, st) || overlap(sh, sw) ||
        (!sh.empty() && (!same_or_disjoint(sh, sx) || !same_or_disjoint(sh, sr))))
        return RMSNORM_ERR_ALIAS;
    const Fp8RowsParams p = {x, r, w, q, scale, h, rstd, M, (int)H, (int)G, eps,
                             qtype == RMSNORM_E5M2 ? 1 : 0, ldx, ldr, ldq, ldh};
    if (block_rows != 1)
        return blocks_impl(p, dtype, stream);
    return rows_impl(p, norm ? (res ? 2 : 1) : 0, dtype, stream);
}

} // namespace

extern "C" {

int rmsnorm_fwd_fp8(const void *x, int64_t ldx, const void *r, int64_t ldr, const void *w, void *q,
                    int64_t ldq, float *scale, void *h, int64_t ldh, float *rstd, int64_t M,
                    int64_t H, float eps, int dtype, int qtype, void *stream)
{
    const int st = check_common(M, H, eps, dtype);
    if (st)
        return st;
    if (!fp8_type(qtype))
        return RMSNORM_ERR_BAD_DTYPE;
    return rows_checked(x, ldx, r, ldr, w, true, q, ldq, scale, h, ldh, rstd, M, H, eps, dtype,
                        qtype, 1, static_cast<cudaStream_t>(stream));
}

int rmsnorm_quant_fp8(const void *x, int64_t ldx, void *q, int64_t ldq, float *scale, int64_t M,
                      int64_t H, int block_rows, int dtype, int qtype, void *stream)
{
    if ((dtype != RMSNORM_F32 && dtype != RMSNORM_BF16 && dtype != RMSNORM_F16) || !fp8_type(qtype))
        return RMSNORM_ERR_BAD_DTYPE;
    if (M < 0 || H < 1 || M > INT64_MAX / 8 / H)
        return RMSNORM_ERR_BAD_SHAPE;
    if (H > RMSNORM_FP8_MAX_K || (block_rows != 1 && block_rows != kFp8Group))
        return RMSNORM_ERR_UNSUPPORTED;
    return rows_checked(x, ldx, nullptr, 0, nullptr, false, q, ldq, scale, nullptr, 0, nullptr, M, H,
                        0.f, dtype, qtype, block_rows, static_cast<cudaStream_t>(stream));
}

int rmsnorm_gemm_fp8(const void *a, int64_t lda, const float *a_scale, int a_type, const void *b,
                     int64_t ldb, const float *b_scale, int b_type, void *out, int64_t ldo,
                     int64_t M, int64_t N, int64_t K, int dtype, int flags, void *stream)
{
    if (flags & ~RMSNORM_GEMM_FP8_STATIC_WEIGHTS)
        return RMSNORM_ERR_BAD_FLAGS;
    if ((dtype != RMSNORM_F32 && dtype != RMSNORM_BF16 && dtype != RMSNORM_F16) ||
        !fp8_type(a_type) || !fp8_type(b_type))
        return RMSNORM_ERR_BAD_DTYPE;
    if (M < 0 || N < 1 || K < 1)
        return RMSNORM_ERR_BAD_SHAPE;
    // the grid: at most a CTA to a tile of 128 x 128 (clusters only where all
    // of them run at once)
    if (M > RMSNORM_FP8_MAX_ROWS || N > RMSNORM_FP8_MAX_ROWS || K > RMSNORM_FP8_MAX_K ||
        ((M + 127) / 128) * ((N + 127) / 128) > INT32_MAX)
        return RMSNORM_ERR_UNSUPPORTED;
    // a single row has no stride: any that a tensor map takes
    if (M == 1)
        lda = (K + 15) / 16 * 16;
    if (N == 1)
        ldb = (K + 15) / 16 * 16;
    if (M == 1)
        ldo = std::max(ldo, N);
    if (!stride_ok(lda, M, K) || !stride_ok(ldb, N, K) || !stride_ok(ldo, M, N))
        return RMSNORM_ERR_BAD_STRIDE;
    if (M == 0)
        return RMSNORM_OK;
    if (!a || !a_scale || !b || !b_scale || !out)
        return RMSNORM_ERR_NULLPTR;
    const size_t es = elem_size(dtype);
    if (!aligned(a, 16) || !aligned(b, 16) || lda % 16 || ldb % 16 || !aligned(a_scale, 4) ||
        !aligned(b_scale, 4) || !aligned(out, es))
        return RMSNORM_ERR_MISALIGNED;
    const int64_t G = (K + kFp8Group - 1) / kFp8Group;
    const Span so = rows_span(out, M, N, ldo, es);
    for (Span i : {rows_span(a, M, K, lda, 1), rows_span(b, N, K, ldb, 1),
                   flat(a_scale, (size_t)(M * G) * 4),
                   flat(b_scale, (size_t)((N + kFp8Group - 1) / kFp8Group * G) * 4)})
        if (overlap(so, i))
            return RMSNORM_ERR_ALIAS;
    const Fp8GemmArgs g = {a, b, a_scale, b_scale, out, lda, ldb, ldo, M, N, K, a_type, b_type, dtype,
                           (flags & RMSNORM_GEMM_FP8_STATIC_WEIGHTS) ? 1 : 0};
    return gemm_impl(g, static_cast<cudaStream_t>(stream));
}

void rmsnorm_set_gemm_fp8_test(int path) { g_test_gemm_fp8.store(path); }

} // extern "C"
