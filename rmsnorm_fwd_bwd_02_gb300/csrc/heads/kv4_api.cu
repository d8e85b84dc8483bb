// kv4_api.cu -- attention over a 4-bit cache: host-side argument checks, kernel
// choice and launches of include/rmsnorm.h's rmsnorm_kv4_attention. No
// allocation, no synchronisation, no host copies.
#include "heads_host.h"

#include "../registry.h"

using namespace rmsk;

namespace {

constexpr int kPathKv4Attend = 16, kPathKv4Prompt = 17;

constexpr int kClusterStages = 8;        // most stages a warp in clusters (see below)

// Test hook: the kernel (see rmsnorm.h).
std::atomic<int> g_test_kv4{0};

size_t workspace_bytes(int sms, int64_t D)
{
    size_t most = 0;
    for (int NT = 1; NT <= 2; ++NT)
        most = std::max(most, (size_t)sms * kv4_ctas_per_sm(NT) * kKv4Warps * 2 * kv4_partial((int)D, NT) * 4);
    return most;
}

} // namespace

extern "C" {

size_t rmsnorm_kv4_attention_workspace_bytes(int64_t D)
{
    int dev, sms;
    if ((D != 64 && D != 128) || current_device(&dev) || sm_count(dev, &sms))
        return 0;
    return workspace_bytes(sms, D);
}

int rmsnorm_kv4_attention(const void *q, int64_t q_token, int64_t q_head, void *out, int64_t out_token,
                          int64_t out_head, float *lse, const void *cache, int64_t pages, int64_t page_size,
                          int64_t kv_heads, const float *k_scale, const float *v_scale, const int *block_table,
                          int64_t table_stride, int64_t blocks, const int *seq_lens, const int *q_starts,
                          int64_t B, int64_t T, int64_t heads, int64_t D, float scale, void *workspace,
                          size_t workspace_size, int dtype, void *stream)
{
    if (dtype != RMSNORM_BF16 && dtype != RMSNORM_F16)
        return RMSNORM_ERR_BAD_DTYPE;
    if (B < 0 || T < 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || pages < 0 || page_size < 1 ||
        blocks < 0 || (q_starts == nullptr && T != B))
        return RMSNORM_ERR_BAD_SHAPE;
    if (!std::isfinite(scale))
        return RMSNORM_ERR_BAD_EPS;
    if ((D != 64 && D != 128) || page_size % kKv4Tile || page_size > INT32_MAX || heads > (1 << 20) ||
        pages > INT32_MAX || blocks > INT32_MAX || B > (1 << 20) || T > INT32_MAX ||
        blocks > (INT32_MAX - 1024) / page_size || (T + B) > INT32_MAX / heads ||
        page_size * kv_heads > INT32_MAX / (D * 9 / 8))
        return RMSNORM_ERR_UNSUPPORTED;
    if (!rows_within({T, heads, 1}, {q_token, q_head, 0}, D) ||
        !rows_apart({T, heads, 1}, {out_token, out_head, 0}, D) ||
        (B > 1 && (table_stride < blocks || table_stride > INT32_MAX)))
        return RMSNORM_ERR_BAD_STRIDE;
    if (T == 0 || B == 0)
        return RMSNORM_OK;
    if (!q || !out || !seq_lens || (blocks && !block_table) || (pages && !cache))
        return RMSNORM_ERR_NULLPTR;
    if (!aligned(q, 2) || !aligned(out, 2) || !aligned(lse, 4) || !aligned(cache, 16) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(q_starts, 4) ||
        !aligned(workspace, 16))
        return RMSNORM_ERR_MISALIGNED;
    int dev, sms, st;
    const Span so = heads_span(out, T, heads, D, out_token, out_head, 2);
    const Span sl = flat(lse, (size_t)(T * heads) * 4), sw = flat(workspace, workspace_size);
    const Span in[7] = {heads_span(q, T, heads, D, q_token, q_head, 2),
                        flat(cache, (size_t)(pages * page_size * kv_heads * (D * 9 / 8))),
                        flat(k_scale, (size_t)kv_heads * 4),
                        flat(v_scale, (size_t)kv_heads * 4),
                        blocks ? flat(block_table, (size_t)((B - 1) * (B > 1 ? table_stride : 0) + blocks) * 4)
                               : Span{nullptr, 0, 0, 0},
                        flat(seq_lens, (size_t)B * 4),
                        flat(q_starts, (size_t)(B + 1) * 4)};
    for (const Span &i : in)
        if (overlap(so, i) || overlap(sl, i) || overlap(sw, i))
            return RMSNORM_ERR_ALIAS;
    if (overlap(so, sl) || overlap(so, sw) || overlap(sl, sw))
        return RMSNORM_ERR_ALIAS;
    if ((st = current_device(&dev)) || (st = sm_count(dev, &sms)))
        return st;
    if (workspace == nullptr || workspace_size < workspace_bytes(sms, D))
        return RMSNORM_ERR_WORKSPACE;

    unsigned int *tmo = stream_timeout_counter(dev);
    if (tmo == nullptr)
        return cuda_fail(cudaErrorInvalidSymbol);
    const int64_t G = heads / kv_heads;
    // Eight query rows a tile where a sequence's rows of one key head fit; else
    // sixteen, for which the cache's bytes are widened once (16 x 4 tokens of 32
    // heads of 128 on 8 over 8192: 56 us, in tiles of eight 65; 4 x 4 of 64 heads:
    // 35.9, 38.2). Not for heads of 64, whose kernel of eight rows runs twice on an
    // SM (16 x 5 tokens of 14 heads on 2 over up to 3000: 17.8 us, of sixteen 21.3).
    const int64_t rows = (T + B - 1) / B * G;
    const int NT = rows <= 8 || D == 64 ? 1 : 2, di = D == 128 ? 1 : 0, ti = dtype == RMSNORM_BF16 ? 0 : 1;
    Kv4Params p = {q, q_token, q_head, out, out_token, out_head, lse, static_cast<const uint8_t *>(cache), pages,
                   (int)(page_size / kKv4Tile), k_scale, v_scale, block_table, table_stride, (int)blocks, seq_lens,
                   q_starts, (int)B, (int)T, (int)kv_heads, (int)G, scale,
                   aligned(q, 16) && aligned(out, 16) &&
                           strides_multiple(16, 2, {T > 1 ? q_token : 0, heads > 1 ? q_head : 0,
                                                    T > 1 ? out_token : 0, heads > 1 ? out_head : 0})
                       ? 1
                       : 0,
                   static_cast<float *>(workspace), 0, g_test_extra_tx.load(std::memory_order_relaxed),
                   g_test_wait_us.load(std::memory_order_relaxed), tmo};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Pieces of prompts. For 128 tokens of every sequence the kernel for few
    // rows takes 0.4 ns a row and key head (0.3 with heads of 64), the one for
    // many 1.75 us for each time that its CTAs of 256 rows fill the SMs, however
    // few they are; both grow with the lengths alike. Measured (GB300, 32 heads
    // of 128 on 8): 1 x 128 tokens over 8192 87 / 120 us, 1 x 256 160 / 121; 4 x
    // 32 over 4096 52 / 65, 4 x 64 89 / 70; 16 x 16 over 2048 54 / 39; 14 heads of
    // 64 on 2: 4 x 64 over 4096 36 / 56, 4 x 256 121 / 58, 16 x 64 over 2048 69 / 35.
    // Pieces of one length each: the starts are on the device, so the rule goes by
    // their mean. Where one is long and the others single tokens it may be off: 512
    // tokens beside 63 of one, over 2000 each, take 172 us by the kernel for many,
    // which it picks, and 130 by the other (two calls, one for the piece: 46 + 42).
    const int64_t wide = B * ((rows + kv4_prompt_kernels.rows - 1) / kv4_prompt_kernels.rows) * kv_heads;
    const int ov = g_test_kv4.load(std::memory_order_relaxed);
    if (q_starts && (ov == 2 || (ov == 0 && T * heads >= (D == 128 ? 4400 : 5800) * ((wide + sms - 1) / sms)))) {
        const void *fn = kv4_prompt_kernels.fn[ti][di];
        int bps;
        if ((st = blocks_per_sm(fn, kv4_prompt_kernels.threads, dev, &bps, kv4_prompt_kernels.smem[di])))
            return st;
        void *args[1] = {&p};
        const int64_t tiles = T * G / kv4_prompt_kernels.rows + B;
        const cudaError_t e = launch_pdl(fn, dim3((unsigned)(tiles * kv_heads)), kv4_prompt_kernels.threads,
                                         (size_t)kv4_prompt_kernels.smem[di], s, args);
        if (e != cudaSuccess)
            return cuda_fail(e);
        t_last_path = kPathKv4Prompt;
        return RMSNORM_OK;
    }
    const int64_t tiles = q_starts ? (T * G) / (8 * NT) + B : B * ((G + 8 * NT - 1) / (8 * NT));
    if (tiles * kv_heads > INT32_MAX / (blocks * page_size / kKv4Slot + 4))
        return RMSNORM_ERR_UNSUPPORTED;
    const void *fn = kv4_kernels.attend[ti][di][NT - 1];
    const int smem = kv4_smem((int)D);
    int bps;
    if ((st = blocks_per_sm(fn, kKv4Warps * 32, dev, &bps, smem)))
        return st;
    int ctas = sms * std::min(bps, kv4_ctas_per_sm(NT));
    void *args[1] = {&p};
    cudaError_t e;
    // A cluster a segment, the largest with which all run at once, where a
    // warp then has few stages. Measured (GB300, 32 heads of 128 on 8, all
    // lengths alike, list / clusters): one sequence of 64 tokens 7.9 / 4.3 us,
    // 4096 12.7 / 8.3, 16384 (8 stages a warp) 20.0 / 15.2, 65536 (32) 27 / 42;
    // 16 of 4096 (8) 24.4 / 21.4, of 16384 (32) 61 / 66; 32 of 4096 (16) 40.9 /
    // 36.4, of 16384 (64) 110 / 120. Lengths that differ favour the list,
    // which is even whatever they are.
    const int64_t segs = tiles * kv_heads, stages = (blocks * page_size + kKv4Slot - 1) / kKv4Slot;
    if (ov != 1 && segs <= ctas) {
        int cs = kKv4Cluster, n = 0;
        for (; cs > 1; cs /= 2) {
            if (stages <= (int64_t)(cs / 2) * kKv4Warps)
                continue;                                       // half as many would have a stage a warp
            if ((st = max_active_clusters(fn, kKv4Warps * 32, smem, cs, dev, &n)))
                return st;
            if (segs <= n)
                break;
        }
        if (ov == 3 || stages <= cs * kKv4Warps * kClusterStages) {
            p.cluster = cs;
            e = launch_pdl(fn, dim3((unsigned)(segs * cs)), kKv4Warps * 32, (size_t)smem, s, args, cs);
            if (e != cudaSuccess)
                return cuda_fail(e);
            t_last_path = kPathKv4Attend;
            return RMSNORM_OK;
        }
    }
    e = launch_pdl(fn, dim3((unsigned)ctas), kKv4Warps * 32, (size_t)smem, s, args);
    if (e != cudaSuccess)
        return cuda_fail(e);
    // the parts of segments that were split; none is, where one stage covers any length
    if (blocks * page_size > kKv4Slot) {
        void *cargs[2] = {&p, &ctas};
        e = launch_pdl(kv4_kernels.combine[ti][di][NT - 1], dim3((unsigned)(tiles * kv_heads)), 256, 0, s, cargs);
        if (e != cudaSuccess)
            return cuda_fail(e);
    }
    t_last_path = kPathKv4Attend;
    return RMSNORM_OK;
}

void rmsnorm_set_kv4_test(int kernel) { g_test_kv4.store(kernel); }

} // extern "C"
