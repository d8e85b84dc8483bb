// kv4_prompt.cuh -- attention over a 4-bit cache for pieces of prompts: many
// query rows of a sequence and key head. Same result as kv4_attend.cuh (its
// mathematics: the cache exact in fp16, q scaled by a power of two a row, the
// softmax in powers of two with a reference that moves rarely), on the
// fifth-generation tensor cores. But for fp16 outputs: p is one half here, not
// two, which would be half as many products again; a row's error against 64 bits
// is 2.9e-4 with it (2.1e-4 there), for bf16 1.67e-3 by both.
//
// Why this shape. With hundreds of rows the products bound the call, and
// widening the cache's bytes anew for every 16 rows costs more than they do.
// A CTA holds 256 rows (tokens times heads of one key head) as two tiles of
// 128 and goes through the sequence 128 tokens at a time; the widened keys and
// values in shared memory serve both tiles. Warps have one task each:
//   0-3, 4-7    the softmax of tile 0, of tile 1: a thread a row, which reads
//               its scores from tensor memory (lane = row), keeps the row's
//               reference and denominator, and writes p as fp16;
//   8-11        keys, a thread a token, and values, transposed on the way, a
//               thread eight tokens of 16 features, whose nibbles it
//               interleaves in pairs of tokens; bytes from global memory a
//               tile ahead;
//   12          the products: S_t = Q_t K^T and O_t += P_t V, m128 n128 k16
//               (n64 for O with heads of 64).
// While tile 0's rows are in the softmax the tensor cores work on tile 1's
// scores, and the other way round. Operands from shared memory are K-major in
// the 128-byte swizzled layout (gemv_umma.cuh); the transposed values have the
// tokens as K. Two m128 n128 k16 operands from shared memory take all of its
// bandwidth, and p would be written there besides: p stays in tensor memory,
// over its tile's scores, and is the product's first operand from there
// (tensor memory: two tiles of scores and p, two of outputs, 512 columns).
// That leaves room for keys and values in two buffers each. A row's output is
// scaled in tensor memory when its reference moves.
//
// Measured (GB300): 2 x 512 tokens of 32 heads of 128 on 8 over up to 8192, 118 us,
// 1.05 PFLOP/s (the kernel for few rows: 607). A tile of 128 tokens takes some
// 3100 cycles, 2048 of them MMAs at their rate: a tile's softmax (1400), product
// and next scores wait for one another, and two tiles of rows overlap them. With
// p in shared memory 227 us; products issued by a lone lane, whose descriptors
// then go through vector registers, 140.
//
// Every wait is bounded; one that runs out sets a flag that ends the others,
// counts in the timeout counter and leaves the rows unwritten.
#pragma once

#include "../gemv_umma.cuh"
#include "kv4_attend.cuh"

namespace rmsk {

// p = 2^(x - m + kPromptBase), and a reference holds up to x = m + kPromptRoom,
// p = 2^15. A wider room than the other kernel's 8 and 7: a tile that passes it
// is done twice, for all of its warp's rows.
constexpr float kPromptBase = 4.f, kPromptRoom = 11.f;
constexpr int kPromptRows = 256, kPromptTokens = 128, kPromptThreads = 13 * 32;

// Shared memory: q of both tiles, keys and values (two in turn each), then the
// barriers, the tensor-memory address and the keys' tiles that are there.
template <int D>
struct PromptLayout {
    static constexpr uint32_t kQ = 128 * D * 2, kK = 128 * D * 2, kV = D * 128 * 2;
    static constexpr uint32_t q = 0, k = 2 * kQ, v = k + 2 * kK, bar = v + 2 * kV;
    static constexpr uint32_t kBars = 14;
    static constexpr uint32_t total = bar + 8 * kBars + 32 + 1023;       // with the alignment
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    uint32_t u[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
                   "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
                   "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
                   "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
                   "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
                 : "r"(taddr)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(u[i]);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
                 "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
                 "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]),
                 "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]),
                 "f"(v[30]), "f"(v[31])
                 : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 32 words to as many columns of the warp's lanes, without the wait.
__device__ __forceinline__ void tmem_put32(uint32_t taddr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                 "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
                 "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
                 "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
                 "r"(v[30]), "r"(v[31])
                 : "memory");
}

__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (tensor memory) = A B^T (+ D), kind::f16, with A in tensor memory: a lane a
// row, a column two elements along K.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// One lane of the warp, always the same; all lanes take part.
__device__ __forceinline__ bool elect_lane()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A bounded wait that also ends when another warp's has run out.
__device__ __forceinline__ bool prompt_wait(uint32_t bar, uint32_t parity, volatile int *bad,
                                            unsigned long long limit)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const unsigned long long t0 = global_ns();
    for (int i = 1; !mbar_try_wait(bar, parity); ++i)
        if ((i & 15) == 0 && (*bad || global_ns() - t0 > limit)) {
            *bad = 1;
            return false;
        }
    return true;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(kPromptThreads, 1) kv4_prompt(Kv4Params p)
{
    using L = PromptLayout<D>;
    constexpr int kTile = kv4_tile_bytes(D), G16 = D / 16;
    extern __shared__ uint8_t raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *const sm = raw + (base - smem_addr(raw));
    // barriers: keys full [2], free [2]; values full [2], free [2]; scores full [2]; p full [2]; all done
    const uint32_t kfull = base + L::bar, kfree = kfull + 16, vfull = kfull + 32, vfree = kfull + 48,
                   sfull = kfull + 64, pfull = kfull + 80, done = kfull + 96;
    volatile uint32_t *slots = reinterpret_cast<volatile uint32_t *>(sm + L::bar + 8 * L::kBars);
    volatile int *bad = reinterpret_cast<volatile int *>(slots + 1);
    volatile uint8_t *present = reinterpret_cast<volatile uint8_t *>(sm + L::bar + 8 * L::kBars + 8);   // [4][4]

    griddep_wait();
    // the segment of this CTA: sequences' segments side by side, a key head's
    // tiles from the last (which sees most) to the first
    int64_t segs = 0, seg = -1;
    int seq = 0;
    for (int b0 = 0; b0 < p.B && seg < 0; b0 += 32) {
        int64_t n = 0;
        if (b0 + lane < p.B) {
            const Kv4Seq t = kv4_seq<kPromptRows / 8>(p, b0 + lane);
            n = (int64_t)t.tiles * p.Hk;
        }
        int64_t sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o)
                sum += v;
        }
        const unsigned at = __ballot_sync(0xFFFFFFFFu, segs + sum > blockIdx.x);
        if (at) {
            const int l = __ffs(at) - 1;
            seq = b0 + l;
            seg = blockIdx.x - (segs + __shfl_sync(0xFFFFFFFFu, sum - n, l));
        }
        segs += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (seg < 0)
        return;                                                 // for the whole CTA
    const Kv4Seq s = kv4_seq<kPromptRows / 8>(p, seq);
    const int h = (int)(seg % p.Hk), tile = s.tiles - 1 - (int)(seg / p.Hk);
    if (tile < 0)
        return;                                                 // lengths that change under the call
    const int rows = s.n * p.G;                                 // of this sequence and key head
    const int row0 = tile * kPromptRows, row_last = min(rows, row0 + kPromptRows) - 1;
    const int most = max(0, s.len - s.n + row_last / p.G + 1);  // tokens that the last row sees
    const int count = (most + kPromptTokens - 1) / kPromptTokens;
    const unsigned long long limit = wait_limit_ns(p.wait_limit_us);

    if (warp == 12) {
        if (lane == 0) {
            for (int t = 0; t < 2; ++t) {
                // the test hook: one arrival more than there are, so that the waits run out
                mbar_init(kfull + 8 * t, p.extra_tx ? 129 : 128);
                mbar_init(kfree + 8 * t, 1);
                mbar_init(vfull + 8 * t, 128);
                mbar_init(vfree + 8 * t, 1);
                mbar_init(sfull + 8 * t, 1);
                mbar_init(pfull + 8 * t, 128);
            }
            mbar_init(done, 1);
            mbar_init_fence();
            *bad = 0;
        }
        __syncwarp();
        tmem_alloc(base + L::bar + 8 * L::kBars, 512);
        tmem_relinquish();
    }

    // q, a thread a row: to fp16 with the largest element at 2^14
    float mul = 0.f;
    int lim = 0, row_i = 0, row_h = 0;
    bool real = false;
    if (warp < 8) {
        const int t = tid >> 7, r = tid & 127, row = row0 + t * 128 + r;
        real = row < rows;
        row_i = real ? row / p.G : 0;
        row_h = h * p.G + (real ? row - row_i * p.G : 0);
        lim = real ? max(0, s.len - s.n + row_i + 1) : 0;
        const char *q = static_cast<const char *>(p.q) +
                        ((int64_t)(s.q0 + row_i) * p.qt + row_h * p.qh) * (int64_t)sizeof(T);
        auto word = [&](int j) {
            return (uint32_t)ld_row_b16(q + 4 * j) | (uint32_t)ld_row_b16(q + 4 * j + 2) << 16;
        };
        auto chunk = [&](int c) {
            if (!real)
                return make_uint4(0, 0, 0, 0);
            if (p.vec)
                return __ldg(reinterpret_cast<const uint4 *>(q) + c);
            return make_uint4(word(4 * c), word(4 * c + 1), word(4 * c + 2), word(4 * c + 3));
        };
        float m = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
            const uint4 u = chunk(c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = Half16<T>::wide2(w[j]);
                m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
        const int e = max((int)(__float_as_uint(m) >> 23) - 127, -100);
        const float k = p.scale * 1.4426950408889634f * (p.kscale ? __ldg(p.kscale + h) : 1.f);
        // the factor's sign goes into q: the largest score is then the largest power
        const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - e) << 23), k);
        mul = fabsf(k) * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
            const uint4 u = chunk(c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = Half16<T>::wide2(w[j]);
                o[j] = Half16<f16>::narrow2(f.x * up, f.y * up);
            }
            sts128(base + L::q + t * L::kQ + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4), o[0], o[1],
                   o[2], o[3]);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = slots[0];
    // Not before the CTA holds its tensor memory: a dependent's CTA beside it may
    // take columns first and keep them until this grid ends, which would then
    // wait for them.
    griddep_launch_dependents();

    if (warp < 8) {
        // ------------------------------------------------------ the softmax
        const int t = tid >> 7;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;     // (32 (warp % 4)) << 16
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
        // (a row that sees nothing wants no reference)
        float m = lim > 0 ? kKv4Least : 0.f, l = 0.f;
        int least = real ? lim : INT32_MAX;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
        bool ok = true;
        for (int j = 0; j < count; ++j) {
            ok = __all_sync(0xFFFFFFFFu, prompt_wait(sfull + 8 * t, j & 1, bad, limit));
            if (!ok)
                break;
            tc_fence_after_sync();
            const uint32_t there = *reinterpret_cast<volatile uint32_t *>(sm + L::bar + 8 * L::kBars + 8 + 4 * (j & 3));
            const int tok = j * kPromptTokens;
            const bool whole = tok + kPromptTokens <= least && there == 0x03030303u;
            // column c's token is seen: past neither the row's limit nor in a tile that is not there
            auto seen = [&](int c) { return tok + c < lim && (there >> (8 * (c >> 5) + ((c >> 4) & 1)) & 1u); };
            // p from the reference as it is, where all tokens are seen: most
            // tiles do not pass it
            bool far = m == kKv4Least || !whole;
            if (!__any_sync(0xFFFFFFFFu, far)) {
                const float2 mul2 = make_float2(mul, mul), b2 = make_float2(kPromptBase - m, kPromptBase - m);
                float2 sum = make_float2(0.f, 0.f);
                uint32_t top = 0, w[64];                        // packed p; positive halves compare as integers
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    float x[32];
                    tmem_ld32(ts + 32 * ch, x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), mul2, b2);
                        const float2 e = make_float2(exp2_of(y.x), exp2_of(y.y));
                        sum = __fadd2_rn(sum, e);
                        w[16 * ch + i] = Half16<f16>::narrow2(e.x, e.y);
                        top = __vmaxu2(top, w[16 * ch + i]);
                    }
                }
                far = max(top & 0xFFFFu, top >> 16) > 0x7800u;  // above 2^15, or not a number
                // over the scores, unless they are wanted again
                if (!__any_sync(0xFFFFFFFFu, far)) {
                    l += sum.x + sum.y;
                    tmem_put32(ts, w);
                    tmem_put32(ts + 32, w + 32);
                }
            }
            // a new reference for the rows that want one, and p again
            auto again = [&](auto masked) {
                constexpr bool kMasked = decltype(masked)::value;
                float mx = kKv4Least, f = 1.f;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    float x[32];
                    tmem_ld32(ts + 32 * ch, x);
                    float a = kKv4Least, b = kKv4Least;
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        if (!kMasked || seen(32 * ch + i))
                            a = fmaxf(a, x[i]);
                        if (!kMasked || seen(32 * ch + i + 1))
                            b = fmaxf(b, x[i + 1]);
                    }
                    mx = fmaxf(mx, fmaxf(a, b));
                }
                const float top = mx == kKv4Least ? kKv4Least : mx * mul;
                if (top > m + kPromptRoom) {
                    f = exp2_of(m - top);
                    m = top;
                    l *= f;
                }
                if (j > 0 && __any_sync(0xFFFFFFFFu, f != 1.f)) {
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        float x[32];
                        tmem_ld32(to + 32 * ch, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] *= f;
                        tmem_st32(to + 32 * ch, x);
                    }
                }
                const float2 mul2 = make_float2(mul, mul);
                const float2 b2 = m == kKv4Least ? make_float2(0.f, 0.f)
                                                 : make_float2(kPromptBase - m, kPromptBase - m);
                float2 sum = make_float2(0.f, 0.f);
                // (a chunk's p takes columns of scores that have been read)
#pragma unroll 1
                for (int ch = 0; ch < 4; ch += 2) {
                    uint32_t w[32];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float x[32];
                        tmem_ld32(ts + 32 * (ch + k), x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), mul2, b2);
                            float2 e = make_float2(exp2_of(y.x), exp2_of(y.y));
                            if (kMasked) {
                                e.x = seen(32 * (ch + k) + 2 * i) ? e.x : 0.f;
                                e.y = seen(32 * (ch + k) + 2 * i + 1) ? e.y : 0.f;
                            }
                            sum = __fadd2_rn(sum, e);
                            w[16 * k + i] = Half16<f16>::narrow2(e.x, e.y);
                        }
                    }
                    tmem_put32(ts + 16 * ch, w);
                }
                l += sum.x + sum.y;
            };
            if (__any_sync(0xFFFFFFFFu, far)) {
                if (whole)
                    again(std::false_type{});
                else
                    again(std::true_type{});
            }
            tmem_put_wait();
            tc_fence_before_sync();
            bar_arrive(pfull + 8 * t);
        }
        if (ok && count > 0)
            ok = __all_sync(0xFFFFFFFFu, prompt_wait(done, 0, bad, limit)) && !*bad;
        if (ok) {
            tc_fence_after_sync();
            const float gv = p.vscale ? __ldg(p.vscale + h) : 1.f;
            const float f = l > 0.f || l != l ? gv / l : 0.f;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                float x[32];
                if (count > 0)
                    tmem_ld32(to + 32 * ch, x);
                if (real)
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        kv4_store<T>(p, s.q0 + row_i, row_h, 32 * ch + i,
                                     f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                              : make_float4(x[i] * f, x[i + 1] * f, x[i + 2] * f, x[i + 3] * f));
            }
            if (real && p.lse != nullptr)
                p.lse[(int64_t)(s.q0 + row_i) * p.Hk * p.G + row_h] = kv4_lse(m, l, kPromptBase);
        }
    } else if (warp < 12) {
        // ------------------------------------------------ keys and values
        const int r = tid & 127, g = r >> 4, oct = r & 15;      // a token's keys; a group of eight tokens' values
        const int *row = p.table + seq * p.table_ld;
        const uint8_t *head = p.cache + (int64_t)h * p.tpp * kTile;
        const int64_t page_bytes = (int64_t)p.Hk * p.tpp * kTile;
        const int tiles = (most + kKv4Tile - 1) / kKv4Tile;
        uint4 kcode[D / 32], vcode[4];
        uint2 ksc = make_uint2(0, 0), vsc = make_uint2(0, 0);
        bool khave = false, vhave = false;
        // The cache's tiles of 16 tokens that a thread goes through, eight
        // apart: their block in the table and place in its page, advanced
        // without a division. A page is looked at when it is used, a tile after
        // it was loaded, so that nothing waits for it.
        const int by_blk = 8 / p.tpp, by_in = 8 - by_blk * p.tpp;
        struct Walk {
            int t16, blk, in;                                   // the tile whose page comes next
            int page, place;                                    // the tile before: its page, its place there
        };
        auto ahead = [&](Walk &w) {
            w.place = w.in;
            w.page = w.t16 < tiles ? __ldg(row + w.blk) : -1;
            w.t16 += 8;
            w.blk += by_blk;
            w.in += by_in;
            if (w.in >= p.tpp) {
                w.in -= p.tpp;
                ++w.blk;
            }
        };
        auto at = [&](const Walk &w) { return head + w.page * page_bytes + w.place * kTile; };
        Walk kw = {r >> 4, (r >> 4) / p.tpp, (r >> 4) % p.tpp, -1, 0},
             vw = {oct >> 1, (oct >> 1) / p.tpp, (oct >> 1) % p.tpp, -1, 0};
        auto fetch_k = [&]() {
            khave = kw.page >= 0 && kw.page < p.pages;
            if (!khave)
                return;
            const uint8_t *a = at(kw);
            const uint4 *c = reinterpret_cast<const uint4 *>(a + (r & 15) * (D / 2));
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                kcode[i] = __ldg(c + i);
            if constexpr (D == 128)
                ksc = __ldg(reinterpret_cast<const uint2 *>(a + kv4_kscale(D) + (r & 15) * 8));
            else
                ksc.x = __ldg(reinterpret_cast<const uint32_t *>(a + kv4_kscale(D) + (r & 15) * 4));
        };
        auto fetch_v = [&]() {
            vhave = vw.page >= 0 && vw.page < p.pages && g < G16;
            if (!vhave)
                return;
            const uint8_t *a = at(vw);
            const uint4 *c = reinterpret_cast<const uint4 *>(a + kv4_v(D) + g * 128 + (oct & 1) * 64);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                vcode[i] = __ldg(c + i);
            vsc = __ldg(reinterpret_cast<const uint2 *>(a + kv4_vscale(D) + g * 16 + (oct & 1) * 8));
        };
        auto keys = [&](int j) {
            const unsigned in = __ballot_sync(0xFFFFFFFFu, khave);
            if (lane == 0)
                present[4 * (j & 3) + (warp - 8)] = (in & 1u) | (in >> 15 & 2u);
#pragma unroll
            for (int gg = 0; gg < G16; ++gg) {
                const uint4 u = kcode[gg >> 1];
                const uint32_t w[2] = {khave ? (gg & 1 ? u.z : u.x) : 0u, khave ? (gg & 1 ? u.w : u.y) : 0u};
                const uint32_t sb = ((gg & 4) ? ksc.y : ksc.x) >> (8 * (gg & 3)) & 0xFFu;
                const uint32_t f = khave ? scales2((uint16_t)(sb * 0x0101u)) : 0u;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t e[4];
                    widen4(w[k], e);
                    const int c = 2 * gg + k;
                    sts128(base + L::k + (j & 1) * L::kK + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4), hmul2(e[0], f),
                           hmul2(e[1], f), hmul2(e[2], f), hmul2(e[3], f));
                }
            }
            fence_proxy_async_smem();
            bar_arrive(kfull + 8 * (j & 1));
        };
        auto values = [&](int j) {
            if (g < G16) {
                // tokens past the sequence's end, and those of a page that is
                // not there, count as zeros whatever their bytes
                const int left = vhave ? s.len - (j * kPromptTokens + oct * 8) : 0;
                uint32_t f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = scales2((uint16_t)((i & 2 ? vsc.y : vsc.x) >> (16 * (i & 1))));
                    f[i] = (2 * i < left ? two & 0xFFFFu : 0u) | (2 * i + 1 < left ? two & 0xFFFF0000u : 0u);
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint32_t e[4][4], o[4][4];                  // [pair of tokens][pair of features]
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a = vhave ? (w ? vcode[i].y : vcode[i].x) : 0u,
                                       b = vhave ? (w ? vcode[i].w : vcode[i].z) : 0u;
                        widen4((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), e[i]);
                        widen4(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), o[i]);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int d = g * 16 + 8 * w + 2 * k;
                        const uint32_t to = base + L::v + (j & 1) * L::kV + (oct >> 3) * (D * 128) + d * 128;
                        sts128(to + (((oct & 7) ^ (d & 7)) << 4), hmul2(e[0][k], f[0]), hmul2(e[1][k], f[1]),
                               hmul2(e[2][k], f[2]), hmul2(e[3][k], f[3]));
                        sts128(to + 128 + (((oct & 7) ^ ((d + 1) & 7)) << 4), hmul2(o[0][k], f[0]),
                               hmul2(o[1][k], f[1]), hmul2(o[2][k], f[2]), hmul2(o[3][k], f[3]));
                    }
                }
            }
            fence_proxy_async_smem();
            bar_arrive(vfull + 8 * (j & 1));
        };
        ahead(kw);
        ahead(vw);
        fetch_k();
        fetch_v();
        ahead(kw);
        ahead(vw);
        for (int j = 0; j < count; ++j) {
            const uint32_t again = ((j >> 1) - 1) & 1;          // the phase that frees a buffer
            if (j > 1 && !__all_sync(0xFFFFFFFFu, prompt_wait(kfree + 8 * (j & 1), again, bad, limit)))
                break;
            keys(j);
            fetch_k();
            ahead(kw);
            if (j > 1 && !__all_sync(0xFFFFFFFFu, prompt_wait(vfree + 8 * (j & 1), again, bad, limit)))
                break;
            values(j);
            fetch_v();
            ahead(vw);
        }
    } else if (count > 0) {
        // ------------------------------------------------------ the products
        // The whole warp goes through this, so that the descriptors are
        // computed in uniform registers; one elected lane issues.
        const bool one = elect_lane();
        const uint32_t is = umma_idesc_f16(0, 128, 128), io = umma_idesc_f16(0, 128, D);
        const uint64_t dq = umma_desc_sw128(base + L::q), dk = umma_desc_sw128(base + L::k),
                       dv = umma_desc_sw128(base + L::v);
        auto wait = [&](uint32_t bar, int phase) {
            return __all_sync(0xFFFFFFFFu, prompt_wait(bar, (uint32_t)phase & 1u, bad, limit));
        };
        auto scores = [&](int t, int j) {
            const uint64_t a = dq + t * (L::kQ >> 4), b = dk + (j & 1) * (L::kK >> 4);
            if (one) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t step = (uint64_t)((k >> 2) * (16384 >> 4) + 2 * (k & 3));
                    if (k == 0)
                        umma_f16(tmem + t * 128, a, b, is, 0);
                    else
                        umma_f16(tmem + t * 128, a + step, b + step, is, 1);
                }
                umma_commit(sfull + 8 * t);
                if (t == 1)
                    umma_commit(kfree + 8 * (j & 1));
            }
            __syncwarp();
        };
        bool ok = wait(kfull, 0);
        if (ok) {
            tc_fence_after_sync();
            scores(0, 0);
            scores(1, 0);
        }
        for (int j = 0; ok && j < count; ++j) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                ok = ok && wait(pfull + 8 * t, j) && (t == 1 || wait(vfull + 8 * (j & 1), j >> 1));
                if (!ok)
                    break;
                tc_fence_after_sync();
                if (one) {
                    const uint64_t b = dv + (j & 1) * (L::kV >> 4);
#pragma unroll
                    for (int k = 0; k < kPromptTokens / 16; ++k)
                        umma_f16_ta(tmem + 256 + t * 128, tmem + t * 128 + 8 * k,
                                    b + (k >> 2) * (D * 128 >> 4) + 2 * (k & 3), io, k == 0 ? j > 0 : 1);
                    if (t == 1)
                        umma_commit(vfree + 8 * (j & 1));
                }
                __syncwarp();
                if (j + 1 < count) {
                    ok = t == 1 || wait(kfull + 8 * ((j + 1) & 1), (j + 1) >> 1);
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    scores(t, j + 1);
                }
            }
        }
        // nothing may be in flight when the tensor memory is given back
        if (one)
            umma_commit(done);
        __syncwarp();
        const unsigned long long t0 = global_ns();
        while (!mbar_try_wait(done, 0))
            if (global_ns() - t0 > limit) {
                *bad = 1;
                break;
            }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after_sync();
        if (*bad && lane == 0)
            atomicAdd(p.timeouts, 1u);
        tmem_dealloc(tmem, 512);
    }
}

} // namespace rmsk
