// fp8_gemm.cuh -- the product of two 8-bit tensors with fp32 scales: A [M,K]
// with a scale for each 128 columns of a row, B [N,K] with one for each block
// of 128 x 128, on the fifth-generation tensor cores.
//
// Mathematics. With groups g of 128 columns,
//   out[m,n] = sum_g sa[m,g] sb[n / 128,g] P_g[m,n],
//   P_g[m,n] = sum_{k in g} qa[m,k] qb[n,k],
// so the scales are constant within one step of 128 in K. P_g is formed by
// four tcgen05.mma (K = 32 each, kind::f8f6f4, accumulated in fp32 in tensor
// memory), read back, and added to fp32 sums in registers with one fused
// multiply-add an element. The sums over the groups are thus plain fp32 sums
// of correctly scaled terms; the only rounding to fewer bits is the last, to
// the output's type.
//
// Tiles. One CTA to a tile of 128 rows of the "row operand" (tensor-memory
// lanes) by BN rows of the "column operand" (tensor-memory columns), its K
// split over a cluster of KS CTAs:
//  - few tokens (SWAP): the weight B is the row operand and the tokens are
//    the columns (BN = 16, 32 or 64 >= M), so a tile wastes no tensor-core
//    row and every SM streams its own rows of the weight;
//  - more: the tokens are the rows, 128 rows of B the columns.
//
// Roles (64 + 32 EW threads): warp 0 feeds a ring of stages (tensor copies,
// 128-byte swizzle: a stage is 128 columns, exactly one swizzle span, of both
// operands), warp 1 issues the MMAs into NB buffers of tensor memory in turn,
// the EW other warps read the buffers and keep the sums. At the end each CTA
// of a cluster owns some rows of the tile; the others send it theirs, counted
// on its barrier, by asynchronous 16-byte stores straight from registers (up
// to 32 columns) or through shared memory by one bulk copy an owner. The owner
// adds them in rank order and writes out: the same bits on every run. (With
// the sums left where they were and read by their owners after a cluster
// barrier, 1 x 6144 x 4096 took 8.0 us against 6.7, 64 x 4096 x 4096 9.0
// against 7.9.)
//
// Every wait is bounded (about one second, or the test limit); one that runs
// out counts in the library's timeout counter, and the CTA skips its work but
// still stores its (meaningless) sums into its peers, which count on them,
// meets its cluster, waits (bounded) for its copies, its peers' sums and its
// MMAs in flight and frees its tensor memory.
#pragma once

#include "../gemv_tc.cuh"
#include "fp8.h"

namespace rmsk {

constexpr int kFp8MaxCluster = 8;                      // CTAs that split K
constexpr int kFp8TileR = 128;                          // rows of the row operand
constexpr uint32_t kFp8StageR = kFp8TileR * kFp8Group;  // its bytes in a stage

__host__ __device__ constexpr int fp8_epi_warps(int BN) { return BN >= 128 ? 8 : 4; }
__host__ __device__ constexpr int fp8_gemm_threads(int BN) { return 64 + 32 * fp8_epi_warps(BN); }
// Whether a cluster's sums travel by bulk copies (else by stores from
// registers, which are quicker for few columns).
__host__ __device__ constexpr bool fp8_bulk(int BN) { return BN >= 64; }
__host__ __device__ constexpr int fp8_acc_bufs(int BN) { return BN >= 64 ? 2 : 4; }
__host__ __device__ constexpr int fp8_tmem_cols(int BN) { return BN * fp8_acc_bufs(BN); }

// Shared memory of one CTA, byte offsets from a 1024-byte aligned base: the
// ring (NSt stages of 128 + BN rows of 128 bytes; alone, the sums [128][BN +
// 4] over it at the end), with a cluster the sums received ([rank][own rows]
// [BN + 4]), the scales of the tokens with SWAP ([groups][BN + 4]), the
// mbarriers (full, empty a stage; full, empty a buffer; drain; received),
// eight words (tensor-memory address, failure flag, stages issued, consumed).
struct Fp8GemmLayout {
    int NSt, rpo;                                       // rpo: rows of the tile a CTA owns
    uint32_t stage, recv, sc, bar, slots, total;        // total: with 1023 bytes of alignment
};

__host__ __device__ inline Fp8GemmLayout fp8_gemm_layout(int BN, bool swap, int NSt, int groups,
                                                         int KS)
{
    Fp8GemmLayout L;
    L.NSt = NSt;
    L.rpo = (kFp8TileR + KS - 1) / KS;
    L.stage = kFp8StageR + (uint32_t)BN * kFp8Group;
    const uint32_t ring = (uint32_t)NSt * L.stage, row = (uint32_t)(BN + 4) * 4u;
    const uint32_t sums = (uint32_t)kFp8TileR * row;
    // where the sums go over the ring before anything else: alone, and where
    // they travel by bulk copies
    const uint32_t first = (KS == 1 || fp8_bulk(BN)) && sums > ring ? sums : ring;
    L.recv = KS > 1 ? first : 0u;
    L.sc = first + (KS > 1 ? (uint32_t)(KS * L.rpo) * row : 0u);
    L.bar = L.sc + (swap ? (uint32_t)groups * row : 0u);
    L.slots = L.bar + 8u * (uint32_t)(2 * NSt + 2 * fp8_acc_bufs(BN) + 2);
    L.total = L.slots + 32u + 1023u;
    // An SM has 512 columns of tensor memory. A CTA that waits for its
    // columns while a peer of its cluster holds some elsewhere could wait
    // for ever, so no more CTAs may share an SM than have columns: each
    // takes at least its share of the SM's 228 KB of shared memory (1 KB of
    // it the system's own).
    const uint32_t least = 228u * 1024u / 512u * (uint32_t)fp8_tmem_cols(BN) - 1024u;
    if (L.total < least)
        L.total = least;
    return L;
}

struct Fp8GemmParams {
    const float *sa;   // [M,G]
    const float *sb;   // [ceil(N / 128),G]
    void *out;         // [M,N], row stride ldo
    int64_t ldo;
    int M, N, G;
    int KS;            // CTAs of a cluster, which split the G groups
    int tiles_r;       // tiles along the row operand
    uint32_t idesc;    // instruction descriptor of the MMAs
    int static_w;      // B and sb may be read before the wait on the previous kernel
    int vec;           // rows of out start at multiples of four elements
    uint32_t extra_tx, wait_limit_us;   // test hook of the bounded waits
    Fp8GemmLayout L;
};

// Instruction descriptor of kind::f8f6f4: as umma_idesc_f16, the formats of
// A and B (0 e4m3, 1 e5m2) each on its own.
__host__ __device__ constexpr uint32_t umma_idesc_f8(uint32_t a, uint32_t b, int M, int N)
{
    return (1u << 4) | (a << 7) | (b << 10) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// D (tensor memory) = A B^T (+ D when accumulate != 0), kind::f8f6f4, K = 32.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// One lane of a converged warp. The roles' loops are run by whole warps and
// only the instructions that one thread must issue sit under this predicate:
// descriptors and barriers then stay in uniform registers. (With the loop
// itself under `lane == 0` a group of 128 columns took some 1100 cycles to
// issue.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// Bounded wait of a whole warp, as tc_wait, but the clock is only read once
// in a while (each try already blocks for a time of the hardware's choice).
// `fail` is the flag's shared address; the limit is worked out only where it
// is needed (both to spare the loops' registers).
__device__ __forceinline__ bool fp8_wait(uint32_t bar, uint32_t parity, uint32_t limit_us,
                                         uint32_t fail)
{
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)))
        return true;
    unsigned long long t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)))
                return true;
        int failed;
        asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(failed) : "r"(fail) : "memory");
        const unsigned long long t = global_ns();
        if (t0 == 0)
            t0 = t;
        const bool stop = failed != 0 || t - t0 > wait_limit_ns(limit_us);
        if (__any_sync(0xFFFFFFFFu, stop)) {
            asm volatile("st.volatile.shared.s32 [%0], %1;" ::"r"(fail), "r"(1) : "memory");
            return false;
        }
    }
}

// N consecutive fp32 columns of the warp's 32 lanes (lane = this thread);
// complete only after tmem_wait on the same registers.
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]),
                   "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_wait(uint32_t (&v)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

template <typename T> __device__ __forceinline__ void store_out1(T *p, float v)
{
    if constexpr (sizeof(T) == 4)
        *p = v;
    else
        st_row_b16(p, Half16<T>::narrow1(v));
}

template <typename T> __device__ __forceinline__ void store_out4(T *p, float4 v)
{
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4 *>(p) = v;
    else
        asm volatile("st.global.v2.b32 [%0], {%1,%2};" ::"l"(p), "r"(Half16<T>::narrow2(v.x, v.y)),
                     "r"(Half16<T>::narrow2(v.z, v.w))
                     : "memory");
}

// Columns 4 c4 .. of row `row` of the tile at (r0, c0) to out: with SWAP four
// tokens of a feature, else four features of a token.
template <typename T, bool SWAP>
__device__ __forceinline__ void fp8_store_quad(const Fp8GemmParams &p, int r0, int c0, int row, int c4,
                                               float4 v)
{
    T *out = static_cast<T *>(p.out);
    const float e[4] = {v.x, v.y, v.z, v.w};
    if constexpr (SWAP) {
        const int n = r0 + row, m = c0 + c4 * 4;
        if (n < p.N) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (m + j < p.M)
                    store_out1<T>(out + (int64_t)(m + j) * p.ldo + n, e[j]);
        }
    } else {
        const int m = r0 + row, n = c0 + c4 * 4;
        if (m < p.M) {
            T *to = out + (int64_t)m * p.ldo + n;
            if (p.vec && n + 4 <= p.N) {
                store_out4<T>(to, v);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < p.N)
                        store_out1<T>(to + j, e[j]);
            }
        }
    }
}

// Rows row0 .. row0 + own - 1 of the tile, four columns at a time, to out:
// each the sum, in rank order, of what `KS` CTAs hold of it ([KS][rpo][BN +
// 4]). NT threads, of which this is number t.
template <typename T, int BN, bool SWAP, int NT>
__device__ __forceinline__ void fp8_finish(const Fp8GemmParams &p, const float *sums, int KS, int rpo,
                                           int r0, int c0, int row0, int own, int nc, int t)
{
    constexpr int SROW = BN + 4, UB = 4;                // quads a thread has in hand
    const int units = own * nc;
    for (int ub = t; ub < units; ub += UB * NT) {
        int rl[UB], c4[UB];
        float4 v[UB];
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int u = min(ub + i * NT, units - 1);
            rl[i] = SWAP ? u % own : u / nc;
            c4[i] = SWAP ? u / own : u % nc;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                const float4 w = *reinterpret_cast<const float4 *>(sums + (k * rpo + rl[i]) * SROW +
                                                                   c4[i] * 4);
                v[i].x += w.x;
                v[i].y += w.y;
                v[i].z += w.z;
                v[i].w += w.w;
            }
        }
#pragma unroll
        for (int i = 0; i < UB; ++i)
            if (ub + i * NT < units)
                fp8_store_quad<T, SWAP>(p, r0, c0, row0 + rl[i], c4[i], v[i]);
    }
}

// grid = tiles x KS CTAs (KS consecutive ones a cluster); the tiles along the
// row operand follow one another.
template <typename T, int BN, bool SWAP>
__global__ void __launch_bounds__(fp8_gemm_threads(BN))
rms_fp8_gemm(const Fp8GemmParams p, const __grid_constant__ CUtensorMap tmR,
             const __grid_constant__ CUtensorMap tmC, unsigned int *timeouts)
{
    constexpr int EW = fp8_epi_warps(BN), NB = fp8_acc_bufs(BN);
    constexpr int CW = BN * 4 / EW;                     // columns a thread sums
    constexpr int SROW = BN + 4, kScRow = BN + 4;       // floats a row of the sums, the scales
    constexpr uint32_t kRow = SROW * 4u;
    constexpr bool BULK = fp8_bulk(BN);
    constexpr uint32_t kCols = fp8_tmem_cols(BN);
    extern __shared__ __align__(1024) unsigned char fp8_smem[];

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int KS = p.KS, rank = KS > 1 ? (int)cluster_ctarank() : 0;
    const int g0 = rank * p.G / KS, ng = (rank + 1) * p.G / KS - g0;   // this CTA's groups
    const int tile = (int)(blockIdx.x / KS);
    const int r0 = tile % p.tiles_r * kFp8TileR, c0 = tile / p.tiles_r * BN;
    const Fp8GemmLayout &L = p.L;
    const int NSt = L.NSt;
    const uint32_t raw_s = smem_addr(fp8_smem);
    unsigned char *base = fp8_smem + (((raw_s + 1023u) & ~1023u) - raw_s);
    const uint32_t ring_s = smem_addr(base), recv_s = ring_s + L.recv;
    const int nc = SWAP ? (min(BN, p.M - c0) + 3) / 4 : BN / 4;        // column quads wanted
    // the rows of the tile that this CTA adds up and writes
    const int own = max(0, min(L.rpo, kFp8TileR - rank * L.rpo));
    float *sc = reinterpret_cast<float *>(base + L.sc);
    const uint32_t full0 = smem_addr(base + L.bar), empty0 = full0 + 8u * (uint32_t)NSt;
    const uint32_t accf0 = empty0 + 8u * (uint32_t)NSt, acce0 = accf0 + 8u * NB;
    const uint32_t dbar = acce0 + 8u * NB, rxbar = dbar + 8u;
    int *slots = reinterpret_cast<int *>(base + L.slots);
    volatile int *fail = slots + 1;
    const uint32_t fail_s = smem_addr(slots + 1);

    if (warp == 0) {
        tmem_alloc(smem_addr(slots), kCols);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (int s = 0; s < NSt; ++s) {
            mbar_init(full0 + 8u * s, 1);
            mbar_init(empty0 + 8u * s, 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(accf0 + 8u * b, 1);
            mbar_init(acce0 + 8u * b, EW);
        }
        mbar_init(dbar, 1);
        mbar_init(rxbar, 1);
        if (KS > 1)             // every peer's sums of the own rows
            mbar_expect_tx(rxbar, (uint32_t)((KS - 1) * own) * (BULK ? kRow : (uint32_t)nc * 16u));
        slots[1] = slots[2] = slots[3] = 0;
    }
    if (tid == 64) {
        prefetch_tmap(&tmR);
        prefetch_tmap(&tmC);
    }
    mbar_init_fence();
    tc_fence_before_sync();
    __syncthreads();
    if (KS > 1)                 // the peers' barriers exist once all have arrived
        cluster_arrive_release();
    tc_fence_after_sync();
    const uint32_t tmem = static_cast<uint32_t>(slots[0]);

    if (warp == 0) {
        // ------------------------------------------------------ copies
        const CUtensorMap *tmW = SWAP ? &tmR : &tmC, *tmA = SWAP ? &tmC : &tmR;
        const uint32_t offW = SWAP ? 0u : kFp8StageR, offA = SWAP ? kFp8StageR : 0u;
        const int w0 = SWAP ? r0 : c0, a0 = SWAP ? c0 : r0;
        // the weight's first stages may start before the previous kernel is
        // complete
        const int early = p.static_w ? min(ng, NSt) : 0;
        if (elect_one()) {
            for (int q = 0; q < early; ++q) {
                mbar_expect_tx(full0 + 8u * q, L.stage + p.extra_tx);
                tma_load_2d(ring_s + (uint32_t)q * L.stage + offW, tmW, (g0 + q) * kFp8Group, w0,
                            full0 + 8u * q);
            }
        }
        griddep_wait();
        int q = 0;
        for (int s = 0, u = 0; q < ng; ++q) {
            const uint32_t dst = ring_s + (uint32_t)s * L.stage, bar = full0 + 8u * s;
            const int x = (g0 + q) * kFp8Group;
            if (u > 0 && !fp8_wait(empty0 + 8u * s, (uint32_t)((u - 1) & 1), p.wait_limit_us, fail_s))
                break;
            if (elect_one()) {
                if (q >= early) {
                    mbar_expect_tx(bar, L.stage + p.extra_tx);
                    tma_load_2d(dst + offW, tmW, x, w0, bar);
                }
                tma_load_2d(dst + offA, tmA, x, a0, bar);
            }
            if (++s == NSt) {
                s = 0;
                ++u;
            }
        }
        if (elect_one())
            slots[2] = q;
        griddep_launch_dependents();
    } else if (warp == 1) {
        // -------------------------------------------------------- MMAs
        const uint64_t dr0 = umma_desc_sw128(ring_s);
        int q = 0;
        for (int s = 0, us = 0, b = 0, ub = 0; q < ng; ++q) {
            if (ub > 0 && !fp8_wait(acce0 + 8u * b, (uint32_t)((ub - 1) & 1), p.wait_limit_us, fail_s))
                break;
            if (!fp8_wait(full0 + 8u * s, (uint32_t)(us & 1), p.wait_limit_us, fail_s))
                break;
            tc_fence_after_sync();
            if (elect_one()) {
                const uint64_t da = dr0 + (uint64_t)((uint32_t)s * (L.stage >> 4));
                const uint64_t db = da + (kFp8StageR >> 4);
#pragma unroll
                for (int k4 = 0; k4 < kFp8Group / 32; ++k4)
                    umma_f8(tmem + (uint32_t)(b * BN), da + 2 * k4, db + 2 * k4, p.idesc,
                            k4 != 0 ? 1u : 0u);
                umma_commit(empty0 + 8u * s);
                umma_commit(accf0 + 8u * b);
            }
            __syncwarp();
            if (++s == NSt) {
                s = 0;
                ++us;
            }
            if (++b == NB) {
                b = 0;
                ++ub;
            }
        }
        if (elect_one())
            slots[3] = q;
    } else {
        // ------------------------------------------------------ the sums
        const int etid = tid - 64, q4 = warp & 3, half = (warp - 2) / 4;
        const int row = q4 * 32 + lane;                 // of the row operand's tile
        const int col0 = half * CW;
        griddep_wait();
        const float *sb = p.sb + (int64_t)((SWAP ? r0 : c0) / kFp8Group) * p.G + g0;
        const float *sa = p.sa + (int64_t)min(r0 + row, p.M - 1) * p.G + g0;
        if constexpr (SWAP) {
            // the products of the tokens' scales and the block's: each warp
            // takes every EW-th token, its lanes the groups (neighbours in
            // memory); all of a lane's loads are in flight at once (a round
            // trip takes 1 to 2 us while the weight streams in)
            const int w = warp - 2, nt = min(BN, p.M - c0);
            for (int g = lane; g < ng; g += 32) {
                const float sbg = __ldg(sb + g);
                float v[BN / EW];
#pragma unroll
                for (int j = 0; j < BN / EW; ++j)
                    v[j] = w + j * EW < nt
                               ? __ldcg(p.sa + (int64_t)(c0 + w + j * EW) * p.G + g0 + g)
                               : 0.f;
#pragma unroll
                for (int j = 0; j < BN / EW; ++j)
                    sc[g * kScRow + w + j * EW] = v[j] * sbg;
            }
            named_bar_sync(1, EW * 32);
        }
        float2 acc[CW / 2];
#pragma unroll
        for (int i = 0; i < CW / 2; ++i)
            acc[i] = make_float2(0.f, 0.f);
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        float sa_next = 0.f, sb_next = 0.f;
        if constexpr (!SWAP) {
            sa_next = sa[0];
            sb_next = __ldg(sb);
        }
        for (int q = 0, b = 0, ub = 0; q < ng; ++q) {
            const float s = sa_next * sb_next;
            if constexpr (!SWAP) {
                if (q + 1 < ng) {                   // one group ahead
                    sa_next = sa[q + 1];
                    sb_next = __ldg(sb + q + 1);
                }
            }
            if (!fp8_wait(accf0 + 8u * b, (uint32_t)(ub & 1), p.wait_limit_us, fail_s))
                break;
            tc_fence_after_sync();
            const uint32_t at = tmem + lanes + (uint32_t)(b * BN + col0);
            uint32_t v[2][16];                      // the next 16 columns come while
            tmem_ld_start(at, v[0]);                // these are added
#pragma unroll
            for (int c = 0; c < CW; c += 16) {
                uint32_t(&w)[16] = v[(c / 16) & 1];
                tmem_wait(w);
                if (c + 16 < CW)
                    tmem_ld_start(at + (uint32_t)(c + 16), v[(c / 16 + 1) & 1]);
                if (c + 16 >= CW) {                 // all of the buffer is in registers
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(acce0 + 8u * b);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 s4 = make_float4(s, s, s, s);
                    if constexpr (SWAP)
                        s4 = *reinterpret_cast<const float4 *>(sc + q * kScRow + col0 + c + 4 * j);
                    acc[c / 2 + 2 * j] = vfma(
                        make_float2(__uint_as_float(w[4 * j]), __uint_as_float(w[4 * j + 1])),
                        make_float2(s4.x, s4.y), acc[c / 2 + 2 * j]);
                    acc[c / 2 + 2 * j + 1] = vfma(
                        make_float2(__uint_as_float(w[4 * j + 2]), __uint_as_float(w[4 * j + 3])),
                        make_float2(s4.z, s4.w), acc[c / 2 + 2 * j + 1]);
                }
            }
            if (++b == NB) {
                b = 0;
                ++ub;
            }
        }
        if (KS > 1) {
            cluster_wait_acquire();
            if constexpr (BULK) {
                // the tile's sums over the ring, then each owner's rows in one
                // copy (should the CTA have failed, what still lands in the
                // ring spoils sums that do not matter)
                named_bar_sync(1, EW * 32);             // every warp has seen the last buffer
                float4 *to = reinterpret_cast<float4 *>(base + (row * SROW + col0) * 4);
#pragma unroll
                for (int i = 0; i < CW / 4; ++i)
                    to[i] = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x,
                                        acc[2 * i + 1].y);
                fence_proxy_async_smem();
                named_bar_sync(1, EW * 32);
                if (etid < KS && etid != rank) {
                    const int theirs = min(L.rpo, kFp8TileR - etid * L.rpo);
                    bulk_s2s_cluster(
                        cluster_map(recv_s + (uint32_t)(rank * L.rpo) * kRow, (uint32_t)etid),
                        ring_s + (uint32_t)(etid * L.rpo) * kRow, (uint32_t)theirs * kRow,
                        cluster_map(rxbar, (uint32_t)etid));
                }
                // this CTA's own rows
                for (int i = etid; i < own * (SROW / 4); i += EW * 32)
                    reinterpret_cast<float4 *>(base + L.recv + (uint32_t)(rank * L.rpo) * kRow)[i] =
                        reinterpret_cast<const float4 *>(base + (uint32_t)(rank * L.rpo) * kRow)[i];
                if (etid < KS && etid != rank)
                    bulk_wait_read_all();
                __syncwarp();
            } else {
                // this row's sums to its owner
                const int owner = row / L.rpo;
                const uint32_t at =
                    recv_s + (uint32_t)(((rank * L.rpo + row % L.rpo) * SROW + col0) * 4);
                const uint32_t to = cluster_map(at, (uint32_t)owner);
                const uint32_t bar = cluster_map(rxbar, (uint32_t)owner);
#pragma unroll
                for (int i = 0; i < CW / 4; ++i) {
                    if (col0 / 4 + i >= nc)
                        break;
                    const float4 v =
                        make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
                    if (owner == rank)
                        *reinterpret_cast<float4 *>(base + (at - ring_s) + 16 * i) = v;
                    else
                        st_async_v4(to + 16u * i, v, bar);
                }
                __syncwarp();
            }
            cluster_arrive_relaxed();                   // nothing more goes to a peer
            named_bar_sync(1, EW * 32);                 // this CTA's own part is there
            if (!mbar_wait_bounded_cluster(rxbar, 0, wait_limit_ns(p.wait_limit_us)))
                *fail = 1;
            if (!*fail)
                fp8_finish<T, BN, SWAP, EW * 32>(p, reinterpret_cast<const float *>(base + L.recv),
                                                 KS, L.rpo, r0, c0, rank * L.rpo, own, nc, etid);
        } else if constexpr (SWAP) {
            // alone with a feature a lane: neighbouring lanes write neighbours
            if (!*fail) {
#pragma unroll
                for (int i = 0; i < CW / 4; ++i)
                    if (col0 / 4 + i < nc)
                        fp8_store_quad<T, SWAP>(p, r0, c0, row, col0 / 4 + i,
                                                make_float4(acc[2 * i].x, acc[2 * i].y,
                                                            acc[2 * i + 1].x, acc[2 * i + 1].y));
            }
        } else {
            // the ring is drained: the last buffer was complete, so every
            // copy has landed and every MMA has read it (or the CTA has
            // failed, and copies may still land: write nothing)
            named_bar_sync(1, EW * 32);
            if (!*fail) {
                float4 *to = reinterpret_cast<float4 *>(base + (row * SROW + col0) * 4);
#pragma unroll
                for (int i = 0; i < CW / 4; ++i)
                    to[i] = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x,
                                        acc[2 * i + 1].y);
            }
        }
    }
    if (KS > 1 && warp < 2) {
        cluster_wait_acquire();
        cluster_arrive_relaxed();
    }

    // every role has finished or given up
    __syncthreads();
    if (!SWAP && KS == 1 && !*fail)
        fp8_finish<T, BN, SWAP, fp8_gemm_threads(BN)>(p, reinterpret_cast<const float *>(base), 1,
                                                      kFp8TileR, r0, c0, 0, kFp8TileR, nc, tid);
    if (*fail) {
        const unsigned long long limit = wait_limit_ns(p.wait_limit_us);
        if (tid == 0) {
            for (int q = slots[3]; q < slots[2]; ++q)
                (void)mbar_wait_bounded(full0 + 8u * (q % NSt), (uint32_t)((q / NSt) & 1), limit);
            atomicAdd(timeouts, 1u);
        }
        if (warp == 1) {        // the lane that issued the MMAs commits them
            if (elect_one())
                umma_commit(dbar);
            __syncwarp();
            (void)mbar_wait_bounded(dbar, 0, limit);
        }
    }
    tc_fence_before_sync();
    if (KS > 1) {               // no CTA leaves while a peer may still store into it
        cluster_wait_acquire();
        if (*fail)              // (had its wait run out, what was on its way then)
            (void)mbar_wait_bounded_cluster(rxbar, 0, wait_limit_ns(p.wait_limit_us));
    } else {
        __syncthreads();
    }
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kCols);
    }
}

} // namespace rmsk
