// fp8_gemm_pair.cuh -- the product of fp8_gemm.cuh for many tokens: pairs of
// CTAs that share one tile of 256 x 256 (tcgen05.mma with cta_group::2),
// persistent over the tiles.
//
// Mathematics and rounding: as in fp8_gemm.cuh; each group of 128 columns is
// four MMAs (m256 n256 k32) into one of two buffers of tensor memory, read
// back and added to fp32 sums in registers with the group's scales.
//
// Why this shape. At M = 8192, N = 24576, K = 4096 the tensor cores' time is
// the floor (422 us at twice the measured bf16 rate). An SM alone on a 128 x
// 256 tile would read 48 KB of operands from L2 for every 512 cycles of MMAs
// and as much from shared memory; a pair reads each row of A and of B once
// for both SMs, 32 KB each. Reading the groups back is the other limit: 128 x
// 256 sums a group and SM, 64 fp32 FMAs a cycle of the 128 an SM has, so the
// tensor memory is loaded 32 columns at a time by sixteen warps (four on each
// of the SM's quarters, to hide the loads' latency behind one another's
// arithmetic), and the scale of a row and group is one product a thread. The
// sums take 64 registers a thread.
//
// Roles (kPairThreads threads a CTA): warp 0 copies this CTA's 128 rows of
// A and 128 rows of B into the ring; warp 1 of the leader (rank 0) issues the
// MMAs of both; warps 2 and 3 fetch the scales of this CTA's rows (a row's lie
// beside one another in memory, a thread wants one of a row of its own: read
// by the threads that use them, a warp's 32 came from 32 lines a group); the
// sixteen others keep the sums of this CTA's 128 rows. The copies
// of both CTAs complete on the leader's `full` barrier; the MMAs' completion
// is sent to both CTAs' `empty` and `accf` barriers, and both CTAs' readers
// hand a buffer back on the leader's `acce` barrier. The ring and the two
// buffers run on across tiles, so the stores of one tile overlap the first
// groups of the next.
//
// Waits are bounded as in fp8_gemm.cuh. A CTA that gives up still meets its
// peer; the leader then waits (bounded) for copies in flight and MMAs.
#pragma once

#include "fp8_gemm.cuh"

namespace rmsk {

constexpr int kPairTile = 256;                          // rows of A and of B to a pair's tile
constexpr int kPairEpi = 16;                            // epilogue warps of a CTA
constexpr int kPairLd = 32;                             // columns a load of tensor memory
constexpr int kPairScaleWarps = 2;                      // warps that fetch the scales
constexpr int kPairThreads = 128 + 32 * kPairEpi;
// Registers a thread: what the kernel is launched with, and what its first
// four warps (copies, MMAs, scales) and the sixteen others take of that.
constexpr int kPairRegs = 96, kPairRegsCtl = 32, kPairRegsEpi = 112;
static_assert(128 * kPairRegsCtl + 32 * kPairEpi * kPairRegsEpi <= kPairThreads * kPairRegs,
              "the shares fit what the CTA is launched with");
constexpr int kPairStages = 4;
constexpr uint32_t kPairHalf = 128u * kFp8Group;        // 128 rows of one operand
constexpr uint32_t kPairStage = 2u * kPairHalf;
constexpr int kPairBufs = 2;                            // x 256 columns: all tensor memory
constexpr int kPairTileRun = 16;                        // row tiles that are swept together
constexpr int kPairChunk = 16;                          // groups whose scales come together
constexpr int kPairScRow = 129;                         // floats a group of them (no conflicts)
constexpr uint32_t kPairRowBytes = 64;                  // of a row of out staged at a time
// The ring, two times 32 rows of out for each epilogue warp, two chunks of
// scales (for each of the tile's two blocks of columns, group and row their
// product), the mbarriers (full, empty; accf, acce; scales full, empty;
// drain), eight words. All of an SM's shared memory is taken: no other CTA may
// wait for tensor memory beside this one.
constexpr uint32_t kPairOut = kPairStages * kPairStage;
constexpr uint32_t kPairOutSlot = 32u * kPairRowBytes;
constexpr uint32_t kPairSc = kPairOut + 2u * kPairOutSlot * kPairEpi;
constexpr uint32_t kPairScChunk = 2u * kPairChunk * kPairScRow;   // floats
constexpr uint32_t kPairBar = kPairSc + 2u * kPairScChunk * 4u;
static_assert(kPairOut % 512 == 0 && kPairOutSlot % 512 == 0 && kPairBar % 8 == 0, "alignment");
constexpr uint32_t kPairSlots = kPairBar + 8u * (2 * kPairStages + 2 * kPairBufs + 5);
constexpr uint32_t kPairSmem = 227u * 1024u;
static_assert(kPairSlots + 32u + 1023u <= kPairSmem, "shared memory of a pair's CTA");

struct Fp8PairParams {
    const float *sa;   // [M,G]
    const float *sb;   // [ceil(N / 128),G]
    void *out;         // [M,N], row stride ldo
    int64_t ldo;
    int M, N, G;
    int tiles_m, tiles_n;
    uint32_t idesc;
    int static_w;
    int vec;           // rows of out start at multiples of 16 bytes (1), end there too (2)
    uint32_t extra_tx, wait_limit_us;
};

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// The mbarriers at this offset in both CTAs complete a phase once every
// tcgen05 operation this thread issued before has.
__device__ __forceinline__ void umma_commit_pair(uint32_t mbar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::"
                 "cluster.b64 [%0], %1;" ::"r"(mbar),
                 "h"((uint16_t)3)
                 : "memory");
}

// As tma_load_2d, completing on a barrier of either CTA of the pair (`bar`: a
// cluster address). x is a multiple of 128 one-byte elements.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y,
                                                 uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::"
                 "complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

// 16 bytes of out from floats: four fp32 or eight 16-bit values.
template <typename T> __device__ __forceinline__ uint4 pack_out16(const float *f)
{
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    else
        return make_uint4(Half16<T>::narrow2(f[0], f[1]), Half16<T>::narrow2(f[2], f[3]),
                          Half16<T>::narrow2(f[4], f[5]), Half16<T>::narrow2(f[6], f[7]));
}

// 32 consecutive fp32 columns of the warp's 32 lanes, as for 16.
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait(uint32_t (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                   "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(v[30]), "+r"(v[31]));
}

// Tile t of the sweep: runs of kPairTileRun row tiles, each run over all
// column tiles, so that the pairs at work at one time share rows of both
// operands in L2.
__device__ __forceinline__ void pair_tile(const Fp8PairParams &p, int t, int &m0, int &n0)
{
    const int run = t / (kPairTileRun * p.tiles_n);
    const int first = run * kPairTileRun, rows = min(kPairTileRun, p.tiles_m - first);
    const int r = t - first * p.tiles_n;
    m0 = (first + r % rows) * kPairTile;
    n0 = r / rows * kPairTile;
}

// grid = 2 x pairs, cluster (2, 1, 1), kPairThreads threads, kPairSmem bytes.
template <typename T>
__global__ void __launch_bounds__(kPairThreads, 1)
rms_fp8_gemm_pair(const Fp8PairParams p, const __grid_constant__ CUtensorMap tmA,
                  const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmO, unsigned int *timeouts)
{
    constexpr int CW = kPairTile * 4 / kPairEpi;        // columns a thread sums
    extern __shared__ __align__(1024) unsigned char pair_smem[];

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t rank = cluster_ctarank();
    const int pair = (int)blockIdx.x / 2, npairs = (int)gridDim.x / 2;
    const int ntiles = p.tiles_m * p.tiles_n, G = p.G;
    const uint32_t raw_s = smem_addr(pair_smem);
    unsigned char *base = pair_smem + (((raw_s + 1023u) & ~1023u) - raw_s);
    const uint32_t ring_s = smem_addr(base);
    const uint32_t full0 = ring_s + kPairBar, empty0 = full0 + 8u * kPairStages;
    const uint32_t accf0 = empty0 + 8u * kPairStages, acce0 = accf0 + 8u * kPairBufs;
    const uint32_t scf0 = acce0 + 8u * kPairBufs, sce0 = scf0 + 16u, dbar = sce0 + 16u;
    float *sc = reinterpret_cast<float *>(base + kPairSc);
    int *slots = reinterpret_cast<int *>(base + kPairSlots);
    const uint32_t fail_s = smem_addr(slots + 1);

    if (tid == 32) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(full0 + 8u * s, 1);               // the leader's own arrival
            mbar_init(empty0 + 8u * s, 1);
        }
        for (int b = 0; b < kPairBufs; ++b) {
            mbar_init(accf0 + 8u * b, 1);
            mbar_init(acce0 + 8u * b, 2 * kPairEpi);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(scf0 + 8u * b, kPairScaleWarps);
            mbar_init(sce0 + 8u * b, kPairEpi);
        }
        mbar_init(dbar, 1);
        slots[1] = slots[2] = slots[3] = 0;
    }
    if (tid == 64) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 0)
        tmem_alloc_pair(smem_addr(slots), kPairBufs * kPairTile);
    mbar_init_fence();
    tc_fence_before_sync();
    __syncthreads();
    cluster_arrive_release();                           // the peer's barriers exist
    cluster_wait_acquire();
    tc_fence_after_sync();
    const uint32_t tmem = static_cast<uint32_t>(slots[0]);

    if (warp < 4)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairRegsCtl));
    if (warp == 0) {
        // ------------------------------------------------------ copies
        const uint32_t lead = cluster_map(full0, 0);
        bool waited = p.static_w == 0;
        if (waited)
            griddep_wait();
        int q = 0, s = 0, u = 0;
        bool stop = false;
        for (int t = pair; t < ntiles && !stop; t += npairs) {
            int m0, n0;
            pair_tile(p, t, m0, n0);
            m0 += (int)rank * 128;
            n0 += (int)rank * 128;
            for (int g = 0; g < G; ++g, ++q) {
                if (!waited) {
                    // rows of B may come before the previous kernel is
                    // complete, as many as the ring holds
                    const int early = min(G, kPairStages);
                    if (elect_one()) {
                        for (int e = 0; e < early; ++e) {
                            if (rank == 0)
                                mbar_expect_tx(full0 + 8u * e, 2u * kPairStage + p.extra_tx);
                            tma_load_2d_pair(ring_s + (uint32_t)e * kPairStage + kPairHalf, &tmB,
                                             e * kFp8Group, n0, lead + 8u * e);
                        }
                    }
                    __syncwarp();
                    griddep_wait();
                    waited = true;
                }
                if (u > 0 && !fp8_wait(empty0 + 8u * s, (uint32_t)((u - 1) & 1), p.wait_limit_us,
                                       fail_s)) {
                    stop = true;
                    break;
                }
                const bool have_b = p.static_w && q < min(G, kPairStages);
                if (elect_one()) {
                    const uint32_t dst = ring_s + (uint32_t)s * kPairStage, bar = lead + 8u * s;
                    if (!have_b) {
                        if (rank == 0)
                            mbar_expect_tx(full0 + 8u * s, 2u * kPairStage + p.extra_tx);
                        tma_load_2d_pair(dst + kPairHalf, &tmB, g * kFp8Group, n0, bar);
                    }
                    tma_load_2d_pair(dst, &tmA, g * kFp8Group, m0, bar);
                }
                __syncwarp();
                if (++s == kPairStages) {
                    s = 0;
                    ++u;
                }
            }
        }
        if (lane == 0)
            slots[2] = q;
        griddep_launch_dependents();
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------------------------------------------- MMAs
            const uint64_t dr0 = umma_desc_sw128(ring_s);
            int q = 0, s = 0, us = 0, b = 0, ub = 0;
            const int nq = (ntiles - pair + npairs - 1) / npairs * G;
            for (; q < nq; ++q) {
                if (ub > 0 && !fp8_wait(acce0 + 8u * b, (uint32_t)((ub - 1) & 1), p.wait_limit_us, fail_s))
                    break;
                if (!fp8_wait(full0 + 8u * s, (uint32_t)(us & 1), p.wait_limit_us, fail_s))
                    break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t da = dr0 + (uint64_t)((uint32_t)s * (kPairStage >> 4));
                    const uint64_t db = da + (kPairHalf >> 4);
#pragma unroll
                    for (int k4 = 0; k4 < kFp8Group / 32; ++k4)
                        umma_f8_pair(tmem + (uint32_t)(b * kPairTile), da + 2 * k4, db + 2 * k4,
                                     p.idesc, k4 != 0 ? 1u : 0u);
                    umma_commit_pair(empty0 + 8u * s);
                    umma_commit_pair(accf0 + 8u * b);
                }
                __syncwarp();
                if (++s == kPairStages) {
                    s = 0;
                    ++us;
                }
                if (++b == kPairBufs) {
                    b = 0;
                    ++ub;
                }
            }
            if (lane == 0)
                slots[3] = q;
        }
    } else if (warp < 4) {
        // ------------------------------------------------------ scales
        // sc[chunk % 2][block][group][row]: half a warp reads 16 groups of a
        // row, eight rows at a time
        const int w = warp - 2, gl = lane % kPairChunk, rr = lane / kPairChunk;
        const int nblocks = (p.N + 127) / 128;
        griddep_wait();
        int c = 0;
        bool stop = false;
        for (int t = pair; t < ntiles && !stop; t += npairs) {
            int m0, n0;
            pair_tile(p, t, m0, n0);
            m0 += (int)rank * 128;
            const float *sb0 = p.sb + (int64_t)(n0 / 128) * G + gl;
            const float *sb1 = p.sb + (int64_t)min(n0 / 128 + 1, nblocks - 1) * G + gl;
            for (int g0 = 0; g0 < G; g0 += kPairChunk, ++c) {
                const bool in = g0 + gl < G;
                const float b0 = in ? __ldg(sb0 + g0) : 0.f, b1 = in ? __ldg(sb1 + g0) : 0.f;
                if (c >= 2 &&
                    !fp8_wait(sce0 + 8u * (c & 1), (uint32_t)((c / 2 - 1) & 1), p.wait_limit_us, fail_s)) {
                    stop = true;
                    break;
                }
                float *to = sc + (c & 1) * kPairScChunk + gl * kPairScRow;
                const float *from = p.sa + (int64_t)m0 * G + g0 + gl;
                for (int i0 = w * 64; i0 < w * 64 + 64; i0 += 16) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = i0 + 2 * j + rr;
                        v[j] = m0 + r < p.M && in ? __ldcg(from + (int64_t)r * G) : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        to[i0 + 2 * j + rr] = v[j] * b0;
                        to[kPairChunk * kPairScRow + i0 + 2 * j + rr] = v[j] * b1;
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(scf0 + 8u * (c & 1));
            }
        }
    } else {
        // ------------------------------------------------------ the sums
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairRegsEpi));
        const int q4 = warp & 3, col0 = (warp - 4) / 4 * CW;
        const uint32_t at0 = tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)col0;
        const uint32_t hand_back = cluster_map(acce0, 0);
        const uint32_t sc_row =
            ring_s + kPairSc + 4u * (uint32_t)(col0 / 128 * (kPairChunk * kPairScRow) + q4 * 32 + lane);
        T *out = static_cast<T *>(p.out);
        griddep_wait();
        int q = 0, chunk = 0;                           // groups, chunks of scales so far
        bool stop = false;
        for (int t = pair; t < ntiles && !stop; t += npairs) {
            float2 acc[CW / 2];
#pragma unroll
            for (int i = 0; i < CW / 2; ++i)
                acc[i] = make_float2(0.f, 0.f);
            for (int g0 = 0; g0 < G && !stop; g0 += kPairChunk, ++chunk) {
                if (!fp8_wait(scf0 + 8u * (chunk & 1), (uint32_t)((chunk / 2) & 1), p.wait_limit_us, fail_s)) {
                    stop = true;
                    break;
                }
                uint32_t s_at = sc_row + (uint32_t)(chunk & 1) * (kPairScChunk * 4u);
                const int ng = min(kPairChunk, G - g0);
                for (int g = 0; g < ng; ++g, ++q, s_at += kPairScRow * 4u) {
                    float s;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(s_at) : "memory");
                    const uint32_t b = (uint32_t)q & 1u;
                    if (!fp8_wait(accf0 + 8u * b, (uint32_t)(q >> 1) & 1u, p.wait_limit_us, fail_s)) {
                        stop = true;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t at = at0 + b * kPairTile;
#pragma unroll
                    for (int c = 0; c < CW; c += kPairLd) {
                        uint32_t w[kPairLd];
                        tmem_ld_start(at + (uint32_t)c, w);
                        tmem_wait(w);
                        if (c + kPairLd == CW) {        // this warp is done with the buffer
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive_remote_cta(hand_back + 8u * b);
                        }
#pragma unroll
                        for (int j = 0; j < kPairLd / 2; ++j)
                            acc[c / 2 + j] =
                                vfma(make_float2(__uint_as_float(w[2 * j]),
                                                 __uint_as_float(w[2 * j + 1])),
                                     make_float2(s, s), acc[c / 2 + j]);
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(sce0 + 8u * (chunk & 1));
            }
            if (stop)
                break;
            int m0, n0;
            pair_tile(p, t, m0, n0);
            // out goes through shared memory, 64 bytes of each of the warp's
            // 32 rows a pass, two passes' room in turn: 16-byte chunk c of row
            // r at c ^ (r / 2) % 4 (no conflicts; a tensor copy's 64-byte
            // swizzle), then by one tensor copy, which leaves out what lies
            // past M or N, while the warp goes on
            constexpr int W = 16 / (int)sizeof(T), VP = 4 * W;   // values a chunk, a row and pass
            const int mw = m0 + (int)rank * 128 + q4 * 32;       // the warp's first row
            const int n = n0 + col0;
#pragma unroll
            for (int c0 = 0; c0 < CW; c0 += VP) {
                const uint32_t off =
                    kPairOut + (uint32_t)((warp - 4) * 2 + (c0 / VP & 1)) * kPairOutSlot;
                if (lane == 0)                          // the copy before the last has read it
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
                // a copy leaves out whole 16-byte pieces past N: a row of out
                // that ends inside one is written element by element there
                const bool copy = p.vec == 2 || (p.vec == 1 && n + c0 + VP <= p.N);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[W];
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        f[j] = j & 1 ? acc[(c0 + i * W + j) / 2].y : acc[(c0 + i * W + j) / 2].x;
                    const uint4 u = pack_out16<T>(f);
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                     ring_s + off + (uint32_t)lane * kPairRowBytes +
                                     (uint32_t)((i ^ ((lane >> 1) & 3)) << 4)),
                                 "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w)
                                 : "memory");
                }
                if (copy) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && mw < p.M && n + c0 < p.N) {
                        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group "
                                     "[%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(&tmO)),
                                     "r"(n + c0), "r"(mw), "r"(ring_s + off)
                                     : "memory");
                    }
                } else {
                    __syncwarp();
                    const unsigned char *st = base + off;
                    for (int i = lane; i < 32 * VP; i += 32) {
                        const int r = i / VP, e = i % VP;
                        const T v = *reinterpret_cast<const T *>(
                            st + r * kPairRowBytes + (((e / W) ^ ((r >> 1) & 3)) << 4) +
                            (e % W) * sizeof(T));
                        if (mw + r < p.M && n + c0 + e < p.N)
                            out[(int64_t)(mw + r) * p.ldo + n + c0 + e] = v;
                    }
                    __syncwarp();
                }
                // one group a pass, with a copy in it or without: that is what
                // the wait for all but the last counts
                if (lane == 0)
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        }
        if (lane == 0)                                  // out is written
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    // every role has finished or given up
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    const unsigned long long limit = wait_limit_ns(p.wait_limit_us);
    if (tid == 0 && *reinterpret_cast<volatile int *>(slots + 1))
        atomicAdd(timeouts, 1u);
    if (rank == 0 && warp == 1) {
        // copies of either CTA that no MMA consumed, and the MMAs themselves.
        // A stage that only one of the two asked for never completes: the
        // wait for it is as long as any copy could take.
        int mine = 0, peer = 0;
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(peer)
                     : "r"(cluster_map(smem_addr(slots + 2), 1))
                     : "memory");
        mine = slots[2];
        const int done = slots[3];
        for (int q = done; q < max(mine, peer); ++q)
            if (!mbar_wait_bounded(full0 + 8u * (q % kPairStages), (uint32_t)((q / kPairStages) & 1),
                                   limit))
                break;
        if (max(mine, peer) > done) {
            if (elect_one())
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 "
                             "[%0];" ::"r"(dbar)
                             : "memory");
            __syncwarp();
            (void)mbar_wait_bounded(dbar, 0, limit);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, kPairBufs * kPairTile);
    }
}

} // namespace rmsk
