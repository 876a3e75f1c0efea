// int8_kernel.cuh -- INT8 W8A8 matmul, dense and grouped by experts:
//
//     Y[m,n] = BF16( sA[m] * sW[n] * sum_k a[m,k] * w[n,k] )
//
// a, w are signed 8-bit codes, sA one FP32 scale per token (row of A), sW one per
// output channel (row of W).  The sum over k is an exact INT32 sum (K <= 131056, so
// that even codes of -128 cannot overflow it); in FP32 it is multiplied by sW, then by sA,
// and the result is rounded once to BF16.  (Not by sW * sA: that product can leave FP32's
// range where the result does not.  A sum other than 0 times an sW of 2^-126 .. 2^96 is
// normal, and is then rounded where the result is, whatever sA.  Moving an sW outside by a
// power of two, and the result back, cost 4 to 12 % where the epilogue bounds, in four forms.)
//
// The weights are the MMA's M side (channels in TMEM lanes) and the tokens its N side
// (columns), whatever their number: a tile is 256 channels by up to `bt` tokens on a pair
// of SMs (tcgen05.mma.cta_group::2.kind::i8, M = 256), and the last tile of a group of
// rows runs the MMA only as wide as its tokens need (N in steps of 32).  So a ragged
// expert or a single token costs no MMA rows of padding, and one code path serves all.
//   * Each CTA of the pair loads its own 128 channels and half of the tile's tokens.
//   * With few tiles a cluster of `split` pairs works on one tile, each pair on its own
//     range of K; the INT32 partial sums meet in the owners' shared memory (distributed
//     shared memory, no workspace), every pair finishing its share of the tile's tokens.
//     Integer sums do not depend on order.
// Warp 0 loads (TMA, 128-byte swizzle), warp 1 of the leader issues the MMAs, eight warps
// apply the scales and store.  The accumulator is double-buffered and the clusters are
// persistent, so a tile's epilogue runs under the next tile's MMAs.
//
// What bounds it (B200, zeros where power is not the question): an SM's shared memory
// takes one 128-byte row a clock, for the TMA writes and the MMA's operand reads alike.  A
// 128-byte step of K of a full tile costs 256 clocks for the channels (written, read) and
// bt for the tokens, against 2 bt clocks of MMA: tiles of 256 tokens are the smallest that
// the MMA bounds.  Measured per step: 156 ns at 64 tokens, 201 at 128, 322 at 256 with
// every SM busy.  Large products are bound by power: 4096 x 5376 x 14336 takes 163 us on
// zeros, and on random codes 200 to 212 us in short runs, 236 to 255 us in long ones.  Small
// ones by the weights' bytes (32 rows over 8 experts [14336, 4096]: 74 us, 6.3 TB/s; one token
// at 5376 x 14336: 15.0 us, 5.1 TB/s).  Single SMs instead of pairs (M = 128) took 31 us for
// 333 tokens where pairs take 27 (short runs), and 78 us for 32 tokens over 8 experts where
// pairs take 75.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "grouped_pair_kernel.cuh"
#include "ptx.cuh"
#include "w4a4_pair_kernel.cuh"

namespace nvfp4 {
namespace int8 {

using w4a4::ROLE_DRAIN;
using w4a4::ROLE_EPI;
using w4a4::ROLE_MMA;
using w4a4::ROLE_PRODUCER;

constexpr int MAX_EXPERTS = grouped_pair::MAX_EXPERTS;
constexpr int CTAS = 2;          // a pair of SMs per tile and part of K
constexpr int BW = 128;          // weight rows (channels) per CTA
constexpr int TILE_N = CTAS * BW;
constexpr int BKB = 128;         // bytes (= codes) of K per chunk: one swizzle row
constexpr int KSTEPS = BKB / 32; // K = 32 per kind::i8 MMA
constexpr int MAX_BT = 256;      // token columns of a tile
constexpr int MAX_STAGES = 12;
constexpr int MAX_CHUNKS = 2;
constexpr int MAX_SPLIT_BT = 128;  // token columns of a split tile at most
constexpr int MAX_SPLIT = 4;     // pairs of a split tile (8 CTAs: the portable cluster size)
constexpr int NUM_EPI_WARPS = 8;
constexpr int FIRST_EPI_WARP = 2;
constexpr int NUM_THREADS = 32 * (FIRST_EPI_WARP + NUM_EPI_WARPS);
constexpr int MAX_K = 131056;    // 128 * 128 * K < 2^31

struct Shape {
    int M, N, K, E;
    int bt;      // token columns of a full tile (a multiple of 32)
    int split;   // pairs per tile over K
    int chunks;  // 128-byte chunks of K per stage (1 or 2)
    int stages;
};

// fixed part of shared memory; the stages follow at the next 1024-byte boundary
struct Smem {
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t drain;
    uint64_t red_full;  // split tile: every source's partial sums are here
    uint32_t tmem_base;
    int abort;
    int bad;
    int tb_start[MAX_EXPERTS + 1];   // prefix sums of token blocks per expert
    int row_start[MAX_EXPERTS + 1];  // token offsets
};
constexpr int HEAD_BYTES = (sizeof(Smem) + 1023) / 1024 * 1024;

__host__ __device__ constexpr int tmem_cols(int bt) {  // two accumulators
    int c = 32;
    while (c < 2 * bt) c *= 2;
    return c;
}
__host__ __device__ constexpr int stage_bytes(int bt, int chunks) {
    return chunks * (BW + bt / CTAS) * BKB;
}
// Split tiles: CTA o of the cluster finishes token columns [o*cw, (o+1)*cw), cw columns
// of the tile's `rows`, in whole quads.
__host__ __device__ constexpr int share_cols(int rows, int split) {
    return ((rows + split - 1) / split + 3) / 4 * 4;
}
// bytes of the partial sums such a CTA receives: S sources x its columns x 128 channels
__host__ __device__ constexpr int reduce_bytes(int bt, int split) {
    return split > 1 ? split * share_cols(bt, split) * BW * 4 : 0;
}
constexpr int OUT_BYTES = 32 * BW * 2;  // epilogue staging of a chunk of tokens (whole tiles), twice
// At least the share of an SM's 228 KB that the CTA takes of its 512 TMEM columns: then
// CTAs that fit an SM together never wait for each other's TMEM.  (Two clusters that each
// hold the columns the other one waits for would never end.)
__host__ __device__ constexpr size_t smem_bytes(int bt, int split, int chunks, int stages) {
    const size_t need = 1024 + HEAD_BYTES + (size_t)stages * stage_bytes(bt, chunks) +
                        (split > 1 ? reduce_bytes(bt, split) : 2 * OUT_BYTES);
    const size_t share = (size_t)tmem_cols(bt) * (228 * 1024 / 512);
    const size_t most = 227 * 1024;
    return need >= share ? need : share < most ? share : most;
}

// TMEM -> registers: 16 lanes x 256 bit, four times (32 columns): the MMA's fragment
// layout, row lane / 4 (then row lane / 4 + 8), columns 2 (lane % 4) and the next of each 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32"
        " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Two products rounded to nearest, in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// Four 8 x 8 blocks of 16-bit values (fragment layout), each stored transposed: lane l
// gives the address of row l % 8 of block l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(void* row, const uint32_t (&m)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(smem_u32(row)), "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3]) : "memory");
}

// The pair's D[tmem] (+)= A[smem] * B[smem]^T with signed 8-bit operands and INT32 sums,
// K = 32.
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// Instruction descriptor of kind::i8: S8 x S8 -> S32, K-major, no saturation.
//   bits 4-5 D format (2 = S32)    bits 7-9 / 10-12 A/B format (1 = signed 8-bit)
//   bits 17-22 N >> 3              bits 24-28 M >> 4
__host__ __device__ constexpr uint32_t idesc_i8(uint32_t M, uint32_t N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// A stage and the parity of its barriers, advanced by one stage at a time.
struct Ring {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
};

__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded wait of a whole converged warp (mbar_wait's limit and error record).  Every lane
// polls, so no shuffle or branch stands between the barrier and the work behind it, and
// the clock and the abort flag are looked at once every 32 polls: a K-block of one tile of
// 16 tokens took 0.35 us with a one-lane wait that reads the clock on every poll, 0.21 us
// with this one.
// CLUSTER: acquires what other CTAs of the cluster released on the barrier.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, int role) {
    uint64_t t0 = 0;
    bool ok = true;
    for (uint32_t n = 1; !(CLUSTER ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)); ++n) {
        if ((n & 31) == 0) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (*abort || now - t0 > wait_limit_ns()) {
                if (!*abort) atomicOr(&g_device_error, 1 | (role << 8));
                *abort = 1;
                ok = false;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// Columns of the MMA of a tile of `rows` tokens.
__device__ __forceinline__ int mma_n(int rows) { return (rows + 31) / 32 * 32; }

struct Tile {
    int e;
    int m0;    // first token row
    int rows;  // tokens of the tile, 1..bt
    int n0;    // first channel of the pair's 256
};

// Tile t of the list that runs over the experts; within an expert, groups of GROUP_M
// token blocks sweep the channels together, token blocks fastest (they share weights).
__device__ __forceinline__ Tile decode(const Smem& sm, const Shape& s, int t, int nblk) {
    int lo = 0, hi = s.E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sm.tb_start[mid] * nblk <= t) lo = mid; else hi = mid;
    }
    Tile tl;
    tl.e = lo;
    int mb, nb;
    w4a4_pair::tile_coords(t - sm.tb_start[lo] * nblk, sm.tb_start[lo + 1] - sm.tb_start[lo], nblk, mb, nb);
    tl.m0 = sm.row_start[lo] + mb * s.bt;
    tl.rows = min(s.bt, sm.row_start[lo + 1] - tl.m0);
    tl.n0 = nb * TILE_N;
    return tl;
}

// The token blocks of every expert, from the offsets in device memory (or one group of
// M rows without them).  Offsets that are not a non-decreasing run from 0 to at most M
// give no tile at all and a device error bit.  One warp.
__device__ __forceinline__ void plan_rows(Smem& sm, const Shape& s, const int32_t* __restrict__ offsets) {
    const int lane = threadIdx.x & 31;
    int base = 0, bad = 0;
    for (int e0 = 0; e0 < s.E; e0 += 32) {
        const int e = e0 + lane;
        int r0 = 0, r1 = 0;
        if (e < s.E) {
            r0 = offsets ? __ldg(offsets + e) : 0;
            r1 = offsets ? __ldg(offsets + e + 1) : s.M;
            if (r1 < r0 || r0 < 0 || r1 > s.M || (e == 0 && r0 != 0)) bad = 1;
        }
        const int nb = bad ? 0 : (r1 - r0 + s.bt - 1) / s.bt;
        int incl = nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (e < s.E) {
            sm.tb_start[e] = base + incl - nb;
            sm.row_start[e] = r0;
            if (e == s.E - 1) {
                sm.tb_start[s.E] = base + incl;
                sm.row_start[s.E] = r1;
            }
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        sm.bad = bad;
        if (bad && blockIdx.x == 0) atomicOr(&g_device_error, grouped_pair::BAD_OFFSETS);
    }
}

// named_bar_sync that returns whether `ok` held in every thread.
__device__ __forceinline__ bool named_bar_and(uint32_t id, uint32_t nthreads, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all) : "r"(id), "r"(nthreads), "r"((uint32_t)ok) : "memory");
    return all != 0;
}
// The halves of a cluster barrier that publishes no memory writes.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t map_addr(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// 16 bytes into the shared memory of a CTA of the cluster, counted on a barrier there
// (both addresses shared::cluster): the data is visible to whoever waits on the barrier,
// without a fence on either side.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t bar, uint32_t a, uint32_t b,
                                            uint32_t c, uint32_t d) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];"
        ::"r"(addr), "r"(bar), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int CHUNKS>
__global__ void __launch_bounds__(NUM_THREADS, 1)
int8_kernel(const __grid_constant__ CUtensorMap tmW,  // W codes [E*N][K], box 128 B x 128 rows
            const __grid_constant__ CUtensorMap tmA,  // A codes [M][K], box 128 B x bt/2 rows
            const float* __restrict__ sA, const float* __restrict__ sW,
            const int32_t* __restrict__ offsets,      // device int32 [E+1], or null (E == 1: all M rows)
            __nv_bfloat16* __restrict__ Y, const __grid_constant__ Shape s) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    Smem& sm = *reinterpret_cast<Smem*>(base);
    uint8_t* const stages = base + HEAD_BYTES;
    const int tokbytes = s.bt / CTAS * BKB;            // this CTA's tokens in one chunk
    const int sbytes = CHUNKS * (BW * BKB + tokbytes);  // a stage: CHUNKS of W, then of A
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t prank = rank % CTAS, lead = rank - prank;  // rank in its pair, the pair's leader
    const bool leader = prank == 0;
    const int part = (int)(rank / CTAS);  // this pair's part of K
    const int per = CTAS * s.split;       // CTAs of a cluster
    const int cid = blockIdx.x / per, nclusters = gridDim.x / per;
    const int nblk = (s.N + TILE_N - 1) / TILE_N;
    const int nk = (s.K + CHUNKS * BKB - 1) / (CHUNKS * BKB);
    // this pair's K-blocks (all of them unless the tile is split); a chunk past K is all
    // zeros, as every byte that a box reads out of range
    const int kb0 = (int)((long long)nk * part / s.split);
    const int kb1 = (int)((long long)nk * (part + 1) / s.split);
    const uint32_t acc_stride = (uint32_t)s.bt;
    volatile int* abort = &sm.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], CTAS * NUM_EPI_WARPS);
        }
        mbar_init(&sm.drain, 1);
        mbar_init(&sm.red_full, 1);
        sm.abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmA);
    }
    if (warp == 1) {
        tmem_alloc_pair(&sm.tmem_base, tmem_cols(s.bt));
        tmem_relinquish_pair();
    }
    if (!offsets && warp == FIRST_EPI_WARP) plan_rows(sm, s, offsets);
    tc_fence_before();
    cluster_sync();  // every CTA's barriers exist before any remote arrive
    tc_fence_after();
    // The kernel behind this one may start its own set-up now: not earlier, so that its
    // tensor-memory allocation cannot come before this CTA's.
    grid_dependents_launch();
    // The set-up above overlaps the kernel before this one; its output is read only from here.
    grid_dependency_wait();
    if (offsets) {
        if (warp == FIRST_EPI_WARP) plan_rows(sm, s, offsets);
        __syncthreads();
    }
    const uint32_t tmem = sm.tmem_base;
    const int tiles = sm.bad ? 0 : sm.tb_start[s.E] * nblk;

    if (warp == 0) {
        // ------------------------------------------------------------ producer (every CTA)
        int it = 0;
        Ring ring;
        bool ok = true;
        for (int t = cid; t < tiles && ok; t += nclusters) {
            const Tile tl = decode(sm, s, t, nblk);
            const int wrow = tl.e * s.N + tl.n0 + (int)prank * BW;
            // a pair's MMA takes the first half of its columns from CTA 0, the rest from CTA 1
            const int arow = tl.m0 + (int)prank * (mma_n(tl.rows) / 2);
            for (int kb = kb0; kb < kb1; ++kb, ++it, ring.next(s.stages)) {
                const int st = ring.s;
                if (!wait_bar(&sm.empty[st], ring.parity ^ 1, abort, ROLE_PRODUCER)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    uint8_t* w = stages + (size_t)st * sbytes;
                    if (leader) mbar_arrive_expect_tx(&sm.full[st], CTAS * sbytes);
                    uint8_t* a = w + CHUNKS * BW * BKB;
                    const uint32_t full0 = map_to_rank(&sm.full[st], lead);
#pragma unroll
                    for (int c = 0; c < CHUNKS; ++c) {
                        const int x = (kb * CHUNKS + c) * BKB;
                        tma_load_2d_pair(w + c * BW * BKB, &tmW, full0, x, wrow);
                        tma_load_2d_pair(a + c * tokbytes, &tmA, full0, x, arow);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && leader && lane == 0) {
            // every copy in flight lands before the CTA (or the pair) leaves
            for (int j = max(0, it - s.stages); j < it; ++j) {
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(&sm.full[j % s.stages], (j / s.stages) & 1) &&
                       globaltimer_ns() - t0 < kWaitLimitNs) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (leader)
        if (leader) {
            int tc = 0;
            Ring ring;
            bool ok = true;
#ifdef NVFP4_WAIT_TEST
            // test-only: wait for a commit that has not been issued, so that this bounded
            // wait expires and every role of the cluster takes its abort path
            if (g_wait_test_stall == 1 && !wait_bar(&sm.drain, 0, abort, ROLE_MMA)) ok = false;
#endif
            // descriptors of stage 0; a stage further is sbytes / 16 more in the address field
            const uint64_t w_desc0 = desc_kmajor_sw128(smem_u32(stages));
            const uint64_t a_desc0 = desc_kmajor_sw128(smem_u32(stages) + CHUNKS * BW * BKB);
            for (int t = cid; t < tiles && ok; t += nclusters, ++tc) {
                const Tile tl = decode(sm, s, t, nblk);
                const uint32_t idesc = idesc_i8(TILE_N, mma_n(tl.rows));
                const int buf = tc & 1;
                const uint32_t acc = tmem + buf * acc_stride;
                if (!wait_bar(&sm.acc_empty[buf], ((tc >> 1) & 1) ^ 1, abort, ROLE_MMA)) break;
                tc_fence_after();
                for (int kb = kb0; kb < kb1; ++kb, ring.next(s.stages)) {
                    const int st = ring.s;
                    if (!wait_bar(&sm.full[st], ring.parity, abort, ROLE_MMA)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t step = (uint32_t)(st * (sbytes >> 4));
#pragma unroll
                        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                            for (int ks = 0; ks < KSTEPS; ++ks)
                                mma_i8(acc, w_desc0 + (step + c * (BW * BKB / 16) + ks * 2),
                                       a_desc0 + (step + c * (tokbytes >> 4) + ks * 2), idesc,
                                       kb != kb0 || c != 0 || ks != 0);
                        mma_commit_pair(&sm.empty[st], 0x3 << lead);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (elect_one()) mma_commit_pair(&sm.acc_full[buf], 0x3 << lead);
                __syncwarp();
            }
            if (elect_one()) {
                mma_commit_pair(&sm.drain, 0x1 << lead);
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(&sm.drain, 0)) {
                    if (globaltimer_ns() - t0 > kWaitLimitNs) {
                        atomicOr(&g_device_error, 1 | (ROLE_DRAIN << 8));
                        break;
                    }
                }
            }
            __syncwarp();
        }
    } else if (s.split == 1) {
        // ------------------------------------------------------------ epilogue, whole tiles
        // Four warps (one per 32 channels) take each second chunk of 32 tokens, through a
        // staging buffer of 32 tokens x 128 channels: the accumulator comes in the MMA
        // fragment layout, is stored transposed (stmatrix) and leaves as whole 256-byte
        // runs of a token's channels.  (Two-byte stores straight from the registers, 64
        // bytes of one token per warp, took 6 us for 256 tokens.)
        const int q = warp & 3, half = (warp - FIRST_EPI_WARP) >> 2;
        uint8_t* const out = stages + (size_t)s.stages * sbytes + half * OUT_BYTES;
        const int g = lane >> 2, p2 = (lane & 3) * 2;  // fragment row, first of its two columns
        const bool wide = s.N % 8 == 0;                // 16-byte stores stay in a row
        // What a tile needs beside its accumulator, fetched one tile ahead: the tile itself,
        // the scales of channels g, g + 8, g + 16, g + 24 of the warp's 32, and on lane l the
        // scale of token l of each of the warp's chunks.
        struct Ahead {
            Tile tl;
            float sw[4], sa[MAX_BT / 64];
        };
        auto fetch = [&](int t) {
            Ahead f;
            f.tl = decode(sm, s, t, nblk);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = f.tl.n0 + (int)prank * BW + 32 * q + 8 * i + g;
                f.sw[i] = n < s.N ? __ldg(sW + (size_t)f.tl.e * s.N + n) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < MAX_BT / 64; ++i) {
                const int j = half * 32 + i * 64 + lane;
                f.sa[i] = j < f.tl.rows ? __ldg(sA + f.tl.m0 + j) : 0.f;
            }
            return f;
        };
        int tc = 0;
        Ahead next = {};
        if (cid < tiles) next = fetch(cid);
        for (int t = cid; t < tiles; t += nclusters, ++tc) {
            const Ahead now = next;
            const Tile tl = now.tl;
            const int n0 = tl.n0 + (int)prank * BW;
            const int buf = tc & 1;
            // A warp that gives up here still meets its three others at the tile's first
            // barrier, which tells all four.  Every tile has one in either half, so none of
            // them goes on to a tile that the others will not come to.
            bool ok = wait_bar(&sm.acc_full[buf], (tc >> 1) & 1, abort, ROLE_EPI);
#ifdef NVFP4_WAIT_TEST
            // test-only: one warp's wait counts as expired although the others' did not
            if (g_wait_test_stall == 2 && tc == 0 && warp == FIRST_EPI_WARP + 4) {
                if (lane == 0) atomicOr(&g_device_error, 1 | (ROLE_EPI << 8));
                ok = false;
            }
#endif
            tc_fence_after();
            if (t + nclusters < tiles) next = fetch(t + nclusters);
            const uint32_t acc = tmem + buf * acc_stride + ((uint32_t)(32 * q) << 16);
#pragma unroll
            for (int cc = 0; cc < MAX_BT / 64; ++cc) {
                const int c = half * 32 + cc * 64;
                if (c >= tl.rows) break;
                uint32_t r[32];  // [channels 0-15, 16-31][8 tokens][row g, row g + 8][2 tokens]
                if (ok) {
                    tmem_ld_16x256b_x4(acc + c, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
                    tmem_ld_16x256b_x4(acc + (16u << 16) + c, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
                }
                float2 sa[4];  // the two tokens of each 8
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sa[i] = make_float2(__shfl_sync(0xffffffffu, now.sa[cc], 8 * i + p2),
                                        __shfl_sync(0xffffffffu, now.sa[cc], 8 * i + p2 + 1));
                tmem_ld_wait();
                reg_fence(r);
                ok = named_bar_and(1 + half, 128, ok);  // the buffer's last chunk has left
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // 8 tokens
                    uint32_t m[4];             // 8 x 8 blocks of channels 0, 8, 16, 24
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = (k >> 1) * 16 + i * 4 + (k & 1) * 2;
                        float2 v = make_float2((float)(int)r[at], (float)(int)r[at + 1]);
                        v = mul2(mul2(v, make_float2(now.sw[k], now.sw[k])), sa[i]);
                        __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
                        m[k] = *reinterpret_cast<uint32_t*>(&h);
                    }
                    // lane l gives the address of row l & 7 (a token) of block l >> 3
                    const int tok = 8 * i + (lane & 7), blk = 4 * q + (lane >> 3);
                    stmatrix_x4_trans(out + tok * 256 + ((blk ^ (tok & 7)) << 4), m);
                }
                named_bar_sync(1 + half, 128);
                const int cnt = min(32, tl.rows - c);
                if (wide) {
                    const int n = n0 + (lane & 15) * 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = q * 8 + i * 2 + (lane >> 4);
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            out + tok * 256 + ((((lane & 15)) ^ (tok & 7)) << 4));
                        if (tok < cnt && n < s.N)
                            *reinterpret_cast<uint4*>(Y + (size_t)(tl.m0 + c + tok) * s.N + n) = v;
                    }
                } else {
                    // Rows start anywhere: each leaves as the 16-byte pieces between its first
                    // and last 16-byte boundaries and two bytes at a time around them.
                    // (Two-byte stores alone took 24 us for 700 x 2500 x 6000, four-byte ones
                    // 21.)  The second CTA's columns may all lie past N.
                    const int width = max(0, min(BW, s.N - n0));
                    const int piece = lane & 15;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = q * 8 + i * 2 + (lane >> 4);
                        const uint8_t* const src = out + tok * 256;
                        const int x = (tok & 7) << 4;  // a row's 16-byte blocks are exchanged by it
                        uint16_t* const y = reinterpret_cast<uint16_t*>(Y) + (size_t)(tl.m0 + c + tok) * s.N + n0;
                        // elements before the first boundary, whole pieces, and where they end
                        const int head = min(width, (int)(-(reinterpret_cast<uintptr_t>(y) >> 1) & 7));
                        const int tail = head + ((width - head) & ~7);
                        const int e = head + piece * 8;
                        uint32_t w[5];
#pragma unroll
                        for (int k = 0; k < 5; ++k) {
                            const int byte = min((e >> 1) + k, BW / 2 - 1) * 4;
                            w[k] = *reinterpret_cast<const uint32_t*>(src + (byte ^ x));
                        }
                        const int edge = piece < 8 ? piece : tail + piece - 8;  // one element of the ends
                        const uint16_t h = *reinterpret_cast<const uint16_t*>(src + ((min(edge, BW - 1) * 2) ^ x));
                        if (tok < cnt) {
                            const uint32_t sh = (e & 1) * 16;
                            if (e + 8 <= tail)
                                *reinterpret_cast<uint4*>(y + e) =
                                    make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                                               __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
                            if (piece < 8 ? edge < head : edge < width) y[edge] = h;
                        }
                    }
                }
            }
            if (half * 32 >= tl.rows) ok = named_bar_and(1 + half, 128, ok);  // no chunk, no barrier yet
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            // (a buffer that no later tile takes is not handed back: every remote arrive is
            // one that the MMA warp waits for, so none can reach a CTA that has left)
            if (lane == 0 && t + 2 * nclusters < tiles) mbar_arrive_remote(&sm.acc_empty[buf], lead);
        }
    } else if (cid < tiles) {
        // ------------------------------------------------------------ epilogue, a split tile
        // (one per cluster: the host splits only where all tiles run at once.)  Each CTA
        // sends its INT32 partial sums to the columns' owners, as [source][column
        // quad][channel] int4; an owner adds its columns' sums and stores them.
        const int q = warp & 3, half = (warp - FIRST_EPI_WARP) >> 2;
        const int tid = threadIdx.x - 32 * FIRST_EPI_WARP, ch = tid & (BW - 1);
        uint8_t* const red = stages + (size_t)s.stages * sbytes;
        const Tile tl = decode(sm, s, cid, nblk);
        const int cw = share_cols(tl.rows, s.split), quads = cw / 4;
        const int my_cols = max(0, min(cw, tl.rows - part * cw));
        const int n = tl.n0 + (int)prank * BW + ch;
        const float sw = n < s.N ? __ldg(sW + (size_t)tl.e * s.N + n) : 0.f;
        // lane l: the scales of this pair's tokens l and 32 + l (a share is at most 64)
        const int m0 = tl.m0 + part * cw;
        const float sa0 = lane < my_cols ? __ldg(sA + m0 + lane) : 0.f;
        const float sa1 = 32 + lane < my_cols ? __ldg(sA + m0 + 32 + lane) : 0.f;
        if (tid == 0) mbar_arrive_expect_tx(&sm.red_full, s.split * ((my_cols + 3) / 4) * BW * 16);
        if (wait_bar(&sm.acc_full[0], 0, abort, ROLE_EPI)) {
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
            const uint32_t src = smem_u32(red) + (uint32_t)(part * quads * BW + 32 * q + lane) * 16;
            for (int c = half * 32; c < tl.rows; c += 64) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(acc + c, r);
                tmem_ld_wait();
                reg_fence(r);
                int o = c / cw, quad = (c - o * cw) / 4;
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    if (c + j < tl.rows) {
                        const uint32_t to = (uint32_t)o * CTAS + prank;
                        st_async_v4(map_addr(src + (uint32_t)(quad * BW * 16), to),
                                    map_to_rank(&sm.red_full, to), r[j], r[j + 1], r[j + 2], r[j + 3]);
                    }
                    if (++quad == quads) {
                        quad = 0;
                        ++o;
                    }
                }
            }
            tc_fence_before();
        }
#ifdef NVFP4_WAIT_TEST
        // test-only: the owners' waits count as expired, with sums still on their way to them
        const bool expired = g_wait_test_stall == 3 && my_cols > 0;
        if (expired && tid == 0) atomicOr(&g_device_error, 1 | (ROLE_EPI << 8));
#else
        constexpr bool expired = false;
#endif
        if (!expired && wait_bar<true>(&sm.red_full, 0, abort, ROLE_EPI)) {
            for (int c = tid / BW; c * 4 < my_cols; c += NUM_EPI_WARPS * 32 / BW) {
                int4 v = make_int4(0, 0, 0, 0);
                for (int i = 0; i < s.split; ++i) {
                    const int4 p = *reinterpret_cast<const int4*>(red + ((i * quads + c) * BW + ch) * 16);
                    v.x += p.x;
                    v.y += p.y;
                    v.z += p.z;
                    v.w += p.w;
                }
                const int sum[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = c * 4 + j;
                    const float sa = __shfl_sync(0xffffffffu, col < 32 ? sa0 : sa1, col & 31);
                    if (col < my_cols && n < s.N)
                        Y[(size_t)(m0 + col) * s.N + n] = __float2bfloat16_rn((float)sum[j] * sw * sa);
                }
            }
        }
    }

    // No CTA of a cluster leaves (or frees a pair's TMEM) while another may still use it.
    // Nothing is published here: a release would wait for the output stores (1 to 2 us).
    __syncwarp();
    tc_fence_before();
    cluster_arrive_relaxed();
    cluster_wait();
    tc_fence_after();
    // By now every partial sum of a split tile has been sent, but a CTA whose wait for them
    // expired may still be their target: it stays until they have landed (or until the limit,
    // when some were never sent).  Otherwise this is one look at a completed barrier.
    if (s.split > 1 && warp == 0 && cid < tiles) {
        const uint64_t t0 = globaltimer_ns();
        while (!try_wait_cluster(&sm.red_full, 0) && globaltimer_ns() - t0 < wait_limit_ns()) {
        }
    }
    if (warp == 1) tmem_dealloc_pair(tmem, tmem_cols(s.bt));
}

}  // namespace int8
}  // namespace nvfp4
