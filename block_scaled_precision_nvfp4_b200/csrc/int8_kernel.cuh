// int8_kernel.cuh -- INT8 W8A8 matmul, dense and grouped by experts:
//
//     Y[m,n] = BF16( sA[m] * sW[n] * sum_k a[m,k] * w[n,k] )
//
// a, w are signed 8-bit codes, sA one FP32 scale per token (row of A), sW one per
// output channel (row of W).  The sum over k is an exact INT32 sum (K <= 131056, so
// that even codes of -128 cannot overflow it); the two scales are applied in FP32 and
// the result is rounded once to BF16.
//
// The weights are the MMA's M side (channels in TMEM lanes) and the tokens its N side
// (columns), whatever their number: a tile is 128 channels per CTA by up to `bt`
// tokens, and the last tile of a group of rows runs the MMA only as wide as its
// tokens need (N in steps of 16, or of 32 on a pair of SMs).  So a ragged expert or a
// single token costs no MMA rows of padding, and one code path serves them all.
//   * int8_kernel<true>: pairs of SMs (tcgen05.mma.cta_group::2.kind::i8, M = 256):
//     each CTA loads its own 128 channels and half of the tile's tokens.
//   * int8_kernel<false>: single SMs (M = 128).  With S > 1 a cluster of S CTAs works
//     on one tile, each on its own range of K; the INT32 partial sums meet in the
//     owners' shared memory (distributed shared memory, no workspace), every CTA
//     finishing its share of the tile's tokens.  Integer sums do not depend on order.
// Warp 0 loads (TMA, 128-byte swizzle), warp 1 issues the MMAs, eight warps apply the
// scales and store.  With S == 1 the accumulator is double-buffered and the CTAs are
// persistent, so a tile's epilogue runs under the next tile's MMAs.
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
constexpr int BW = 128;          // weight rows (channels) per CTA
constexpr int BKB = 128;         // bytes (= codes) of K per stage row: one swizzle row
constexpr int KSTEPS = BKB / 32; // K = 32 per kind::i8 MMA
constexpr int MAX_BT = 256;      // token columns of a tile
constexpr int MAX_STAGES = 12;
constexpr int MAX_SPLIT = 8;     // CTAs of a split tile (portable cluster size)
constexpr int NUM_EPI_WARPS = 8;
constexpr int FIRST_EPI_WARP = 2;
constexpr int NUM_THREADS = 32 * (FIRST_EPI_WARP + NUM_EPI_WARPS);
constexpr int MAX_K = 131056;    // 128 * 128 * K < 2^31

struct Shape {
    int M, N, K, E;
    int bt;      // token columns of a full tile (a multiple of 16; of 32 on pairs)
    int split;   // CTAs per tile over K (1 on pairs)
    int stages;
};

// fixed part of shared memory; the stages follow at the next 1024-byte boundary
struct Smem {
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int bad;
    int tb_start[MAX_EXPERTS + 1];   // prefix sums of token blocks per expert
    int row_start[MAX_EXPERTS + 1];  // token offsets
};
constexpr int HEAD_BYTES = (sizeof(Smem) + 1023) / 1024 * 1024;

__host__ __device__ constexpr int acc_cols(int bt) { return (bt + 31) / 32 * 32; }
__host__ __device__ constexpr int tmem_cols(int bt, int split) {
    const int need = acc_cols(bt) * (split > 1 ? 1 : 2);
    int c = 32;
    while (c < need) c *= 2;
    return c;
}
__host__ __device__ constexpr int stage_bytes(bool pair, int bt) {
    return BW * BKB + (pair ? bt / 2 : bt) * BKB;
}
// bytes of the partial sums a CTA of a split tile receives, S sources x its columns x 128
__host__ __device__ constexpr int reduce_bytes(int bt, int split) {
    return split > 1 ? split * ((bt + split - 1) / split) * BW * 4 : 0;
}
// a reduce buffer of its own up to this size; a larger one reuses the stages, which
// costs one more cluster barrier (all of the cluster's MMAs must be over first)
constexpr int REDUCE_OWN_BYTES = 36 * 1024;
__host__ __device__ constexpr bool reduce_aliased(int bt, int split) {
    return reduce_bytes(bt, split) > REDUCE_OWN_BYTES;
}
__host__ __device__ constexpr size_t smem_bytes(bool pair, int bt, int split, int stages) {
    return 1024 + HEAD_BYTES + (size_t)stages * stage_bytes(pair, bt) +
           (reduce_aliased(bt, split) ? 0 : reduce_bytes(bt, split));
}

// D[tmem] (+)= A[smem] * B[smem]^T with signed 8-bit operands and INT32 sums, K = 32.
template <bool PAIR>
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
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

// Bounded wait of a whole converged warp (mbar_wait's limit and error record).  Every lane
// polls, so no shuffle or branch stands between the barrier and the work behind it, and
// the clock and the abort flag are looked at once every 32 polls: a K-block of one tile of
// 16 tokens took 0.35 us with a one-lane wait that reads the clock on every poll, 0.21 us
// with this one.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, int role) {
    uint64_t t0 = 0;
    bool ok = true;
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
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

struct Tile {
    int e;
    int m0;    // first token row
    int rows;  // tokens of the tile, 1..bt
    int n0;    // first channel (of the pair's 256, or of the CTA's 128)
};

// Tile t of the list that runs over the experts; within an expert, groups of GROUP_M
// token blocks sweep the channels together, token blocks fastest (they share weights).
__device__ __forceinline__ Tile decode(const Smem& sm, const Shape& s, int t, int nblk, int tile_n) {
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
    tl.n0 = nb * tile_n;
    return tl;
}

// The token blocks of every expert, from the offsets in device memory (or one group of
// M rows without them).  Offsets that are not a non-decreasing run from 0 to at most M
// give no tile at all and a device error bit.  One warp; bad is 0 on entry.
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
    if (bad && lane == 0) {
        sm.bad = 1;
        if (blockIdx.x == 0) atomicOr(&g_device_error, grouped_pair::BAD_OFFSETS);
    }
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <bool PAIR>
__global__ void __launch_bounds__(NUM_THREADS, PAIR ? 1 : 2)
int8_kernel(const __grid_constant__ CUtensorMap tmW,  // W codes [E*N][K], box 128 B x 128 rows
            const __grid_constant__ CUtensorMap tmA,  // A codes [M][K], box 128 B x bt (pair: bt/2) rows
            const float* __restrict__ sA, const float* __restrict__ sW,
            const int32_t* __restrict__ offsets,      // device int32 [E+1], or null (E == 1: all M rows)
            __nv_bfloat16* __restrict__ Y, const __grid_constant__ Shape s) {
    constexpr int CTAS = PAIR ? 2 : 1;
    constexpr int TILE_N = BW * CTAS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    Smem& sm = *reinterpret_cast<Smem*>(base);
    uint8_t* const stages = base + HEAD_BYTES;
    const int sbytes = stage_bytes(PAIR, s.bt);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool clustered = PAIR || s.split > 1;
    const uint32_t rank = clustered ? cluster_ctarank() : 0;
    const bool leader = !PAIR || rank == 0;
    const int per = PAIR ? 2 : s.split;  // CTAs of a cluster
    const int cid = blockIdx.x / per, nclusters = gridDim.x / per;
    const int nblk = (s.N + TILE_N - 1) / TILE_N;
    const int nk = (s.K + BKB - 1) / BKB;
    // this CTA's K-blocks (all of them unless the tile is split)
    const int kb0 = PAIR ? 0 : (int)((long long)nk * rank / s.split);
    const int kb1 = PAIR ? nk : (int)((long long)nk * (rank + 1) / s.split);
    const int bufs = s.split > 1 ? 1 : 2;
    const uint32_t acc_stride = (uint32_t)acc_cols(s.bt);
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
        sm.abort = 0;
        sm.bad = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmA);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(&sm.tmem_base, tmem_cols(s.bt, s.split));
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&sm.tmem_base, tmem_cols(s.bt, s.split));
            tmem_relinquish();
        }
    }
    __syncthreads();
    // the set-up above overlaps the kernel before this one; its output is read only from here
    grid_dependency_wait();
    if (warp == FIRST_EPI_WARP) plan_rows(sm, s, offsets);
    tc_fence_before();
    if (clustered) cluster_sync(); else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const int tiles = sm.bad ? 0 : sm.tb_start[s.E] * nblk;

    if (warp == 0) {
        // ------------------------------------------------------------ producer (every CTA)
        int it = 0;
        Ring ring;
        bool ok = true;
        for (int t = cid; t < tiles && ok; t += nclusters) {
            const Tile tl = decode(sm, s, t, nblk, TILE_N);
            const int wrow = tl.e * s.N + tl.n0 + (PAIR ? (int)rank * BW : 0);
            // a pair's MMA takes the first half of its columns from CTA 0, the rest from CTA 1
            const int arow = tl.m0 + (PAIR ? (int)rank * ((tl.rows + 31) / 32 * 16) : 0);
            for (int kb = kb0; kb < kb1; ++kb, ++it, ring.next(s.stages)) {
                const int st = ring.s;
                if (!wait_bar(&sm.empty[st], ring.parity ^ 1, abort, ROLE_PRODUCER)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    uint8_t* w = stages + (size_t)st * sbytes;
                    if (leader) mbar_arrive_expect_tx(&sm.full[st], CTAS * sbytes);
                    if constexpr (PAIR) {
                        const uint32_t full0 = map_to_rank(&sm.full[st], 0);
                        tma_load_2d_pair(w, &tmW, full0, kb * BKB, wrow);
                        tma_load_2d_pair(w + BW * BKB, &tmA, full0, kb * BKB, arow);
                    } else {
                        tma_load_2d(w, &tmW, &sm.full[st], kb * BKB, wrow);
                        tma_load_2d(w + BW * BKB, &tmA, &sm.full[st], kb * BKB, arow);
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
            // descriptors of stage 0; a stage further is sbytes / 16 more in the address field
            const uint64_t w_desc0 = desc_kmajor_sw128(smem_u32(stages));
            const uint64_t a_desc0 = desc_kmajor_sw128(smem_u32(stages) + BW * BKB);
            for (int t = cid; t < tiles && ok; t += nclusters, ++tc) {
                const Tile tl = decode(sm, s, t, nblk, TILE_N);
                const uint32_t idesc = PAIR ? idesc_i8(TILE_N, (tl.rows + 31) / 32 * 32)
                                            : idesc_i8(TILE_N, (tl.rows + 15) / 16 * 16);
                const int buf = tc % bufs;
                const uint32_t acc = tmem + buf * acc_stride;
                if (!wait_bar(&sm.acc_empty[buf], ((tc / bufs) & 1) ^ 1, abort, ROLE_MMA)) break;
                tc_fence_after();
                for (int kb = kb0; kb < kb1; ++kb, ring.next(s.stages)) {
                    const int st = ring.s;
                    if (!wait_bar(&sm.full[st], ring.parity, abort, ROLE_MMA)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t step = (uint32_t)(st * (sbytes >> 4));
#pragma unroll
                        for (int ks = 0; ks < KSTEPS; ++ks)
                            mma_i8<PAIR>(acc, w_desc0 + (step + ks * 2), a_desc0 + (step + ks * 2),
                                         idesc, kb != kb0 || ks != 0);
                        if constexpr (PAIR) mma_commit_pair(&sm.empty[st], 0x3);
                        else mma_commit(&sm.empty[st]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (elect_one()) {
                    if constexpr (PAIR) mma_commit_pair(&sm.acc_full[buf], 0x3);
                    else mma_commit(&sm.acc_full[buf]);
                }
                __syncwarp();
            }
            if (elect_one()) {
                if constexpr (PAIR) mma_commit_pair(&sm.drain, 0x1);
                else mma_commit(&sm.drain);
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
        // lane = channel; the warp's half of the 32-token chunks.  One token's 32 channels
        // leave as one 64-byte store.
        const int q = warp & 3, half = (warp - FIRST_EPI_WARP) >> 2;
        int tc = 0;
        for (int t = cid; t < tiles; t += nclusters, ++tc) {
            const Tile tl = decode(sm, s, t, nblk, TILE_N);
            const int n = tl.n0 + (PAIR ? (int)rank * BW : 0) + 32 * q + lane;
            const bool nok = n < s.N;
            const float sw = nok ? __ldg(sW + (size_t)tl.e * s.N + n) : 0.f;
            const int buf = tc % bufs;
            if (!wait_bar(&sm.acc_full[buf], (tc / bufs) & 1, abort, ROLE_EPI)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * acc_stride + ((uint32_t)(32 * q) << 16);
            for (int c = half * 32; c < tl.rows; c += 64) {
                const float sa = c + lane < tl.rows ? __ldg(sA + tl.m0 + c + lane) : 0.f;
                uint32_t r[32];
                tmem_ld_32x32b_x32(acc + c, r);
                tmem_ld_wait();
                reg_fence(r);
                __nv_bfloat16* y = Y + (size_t)(tl.m0 + c) * s.N + n;
                const int cnt = min(32, tl.rows - c);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float f = sw * __shfl_sync(0xffffffffu, sa, j);
                    if (j < cnt && nok) y[(size_t)j * s.N] = __float2bfloat16_rn((float)(int)r[j] * f);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_remote(&sm.acc_empty[buf], 0);
                else mbar_arrive(&sm.acc_empty[buf]);
            }
        }
    }

    if (!PAIR && s.split > 1 && cid < tiles) {
        // ------------------------------------------------------------ split tile: join the K ranges
        // CTA `o` of the cluster finishes token columns [o*cw, (o+1)*cw); each CTA leaves
        // its INT32 partial sums of those columns in o's buffer [source][column][128].
        const Tile tl = decode(sm, s, cid, nblk, TILE_N);
        const int cw = (tl.rows + s.split - 1) / s.split;
        int32_t* red = reinterpret_cast<int32_t*>(
            stages + (reduce_aliased(s.bt, s.split) ? 0 : (size_t)s.stages * sbytes));
        if (reduce_aliased(s.bt, s.split)) {
            __syncwarp();
            if (warp >= FIRST_EPI_WARP) wait_bar(&sm.acc_full[0], 0, abort, ROLE_EPI);
            cluster_sync();  // every CTA's MMAs have read their stages
        }
        if (warp >= FIRST_EPI_WARP) {
            const int q = warp & 3, half = (warp - FIRST_EPI_WARP) >> 2;
            if (wait_bar(&sm.acc_full[0], 0, abort, ROLE_EPI)) {
                tc_fence_after();
                const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
                for (int c = half * 32; c < tl.rows; c += 64) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(acc + c, r);
                    tmem_ld_wait();
                    reg_fence(r);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int col = c + j, o = col / cw;
                        if (col < tl.rows)
                            st_cluster_u32(map_to_rank(red + ((int)rank * cw + col - o * cw) * BW + 32 * q + lane,
                                                       (uint32_t)o),
                                           r[j]);
                    }
                }
                tc_fence_before();
            }
        }
        __syncwarp();
        cluster_sync();  // release/acquire: the partial sums are in place
        if (warp >= FIRST_EPI_WARP && !*abort) {
            const int tid = threadIdx.x - 32 * FIRST_EPI_WARP;
            const int n = tl.n0 + (tid & (BW - 1));
            const int c0 = (int)rank * cw, cnt = min(cw, tl.rows - c0);
            if (n < s.N) {
                const float sw = __ldg(sW + (size_t)tl.e * s.N + n);
                for (int c = tid / BW; c < cnt; c += NUM_EPI_WARPS * 32 / BW) {
                    int32_t v = 0;
                    for (int i = 0; i < s.split; ++i) v += red[(i * cw + c) * BW + (tid & (BW - 1))];
                    const int m = tl.m0 + c0 + c;
                    Y[(size_t)m * s.N + n] = __float2bfloat16_rn((float)v * (sw * __ldg(sA + m)));
                }
            }
        }
    }

    // No CTA of a pair leaves (or frees TMEM) while the other may still use it.
    tc_fence_before();
    if constexpr (PAIR) cluster_sync(); else __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if constexpr (PAIR) tmem_dealloc_pair(tmem, tmem_cols(s.bt, s.split));
        else tmem_dealloc(tmem, tmem_cols(s.bt, s.split));
    }
}

}  // namespace int8
}  // namespace nvfp4
