// lora_pair_gemm.cuh -- the product of two bf16 matrices on CTA pairs, as a
// loop that kernels with different epilogues share.
//
// D[256 x 256] = A[256 x K] * B[256 x K]^T per cluster of two CTAs
// (cta_group::2): each CTA holds 128 rows of A, 128 rows of B and, in its
// TMEM, 128 rows of D.  Either operand may be stored with K contiguous, or
// with its rows contiguous (a transposed matrix): a 64-wide K block of such
// an operand is two panels of 64 K rows x 64 elements, which the matrix
// descriptors address as MN-major.
//
// What bounds it: one pair of 128 x 256 x 64 UMMAs takes 512 clocks on an SM
// (4096 multiply-adds a clock) and reads 32 KB of shared memory in that
// time; with one CTA per tile (128 x 256) it would be 48 KB, and each SM
// would draw 1.5 times the bytes from L2.
//
// Warps: 0 loads (TMA), 1 issues the UMMAs (even CTA only), 2..9 run the
// epilogue of one accumulator (a half of its columns each four) while the
// next tile fills the other.
// Both CTAs' loads signal the even CTA's "full" barrier; the UMMAs' commits
// free the stage in both.
#pragma once

#include "lora_common.cuh"
#include "lora_umma.cuh"

namespace lora {

constexpr int PG_TILE = 256;          // rows and columns of a pair's tile
constexpr int PG_HALF = 128;          // of them in one CTA
constexpr int PG_BK = 64;
constexpr int PG_STAGES = 6;
constexpr int PG_STAGE_BYTES = 2 * PG_HALF * PG_BK * 2;     // A and B, 32 KB
constexpr int PG_THREADS = 320;
constexpr int PG_EPI_WARP0 = 2;
constexpr int PG_SMEM = PG_STAGES * PG_STAGE_BYTES + 1024 + 256;
constexpr long long PG_TIMEOUT_CYCLES = 2000000000ll;
constexpr int LORA_TIMEOUT_BIT = 1 << 30;

// TMA tile load into this CTA whose bytes are counted on a barrier of either
// CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int c0,
                                                 int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// The same for a box of one matrix of a stack (encode_stack_map).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int c0,
                                                 int c1, int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// Arrive on the barrier at this shared-memory offset in both CTAs of the
// pair once every pair UMMA issued so far by this thread has completed.
__device__ __forceinline__ void umma_commit_both(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
        ".multicast::cluster.b64 [%0], %1;\n"
        :: "r"(bar), "h"(uint16_t(3)) : "memory");
}

// Waits for a phase, at most PG_TIMEOUT_CYCLES from the first failed poll;
// false once *abort is set or the time is over (then *abort is set).
__device__ __forceinline__ bool pg_wait(uint32_t bar, uint32_t parity, volatile int *abort)
{
    if (mbar_try_wait_cluster(bar, parity)) return true;
    return mbar_wait_bounded_cluster(bar, parity, abort, clock64() + PG_TIMEOUT_CYCLES);
}

// Descriptor of an MN-major operand: panels of K rows x 64 elements
// (128-byte rows, 128-byte swizzle).  Eight K rows are 1024 bytes (stride
// offset); the next 64 elements along M or N begin `panel` bytes on (leading
// offset; 8192 for 64 K rows).  Advancing K by 16 adds 2048 bytes to the
// start.
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t saddr, uint32_t panel = 8192)
{
    uint64_t d = 0;
    d |= uint64_t((saddr & 0x3FFFFu) >> 4);
    d |= uint64_t(panel >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

// One tile of work: its first row of A and of B, its K blocks, and, where A is
// a stack of matrices, which of them and how many rows of B there are (a
// multiple of 32, at most PG_TILE).
struct PairItem {
    int row_a, row_b, kb0, kb1;
    int mat = 0, n = PG_TILE;
};

// What the warps behind the epilogue's do meanwhile: nothing.
struct NoSideJob {
    __device__ __forceinline__ void operator()(int) const {}
};

// Runs `total` items on the grid's pairs.  A_T / B_T: the operand is stored
// with its rows contiguous.  A_STACK: map_a is a stack's (encode_stack_map), and
// a tile is 256 rows of A by the item's n of B.  item(i) -> PairItem (every thread computes the
// same); epilogue(i, item, tmem address of this warp's 32 lanes, row of this
// thread within the CTA's 128 rows, first of its 128 columns, CTA rank,
// whether the item has no K blocks).  side(warp): what further warps of the
// launch do beside the products.
template <bool A_T, bool B_T, bool A_STACK = false, typename ItemFn, typename EpiFn, typename SideFn = NoSideJob>
__device__ __forceinline__ void pair_gemm(const CUtensorMap *map_a, const CUtensorMap *map_b,
                                          int total, int32_t *error_word, ItemFn item_of,
                                          EpiFn epilogue, SideFn side = SideFn())
{
    extern __shared__ uint8_t pg_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(pg_smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_addr(smem);
    const uint32_t bars = base + PG_STAGES * PG_STAGE_BYTES;
    const uint32_t bar_full = bars, bar_empty = bars + 8 * PG_STAGES;
    const uint32_t bar_accf = bar_empty + 8 * PG_STAGES;      // [2]
    const uint32_t bar_acce = bar_accf + 16;                  // [2]
    const uint32_t bar_odd = bar_acce + 16;                   // [2], the odd CTA's in the even one
    const uint32_t bar_drain = bar_odd + 16;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + (bar_drain + 8 - base));
    volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
    // the warp as a value that the compiler knows to be the same in its lanes
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = int(blockIdx.x >> 1), npairs = int(gridDim.x >> 1);

    if (tid == 0) {
        for (int i = 0; i < PG_STAGES; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_accf + 8 * i, 1);
            mbar_init(bar_acce + 8 * i, 8);       // this CTA's epilogue warps
            mbar_init(bar_odd + 8 * i, 1);
        }
        mbar_init(bar_drain, 1);
        mbar_fence_init();
        *s_abort = 0;
        tma_prefetch_map(map_a);
        tma_prefetch_map(map_b);
    }
    if (warp == 1) tmem_alloc_pair(smem_addr(s_tmem), 512);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);

    if (warp == 0) {
        // ---------------------------------------------------------- loads
        if (lane == 0) {
            // the operands may have been written by the stream's previous
            // kernel with ordinary stores
            asm volatile("fence.proxy.async.global;\n" ::: "memory");
            const uint32_t full0 = cluster_map(bar_full, 0);
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = pair; ok && i < total; i += npairs) {
                const PairItem it = item_of(i);
                const int ra = it.row_a + int(rank) * PG_HALF;
                const int rb = it.row_b + int(rank) * (A_STACK ? it.n / 2 : PG_HALF);
                for (int kb = it.kb0; kb < it.kb1; ++kb) {
                    if (!pg_wait(bar_empty + 8 * stage, phase ^ 1u, s_abort)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0)
                        mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * PG_STAGE_BYTES);
                    const uint32_t sa = base + stage * PG_STAGE_BYTES, sb = sa + PG_STAGE_BYTES / 2;
                    const uint32_t full = full0 + 8 * stage;
                    if constexpr (A_STACK && A_T) {
                        tma_load_3d_pair(sa, map_a, ra, kb * PG_BK, it.mat, full);
                        tma_load_3d_pair(sa + 8192, map_a, ra + 64, kb * PG_BK, it.mat, full);
                    } else if constexpr (A_STACK) {
                        tma_load_3d_pair(sa, map_a, kb * PG_BK, ra, it.mat, full);
                    } else if constexpr (A_T) {
                        tma_load_2d_pair(sa, map_a, ra, kb * PG_BK, full);
                        tma_load_2d_pair(sa + 8192, map_a, ra + 64, kb * PG_BK, full);
                    } else {
                        tma_load_2d_pair(sa, map_a, kb * PG_BK, ra, full);
                    }
                    if constexpr (B_T) {
                        tma_load_2d_pair(sb, map_b, rb, kb * PG_BK, full);
                        tma_load_2d_pair(sb + 8192, map_b, rb + 64, kb * PG_BK, full);
                    } else {
                        tma_load_2d_pair(sb, map_b, kb * PG_BK, rb, full);
                    }
                    ++issued;
                    if (++stage == PG_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // No copy and no commit may still target this CTA when it exits:
            // wait (bounded) for the last fills to be consumed or, after an
            // abort, at least to have landed.
            const long long dd = clock64() + PG_TIMEOUT_CYCLES;
            for (int i = max(0, issued - PG_STAGES); i < issued; ++i) {
                const uint32_t ph = uint32_t(i / PG_STAGES) & 1u;
                const uint32_t b8 = 8 * (i % PG_STAGES);
                if (rank == 0)
                    while (!mbar_try_wait_cluster(bar_full + b8, ph) && clock64() < dd) {
                    }
                while (!mbar_try_wait_cluster(bar_empty + b8, ph) && !*s_abort && clock64() < dd) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- UMMAs
        if (rank == 0) {
            // The whole warp walks the items and one lane issues, so that
            // what the products are addressed by is in uniform registers:
            // from a branch of one lane a product takes 75 clocks to issue,
            // four of them and the waits nearly as long as they run.
            constexpr uint32_t turned = (A_T ? 1u << 15 : 0u) | (B_T ? 1u << 16 : 0u);
            const bool leader = elect_one();
            // the lanes give up together
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, pg_wait(bar, parity, s_abort));
            };
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int i = pair; ok && i < total; i += npairs) {
                const PairItem it = item_of(i);
                if (it.kb0 >= it.kb1) continue;
                const uint32_t idesc =
                    __shfl_sync(0xffffffffu, umma_idesc_bf16(PG_TILE, A_STACK ? it.n : PG_TILE) | turned, 0);
                if (!wait(bar_acce + 8 * acc, acc_phase ^ 1u) ||
                    !wait(bar_odd + 8 * acc, acc_phase ^ 1u))
                    break;
                tc_fence_after();
                const int blocks = __shfl_sync(0xffffffffu, it.kb1 - it.kb0, 0);
                for (int kb = 0; kb < blocks; ++kb) {
                    if (!wait(bar_full + 8 * stage, phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + stage * PG_STAGE_BYTES, sb = sa + PG_STAGE_BYTES / 2;
                    if (leader) {
                        const uint64_t da = A_T ? umma_desc_mn(sa) : umma_desc_sw128(sa);
                        const uint64_t db = B_T ? umma_desc_mn(sb) : umma_desc_sw128(sb);
#pragma unroll
                        for (int kk = 0; kk < PG_BK / 16; ++kk)
                            umma_bf16_pair(tmem + uint32_t(acc * PG_TILE), da + kk * (A_T ? 128 : 2),
                                           db + kk * (B_T ? 128 : 2), idesc, kb != 0 || kk != 0);
                        umma_commit_both(bar_empty + 8 * stage);
                    }
                    __syncwarp();
                    if (++stage == PG_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (leader) umma_commit_both(bar_accf + 8 * acc);
                __syncwarp();
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (leader && *s_abort) {       // nothing in flight when TMEM is released
                umma_commit_pair(cluster_map(bar_drain, 0));
                const long long dd = clock64() + PG_TIMEOUT_CYCLES;
                while (!mbar_try_wait_cluster(bar_drain, 0) && clock64() < dd) {
                }
            }
        } else if (lane == 0) {
            // tells the even CTA which accumulators the odd one has read.
            // The epilogue warps arrive in their own CTA: an arrival at
            // cluster scope waits for the warp's loads and stores in flight.
            const uint32_t to = cluster_map(bar_odd, 0);
            int acc = 0;
            uint32_t acc_phase = 0;
            for (int i = pair; i < total; i += npairs) {
                const PairItem it = item_of(i);
                if (it.kb0 >= it.kb1) continue;
                if (!pg_wait(bar_acce + 8 * acc, acc_phase, s_abort)) break;
                tc_fence_after();
                tc_fence_before();
                mbar_arrive_cluster(to + 8 * acc);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
        __syncwarp();
    } else if (warp >= PG_THREADS / 32) {
        side(warp - PG_THREADS / 32);
    } else {
        // ------------------------------------------------------- epilogue
        const int q = warp & 3;                   // TMEM lane quarter of this warp
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int i = pair; i < total; i += npairs) {
            const PairItem it = item_of(i);
            const bool empty = it.kb0 >= it.kb1;
            if (!empty) {
                const bool got = pg_wait(bar_accf + 8 * acc, acc_phase, s_abort);
                if (__all_sync(0xffffffffu, got) == 0) break;
                tc_fence_after();
            }
            epilogue(i, it, tmem + uint32_t(acc * PG_TILE) + (uint32_t(q * 32) << 16),
                     q * 32 + lane, (warp - PG_EPI_WARP0) / 4 * PG_HALF, int(rank), empty);
            if (!empty) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_acce + 8 * acc);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
    }

    if (tid == 0 && *s_abort && error_word != nullptr) atomicOr(error_word, LORA_TIMEOUT_BIT);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Launch of `clusters` clusters of `size` CTAs.
template <typename Kern, typename Arg>
cudaError_t launch_clusters(Kern kernel, int size, int clusters, cudaStream_t stream, const Arg &arg, int threads,
                            int smem)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(size * clusters));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, arg);
}

// Launch with clusters of two CTAs.
template <typename Kern, typename Arg>
cudaError_t launch_pair_kernel(Kern kernel, int pairs, cudaStream_t stream, const Arg &arg,
                               int threads = PG_THREADS, int smem = PG_SMEM)
{
    return launch_clusters(kernel, 2, pairs, stream, arg, threads, smem);
}

}  // namespace lora
