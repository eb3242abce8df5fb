// lora_backward_tc.cu -- the three products of lora_linear_backward on the
// tensor cores (tcgen05), for padded ranks 64 and 128; see lora_backward.cu
// for the formulas and the layout of g and u.
//
// Rows of dy and x are fetched through the token order by TMA: each lane of
// the loading warp has four rows; lanes whose rows follow one another join
// into one box of up to 128 rows (a sequence's tokens do), the others take
// their four rows by a gather.  A gather moves 512 bytes in about 90 clocks,
// so a tile of one box loads many times faster (the whole of grad_u at 16384
// tokens, rank 128: 197 us by gathers alone).  A row past an adapter's last
// token gets an index past the matrix and arrives as zeros.  Weights are mapped
// with a dimension of their own for the adapter, so that what lies behind a
// slice's last row or column arrives as zeros too, never as a neighbour's
// values.  Products over tokens take both operands with their rows
// contiguous (MN-major), so nothing is transposed.
//
// One CTA an SM (dA and dB: pairs of them); warps: 0 gathers, 1 loads boxes,
// 2 issues UMMAs, 4..7 run the epilogue (thread = TMEM lane = row of the
// result).
#include "lora_backward.cuh"
#include "lora_tc.cuh"

namespace lora {

constexpr int TC_ONES = 2048;                    // 16 rows of a panel
constexpr int TC_ROWS = 128;                     // tokens of a tile of g and dx
constexpr int TC_MAX_N = 384;                    // slices x rank of one dA product

// Four rows of a 2-D tensor, one 64-column box each.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int col, int r0,
                                            int r1, int r2, int r3, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(r0), "r"(r1), "r"(r2),
           "r"(r3), "r"(bar) : "memory");
}

constexpr int TC_HEIGHTS = 6;                    // boxes of 4, 8, ... 128 rows

// The rows a lane loads: its four tokens, or a box of 4 << level rows from
// the first of them (level 0 .. 5), or nothing (another lane's box holds
// them).
struct TcRows {
    int t[4];
    int level;              // -1: a gather, -2: nothing
};

// Joins the lanes' runs of four tokens; lanes that differ in the bits below
// `stride` load other columns of the same rows.  Called by the whole warp.
__device__ __forceinline__ void join_rows(TcRows &r, int stride)
{
    const int lane = threadIdx.x & 31;
    bool run = r.t[1] == r.t[0] + 1 && r.t[2] == r.t[0] + 2 && r.t[3] == r.t[0] + 3;
    r.level = run ? 0 : -1;
#pragma unroll
    for (int k = 0; k < TC_HEIGHTS - 1; ++k) {
        const int bit = stride << k;
        if (bit >= 32) break;
        const int other = __shfl_xor_sync(0xffffffffu, r.t[0], bit);
        const int orun = __shfl_xor_sync(0xffffffffu, int(run), bit);
        const int first = (lane & bit) ? other : r.t[0], second = (lane & bit) ? r.t[0] : other;
        run = run && orun && second == first + (4 << k);
        if (run) {
            r.t[0] = first;
            r.level = (lane & bit) ? -2 : (r.level >= 0 ? k + 1 : r.level);
        }
    }
}

// The row number a lane's row has past an adapter's tokens: outside the
// matrix, and running on, so that such rows join too.
__device__ __forceinline__ int tc_no_row(int T, int row) { return T + row; }

__device__ __forceinline__ void tc_load_rows(const TcRows &r, uint32_t dst, const CUtensorMap *gather,
                                             const CUtensorMap *boxes, int col, uint32_t bar)
{
    if (r.level >= 0) tma_load_2d(dst, boxes + r.level, col, r.t[0], bar);
    else if (r.level == -1) tma_gather4(dst, gather, col, r.t[0], r.t[1], r.t[2], r.t[3], bar);
}

// The same into this CTA, counted on a barrier of either CTA of a pair.
__device__ __forceinline__ void tc_load_rows_pair(const TcRows &r, uint32_t dst, const CUtensorMap *gather,
                                                  const CUtensorMap *boxes, int col, uint32_t bar)
{
    if (r.level >= 0) {
        tma_load_2d_pair(dst, boxes + r.level, col, r.t[0], bar);
    } else if (r.level == -1) {
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n"
            :: "r"(dst), "l"(reinterpret_cast<uint64_t>(gather)), "r"(col), "r"(r.t[0]), "r"(r.t[1]),
               "r"(r.t[2]), "r"(r.t[3]), "r"(bar) : "memory");
    }
}

// Host: the maps of one matrix's rows: the gather's, then the boxes'.
struct TcRowMaps {
    CUtensorMap gather, box[TC_HEIGHTS];
};
static bool encode_row_maps(TcRowMaps *m, const uint16_t *ptr, int64_t rows, int64_t cols, int64_t ld)
{
    if (!encode_tile_map(&m->gather, ptr, uint64_t(rows), uint64_t(cols), uint64_t(ld), 64, 1,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return false;
    for (int k = 0; k < TC_HEIGHTS; ++k)
        if (!encode_tile_map(&m->box[k], ptr, uint64_t(rows), uint64_t(cols), uint64_t(ld), 64, 4u << k,
                             CU_TENSOR_MAP_SWIZZLE_128B))
            return false;
    return true;
}

// ---------------------------------------------------------------- dA, dB, dbias

struct GradWTcArgs {
    BackwardArgs b;
    TcRowMaps dy, x;
    CUtensorMap u, g;          // boxes 64 columns x 64 rows of [S * rows][RP]
    int32_t rp, group, groups; // slices of one dA product
    int32_t end[2 * LORA_MAX_SLICES];   // blocks of one adapter: dA groups, then dB slices
    int32_t kinds, ring, stage_bytes, stages, buffers;
};
constexpr int TC_W_COLS = 256;           // columns of dy or x of an item
constexpr int TC_W_THREADS = TC_THREADS + 128;

// The gradients of an adapter without tokens: zeros, written by 128 threads
// along the rows.
__device__ __forceinline__ void clear_item(const BackwardArgs &p, bool is_a, int id, int s0, int slices,
                                           int c0, int thread)
{
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (is_a) {
        const int chunks = min(16, (p.H - c0) / 8);
        for (int s = s0; s < s0 + slices; ++s) {
            if (p.da[s] == nullptr || (thread & 15) >= chunks) continue;
            uint16_t *out = p.da[s] + int64_t(id) * p.r * p.H + c0 + (thread & 15) * 8;
            for (int r = thread >> 4; r < p.r; r += 8) *reinterpret_cast<uint4 *>(out + int64_t(r) * p.H) = zero;
        }
    } else {
        const int n = p.n[s0], lo = max(0, c0 - p.off[s0]), hi = min(n, c0 + 128 - p.off[s0]);
        if (p.db[s0] != nullptr) {
            uint4 *out = reinterpret_cast<uint4 *>(p.db[s0] + (int64_t(id) * n + lo) * p.r);
            for (int i = thread; i < (hi - lo) * p.r / 8; i += 128) out[i] = zero;
        }
        if (p.dbias[s0] != nullptr && thread < hi - lo) p.dbias[s0][int64_t(id) * n + lo + thread] = 0;
    }
}

// Writes a warp's 32 columns of 64 rows of a row-major matrix: lane l holds
// column l (64 values, 32 words from the first row down); row r, if below
// `rows`, goes to dst + r * ld.  `many`: columns that exist.
__device__ __forceinline__ void store_columns(uint8_t *stage, const uint32_t (&o)[32], uint16_t *dst,
                                              int64_t ld, int rows, int many)
{
    const int lane = threadIdx.x & 31;
    uint16_t *at = reinterpret_cast<uint16_t *>(stage);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        at[(2 * j) * 32 + lane] = uint16_t(o[j] & 0xFFFFu);
        at[(2 * j + 1) * 32 + lane] = uint16_t(o[j] >> 16);
    }
    __syncwarp();
    const int c = (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * i + (lane >> 2);
        if (r < rows && c < many)
            *reinterpret_cast<uint4 *>(dst + r * ld + c) = *reinterpret_cast<const uint4 *>(at + r * 32 + c);
    }
}

// An item is an adapter x 256 columns of x or dy on a CTA pair: D[256
// columns x N] += (64 tokens of the columns)^T (64 tokens of g or u), N = the
// slices' ranks side by side for dA, one slice's for dB; dbias is one more
// product, with ones.  K is the adapter's tokens.  As single CTAs with 128
// columns each SM read 8 KB of shared memory for every 64 clocks of UMMA and
// filled 64 KB a stage beside it, twice what it has (dA and dB at 16384
// tokens, rank 128: 282 us); a pair shares the g and u panels.
//
// Adapters are taken by falling token count, so that the CTAs' shares come
// out even.  Warps 8 to 11 write the zeros of the adapters without tokens
// meanwhile (with 8 of 64 adapters in use they are most of the bytes).
__global__ void __launch_bounds__(TC_W_THREADS, 1) grad_w_tc_kernel(const __grid_constant__ GradWTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = int(blockIdx.x >> 1), pairs = int(gridDim.x >> 1);
    const int PPS = q.rp / 64;                          // panels a slice
    for (int i = tid; i < TC_ONES / 4; i += TC_W_THREADS)
        reinterpret_cast<uint32_t *>(smem + q.ring - TC_ONES)[i] = 0x3F803F80u;
    fence_proxy_async_smem();
    const uint32_t base = smem_addr(smem), ones = base + q.ring - TC_ONES;
    const uint32_t full = base + q.ring + TC_STAGE_ROWS, empty = full + 8 * TC_MAX_STAGES;
    const uint32_t accf = empty + 8 * TC_MAX_STAGES, acce = accf + 16, drain = acce + 16;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + q.ring + TC_STAGE_ROWS + 16 * TC_MAX_STAGES + 40);
    volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
    if (tid == 0) {
        for (int i = 0; i < q.stages; ++i) {
            mbar_init(full + 8 * i, 2);                 // the even CTA's two loading warps
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf + 8 * i, 1);
            mbar_init(acce + 8 * i, 8);                 // four epilogue warps of each CTA
        }
        mbar_init(drain, 1);
        mbar_fence_init();
        *s_abort = 0;
    }
    if (warp == 3) tmem_alloc_pair(smem_addr(s_tmem), 512);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_wait();
    int tiles;
    int *mem = reinterpret_cast<int *>(smem + q.ring + TC_STAGE_ROWS + TC_BAR_BYTES);
    const SegTab tab = load_tab(p, mem, tiles);
    const int *seg_of = load_seg_of(p, tab, tiles, mem);
    // order: the segments of the adapters with tokens, then the adapters without
    int *order = mem + backward_tab_words(p.nbins, p.L);
    if (warp == 0) {
        int used = 0, rest = 0;
        for (int i0 = 0; i0 < p.L; i0 += 32)
            used += __popc(__ballot_sync(0xffffffffu, i0 + lane < p.L && seg_of[i0 + lane] >= 0));
        if (lane == 0) order[p.L] = used;
        for (int i0 = 0; i0 < p.L; i0 += 32) {
            const bool none = i0 + lane < p.L && seg_of[i0 + lane] < 0;
            const uint32_t m = __ballot_sync(0xffffffffu, none);
            if (none) order[used + rest + __popc(m & ((1u << lane) - 1u))] = i0 + lane;
            rest += __popc(m);
        }
    }
    __syncthreads();
    const int active = order[p.L];
    for (int i = tid; i < p.L; i += TC_W_THREADS) {
        const int seg = seg_of[i];
        if (seg < 0) continue;
        // its place by falling count; among many adapters, as they come
        // (finding it would take longer than it saves)
        int at = 0;
        for (int k = 0; k < p.nbins; ++k) {
            if (tab.id[k] < 0 || tab.count[k] <= 0) continue;
            if (active > 256) at += k < seg;
            else at += tab.count[k] > tab.count[seg] || (tab.count[k] == tab.count[seg] && k < seg);
        }
        order[at] = seg;
    }
    __syncthreads();
    const int blocks = q.end[q.kinds - 1];
    const int items = active * blocks;          // the weights fit the memory: below 2^31

    struct Item {
        bool is_a;
        int id, s, slices, start, count, steps, c0, panels;     // c0: this CTA's columns
        int64_t row0;                                           // in g and u, within a slice
    };
    auto kind = [&](int blk, Item &it) {
        int k = 0;
        while (blk >= q.end[k]) ++k;
        it.is_a = k < q.groups;
        it.s = it.is_a ? k * q.group : k - q.groups;
        it.slices = it.is_a ? min(q.group, p.S - it.s) : 1;
        it.c0 = (it.is_a ? 0 : p.off[it.s] & ~7) + (blk - (k > 0 ? q.end[k - 1] : 0)) * TC_W_COLS +
                int(rank) * 128;
        it.panels = (it.slices * PPS + 1) / 2 * 2;              // an odd last one is loaded twice
    };
    auto decode = [&](int i) {
        Item it;
        const int seg = order[i / blocks];
        kind(i % blocks, it);
        it.id = tab.id[seg];
        it.start = tab.start[seg];
        it.count = tab.count[seg];
        it.steps = (it.count + 63) / 64;
        it.row0 = int64_t(tab.tile[seg]) * 64;
        return it;
    };
    // A loading warp's thread, after its last fill: no copy and no commit
    // may still target this CTA when it exits.
    auto drain_loads = [&](int issued) {
        const long long dd = clock64() + PG_TIMEOUT_CYCLES;
        for (int i = max(0, issued - q.stages); i < issued; ++i) {
            const uint32_t ph = uint32_t(i / q.stages) & 1u, b8 = 8u * uint32_t(i % q.stages);
            if (rank == 0)
                while (!mbar_try_wait_cluster(full + b8, ph) && clock64() < dd) {
                }
            while (!mbar_try_wait_cluster(empty + b8, ph) && !*s_abort && clock64() < dd) {
            }
        }
    };
    if (warp == 0) {
        // ------------------------------------------------ columns of dy or x
        const uint32_t full0 = cluster_map(full, 0);
        TcPos pos;
        int issued = 0;
        bool ok = true;
        const int panel = lane & 1, r4 = (lane >> 1) * 4;
        for (int i = pair; ok && i < items; i += pairs) {
            const Item it = decode(i);
            const TcRowMaps *map = it.is_a ? &q.x : &q.dy;
            TcRows rows;
            auto tokens = [&](int k) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = k * 64 + r4 + j;
                    rows.t[j] = row < it.count ? p.sorted[it.start + row] : tc_no_row(p.T, row);
                }
            };
            tokens(0);
            for (int k = 0; k < it.steps; ++k) {
                const bool got = pg_wait(empty + 8 * pos.stage, pos.phase ^ 1u, s_abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                join_rows(rows, 2);
                if (lane == 0 && rank == 0) mbar_arrive_expect_tx(full + 8 * pos.stage, 4 * TC_PANEL);
                __syncwarp();
                tc_load_rows_pair(rows, base + pos.stage * q.stage_bytes + panel * TC_PANEL + r4 * 128, &map->gather,
                                  map->box, it.c0 + panel * 64, full0 + 8 * pos.stage);
                if (k + 1 < it.steps) tokens(k + 1);
                ++issued;
                pos.next(q.stages);
            }
        }
        if (lane == 0) drain_loads(issued);
    } else if (warp == 1) {
        // ------------------------------------------------ g or u: every fourth panel pair's half
        // g and u were written by the stream's previous kernel with ordinary stores
        asm volatile("fence.proxy.async.global;\n" ::: "memory");
        const uint32_t full0 = cluster_map(full, 0);
        TcPos pos;
        int issued = 0;
        bool ok = true;
        for (int i = pair; ok && i < items; i += pairs) {
            const Item it = decode(i);
            const CUtensorMap *map = it.is_a ? &q.g : &q.u;
            // Products take up to four panels, the first half of them from the
            // even CTA: lane j loads this CTA's j-th.
            const int chunk = lane >> 1, in_chunk = min(4, it.panels - 4 * chunk);
            const bool mine = lane < it.panels / 2;
            const int panel = min(it.slices * PPS - 1,
                                  4 * chunk + int(rank) * (in_chunk / 2) + (lane & 1));
            for (int k = 0; k < it.steps; ++k) {
                const bool got = pg_wait(empty + 8 * pos.stage, pos.phase ^ 1u, s_abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                if (lane == 0 && rank == 0)
                    mbar_arrive_expect_tx(full + 8 * pos.stage, uint32_t(it.panels * TC_PANEL));
                __syncwarp();
                if (mine)
                    tma_load_2d_pair(base + pos.stage * q.stage_bytes + (2 + lane) * TC_PANEL, map, panel % PPS * 64,
                                     int((it.s + panel / PPS) * p.rows + it.row0) + k * 64, full0 + 8 * pos.stage);
                ++issued;
                pos.next(q.stages);
            }
        }
        if (lane == 0) drain_loads(issued);
    } else if (warp == 2) {
        // ------------------------------------------------ UMMAs (even CTA)
        if (lane == 0 && rank == 0) {
            constexpr uint32_t T_AB = (1u << 15) | (1u << 16);
            TcPos pos;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int i = pair; ok && i < items; i += pairs) {
                const Item it = decode(i);
                if (!pg_wait(acce + 8 * buf, bphase ^ 1u, s_abort)) break;
                tc_fence_after();
                const uint32_t d = tmem + uint32_t(buf * (512 / q.buffers));
                const bool bias = !it.is_a && p.dbias[it.s] != nullptr;
                for (int k = 0; k < it.steps; ++k) {
                    if (!pg_wait(full + 8 * pos.stage, pos.phase, s_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t z = base + pos.stage * q.stage_bytes, v = z + 2 * TC_PANEL;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t acc = k != 0 || kk != 0;
                        const uint64_t dz = umma_desc_mn(z + kk * 2048);
                        for (int c = 0; c < it.panels; c += 4)
                            umma_bf16_pair(d + uint32_t(c * 64), dz, umma_desc_mn(v + c / 2 * TC_PANEL + kk * 2048),
                                           umma_idesc_bf16(256, min(4, it.panels - c) * 64) | T_AB, acc);
                        if (bias)
                            umma_bf16_pair(d + uint32_t(it.panels * 64), dz, umma_desc_mn(ones),
                                           umma_idesc_bf16(256, 32) | T_AB, acc);
                    }
                    umma_commit_both(empty + 8 * pos.stage);
                    pos.next(q.stages);
                }
                if (!ok) break;
                umma_commit_both(accf + 8 * buf);
                if (++buf == q.buffers) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
            if (*s_abort) {       // nothing in flight when TMEM is released
                umma_commit_pair(cluster_map(drain, 0));
                const long long dd = clock64() + PG_TIMEOUT_CYCLES;
                while (!mbar_try_wait_cluster(drain, 0) && clock64() < dd) {
                }
            }
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------ epilogue
        const int row = (warp - 4) * 32 + lane;         // this thread's column of x or dy
        const uint32_t acce0 = cluster_map(acce, 0);
        uint8_t *stage = smem + q.ring + (warp - 4) * (TC_STAGE_ROWS / 4);
        int buf = 0;
        uint32_t bphase = 0;
        for (int i = pair; i < items; i += pairs) {
            const Item it = decode(i);
            const uint32_t d = tmem + uint32_t(buf * (512 / q.buffers)) + (uint32_t((warp - 4) * 32) << 16);
            const bool got = pg_wait(accf + 8 * buf, bphase, s_abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            uint32_t o[32];
            if (it.is_a) {
                const int h0 = it.c0 + (warp - 4) * 32;
                for (int j = 0; j < it.slices * PPS; ++j) {
                    const int s = it.s + j / PPS, r0 = j % PPS * 64;
                    if (p.da[s] == nullptr || h0 >= p.H) continue;
                    load64(d + uint32_t(j * 64), p.scale, o);
                    store_columns(stage, o, p.da[s] + (int64_t(it.id) * p.r + r0) * p.H + h0, p.H, p.r - r0,
                                  p.H - h0);
                }
            } else {
                const int n = p.n[it.s], at = it.c0 + row - p.off[it.s];
                const bool in = at >= 0 && at < n;
                if (p.db[it.s] != nullptr) {
                    uint16_t *out = p.db[it.s] + (int64_t(it.id) * n + at) * p.r;
                    for (int c = 0; c < p.r; c += 64) {
                        load64(d + uint32_t(c), 1.0f, o);
                        store_rows(stage, o, in ? out + c : nullptr, p.r - c);
                    }
                }
                if (p.dbias[it.s] != nullptr) {
                    uint32_t one[16];
                    tmem_ld16_nowait(d + uint32_t(it.panels * 64), one);
                    tmem_wait_ld();
                    if (in)
                        p.dbias[it.s][int64_t(it.id) * n + at] =
                            uint16_t(pack_bf16x2(__uint_as_float(one[0]), 0.0f) & 0xFFFFu);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acce0 + 8 * buf);
            if (++buf == q.buffers) {
                buf = 0;
                bphase ^= 1u;
            }
        }
    } else if (warp >= 8) {
        // ------------------------------------------------ adapters without tokens
        for (int i = pair; i < (p.L - active) * blocks; i += pairs) {
            Item it;
            kind(i % blocks, it);
            clear_item(p, it.is_a, order[active + i / blocks], it.s, it.slices, it.c0, tid - TC_THREADS);
        }
    }
    __syncwarp();
    if (tid == 0 && *s_abort) atomicOr(p.error_word, LORA_TIMEOUT_BIT);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 3) tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------- dx

struct GradXTcArgs {
    BackwardArgs b;
    CUtensorMap g;                       // boxes 64 columns x 128 rows of [S * rows][RP]
    CUtensorMap a[LORA_MAX_SLICES];      // [L][r][H], boxes 64 x 64 x 1
    int32_t rp;
    int32_t keep;                        // the tile's g stays in shared memory
    int32_t ring, stages;
};
constexpr int TC_X_COLS = 256;

// Both segment tables: 64-token tiles (rows of g and u) and 128-token tiles.
__device__ __forceinline__ int load_tabs(const BackwardArgs &p, int *mem, SegTab &t64, SegTab &t128)
{
    int tiles;
    t64 = load_tab(p, mem, tiles);
    t128 = seg_tab(mem + 4 * p.nbins + 2, p.nbins);
    return load_segments(p.no_lora, p.active, p.counts, p.start_loc, p.nbins, TC_ROWS, t128, false, 0,
                         p.T, p.error_word);
}

// Item: (128-token tile, 256 columns); K = slices x rank.  A CTA takes a run
// of consecutive items, so it meets few tiles; where the tile's rows of g
// fit beside three stages of A (slices x rank <= 384) they are loaded once a
// tile and only A streams (192 instead of 288 KB an item at 384).
__global__ void __launch_bounds__(TC_THREADS, 1) grad_x_tc_kernel(const __grid_constant__ GradXTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kps = q.rp / 64, steps = p.S * kps;
    constexpr int G_BYTES = 2 * TC_PANEL, A_BYTES = 4 * TC_PANEL;
    const uint32_t stage_bytes = q.keep ? A_BYTES : A_BYTES + G_BYTES;
    const TcRing ring = tc_setup(smem, q.ring, int(stage_bytes), q.stages, 1);
    // g of the tile lies behind the ring's stages, one 16 KB block a step
    const uint32_t g_at = ring.ring + q.stages * stage_bytes;
    const uint32_t g_full = ring.drain + 24, g_empty = g_full + 8;
    if (threadIdx.x == 0) {
        mbar_init(g_full, 1);
        mbar_init(g_empty, 1);
        mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();
    SegTab t64, t128;
    const int tiles = load_tabs(p, reinterpret_cast<int *>(smem + q.ring + TC_STAGE_ROWS + TC_BAR_BYTES), t64, t128);
    const int hb = (p.H + TC_X_COLS - 1) / TC_X_COLS;
    const int items = tiles * hb;               // T x H fits the memory: below 2^31
    const int first = int(int64_t(items) * blockIdx.x / gridDim.x);
    const int end = int(int64_t(items) * (blockIdx.x + 1) / gridDim.x);

    if (warp == 0) {
        // g and u were written by the stream's previous kernel with ordinary stores
        asm volatile("fence.proxy.async.global;\n" ::: "memory");
        TcPos pos;
        int issued = 0, loaded = -1;
        uint32_t gphase = 0;
        bool ok = true;
        for (int i = first; ok && i < end; ++i) {
            const int tile = i / hb, h0 = i % hb * TC_X_COLS;
            const int seg = find_segment(t128.tile, p.nbins, tile);
            const int64_t row0 = int64_t(t64.tile[seg]) * 64 + int64_t(tile - t128.tile[seg]) * TC_ROWS;
            const int id = t128.id[seg];
            if (q.keep && tile != loaded) {
                const bool got = pg_wait(g_empty, gphase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) break;
                if (lane == 0) mbar_arrive_expect_tx(g_full, uint32_t(steps * G_BYTES));
                __syncwarp();
                for (int k = lane; k < steps; k += 32)
                    tma_load_2d(g_at + k * G_BYTES, &q.g, k % kps * 64, int(k / kps * p.rows + row0), g_full);
                gphase ^= 1u;
                loaded = tile;
            }
            for (int k = 0; k < steps; ++k) {
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                const uint32_t full = ring.full + 8 * pos.stage;
                const uint32_t at = ring.ring + pos.stage * stage_bytes;
                const int s = k / kps, kc = k % kps * 64;
                if (lane == 0) mbar_arrive_expect_tx(full, stage_bytes);
                __syncwarp();
                if (lane < 4) tma_load_3d(at + lane * TC_PANEL, &q.a[s], h0 + lane * 64, kc, id, full);
                else if (lane == 4 && !q.keep)
                    tma_load_2d(at + A_BYTES, &q.g, kc, int(s * p.rows + row0), full);
                ++issued;
                pos.next(q.stages);
            }
        }
        if (lane == 0) {
            tc_drain_loads(ring, issued);
            // the last tile's g has landed
            if (loaded >= 0) {
                const long long dd = clock64() + PG_TIMEOUT_CYCLES;
                while (!mbar_try_wait(g_full, gphase ^ 1u) && clock64() < dd) {
                }
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            TcPos pos;
            int buf = 0, tile = -1;
            uint32_t bphase = 0, gphase = 0;
            bool ok = true;
            for (int i = first; ok && i < end; ++i) {
                if (!pg_wait(ring.acce + 8 * buf, bphase ^ 1u, ring.abort)) break;
                if (q.keep && i / hb != tile) {
                    tile = i / hb;
                    if (!pg_wait(g_full, gphase, ring.abort)) break;
                    gphase ^= 1u;
                }
                tc_fence_after();
                const uint32_t d = ring.tmem + uint32_t(buf * TC_X_COLS);
                for (int k = 0; k < steps; ++k) {
                    if (!pg_wait(ring.full + 8 * pos.stage, pos.phase, ring.abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sb = ring.ring + pos.stage * stage_bytes;
                    const uint32_t sa = q.keep ? g_at + k * G_BYTES : sb + A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(d, umma_desc_sw128(sa + kk * 32), umma_desc_mn(sb + kk * 2048),
                                  umma_idesc_bf16(128, TC_X_COLS) | 1u << 16, k != 0 || kk != 0);
                    umma_commit(ring.empty + 8 * pos.stage);
                    pos.next(q.stages);
                }
                if (!ok) break;
                umma_commit(ring.accf + 8 * buf);
                if (q.keep && i + 1 < end && (i + 1) / hb != tile) umma_commit(g_empty);
                buf ^= 1;
                if (buf == 0) bphase ^= 1u;
            }
        }
    } else if (warp >= 4) {
        const int row = (warp - 4) * 32 + lane;
        uint8_t *stage = smem + q.ring + (warp - 4) * (TC_STAGE_ROWS / 4);
        int buf = 0;
        uint32_t bphase = 0;
        for (int i = first; i < end; ++i) {
            const int tile = i / hb, h0 = i % hb * TC_X_COLS;
            const int seg = find_segment(t128.tile, p.nbins, tile);
            const int r0 = (tile - t128.tile[seg]) * TC_ROWS;
            const int tok = r0 + row < t128.count[seg]
                                ? checked_token(p.sorted[t128.start[seg] + r0 + row], p.T, p.error_word) : -1;
            uint16_t *dst = p.dx + int64_t(tok < 0 ? 0 : tok) * p.dx_ld + h0;
            const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            const uint32_t d = ring.tmem + uint32_t(buf * TC_X_COLS) + (uint32_t((warp - 4) * 32) << 16);
            if (p.add) {
                for (int c = 0; c < TC_X_COLS && h0 + c < p.H; c += 32) {
                    uint32_t v[32];
                    tmem_ld32_nowait(d + uint32_t(c), v);
                    tmem_wait_ld();
                    add_rows(stage, v, p.scale, tok < 0 ? nullptr : dst + c, p.H - h0 - c);
                }
            } else {
                for (int c = 0; c < TC_X_COLS && h0 + c < p.H; c += 64) {
                    uint32_t o[32];
                    load64(d + uint32_t(c), p.scale, o);
                    store_rows(stage, o, tok < 0 ? nullptr : dst + c, p.H - h0 - c);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.acce + 8 * buf);
            buf ^= 1;
            if (buf == 0) bphase ^= 1u;
        }
    }
    tc_finish(ring, p.error_word);
    if (!p.add) clear_rest(p, t64);
}

// ---------------------------------------------------------------- g and u

struct GradUTcArgs {
    BackwardArgs b;
    TcRowMaps dy[LORA_MAX_SLICES];       // [T][n_s] of each slice
    CUtensorMap w[LORA_MAX_SLICES];      // [L][n_s][r], boxes 64 x 64 x 1
    int32_t by_width[LORA_MAX_SLICES];   // slices, widest first
    int32_t rp, ring, stage_bytes, stages;
};

// Item: (slice, 128-token tile), widest slices first; K = the slice's width.
__global__ void __launch_bounds__(TC_THREADS, 1) grad_u_tc_kernel(const __grid_constant__ GradUTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const TcRing ring = tc_setup(smem, q.ring, q.stage_bytes, q.stages, 2);
    pdl_wait();
    SegTab t64, t128;
    const int tiles = load_tabs(p, reinterpret_cast<int *>(smem + q.ring + TC_STAGE_ROWS + TC_BAR_BYTES), t64, t128);
    const int items = tiles * p.S;
    const int RP = q.rp, panels = RP / 64;

    if (warp == 0) {
        TcPos pos;
        int issued = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const int s = q.by_width[i / tiles], tile = i % tiles;
            const int seg = find_segment(t128.tile, p.nbins, tile);
            const int r0 = (tile - t128.tile[seg]) * TC_ROWS + lane * 4;
            TcRows rows;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                rows.t[j] = r0 + j < t128.count[seg] ? p.sorted[t128.start[seg] + r0 + j]
                                                     : tc_no_row(p.T, r0 + j);
            join_rows(rows, 1);
            const int steps = (p.n[s] + 63) / 64;
            for (int k = 0; k < steps; ++k) {
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                const uint32_t full = ring.full + 8 * pos.stage;
                if (lane == 0) mbar_arrive_expect_tx(full, 2 * TC_PANEL);
                __syncwarp();
                tc_load_rows(rows, ring.ring + pos.stage * ring.stage_bytes + lane * 512, &q.dy[s].gather,
                             q.dy[s].box, k * 64, full);
                ++issued;
                pos.next(ring.stages);
            }
        }
        if (lane == 0) tc_drain_loads(ring, issued);
    } else if (warp == 1) {
        TcPos pos;
        int issued = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const int s = q.by_width[i / tiles], tile = i % tiles;
            const int id = t128.id[find_segment(t128.tile, p.nbins, tile)];
            const int steps = (p.n[s] + 63) / 64;
            for (int k = 0; k < steps; ++k) {
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                const uint32_t full = ring.full + 8 * pos.stage;
                if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(panels * TC_PANEL));
                __syncwarp();
                if (lane < panels)
                    tma_load_3d(ring.ring + pos.stage * ring.stage_bytes + (2 + lane) * TC_PANEL, &q.w[s],
                                lane * 64, k * 64, id, full);
                ++issued;
                pos.next(ring.stages);
            }
        }
        if (lane == 0) tc_drain_loads(ring, issued);
    } else if (warp == 2) {
        if (lane == 0) {
            TcPos pos;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const int steps = (p.n[q.by_width[i / tiles]] + 63) / 64;
                if (!pg_wait(ring.acce + 8 * buf, bphase ^ 1u, ring.abort)) break;
                tc_fence_after();
                const uint32_t d = ring.tmem + uint32_t(buf * 128);
                for (int k = 0; k < steps; ++k) {
                    if (!pg_wait(ring.full + 8 * pos.stage, pos.phase, ring.abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = ring.ring + pos.stage * ring.stage_bytes, sb = sa + 2 * TC_PANEL;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(d, umma_desc_sw128(sa + kk * 32), umma_desc_mn(sb + kk * 2048),
                                  umma_idesc_bf16(128, RP) | 1u << 16, k != 0 || kk != 0);
                    umma_commit(ring.empty + 8 * pos.stage);
                    pos.next(ring.stages);
                }
                if (!ok) break;
                umma_commit(ring.accf + 8 * buf);
                buf ^= 1;
                if (buf == 0) bphase ^= 1u;
            }
        }
    } else if (warp >= 4) {
        const int row = (warp - 4) * 32 + lane;
        uint8_t *stage = smem + q.ring + (warp - 4) * (TC_STAGE_ROWS / 4);
        int buf = 0;
        uint32_t bphase = 0;
        for (int i = blockIdx.x; i < items; i += gridDim.x) {
            const int s = q.by_width[i / tiles], tile = i % tiles;
            const int seg = find_segment(t128.tile, p.nbins, tile);
            const int r0 = (tile - t128.tile[seg]) * TC_ROWS, count = t128.count[seg];
            // rows up to the end of the 64-token tile are written (zeros)
            const bool laid = r0 + row < (count + 63) / 64 * 64;
            const int tok = r0 + row < count
                                ? checked_token(p.sorted[t128.start[seg] + r0 + row], p.T, p.error_word) : -1;
            const int64_t at = (int64_t(s) * p.rows + int64_t(t64.tile[seg]) * 64 + r0 + row) * RP;
            const float *src = p.buf + (int64_t(s) * p.T + (tok < 0 ? 0 : tok)) * p.r;
            uint32_t o[32];
            for (int c = 0; c < RP; c += 64) {
                float4 f[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    f[j] = make_float4(0, 0, 0, 0);
                    if (tok >= 0 && c + 4 * j < p.r) f[j] = *reinterpret_cast<const float4 *>(src + c + 4 * j);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    o[2 * j] = pack_bf16x2(f[j].x, f[j].y);
                    o[2 * j + 1] = pack_bf16x2(f[j].z, f[j].w);
                }
                store_rows(stage, o, laid ? p.u + at + c : nullptr, 64);
            }
            const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            const uint32_t d = ring.tmem + uint32_t(buf * 128) + (uint32_t((warp - 4) * 32) << 16);
            for (int c = 0; c < RP; c += 64) {
                load64(d + uint32_t(c), 1.0f, o);
                store_rows(stage, o, laid ? p.g + at + c : nullptr, 64);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.acce + 8 * buf);
            buf ^= 1;
            if (buf == 0) bphase ^= 1u;
        }
    }
    tc_finish(ring, p.error_word);
}

// ---------------------------------------------------------------- host

static int tc_configure()
{
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    if (dev < 64 && configured[dev]) return 0;
    const void *fns[] = {(const void *)grad_w_tc_kernel, (const void *)grad_x_tc_kernel,
                         (const void *)grad_u_tc_kernel};
    for (const void *f : fns)
        if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, TC_SMEM)) != cudaSuccess)
            return int(e);
    if (dev < 64) configured[dev] = 1;
    return 0;
}

int launch_grad_w_tc(const BackwardArgs &p, int rp, cudaStream_t st)
{
    if (rp < 64 || !p.dy_vec || !p.x_vec || p.T < 1 || p.rows * p.S >= (int64_t(1) << 31)) return -1;
    static thread_local GradWTcArgs q;
    q.b = p;
    q.rp = rp;
    q.group = TC_MAX_N / rp < p.S ? TC_MAX_N / rp : p.S;
    q.groups = (p.S + q.group - 1) / q.group;
    int blocks = 0;
    for (int k = 0; k < q.groups; ++k) {
        bool any = false;
        for (int s = k * q.group; s < (k + 1) * q.group && s < p.S; ++s) any = any || p.da[s] != nullptr;
        if (any) blocks += (p.H + TC_W_COLS - 1) / TC_W_COLS;
        q.end[k] = blocks;
    }
    const bool has_a = blocks > 0;
    for (int s = 0; s < p.S; ++s) {
        if (p.db[s] != nullptr || p.dbias[s] != nullptr)
            blocks += ((p.off[s] & 7) + p.n[s] + TC_W_COLS - 1) / TC_W_COLS;
        q.end[q.groups + s] = blocks;
    }
    q.kinds = q.groups + p.S;
    if (blocks == 0) return 0;
    const int panels = ((has_a ? q.group : 1) * (rp / 64) + 1) / 2 * 2;
    q.stage_bytes = (2 + panels / 2) * TC_PANEL;
    q.ring = tc_ring_bytes(backward_tab_words(p.nbins, p.L) + p.L + 1);
    q.stages = tc_stages(q.ring - TC_ONES, q.stage_bytes);
    if (q.stages < 2) return -1;
    q.buffers = panels * 64 + 32 <= 256 ? 2 : 1;
    if (!encode_row_maps(&q.dy, p.dy, p.T, p.width, p.dy_ld) ||
        !encode_row_maps(&q.x, p.x, p.T, p.H, p.x_ld) ||
        !encode_tile_map(&q.u, p.u, uint64_t(p.S) * p.rows, uint64_t(rp), uint64_t(rp), 64, 64,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&q.g, p.g, uint64_t(p.S) * p.rows, uint64_t(rp), uint64_t(rp), 64, 64,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    if (int e = tc_configure()) return e;
    const int64_t items = int64_t(p.L) * blocks, most = device_sm_count() / 2;
    if (most < 1) return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(2 * (items < most ? items : most)));
    cfg.blockDim = dim3(TC_W_THREADS);
    cfg.dynamicSmemBytes = TC_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return int(cudaLaunchKernelEx(&cfg, grad_w_tc_kernel, q));
}

int launch_grad_x_tc(const BackwardArgs &p, int rp, cudaStream_t st)
{
    if (rp < 64 || !p.dx_vec || p.T < 1 || p.rows * p.S >= (int64_t(1) << 31)) return -1;
    static thread_local GradXTcArgs q;
    q.b = p;
    q.rp = rp;
    if (!encode_tile_map(&q.g, p.g, uint64_t(p.S) * p.rows, uint64_t(rp), uint64_t(rp), 64, 128,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    for (int s = 0; s < p.S; ++s)
        if (!encode_stack_map(&q.a[s], p.a[s], uint64_t(p.L), uint64_t(p.r), uint64_t(p.H), 64, 64)) return -1;
    const int g_bytes = p.S * (rp / 64) * 2 * TC_PANEL;
    q.ring = tc_ring_bytes(2 * (4 * p.nbins + 2));
    q.keep = q.ring - g_bytes >= 2 * 4 * TC_PANEL;
    q.stages = q.keep ? tc_stages(q.ring - g_bytes, 4 * TC_PANEL) : tc_stages(q.ring, 6 * TC_PANEL);
    if (int e = tc_configure()) return e;
    return int(launch_kernel(grad_x_tc_kernel, dim3(unsigned(device_sm_count())), dim3(TC_THREADS),
                             size_t(TC_SMEM), st, q));
}

int launch_grad_u_tc(const BackwardArgs &p, int rp, cudaStream_t st)
{
    if (rp < 64 || !p.dy_vec || p.T < 1 || p.rows * p.S >= (int64_t(1) << 31)) return -1;
    // One CTA walks a tile's whole width: with fewer tiles than half the SMs
    // the cluster kernel, which shares a tile's columns, is faster.
    if (int64_t(p.T) / TC_ROWS * p.S < device_sm_count() / 2) return -1;
    static thread_local GradUTcArgs q;
    q.b = p;
    q.rp = rp;
    for (int s = 0; s < p.S; ++s) {
        if (p.off[s] % 8 != 0) return -1;            // a gather starts on a 16-byte boundary
        if (!encode_row_maps(&q.dy[s], p.dy + p.off[s], p.T, p.n[s], p.dy_ld) ||
            !encode_stack_map(&q.w[s], p.b[s], uint64_t(p.L), uint64_t(p.n[s]), uint64_t(p.r), 64, 64))
            return -1;
        int at = s;
        for (; at > 0 && p.n[q.by_width[at - 1]] < p.n[s]; --at) q.by_width[at] = q.by_width[at - 1];
        q.by_width[at] = s;
    }
    q.stage_bytes = (2 + rp / 64) * TC_PANEL;
    q.ring = tc_ring_bytes(2 * (4 * p.nbins + 2));
    q.stages = tc_stages(q.ring, q.stage_bytes);
    if (int e = tc_configure()) return e;
    return int(launch_kernel(grad_u_tc_kernel, dim3(unsigned(device_sm_count())), dim3(TC_THREADS),
                             size_t(TC_SMEM), st, q));
}

}  // namespace lora
