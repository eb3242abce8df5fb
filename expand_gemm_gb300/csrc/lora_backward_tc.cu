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
// values.
//
// One CTA an SM; warps: 0 gathers, 1 loads boxes, 2 issues UMMAs, 4..7 run
// the epilogue (thread = TMEM lane = row of the result).
//
// 16384 tokens in sequences, 8 of 64 adapters in use, rank 128, 8192 to
// 8192, 1024, 1024: g 76 us (323 MB, 4.3 TB/s: 104 tiles of the wide slice
// on 152 SMs), dx 93 us (451 MB, 4.8 TB/s), dA and dB 208 us.  By token
// the gathers bound all three (16384 tokens, 4096 to 4096, 1024, 1024: g 60
// us in sequences, 209 by token; dA and dB 123 and 294).
#include "lora_backward.cuh"
#include "lora_tc.cuh"

namespace lora {

constexpr int TC_ROWS = 128;                     // tokens of a tile of g and dx

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

// The row to load for `tok`, read from the sorted list (a debug build takes
// one outside the batch as none; TMA's own bounds would give zeros, silently).
__device__ __forceinline__ int tc_row(const BackwardArgs &p, int tok, int row)
{
    if constexpr (kDebugChecks) {
        if (checked_token(tok, p.T, p.error_word) < 0) return tc_no_row(p.T, row);
    }
    return tok;
}

__device__ __forceinline__ void tc_load_rows(const TcRows &r, uint32_t dst, const CUtensorMap *gather,
                                             const CUtensorMap *boxes, int col, uint32_t bar)
{
    if (r.level >= 0) tma_load_2d(dst, boxes + r.level, col, r.t[0], bar);
    else if (r.level == -1) tma_gather4(dst, gather, col, r.t[0], r.t[1], r.t[2], r.t[3], bar);
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
    // [S * rows / 64 * RP][64], boxes 64 x RP: a tile's u or g, transposed (and
    // their second terms behind them)
    CUtensorMap ut, gt;
    int32_t rp, group, groups; // slices of one dA product
    int32_t end[2 * LORA_MAX_SLICES];   // blocks of one adapter: dA groups, then dB slices
    int32_t kinds, ring, stage_bytes, stages, buffers, ones;
};
constexpr int TC_W_COLS = 256;           // columns of dy or x of an item
constexpr int TC_W_THREADS = TC_THREADS + 128;
constexpr int TC_W_SLOTS = 8;            // steps' tokens in shared memory
constexpr int TC_W_AHEAD = 6;            // of them on their way

// The gradients of an adapter without tokens: zeros, written by 128 threads
// along the rows.
__device__ __forceinline__ void clear_item(const BackwardArgs &p, bool is_a, int id, int s0, int slices,
                                           int c0, int thread)
{
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (is_a) {
        const int chunks = min(TC_W_COLS / 8, (p.H - c0) / 8);
        for (int s = s0; s < s0 + slices; ++s) {
            if (p.da[s] == nullptr || (thread & 31) >= chunks) continue;
            uint16_t *out = p.da[s] + int64_t(id) * p.r * p.H + c0 + (thread & 31) * 8;
            for (int r = thread >> 5; r < p.r; r += 4) *reinterpret_cast<uint4 *>(out + int64_t(r) * p.H) = zero;
        }
    } else {
        const int n = p.n[s0], lo = max(0, c0 - p.off[s0]), hi = min(n, c0 + TC_W_COLS - p.off[s0]);
        if (p.db[s0] != nullptr) {
            uint4 *out = reinterpret_cast<uint4 *>(p.db[s0] + (int64_t(id) * n + lo) * p.r);
            for (int i = thread; i < (hi - lo) * p.r / 8; i += 128) out[i] = zero;
        }
        if (p.dbias[s0] != nullptr)
            for (int i = thread; i < hi - lo; i += 128) p.dbias[s0][int64_t(id) * n + lo + i] = 0;
    }
}

// An item is an adapter x 256 columns of x or dy: D[r x 256] += (g or u of
// 64 tokens)^T (64 tokens of the columns); dA of up to two slices at once
// (one under the other at rank 64; one at a time took 216 us in place of 208
// at rank 128, 374 in place of 294 by token), dB of one, dbias as one more
// product, with ones.  K is the adapter's tokens.
//
// K, the tokens, runs along the rows of x and dy: they are the MN-major B.
// g and u are the K-major A, laid out transposed by the kernel that computes
// them, 64 tokens a row: D then has a slice's r along its lanes, so that dA
// leaves in whole rows.  With x or dy as A, on CTA pairs, rank 128 took 279 us
// in place of 231.
//
// At 16384 tokens, hidden 8192, widths 8192, 1024, 1024, 64 adapters: 208 us
// for the 1.27 GB that it moves, 6.1 TB/s (x is read once for each group of
// slices).
//
// TERMS: the same steps again for the second terms of g and u.
//
// Adapters are taken by falling token count, so that the CTAs' shares come
// out even.  Warps 8 to 11 write the zeros of the adapters without tokens
// meanwhile (with 8 of 64 adapters in use they are most of the bytes).
template <bool TERMS>
__global__ void __launch_bounds__(TC_W_THREADS, 1) grad_w_tc_kernel(const __grid_constant__ GradWTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int RP = q.rp, A_BYTES = RP * 128;                // one slice's tile of g or u
    constexpr int Z_BYTES = 4 * TC_PANEL;
    for (int i = tid; i < q.ones / 4; i += TC_W_THREADS)
        reinterpret_cast<uint32_t *>(smem + q.ring - q.ones)[i] = 0x3F803F80u;
    fence_proxy_async_smem();
    const TcRing ring = tc_setup(smem, q.ring, q.stage_bytes, q.stages, 2);
    const uint32_t ones = ring.ring + q.ring - q.ones;
    pdl_wait();
    int tiles;
    int *mem = reinterpret_cast<int *>(smem + q.ring + TC_STAGE_ROWS + TC_BAR_BYTES);
    const SegTab tab = load_tab(p, mem, tiles);
    const int *seg_of = load_seg_of(p, tab, tiles, mem);
    // order: the segments of the adapters with tokens, then the adapters without
    int *order = mem + backward_tab_words(p.nbins, p.L);
    int slot_at = p.L + 1;
    slot_at += -(slot_at + backward_tab_words(p.nbins, p.L)) & 3;
    int *slots = order + slot_at;                           // steps' tokens, 16-byte aligned
    volatile int *done = slots + TC_W_SLOTS * 64;           // steps loaded
    if (tid == 0) *done = 0;
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
    const int slice_tiles = int(p.rows / BW_TOK);

    struct Item {
        bool is_a;
        int id, s, slices, start, count, steps, c0, tile0;
    };
    auto steps_of = [](int count) { return (TERMS ? 2 : 1) * ((count + 63) / 64); };
    auto kind = [&](int blk, Item &it) {
        int k = 0;
        while (blk >= q.end[k]) ++k;
        it.is_a = k < q.groups;
        it.s = it.is_a ? k * q.group : k - q.groups;
        it.slices = it.is_a ? min(q.group, p.S - it.s) : 1;
        it.c0 = (it.is_a ? 0 : p.off[it.s] & ~7) + (blk - (k > 0 ? q.end[k - 1] : 0)) * TC_W_COLS;
    };
    auto decode = [&](int i) {
        Item it;
        const int seg = order[i / blocks];
        kind(i % blocks, it);
        it.id = tab.id[seg];
        it.start = tab.start[seg];
        it.count = tab.count[seg];
        it.steps = steps_of(it.count);
        it.tile0 = tab.tile[seg];
        return it;
    };
    // a step's 64 tokens of the adapter (the second terms' steps come last)
    auto tokens_of = [](const Item &it, int k) { return TERMS && 2 * k >= it.steps ? k - it.steps / 2 : k; };
    if (warp == 0) {
        // ------------------------------------------------ columns of dy or x
        // The steps' tokens come by cp.async, six steps ahead and across the
        // items' ends (loaded one step ahead, into registers, their latency
        // of 1200 clocks beside the other traffic was over half of this
        // warp's time: 225 us in place of 208).
        const uint32_t slots_at = smem_addr(slots);
        int a_item = blockIdx.x, a_k = 0, a_slot = 0, a_start = 0, a_count = 0;
        auto enter = [&]() {
            if (a_item >= items) return;
            const int seg = order[a_item / blocks];
            a_start = tab.start[seg];
            a_count = tab.count[seg];
        };
        auto ahead = [&]() {
            if (a_item < items) {
                const int t0 = (TERMS && 2 * a_k >= steps_of(a_count) ? a_k - steps_of(a_count) / 2 : a_k) * 64;
#pragma unroll
                for (int j = lane; j < 64; j += 32)
                    if (t0 + j < a_count)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n"
                                     :: "r"(slots_at + (a_slot * 64 + j) * 4), "l"(p.sorted + a_start + t0 + j)
                                     : "memory");
                if (TERMS ? ++a_k >= steps_of(a_count) : ++a_k * 64 >= a_count) {
                    a_k = 0;
                    a_item += gridDim.x;
                    enter();
                }
            }
            cp_async_commit();
            a_slot = a_slot + 1 == TC_W_SLOTS ? 0 : a_slot + 1;
        };
        enter();
        for (int i = 0; i < TC_W_AHEAD; ++i) ahead();
        TcPos pos;
        int issued = 0, slot = 0;
        bool ok = true;
        const int panel = lane & 1, r4 = (lane >> 1) * 4;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = decode(i);
            const TcRowMaps *map = it.is_a ? &q.x : &q.dy;
            for (int k = 0; k < it.steps; ++k) {
                cp_async_wait<TC_W_AHEAD - 1>();
                __syncwarp();
                const int4 own = *reinterpret_cast<const int4 *>(slots + slot * 64 + r4);
                slot = slot + 1 == TC_W_SLOTS ? 0 : slot + 1;
                const int row = tokens_of(it, k) * 64 + r4;
                TcRows rows;
                rows.t[0] = row < it.count ? tc_row(p, own.x, row) : tc_no_row(p.T, row);
                rows.t[1] = row + 1 < it.count ? tc_row(p, own.y, row + 1) : tc_no_row(p.T, row + 1);
                rows.t[2] = row + 2 < it.count ? tc_row(p, own.z, row + 2) : tc_no_row(p.T, row + 2);
                rows.t[3] = row + 3 < it.count ? tc_row(p, own.w, row + 3) : tc_no_row(p.T, row + 3);
                join_rows(rows, 2);
                ahead();
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                const uint32_t full = ring.full + 8 * pos.stage;
                if (lane == 0) mbar_arrive_expect_tx(full, Z_BYTES);
                __syncwarp();
#pragma unroll
                for (int j = panel; j < 4; j += 2)
                    tc_load_rows(rows, ring.ring + pos.stage * ring.stage_bytes + j * TC_PANEL + r4 * 128,
                                 &map->gather, map->box, it.c0 + j * 64, full);
                ++issued;
                if (lane == 0) *done = issued;
                pos.next(ring.stages);
            }
        }
        cp_async_wait<0>();
        if (lane == 0) tc_drain_loads(ring, issued);
    } else if (warp == 1) {
        // ------------------------------------------------ u or g
        // written by the stream's previous kernel with ordinary stores
        asm volatile("fence.proxy.async.global;\n" ::: "memory");
        TcPos pos;
        int issued = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = decode(i);
            const CUtensorMap *map = it.is_a ? &q.gt : &q.ut;
            for (int k = 0; k < it.steps; ++k) {
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                const uint32_t full = ring.full + 8 * pos.stage;
                if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(it.slices * A_BYTES));
                __syncwarp();
                if (lane < it.slices)
                    tma_load_2d(ring.ring + pos.stage * ring.stage_bytes + Z_BYTES + lane * A_BYTES, map, 0,
                                ((it.s + lane + (tokens_of(it, k) < k ? p.S : 0)) * slice_tiles + it.tile0 +
                                 tokens_of(it, k)) * RP, full);
                ++issued;
                pos.next(ring.stages);
            }
        }
        if (lane == 0) tc_drain_loads(ring, issued);
    } else if (warp == 2) {
        // ------------------------------------------------ UMMAs
        if (lane == 0) {
            constexpr uint32_t IDESC = umma_idesc_bf16(128, TC_W_COLS) | 1u << 16;
            TcPos pos;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const Item it = decode(i);
                if (!pg_wait(ring.acce + 8 * buf, bphase ^ 1u, ring.abort)) break;
                tc_fence_after();
                const uint32_t d = ring.tmem + uint32_t(buf * (512 / q.buffers));
                const int mt = (it.slices * RP + 127) / 128;
                const bool bias = !it.is_a && p.dbias[it.s] != nullptr;
                for (int k = 0; k < it.steps; ++k) {
                    if (!pg_wait(ring.full + 8 * pos.stage, pos.phase, ring.abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t z = ring.ring + pos.stage * ring.stage_bytes, a = z + Z_BYTES;
                    umma_k64(d, a, z, IDESC, k != 0);
                    if (mt > 1) umma_k64(d + uint32_t(TC_W_COLS), a + 2 * TC_PANEL, z, IDESC, k != 0);
                    if (bias && tokens_of(it, k) == k) umma_k64(d + uint32_t(TC_W_COLS), ones, z, IDESC, k != 0);
                    umma_commit(ring.empty + 8 * pos.stage);
                    pos.next(ring.stages);
                }
                if (!ok) break;
                umma_commit(ring.accf + 8 * buf);
                if (++buf == q.buffers) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------ epilogue
        const int row = (warp - 4) * 32 + lane;         // slice and r
        uint8_t *stage = smem + q.ring + (warp - 4) * (TC_STAGE_ROWS / 4);
        int buf = 0;
        uint32_t bphase = 0;
        for (int i = blockIdx.x; i < items; i += gridDim.x) {
            const Item it = decode(i);
            const uint32_t d = ring.tmem + uint32_t(buf * (512 / q.buffers)) + (uint32_t((warp - 4) * 32) << 16);
            const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            uint32_t o[32];
            if (it.is_a) {
                const int mt = (it.slices * RP + 127) / 128;
                for (int m = 0; m < mt; ++m) {
                    const int R = m * 128 + row, s = it.s + R / RP, r = R % RP;
                    uint16_t *out = R < it.slices * RP && r < p.r ? p.da[s] : nullptr;
                    if (out != nullptr) out += (int64_t(it.id) * p.r + r) * p.H + it.c0;
                    for (int c = 0; c < TC_W_COLS && it.c0 + c < p.H; c += 64) {
                        load64(d + uint32_t(m * TC_W_COLS + c), p.scale, o);
                        store_rows(stage, o, out != nullptr ? out + c : nullptr, p.H - it.c0 - c);
                    }
                }
            } else {
                const int n = p.n[it.s], r0 = (warp - 4) * 32, n0 = it.c0 - p.off[it.s];
                uint16_t *out = p.db[it.s];
                if (out != nullptr && r0 < p.r) {
                    out += (int64_t(it.id) * n + n0) * p.r + r0;
                    for (int c = 0; c < TC_W_COLS && n0 + c < n; c += 64) {
                        load64(d + uint32_t(c), 1.0f, o);
                        store_columns(stage, o, out + int64_t(c) * p.r, p.r, -(n0 + c), n - n0 - c, p.r - r0);
                    }
                }
                uint16_t *bias = p.dbias[it.s];
                if (bias != nullptr && warp == 4) {
                    // every row of the product with ones holds the sums: lane l
                    // keeps column c + l of each 32
                    for (int c = 0; c < TC_W_COLS; c += 32) {
                        uint32_t v[32];
                        tmem_ld32_nowait(d + uint32_t(TC_W_COLS + c), v);
                        tmem_wait_ld();
                        uint32_t mine = 0;
#pragma unroll
                        for (int j = 0; j < 32; ++j) mine = lane == j ? v[j] : mine;
                        const int at = n0 + c + lane;
                        if (at >= 0 && at < n)
                            bias[int64_t(it.id) * n + at] =
                                uint16_t(pack_bf16x2(__uint_as_float(mine), 0.0f) & 0xFFFFu);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.acce + 8 * buf);
            if (++buf == q.buffers) {
                buf = 0;
                bphase ^= 1u;
            }
        }
    } else if (warp >= 8) {
        // ------------------------------------------------ adapters without tokens
        // Written in step with the products: at full speed the zeros take the
        // memory from the first half of the products, whose loads wait for
        // it (231 us in place of 208; 156 without zeros).
        int steps = 0;
        for (int i = blockIdx.x + lane * gridDim.x; i < items; i += 32 * gridDim.x)
            steps += steps_of(tab.count[order[i / blocks]]);
        steps = int(__reduce_add_sync(0xffffffffu, unsigned(steps)));
        const int empty = (p.L - active) * blocks;
        const int mine = empty > int(blockIdx.x) ? (empty - int(blockIdx.x) + int(gridDim.x) - 1) / int(gridDim.x) : 0;
        for (int c = 0; c < mine; ++c) {
            const int first = int(int64_t(steps) * c / mine);
            // a hundred sleeps at most, each up to 1 us, for each item: the
            // order matters, not the wait
            for (int tries = 0; *done < first && tries < 100 && !*ring.abort; ++tries) __nanosleep(500);
            const int i = blockIdx.x + c * gridDim.x;
            Item it;
            kind(i % blocks, it);
            clear_item(p, it.is_a, order[active + i / blocks], it.s, it.slices, it.c0, tid - TC_THREADS);
        }
    }
    tc_finish(ring, p.error_word);
}

// ---------------------------------------------------------------- dx

struct GradXTcArgs {
    BackwardArgs b;
    CUtensorMap g;                       // boxes 64 columns x 128 rows of [S * rows][RP]
    CUtensorMap a[LORA_MAX_SLICES];      // [L][r][H], boxes 64 x 64 x 1
    int32_t rp;
    int32_t ring, stages;
};
constexpr int TC_X_COLS = 256;

// Both segment tables: 64-token tiles (rows of g and u) and tiles of `rows`.
__device__ __forceinline__ int load_tabs(const BackwardArgs &p, int *mem, SegTab &t64, SegTab &tile_tab,
                                         int rows = TC_ROWS)
{
    int tiles;
    t64 = load_tab(p, mem, tiles);
    tile_tab = seg_tab(mem + 4 * p.nbins + 2, p.nbins);
    return load_segments(p.no_lora, p.active, p.counts, p.start_loc, p.nbins, rows, tile_tab, false, 0,
                         p.T, p.error_word);
}

// Item: (128-token tile, 256 columns); K = slices x rank.  For products whose
// g does not fit shared memory beside A (slices x rank above 512): both
// stream.  The others run on grad_x_pair_kernel.
__global__ void __launch_bounds__(TC_THREADS, 1) grad_x_tc_kernel(const __grid_constant__ GradXTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kps = q.rp / 64, steps = p.S * kps;
    constexpr int G_BYTES = 2 * TC_PANEL, A_BYTES = 4 * TC_PANEL;
    constexpr uint32_t STAGE = A_BYTES + G_BYTES;
    const TcRing ring = tc_setup(smem, q.ring, int(STAGE), q.stages, 1);
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
        if (lane == 0) {
            TcPos pos;
            int issued = 0, tile = first / hb, h0 = first % hb * TC_X_COLS;
            bool ok = true;
            for (int i = first; ok && i < end; ++tile, h0 = 0) {
                const int seg = find_segment(t128.tile, p.nbins, tile);
                const int row0 = t64.tile[seg] * 64 + (tile - t128.tile[seg]) * TC_ROWS;
                const int id = t128.id[seg];
                for (; ok && i < end && h0 < p.H; ++i, h0 += TC_X_COLS) {
                    int grow = row0;
                    for (int s = 0; ok && s < p.S; ++s, grow += int(p.rows)) {
                        const CUtensorMap *map = &q.a[s];
                        for (int kc = 0; kc < q.rp; kc += 64) {
                            if (!pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort)) {
                                ok = false;
                                break;
                            }
                            const uint32_t full = ring.full + 8 * pos.stage;
                            const uint32_t at = ring.ring + pos.stage * STAGE;
                            mbar_arrive_expect_tx(full, STAGE);
#pragma unroll
                            for (int j = 0; j < 4; ++j) tma_load_3d(at + j * TC_PANEL, map, h0 + j * 64, kc, id, full);
                            tma_load_2d(at + A_BYTES, &q.g, kc, grow, full);
                            ++issued;
                            pos.next(q.stages);
                        }
                    }
                }
            }
            tc_drain_loads(ring, issued);
        }
    } else if (warp == 1 || warp == 3) {
        if (!p.add) clear_rest(p, t64, warp >> 1, 2);
    } else if (warp == 2) {
        if (lane == 0) {
            TcPos pos;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int i = first; ok && i < end; ++i) {
                if (!pg_wait(ring.acce + 8 * buf, bphase ^ 1u, ring.abort)) break;
                tc_fence_after();
                const uint32_t d = ring.tmem + uint32_t(buf * TC_X_COLS);
                for (int k = 0; k < steps; ++k) {
                    if (!pg_wait(ring.full + 8 * pos.stage, pos.phase, ring.abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sb = ring.ring + pos.stage * STAGE, sa = sb + A_BYTES;
                    umma_k64(d, sa, sb, umma_idesc_bf16(128, TC_X_COLS) | 1u << 16, k != 0);
                    umma_commit(ring.empty + 8 * pos.stage);
                    pos.next(q.stages);
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
}

// dx on CTA pairs: 256 tokens of one adapter, 128 of them in each CTA
// with their g, and half of A's 256 columns in each, which leaves room for
// more of A in flight and for eight epilogue warps (a half of the columns
// each four): with four, one on each scheduler, the chain from TMEM through
// shared memory to dx bounded the kernel: 113 us in place of 75 for 16384
// tokens, rank 128, 4096 to 4096, 1024, 1024.
constexpr int TC_XP_THREADS = 384;
constexpr int TC_XP_SLOT = 32 * 128;             // 32 rows of 64 columns
constexpr int TC_XP_STAGE = 8 * TC_XP_SLOT;

__global__ void __launch_bounds__(TC_XP_THREADS, 1) grad_x_pair_kernel(const __grid_constant__ GradXTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kps = q.rp / 64, steps = p.S * kps;
    constexpr int G_BYTES = 2 * TC_PANEL, A_BYTES = 2 * TC_PANEL;
    const uint32_t base = smem_addr(smem);
    const uint32_t full = base + q.ring + TC_XP_STAGE, empty = full + 8 * TC_MAX_STAGES;
    const uint32_t accf = empty + 8 * TC_MAX_STAGES, acce = accf + 16, drain = acce + 16;
    const uint32_t g_full = drain + 24, g_empty = g_full + 8, acce_odd = g_empty + 8;
    const uint32_t g_at = base + q.stages * A_BYTES;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + (drain + 8 - base));
    volatile int *abort = reinterpret_cast<volatile int *>(misc + 1);
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < q.stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf + 8 * i, 1);
            mbar_init(acce + 8 * i, 8);           // this CTA's epilogue warps
            mbar_init(acce_odd + 8 * i, 1);       // the odd CTA's, in the even one
        }
        mbar_init(drain, 1);
        mbar_init(g_full, 1);
        mbar_init(g_empty, 1);
        mbar_fence_init();
        *abort = 0;
    }
    if (warp == 3) tmem_alloc_pair(smem_addr(misc), 512);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *misc;
    pdl_wait();
    SegTab t64, t256;
    const int tiles = load_tabs(p, reinterpret_cast<int *>(smem + q.ring + TC_XP_STAGE + TC_BAR_BYTES), t64, t256,
                                2 * TC_ROWS);
    const int hb = (p.H + TC_X_COLS - 1) / TC_X_COLS;
    const int items = tiles * hb, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int first = int(int64_t(items) * pair / pairs);
    const int end = int(int64_t(items) * (pair + 1) / pairs);

    if (warp == 0) {
        // g and u were written by the stream's previous kernel with ordinary stores
        asm volatile("fence.proxy.async.global;\n" ::: "memory");
        if (lane == 0) {
            const uint32_t full0 = cluster_map(full, 0), g_full0 = cluster_map(g_full, 0);
            TcPos pos;
            int issued = 0, tile = first / hb, h0 = first % hb * TC_X_COLS;
            uint32_t gphase = 0;
            bool ok = true, loaded = false;
            for (int i = first; ok && i < end; ++tile, h0 = 0) {
                const int seg = find_segment(t256.tile, p.nbins, tile);
                const int row0 = t64.tile[seg] * 64 + (tile - t256.tile[seg]) * 2 * TC_ROWS + int(rank) * TC_ROWS;
                const int id = t256.id[seg];
                if (!pg_wait(g_empty, gphase ^ 1u, abort)) break;
                if (rank == 0) mbar_arrive_expect_tx(g_full, uint32_t(2 * steps * G_BYTES));
                for (int k = 0; k < steps; ++k)
                    tma_load_2d_pair(g_at + k * G_BYTES, &q.g, k % kps * 64, int(k / kps * p.rows) + row0, g_full0);
                gphase ^= 1u;
                loaded = true;
                for (; ok && i < end && h0 < p.H; ++i, h0 += TC_X_COLS) {
                    for (int s = 0; ok && s < p.S; ++s) {
                        const CUtensorMap *map = &q.a[s];
                        for (int kc = 0; kc < q.rp; kc += 64) {
                            if (!pg_wait(empty + 8 * pos.stage, pos.phase ^ 1u, abort)) {
                                ok = false;
                                break;
                            }
                            if (rank == 0) mbar_arrive_expect_tx(full + 8 * pos.stage, 2 * A_BYTES);
                            const uint32_t at = base + pos.stage * A_BYTES;
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                tma_load_3d_pair(at + j * TC_PANEL, map, h0 + int(rank) * 128 + j * 64, kc, id,
                                                 full0 + 8 * pos.stage);
                            ++issued;
                            pos.next(q.stages);
                        }
                    }
                }
            }
            // No copy and no commit may still target this CTA when it exits
            // (the leader's barriers count both CTAs' copies).
            const long long dd = clock64() + PG_TIMEOUT_CYCLES;
            for (int i = max(0, issued - q.stages); i < issued; ++i) {
                const uint32_t ph = uint32_t(i / q.stages) & 1u, b8 = 8u * uint32_t(i % q.stages);
                if (rank == 0)
                    while (!mbar_try_wait_cluster(full + b8, ph) && clock64() < dd) {
                    }
                while (!mbar_try_wait_cluster(empty + b8, ph) && !*abort && clock64() < dd) {
                }
            }
            if (loaded && rank == 0)
                while (!mbar_try_wait_cluster(g_full, gphase ^ 1u) && clock64() < dd) {
                }
        }
    } else if (warp == 1 || warp == 3) {
        if (!p.add) clear_rest(p, t64, warp >> 1, 2);
    } else if (warp == 2) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t IDESC = umma_idesc_bf16(2 * TC_ROWS, TC_X_COLS) | 1u << 16;
            TcPos pos;
            int buf = 0, tile = -1;
            uint32_t bphase = 0, gphase = 0;
            bool ok = true;
            for (int i = first; ok && i < end; ++i) {
                if (!pg_wait(acce + 8 * buf, bphase ^ 1u, abort) ||
                    !pg_wait(acce_odd + 8 * buf, bphase ^ 1u, abort))
                    break;
                if (i / hb != tile) {
                    tile = i / hb;
                    if (!pg_wait(g_full, gphase, abort)) break;
                    gphase ^= 1u;
                }
                tc_fence_after();
                const uint32_t d = tmem + uint32_t(buf * TC_X_COLS);
                for (int k = 0; k < steps; ++k) {
                    if (!pg_wait(full + 8 * pos.stage, pos.phase, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = g_at + k * G_BYTES, sb = base + pos.stage * A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_pair(d, umma_desc_sw128(sa + kk * 32), umma_desc_mn(sb + kk * 2048), IDESC,
                                       k != 0 || kk != 0);
                    umma_commit_both(empty + 8 * pos.stage);
                    pos.next(q.stages);
                }
                if (!ok) break;
                umma_commit_both(accf + 8 * buf);
                if (i + 1 < end && (i + 1) / hb != tile) umma_commit_both(g_empty);
                buf ^= 1;
                if (buf == 0) bphase ^= 1u;
            }
            if (*abort) {       // nothing in flight when TMEM is released
                umma_commit_pair(cluster_map(drain, 0));
                const long long dd = clock64() + PG_TIMEOUT_CYCLES;
                while (!mbar_try_wait_cluster(drain, 0) && clock64() < dd) {
                }
            }
        }
        if (lane == 0 && rank == 1) {
            // tells the even CTA which accumulators are read.  The epilogue
            // warps arrive in their own CTA: an arrival at cluster scope
            // waits for the warp's loads and stores in flight (103 us in
            // place of 93)
            const uint32_t to = cluster_map(acce_odd, 0);
            int buf = 0;
            uint32_t bphase = 0;
            for (int i = first; i < end; ++i) {
                if (!pg_wait(acce + 8 * buf, bphase, abort)) break;
                tc_fence_after();
                tc_fence_before();
                mbar_arrive_cluster(to + 8 * buf);
                buf ^= 1;
                if (buf == 0) bphase ^= 1u;
            }
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) / 4 * (TC_X_COLS / 2);
        const int row = int(rank) * TC_ROWS + quarter * 32 + lane;
        uint8_t *slot = smem + q.ring + (warp - 4) * TC_XP_SLOT;
        int buf = 0, tile = first / hb, h0 = first % hb * TC_X_COLS + half;
        uint32_t bphase = 0;
        // the tokens of rows 4 k + lane / 8 of this warp's 32 (negative: none)
        int token[8];
        auto find = [&](int of) {
            const int seg = find_segment(t256.tile, p.nbins, of);
            const int r = (of - t256.tile[seg]) * 2 * TC_ROWS + row;
            const int tok =
                r < t256.count[seg] ? checked_token(p.sorted[t256.start[seg] + r], p.T, p.error_word) : -1;
#pragma unroll
            for (int k = 0; k < 8; ++k) token[k] = __shfl_sync(0xffffffffu, tok, 4 * k + (lane >> 3));
        };
        uint4 was[8] = {};
        auto fetch = [&](int c) {               // what dx holds of 64 columns
            const int col = c + (lane & 7) * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (token[k] >= 0 && col < p.H)
                    was[k] = *reinterpret_cast<const uint4 *>(p.dx + int64_t(token[k]) * p.dx_ld + col);
        };
        if (first < end) find(tile);
        if (p.add && first < end) fetch(h0);
        for (int i = first; i < end; ++i) {
            const bool got = pg_wait(accf + 8 * buf, bphase, abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            const uint32_t d = tmem + uint32_t(buf * TC_X_COLS + half) + (uint32_t(quarter * 32) << 16);
            const bool turn = h0 - half + TC_X_COLS >= p.H;         // the next item is another tile's
#pragma unroll
            for (int c = 0; c < TC_X_COLS / 2; c += 64) {
                if (p.add) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int r = 4 * k + (lane >> 3);
                        *reinterpret_cast<uint4 *>(slot + r * 128 + ((lane ^ r) & 7) * 16) = was[k];
                    }
                    if (c == 0) fetch(h0 + 64);
                    else if (!turn) fetch(h0 + TC_X_COLS);
                    __syncwarp();
                }
                // a lane's own row: the sums and what dx holds, one rounding
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t v[32];
                    tmem_ld32_nowait(d + uint32_t(c + 32 * e), v);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint4 *piece = reinterpret_cast<uint4 *>(slot + lane * 128 + (((4 * e + k) ^ lane) & 7) * 16);
                        uint32_t o[4];
                        if (p.add) {
                            const uint4 x = *piece;
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                o[j] = pack_bf16x2(
                                    fmaf(p.scale, __uint_as_float(v[8 * k + 2 * j]), bf16_lo(w[j])),
                                    fmaf(p.scale, __uint_as_float(v[8 * k + 2 * j + 1]), bf16_hi(w[j])));
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                o[j] = pack_bf16x2(p.scale * __uint_as_float(v[8 * k + 2 * j]),
                                                   p.scale * __uint_as_float(v[8 * k + 2 * j + 1]));
                        }
                        *piece = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                if (c + 64 == TC_X_COLS / 2) {
                    tc_fence_before();                          // the accumulator is read
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acce + 8 * buf);
                }
                __syncwarp();
                const int col = h0 + c + (lane & 7) * 8;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = 4 * k + (lane >> 3);
                    const uint4 x = *reinterpret_cast<const uint4 *>(slot + r * 128 + ((lane ^ r) & 7) * 16);
                    if (token[k] >= 0 && col < p.H)
                        *reinterpret_cast<uint4 *>(p.dx + int64_t(token[k]) * p.dx_ld + col) = x;
                }
                __syncwarp();
            }
            buf ^= 1;
            if (buf == 0) bphase ^= 1u;
            h0 += TC_X_COLS;
            if (turn && i + 1 < end) {
                h0 = half;
                find(++tile);
                if (p.add) fetch(h0);
            }
        }
    }
    __syncwarp();
    if (threadIdx.x == 0 && *abort && p.error_word != nullptr) atomicOr(p.error_word, LORA_TIMEOUT_BIT);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 3) tmem_dealloc_pair(tmem, 512);
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
                rows.t[j] = r0 + j < t128.count[seg] ? tc_row(p, p.sorted[t128.start[seg] + r0 + j], r0 + j)
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
                    umma_k64(d, sa, sb, umma_idesc_bf16(128, RP) | 1u << 16, k != 0);
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
            // the transposed tiles [r][64 tokens]: this warp's 32 tokens of one
            const int64_t tile64 = int64_t(s) * (p.rows / BW_TOK) + t64.tile[seg] + (r0 + row) / BW_TOK;
            const int64_t turned = tile64 * RP * BW_TOK + row % BW_TOK / 32 * 32;
            const bool laid_warp = r0 + row / 32 * 32 < (count + 63) / 64 * 64;
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
                if (p.ut != nullptr) store_columns(stage, o, p.ut + turned + c * 64, 64, 0, laid_warp ? RP - c : 0, 32);
                else store_rows(stage, o, laid ? p.u + at + c : nullptr, 64);
            }
            const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            const uint32_t d = ring.tmem + uint32_t(buf * 128) + (uint32_t((warp - 4) * 32) << 16);
            for (int c = 0; c < RP; c += 64) {
                load64(d + uint32_t(c), 1.0f, o);
                store_rows(stage, o, laid ? p.g + at + c : nullptr, 64);
                if (p.gt != nullptr) store_columns(stage, o, p.gt + turned + c * 64, 64, 0, laid_warp ? RP - c : 0, 32);
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
    const void *fns[] = {(const void *)grad_w_tc_kernel<false>, (const void *)grad_w_tc_kernel<true>,
                         (const void *)grad_x_tc_kernel, (const void *)grad_x_pair_kernel, (const void *)grad_u_tc_kernel};
    for (const void *f : fns)
        if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, TC_SMEM)) != cudaSuccess)
            return int(e);
    if (dev < 64) configured[dev] = 1;
    return 0;
}

bool grad_w_tc_fits(const BackwardArgs &p, int rp)
{
    if (rp < 64 || !p.dy_vec || !p.x_vec || p.T < 1 || p.rows * p.S * 2 >= (int64_t(1) << 31)) return false;
    // At rank 64 a small batch is faster on mma.sync, whose CTAs are three an
    // SM: 512 tokens x 4096 to 4096 8.8 us there, 10.7 here (32 adapters by
    // token 19.5 and 25.2); 2048 tokens 24.4 there, 16.8 here.  At rank 128
    // it never is (128 tokens 15.2 there, 13.0 here).
    return rp > 64 || int64_t(p.T) / TC_ROWS * ((p.H + p.width) / TC_W_COLS) >= device_sm_count();
}

int launch_grad_w_tc(const BackwardArgs &p, int rp, cudaStream_t st)
{
    static thread_local GradWTcArgs q;
    q.b = p;
    q.rp = rp;
    q.group = p.S < 2 ? p.S : 2;
    q.groups = (p.S + q.group - 1) / q.group;
    int blocks = 0;
    bool bias = false;
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
        bias = bias || p.dbias[s] != nullptr;
        q.end[q.groups + s] = blocks;
    }
    q.kinds = q.groups + p.S;
    if (blocks == 0) return 0;
    // products of 128 rows: two slices at rank 128, or one and the bias, take
    // all of TMEM
    const int slices = has_a ? q.group : 1;
    q.buffers = slices * rp > 128 || bias ? 1 : 2;
    q.stage_bytes = 4 * TC_PANEL + (slices * rp > 128 ? slices * rp * 128 : 2 * TC_PANEL);
    q.ones = bias ? 2 * TC_PANEL : 0;
    q.ring = tc_ring_bytes(backward_tab_words(p.nbins, p.L) + p.L + 1 + 3 + TC_W_SLOTS * 64 + 1);
    q.stages = tc_stages(q.ring - q.ones, q.stage_bytes);
    const uint64_t rows = uint64_t(p.low != 0 ? 2 : 1) * uint64_t(p.S) * uint64_t(p.rows / BW_TOK) * uint64_t(rp);
    if (!encode_row_maps(&q.dy, p.dy, p.T, p.width, p.dy_ld) ||
        !encode_row_maps(&q.x, p.x, p.T, p.H, p.x_ld) ||
        !encode_tile_map(&q.ut, p.ut, rows, 64, 64, 64, uint32_t(rp), CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&q.gt, p.gt, rows, 64, 64, 64, uint32_t(rp), CU_TENSOR_MAP_SWIZZLE_128B))
        return LORA_ERR_DEVICE;
    if (int e = tc_configure()) return e;
    const int64_t items = int64_t(p.L) * blocks;
    const int sms = device_sm_count();
    return int(launch_kernel(p.low != 0 ? grad_w_tc_kernel<true> : grad_w_tc_kernel<false>, dim3(unsigned(items < sms ? items : sms)), dim3(TC_W_THREADS),
                             size_t(TC_SMEM), st, q));
}

int launch_grad_x_tc(const BackwardArgs &p, int rp, cudaStream_t st)
{
    if (rp < 64 || p.low != 0 || !p.dx_vec || p.T < 1 || p.rows * p.S >= (int64_t(1) << 31)) return -1;
    // Fewer items than SMs: smaller ones on mma.sync are faster.  4096 to
    // 4096 at rank 64: 1024 tokens 15.3 us here, 14.0 there; 2048 tokens 15.9
    // here, 22.6 there; at rank 128 16.4 and 15.4, 17.1 and 25.4.
    if (int64_t(p.T) / TC_ROWS * ((p.H + TC_X_COLS - 1) / TC_X_COLS) < device_sm_count()) return -1;
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
    const int pair_ring = q.ring - (TC_XP_STAGE - TC_STAGE_ROWS);
    if (pair_ring - g_bytes >= 4 * 2 * TC_PANEL && device_sm_count() > 1) {
        q.ring = pair_ring;
        q.stages = tc_stages(q.ring - g_bytes, 2 * TC_PANEL);
        if (int e = tc_configure()) return e;
        return int(launch_pair_kernel(grad_x_pair_kernel, device_sm_count() / 2, st, q, TC_XP_THREADS, TC_SMEM));
    }
    q.stages = tc_stages(q.ring, 6 * TC_PANEL);
    if (int e = tc_configure()) return e;
    return int(launch_kernel(grad_x_tc_kernel, dim3(unsigned(device_sm_count())), dim3(TC_THREADS),
                             size_t(TC_SMEM), st, q));
}

int launch_grad_u_tc(const BackwardArgs &p, int rp, cudaStream_t st)
{
    if (rp < 64 || p.low != 0 || !p.dy_vec || p.T < 1 || p.rows * p.S >= (int64_t(1) << 31)) return -1;
    // One CTA walks a tile's whole width; the kernel of lora_backward.cu cuts
    // the width among CTAs and joins.  Widths 4096, 1024, 1024 at rank 128:
    // 1024 tokens (24 tiles) 26.6 us here, 23.5 there; 2048 (48 tiles) 27.2
    // here, 34.3 there; width 4096 at rank 64: 16 tiles 24.9 and 18.8, 64
    // tiles 27.6 and 35.8.
    if (int64_t(p.T) / TC_ROWS * p.S < device_sm_count() / 4) return -1;
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
