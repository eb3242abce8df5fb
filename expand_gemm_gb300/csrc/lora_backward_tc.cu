// lora_backward_tc.cu -- the three products of lora_linear_backward on the
// tensor cores (tcgen05), for padded ranks 64 and 128; see lora_backward.cu
// for the formulas and the layout of g and u.
//
// Rows of dy and x are fetched through the token order by TMA gathers (four
// rows of 64 columns an instruction): a row past an adapter's last token
// gets an index past the matrix and arrives as zeros.  Weights are mapped
// with a dimension of their own for the adapter, so that what lies behind a
// slice's last row or column arrives as zeros too, never as a neighbour's
// values.  Products over tokens take both operands with their rows
// contiguous (MN-major), so nothing is transposed.
//
// One CTA an SM; warps: 0 gathers, 1 loads boxes, 2 issues UMMAs, 4..7 run
// the epilogue (thread = TMEM lane = row of the result).
#include "lora_backward.cuh"
#include "lora_pair_gemm.cuh"

namespace lora {

constexpr int TC_THREADS = 256;
constexpr int TC_PANEL = 64 * 64 * 2;            // 64 rows of 64 bf16
constexpr int TC_RING = 192 * 1024;
constexpr int TC_MAX_STAGES = 8;
constexpr int TC_BAR_BYTES = 256;
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

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                            int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];\n"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// The ring of operand stages and the accumulators' barriers of one CTA.
struct TcRing {
    uint32_t ring, full, empty, accf, acce, drain, stage_bytes;
    int stages;
    volatile int *abort;
    uint32_t tmem;
};

// Position in the ring.
struct TcPos {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// Shared memory: ring, `extra` bytes, barriers; then the caller's tables.
__device__ __forceinline__ TcRing tc_setup(uint8_t *smem, int stage_bytes, int stages, int extra,
                                           int loaders)
{
    TcRing r;
    r.ring = smem_addr(smem);
    r.full = r.ring + TC_RING + extra;
    r.empty = r.full + 8 * TC_MAX_STAGES;
    r.accf = r.empty + 8 * TC_MAX_STAGES;
    r.acce = r.accf + 16;
    r.drain = r.acce + 16;
    r.stage_bytes = uint32_t(stage_bytes);
    r.stages = stages;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + TC_RING + extra + 16 * TC_MAX_STAGES + 40);
    r.abort = reinterpret_cast<volatile int *>(misc + 1);
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(r.full + 8 * i, uint32_t(loaders));
            mbar_init(r.empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(r.accf + 8 * i, 1);
            mbar_init(r.acce + 8 * i, 4);
        }
        mbar_init(r.drain, 1);
        mbar_fence_init();
        *r.abort = 0;
    }
    if (threadIdx.x / 32 == 3) tmem_alloc(smem_addr(misc), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    r.tmem = *misc;
    return r;
}

// One thread of a loading warp, after its last fill: the fills of the last
// stages have landed and been consumed before the CTA may exit.
__device__ __forceinline__ void tc_drain_loads(const TcRing &r, int issued)
{
    const long long dd = clock64() + PG_TIMEOUT_CYCLES;
    for (int i = max(0, issued - r.stages); i < issued; ++i) {
        const uint32_t ph = uint32_t(i / r.stages) & 1u, b8 = 8u * uint32_t(i % r.stages);
        while (!mbar_try_wait(r.full + b8, ph) && clock64() < dd) {
        }
        while (!mbar_try_wait(r.empty + b8, ph) && !*r.abort && clock64() < dd) {
        }
    }
}

__device__ __forceinline__ void tc_finish(const TcRing &r, int32_t *error_word)
{
    __syncwarp();
    if (threadIdx.x == 64 && *r.abort) {              // the thread that issues UMMAs
        umma_commit(r.drain);
        const long long dd = clock64() + PG_TIMEOUT_CYCLES;
        while (!mbar_try_wait(r.drain, 0) && clock64() < dd) {
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && *r.abort) atomicOr(error_word, LORA_TIMEOUT_BIT);
    if (threadIdx.x / 32 == 3) tmem_dealloc(r.tmem, 512);
}

// 32 accumulators of this thread's row as 32 bf16, times f.
__device__ __forceinline__ void pack32(const uint32_t (&v)[32], float f, uint32_t (&o)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j)
        o[j] = pack_bf16x2(f * __uint_as_float(v[2 * j]), f * __uint_as_float(v[2 * j + 1]));
}

// Writes the first `many` (a multiple of 8, at most 32) of 32 bf16 values.
__device__ __forceinline__ void store32(uint16_t *dst, const uint32_t (&o)[16], int many)
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (8 * j < many)
            *reinterpret_cast<uint4 *>(dst + 8 * j) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
}

__device__ __forceinline__ uint8_t *tc_smem()
{
    extern __shared__ uint8_t tc_smem_raw[];
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tc_smem_raw) + 1023) & ~uintptr_t(1023));
}

// ---------------------------------------------------------------- dA, dB, dbias

struct GradWTcArgs {
    BackwardArgs b;
    CUtensorMap dy, x;         // gathers, box 64 columns x 1 row
    CUtensorMap u, g;          // boxes 64 columns x 64 rows of [S * rows][RP]
    int32_t rp, group, groups; // slices of one dA product
    int32_t end[2 * LORA_MAX_SLICES];   // blocks of one adapter: dA groups, then dB slices
    int32_t kinds, stage_bytes, stages, buffers;
};

// dA: rows = (slice, r) in products of 128, columns = 128 of x.
// dB: rows = 128 columns of dy, columns = r; dbias: one more product with
// ones.  An item's K is its adapter's tokens, 64 a stage.  Adapters are
// taken by falling token count, so that the CTAs' shares come out even.
__global__ void __launch_bounds__(TC_THREADS, 1) grad_w_tc_kernel(const __grid_constant__ GradWTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int RP = q.rp, PPS = RP / 64;                 // panels a slice
    for (int i = tid; i < TC_PANEL / 4; i += TC_THREADS)
        reinterpret_cast<uint32_t *>(smem + TC_RING)[i] = 0x3F803F80u;
    fence_proxy_async_smem();
    const TcRing ring = tc_setup(smem, q.stage_bytes, q.stages, TC_PANEL, 2);
    const uint32_t ones = ring.ring + TC_RING;
    pdl_wait();
    pdl_launch_dependents();
    int tiles;
    int *mem = reinterpret_cast<int *>(smem + TC_RING + TC_PANEL + TC_BAR_BYTES);
    const SegTab tab = load_tab(p, mem, tiles);
    const int *seg_of = load_seg_of(p, tab, tiles, mem);
    int *order = mem + backward_tab_words(p.nbins, p.L);
    for (int i = tid; i < p.L; i += TC_THREADS) {
        int at = i;
        if (p.L <= 256) {                               // more would take longer than it saves
            const int mine = seg_of[i] >= 0 ? tab.count[seg_of[i]] : 0;
            at = 0;
            for (int j = 0; j < p.L; ++j) {
                const int c = seg_of[j] >= 0 ? tab.count[seg_of[j]] : 0;
                at += c > mine || (c == mine && j < i);
            }
        }
        order[at] = i;
    }
    __syncthreads();
    const int blocks = q.end[q.kinds - 1];
    const int64_t items = int64_t(p.L) * blocks;

    struct Item {
        bool is_a;
        int id, s, slices, seg, start, count, steps, c0;
        int64_t row0;                                   // in g and u, within a slice
    };
    auto decode = [&](int64_t i) {
        Item it;
        it.id = order[i / blocks];
        const int blk = int(i % blocks);
        int k = 0;
        while (blk >= q.end[k]) ++k;
        const int j0 = blk - (k > 0 ? q.end[k - 1] : 0);
        it.is_a = k < q.groups;
        it.s = it.is_a ? k * q.group : k - q.groups;
        it.slices = it.is_a ? min(q.group, p.S - it.s) : 1;
        it.seg = seg_of[it.id];
        it.start = it.seg >= 0 ? tab.start[it.seg] : 0;
        it.count = it.seg >= 0 ? tab.count[it.seg] : 0;
        it.steps = (it.count + 63) / 64;
        it.c0 = (it.is_a ? 0 : p.off[it.s] & ~7) + j0 * 128;
        it.row0 = it.seg >= 0 ? int64_t(tab.tile[it.seg]) * 64 : 0;
        return it;
    };
    if (warp == 0) {
        // ------------------------------------------------ gathers of dy or x
        TcPos pos;
        int issued = 0;
        bool ok = true;
        const int panel = lane & 1, r4 = (lane >> 1) * 4;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = decode(i);
            const CUtensorMap *map = it.is_a ? &q.x : &q.dy;
            int t[4];
            auto tokens = [&](int k) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = k * 64 + r4 + j;
                    t[j] = row < it.count ? p.sorted[it.start + row] : p.T;
                }
            };
            if (it.steps > 0) tokens(0);
            for (int k = 0; k < it.steps; ++k) {
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                const uint32_t full = ring.full + 8 * pos.stage;
                if (lane == 0) mbar_arrive_expect_tx(full, 2 * TC_PANEL);
                __syncwarp();
                tma_gather4(ring.ring + pos.stage * ring.stage_bytes + panel * TC_PANEL + r4 * 128, map,
                            it.c0 + panel * 64, t[0], t[1], t[2], t[3], full);
                if (k + 1 < it.steps) tokens(k + 1);
                ++issued;
                pos.next(ring.stages);
            }
        }
        if (lane == 0) tc_drain_loads(ring, issued);
    } else if (warp == 1) {
        // ------------------------------------------------ u or g
        // g and u were written by the stream's previous kernel with ordinary stores
        asm volatile("fence.proxy.async.global;\n" ::: "memory");
        TcPos pos;
        int issued = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = decode(i);
            const CUtensorMap *map = it.is_a ? &q.g : &q.u;
            const int panels = it.slices * PPS;
            for (int k = 0; k < it.steps; ++k) {
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                const uint32_t full = ring.full + 8 * pos.stage;
                if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(panels * TC_PANEL));
                __syncwarp();
                if (lane < panels)
                    tma_load_2d(ring.ring + pos.stage * ring.stage_bytes + (2 + lane) * TC_PANEL, map,
                                lane % PPS * 64, int((it.s + lane / PPS) * p.rows + it.row0) + k * 64, full);
                ++issued;
                pos.next(ring.stages);
            }
        }
        if (lane == 0) tc_drain_loads(ring, issued);
    } else if (warp == 2) {
        // ------------------------------------------------ UMMAs
        if (lane == 0) {
            constexpr uint32_t T_AB = (1u << 15) | (1u << 16);
            TcPos pos;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const Item it = decode(i);
                if (it.steps == 0) continue;
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
                    const uint32_t z = ring.ring + pos.stage * ring.stage_bytes, v = z + 2 * TC_PANEL;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t acc = k != 0 || kk != 0;
                        const uint64_t dz = umma_desc_mn(z + kk * 2048);
                        if (it.is_a) {
                            for (int m = 0; m < mt; ++m)
                                umma_bf16(d + uint32_t(m * 128), umma_desc_mn(v + m * 2 * TC_PANEL + kk * 2048),
                                          dz, umma_idesc_bf16(128, 128) | T_AB, acc);
                        } else {
                            umma_bf16(d, dz, umma_desc_mn(v + kk * 2048), umma_idesc_bf16(128, RP) | T_AB, acc);
                            if (bias)
                                umma_bf16(d + uint32_t(RP), dz, umma_desc_mn(ones + kk * 2048),
                                          umma_idesc_bf16(128, 16) | T_AB, acc);
                        }
                    }
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
    } else if (warp >= 4) {
        // ------------------------------------------------ epilogue
        const int row = (warp - 4) * 32 + lane;
        int buf = 0;
        uint32_t bphase = 0;
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            const Item it = decode(i);
            const bool zero = it.steps == 0;
            const uint32_t d = ring.tmem + uint32_t(buf * (512 / q.buffers)) + (uint32_t((warp - 4) * 32) << 16);
            if (!zero) {
                const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) break;
                tc_fence_after();
            }
            uint32_t v[32], o[16];
            auto load = [&](uint32_t at) {
                if (zero) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                } else {
                    tmem_ld32_nowait(at, v);
                    tmem_wait_ld();
                }
            };
            if (it.is_a) {
                const int mt = (it.slices * RP + 127) / 128;
                for (int m = 0; m < mt; ++m) {
                    const int R = m * 128 + row, s = it.s + R / RP, r = R % RP;
                    uint16_t *out = R < it.slices * RP && r < p.r ? p.da[s] : nullptr;
                    if (out != nullptr) out += (int64_t(it.id) * p.r + r) * p.H + it.c0;
                    for (int c = 0; c < 128 && it.c0 + c < p.H; c += 32) {
                        load(d + uint32_t(m * 128 + c));
                        pack32(v, p.scale, o);
                        if (out != nullptr) store32(out + c, o, min(32, p.H - it.c0 - c));
                    }
                }
            } else {
                const int n = p.n[it.s], at = it.c0 + row - p.off[it.s];
                const bool in = at >= 0 && at < n;
                if (p.db[it.s] != nullptr) {
                    uint16_t *out = p.db[it.s] + (int64_t(it.id) * n + at) * p.r;
                    for (int c = 0; c < p.r; c += 32) {
                        load(d + uint32_t(c));
                        pack32(v, 1.0f, o);
                        if (in) store32(out + c, o, min(32, p.r - c));
                    }
                }
                if (p.dbias[it.s] != nullptr) {
                    uint32_t one[16];
                    one[0] = 0u;
                    if (!zero) {
                        tmem_ld16_nowait(d + uint32_t(RP), one);
                        tmem_wait_ld();
                    }
                    if (in)
                        p.dbias[it.s][int64_t(it.id) * n + at] =
                            uint16_t(pack_bf16x2(__uint_as_float(one[0]), 0.0f) & 0xFFFFu);
                }
            }
            if (!zero) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ring.acce + 8 * buf);
                if (++buf == q.buffers) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
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
};
constexpr int TC_X_COLS = 256;
constexpr int TC_X_STAGE = 6 * TC_PANEL;
constexpr int TC_X_STAGES = TC_RING / TC_X_STAGE;

// Both segment tables: 64-token tiles (rows of g and u) and 128-token tiles.
__device__ __forceinline__ int load_tabs(const BackwardArgs &p, int *mem, SegTab &t64, SegTab &t128)
{
    int tiles;
    t64 = load_tab(p, mem, tiles);
    t128 = seg_tab(mem + 4 * p.nbins + 2, p.nbins);
    return load_segments(p.no_lora, p.active, p.counts, p.start_loc, p.nbins, TC_ROWS, t128, false, 0,
                         p.T, p.error_word);
}

// Item: (128-token tile, 256 columns); K = slices x rank.
__global__ void __launch_bounds__(TC_THREADS, 1) grad_x_tc_kernel(const __grid_constant__ GradXTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const TcRing ring = tc_setup(smem, TC_X_STAGE, TC_X_STAGES, 0, 1);
    pdl_wait();
    pdl_launch_dependents();
    SegTab t64, t128;
    const int tiles = load_tabs(p, reinterpret_cast<int *>(smem + TC_RING + TC_BAR_BYTES), t64, t128);
    const int hb = (p.H + TC_X_COLS - 1) / TC_X_COLS;
    const int64_t items = int64_t(tiles) * hb;
    const int kps = q.rp / 64, steps = p.S * kps;

    if (warp == 0) {
        // g and u were written by the stream's previous kernel with ordinary stores
        asm volatile("fence.proxy.async.global;\n" ::: "memory");
        TcPos pos;
        int issued = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const int tile = int(i / hb), h0 = int(i % hb) * TC_X_COLS;
            const int seg = find_segment(t128.tile, p.nbins, tile);
            const int64_t row0 = int64_t(t64.tile[seg]) * 64 + int64_t(tile - t128.tile[seg]) * TC_ROWS;
            const int id = t128.id[seg];
            for (int k = 0; k < steps; ++k) {
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) {
                    ok = false;
                    break;
                }
                const uint32_t full = ring.full + 8 * pos.stage;
                const uint32_t at = ring.ring + pos.stage * TC_X_STAGE;
                const int s = k / kps, kc = k % kps * 64;
                if (lane == 0) mbar_arrive_expect_tx(full, TC_X_STAGE);
                __syncwarp();
                if (lane == 0) tma_load_2d(at, &q.g, kc, int(s * p.rows + row0), full);
                else if (lane <= 4)
                    tma_load_3d(at + (1 + lane) * TC_PANEL, &q.a[s], h0 + (lane - 1) * 64, kc, id, full);
                ++issued;
                pos.next(TC_X_STAGES);
            }
        }
        if (lane == 0) tc_drain_loads(ring, issued);
    } else if (warp == 2) {
        if (lane == 0) {
            TcPos pos;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
                if (!pg_wait(ring.acce + 8 * buf, bphase ^ 1u, ring.abort)) break;
                tc_fence_after();
                const uint32_t d = ring.tmem + uint32_t(buf * TC_X_COLS);
                for (int k = 0; k < steps; ++k) {
                    if (!pg_wait(ring.full + 8 * pos.stage, pos.phase, ring.abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = ring.ring + pos.stage * TC_X_STAGE, sb = sa + 2 * TC_PANEL;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(d, umma_desc_sw128(sa + kk * 32), umma_desc_mn(sb + kk * 2048),
                                  umma_idesc_bf16(128, TC_X_COLS) | 1u << 16, k != 0 || kk != 0);
                    umma_commit(ring.empty + 8 * pos.stage);
                    pos.next(TC_X_STAGES);
                }
                if (!ok) break;
                umma_commit(ring.accf + 8 * buf);
                buf ^= 1;
                if (buf == 0) bphase ^= 1u;
            }
        }
    } else if (warp >= 4) {
        const int row = (warp - 4) * 32 + lane;
        int buf = 0;
        uint32_t bphase = 0;
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            const int tile = int(i / hb), h0 = int(i % hb) * TC_X_COLS;
            const int seg = find_segment(t128.tile, p.nbins, tile);
            const int r0 = (tile - t128.tile[seg]) * TC_ROWS;
            const int tok = r0 + row < t128.count[seg]
                                ? checked_token(p.sorted[t128.start[seg] + r0 + row], p.T, p.error_word) : -1;
            uint16_t *dst = p.dx + int64_t(tok < 0 ? 0 : tok) * p.dx_ld + h0;
            const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            const uint32_t d = ring.tmem + uint32_t(buf * TC_X_COLS) + (uint32_t((warp - 4) * 32) << 16);
            for (int c = 0; c < TC_X_COLS && h0 + c < p.H; c += 32) {
                const int many = min(32, p.H - h0 - c);
                uint32_t v[32], o[16];
                tmem_ld32_nowait(d + uint32_t(c), v);
                uint4 was[4];
                if (p.add && tok >= 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (8 * j < many) was[j] = *reinterpret_cast<const uint4 *>(dst + c + 8 * j);
                }
                tmem_wait_ld();
                if (tok < 0) continue;
                if (p.add) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w[4] = {was[j].x, was[j].y, was[j].z, was[j].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[4 * j + e] = pack_bf16x2(
                                fmaf(p.scale, __uint_as_float(v[8 * j + 2 * e]), bf16_lo(w[e])),
                                fmaf(p.scale, __uint_as_float(v[8 * j + 2 * e + 1]), bf16_hi(w[e])));
                    }
                } else {
                    pack32(v, p.scale, o);
                }
                store32(dst + c, o, many);
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
    CUtensorMap dy[LORA_MAX_SLICES];     // [T][n_s] of each slice, gathers
    CUtensorMap w[LORA_MAX_SLICES];      // [L][n_s][r], boxes 64 x 64 x 1
    int32_t by_width[LORA_MAX_SLICES];   // slices, widest first
    int32_t rp, stage_bytes, stages;
};

// Item: (slice, 128-token tile), widest slices first; K = the slice's width.
__global__ void __launch_bounds__(TC_THREADS, 1) grad_u_tc_kernel(const __grid_constant__ GradUTcArgs q)
{
    const BackwardArgs &p = q.b;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const TcRing ring = tc_setup(smem, q.stage_bytes, q.stages, 0, 2);
    pdl_wait();
    pdl_launch_dependents();
    SegTab t64, t128;
    const int tiles = load_tabs(p, reinterpret_cast<int *>(smem + TC_RING + TC_BAR_BYTES), t64, t128);
    const int64_t items = int64_t(tiles) * p.S;
    const int RP = q.rp, panels = RP / 64;

    if (warp == 0) {
        TcPos pos;
        int issued = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const int s = q.by_width[i / tiles], tile = int(i % tiles);
            const int seg = find_segment(t128.tile, p.nbins, tile);
            const int r0 = (tile - t128.tile[seg]) * TC_ROWS + lane * 4;
            int t[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                t[j] = r0 + j < t128.count[seg] ? p.sorted[t128.start[seg] + r0 + j] : p.T;
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
                tma_gather4(ring.ring + pos.stage * ring.stage_bytes + lane * 512, &q.dy[s], k * 64, t[0],
                            t[1], t[2], t[3], full);
                ++issued;
                pos.next(ring.stages);
            }
        }
        if (lane == 0) tc_drain_loads(ring, issued);
    } else if (warp == 1) {
        TcPos pos;
        int issued = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const int s = q.by_width[i / tiles], tile = int(i % tiles);
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
            for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
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
        int buf = 0;
        uint32_t bphase = 0;
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            const int s = q.by_width[i / tiles], tile = int(i % tiles);
            const int seg = find_segment(t128.tile, p.nbins, tile);
            const int r0 = (tile - t128.tile[seg]) * TC_ROWS, count = t128.count[seg];
            // rows up to the end of the 64-token tile are written (zeros)
            const bool laid = r0 + row < (count + 63) / 64 * 64;
            const int tok = r0 + row < count
                                ? checked_token(p.sorted[t128.start[seg] + r0 + row], p.T, p.error_word) : -1;
            const int64_t at = (int64_t(s) * p.rows + int64_t(t64.tile[seg]) * 64 + r0 + row) * RP;
            const float *src = p.buf + (int64_t(s) * p.T + (tok < 0 ? 0 : tok)) * p.r;
            uint32_t v[32], o[16];
            for (int c = 0; c < RP; c += 32) {
                float4 f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    f[j] = make_float4(0, 0, 0, 0);
                    if (tok >= 0 && c + 4 * j < p.r) f[j] = *reinterpret_cast<const float4 *>(src + c + 4 * j);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[2 * j] = pack_bf16x2(f[j].x, f[j].y);
                    o[2 * j + 1] = pack_bf16x2(f[j].z, f[j].w);
                }
                if (laid) store32(p.u + at + c, o, 32);
            }
            const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            const uint32_t d = ring.tmem + uint32_t(buf * 128) + (uint32_t((warp - 4) * 32) << 16);
            for (int c = 0; c < RP; c += 32) {
                tmem_ld32_nowait(d + uint32_t(c), v);
                tmem_wait_ld();
                pack32(v, 1.0f, o);
                if (laid) store32(p.g + at + c, o, 32);
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
        if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024)) != cudaSuccess)
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
        if (any) blocks += (p.H + 127) / 128;
        q.end[k] = blocks;
    }
    const bool has_a = blocks > 0;
    for (int s = 0; s < p.S; ++s) {
        if (p.db[s] != nullptr || p.dbias[s] != nullptr) blocks += ((p.off[s] & 7) + p.n[s] + 127) / 128;
        q.end[q.groups + s] = blocks;
    }
    q.kinds = q.groups + p.S;
    if (blocks == 0) return 0;
    // an odd number of panels of rank 64 leaves the last product of dA half
    // empty: its second half reads the (unused) next panel of the stage
    const int panels = has_a ? (q.group * (rp / 64) + 1) / 2 * 2 : rp / 64;
    q.stage_bytes = (2 + panels) * TC_PANEL;
    q.stages = TC_RING / q.stage_bytes < TC_MAX_STAGES ? TC_RING / q.stage_bytes : TC_MAX_STAGES;
    const int cols_a = has_a ? (q.group * rp + 127) / 128 * 128 : 0;
    q.buffers = cols_a <= 256 ? 2 : 1;
    const int smem = TC_RING + TC_PANEL + TC_BAR_BYTES + 1024 +
                     (backward_tab_words(p.nbins, p.L) + p.L) * 4;
    if (smem > 227 * 1024) return -1;
    if (!encode_tile_map(&q.dy, p.dy, uint64_t(p.T), uint64_t(p.width), uint64_t(p.dy_ld), 64, 1,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&q.x, p.x, uint64_t(p.T), uint64_t(p.H), uint64_t(p.x_ld), 64, 1,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&q.u, p.u, uint64_t(p.S) * p.rows, uint64_t(rp), uint64_t(rp), 64, 64,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&q.g, p.g, uint64_t(p.S) * p.rows, uint64_t(rp), uint64_t(rp), 64, 64,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    if (int e = tc_configure()) return e;
    const int64_t items = int64_t(p.L) * blocks;
    const int sms = device_sm_count();
    return int(launch_kernel(grad_w_tc_kernel, dim3(unsigned(items < sms ? items : sms)), dim3(TC_THREADS),
                             size_t(smem), st, q));
}

int launch_grad_x_tc(const BackwardArgs &p, int rp, cudaStream_t st)
{
    if (rp < 64 || !p.dx_vec || p.T < 1 || p.rows * p.S >= (int64_t(1) << 31)) return -1;
    static thread_local GradXTcArgs q;
    q.b = p;
    q.rp = rp;
    const int smem = TC_RING + TC_BAR_BYTES + 1024 + 2 * int(seg_tab_bytes(p.nbins));
    if (smem > 227 * 1024) return -1;
    if (!encode_tile_map(&q.g, p.g, uint64_t(p.S) * p.rows, uint64_t(rp), uint64_t(rp), 64, 128,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    for (int s = 0; s < p.S; ++s)
        if (!encode_stack_map(&q.a[s], p.a[s], uint64_t(p.L), uint64_t(p.r), uint64_t(p.H), 64, 64)) return -1;
    if (int e = tc_configure()) return e;
    return int(launch_kernel(grad_x_tc_kernel, dim3(unsigned(device_sm_count())), dim3(TC_THREADS),
                             size_t(smem), st, q));
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
    const int smem = TC_RING + TC_BAR_BYTES + 1024 + 2 * int(seg_tab_bytes(p.nbins));
    if (smem > 227 * 1024) return -1;
    for (int s = 0; s < p.S; ++s) {
        if (p.off[s] % 8 != 0) return -1;            // a gather starts on a 16-byte boundary
        if (!encode_tile_map(&q.dy[s], p.dy + p.off[s], uint64_t(p.T), uint64_t(p.n[s]), uint64_t(p.dy_ld),
                             64, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_stack_map(&q.w[s], p.b[s], uint64_t(p.L), uint64_t(p.n[s]), uint64_t(p.r), 64, 64))
            return -1;
        int at = s;
        for (; at > 0 && p.n[q.by_width[at - 1]] < p.n[s]; --at) q.by_width[at] = q.by_width[at - 1];
        q.by_width[at] = s;
    }
    q.stage_bytes = (2 + rp / 64) * TC_PANEL;
    q.stages = TC_RING / q.stage_bytes < TC_MAX_STAGES ? TC_RING / q.stage_bytes : TC_MAX_STAGES;
    if (int e = tc_configure()) return e;
    return int(launch_kernel(grad_u_tc_kernel, dim3(unsigned(device_sm_count())), dim3(TC_THREADS),
                             size_t(smem), st, q));
}

}  // namespace lora
