// lora_expert_stream.cu -- the forward product of a mixture of experts for few
// rows an expert, where reading the weights bounds it: a tile is 128 rows of
// W[e] (the UMMA's M) by up to NT rows of x (its N), so that the tensor core
// does no more than the rows need and every SM streams weights through one
// ring, across tiles.
//
// Weights in bf16 come by TMA as the operand in shared memory.  Weights in 4
// bits come as codes, 128 rows of 256 elements a stage; sixteen warps decode
// them, a thread a row, into TMEM, from where the UMMA reads that operand:
// through shared memory the decoded tile would be written and read once more
// (8 bytes for each byte of codes).  A byte's two elements are looked up in a
// table that each lane has in a bank of its own, and multiplied by their
// scale.  The table's rows are 256 bytes apart and it begins on a 64 KB
// boundary, so that one byte permutation puts a byte of codes into its
// address: 12 instructions for eight elements.  (With a row every 128 bytes
// and a multiply-add for the address it was 16; with masks and shifts in the
// table's place 21, and a quarter of the words decoded so beside the table 2%
// slower in all.)  The ring's stages lie on both sides of the table, the
// barriers in the rows' second halves.
//
// Warps: 0 loads, 1 issues UMMAs and owns TMEM, 2..5 run the epilogue (thread
// = TMEM lane = row of W); with 4-bit weights 6..21 decode, 22 fetches scales
// and 23 loads x, into a ring of its own: codes are done with when they are
// decoded, x when the products have run (in one ring the decoding waited for
// codes: 256 tokens of 16 experts 4096 x 4096 75 us in place of 66).  Two
// accumulators: the epilogue of one tile runs under the next one's products.
//
// Batches of a few rows need no copy of x: the kernel walks the metadata's
// segments itself and gathers rows by TMA (90 clocks for four rows of 128
// bytes: with more rows that would be what bounds it).
//
// Where the tiles are fewer than the SMs, a cluster of CTAs shares a tile, each
// a run of its K: the others write their sums into the first one's shared
// memory, which adds them in order.
//
// One GB300, whole calls, cold: 256 tokens, 2 of 16 experts 4096 x 4096 in bf16:
// 99 to 103 us, 5.4 TB/s; 32 tokens, 4 of 32 experts 4096 to 11008 in 4 bits: 156
// to 160, 4.9 TB/s, bound by the decoding; one token, two experts 4096 x 4096 in
// bf16: 21 (64 tiles, two CTAs each: 24 of 152 SMs have none).
#include "lora_expert.cuh"
#include "lora_tc.cuh"

namespace lora {

struct StreamArgs {
    ExpertArgs p;
    CUtensorMap w, x, s;
    int32_t stages;               // of the ring
    int32_t boxed;                // scales come by TMA
};

constexpr int ST_ROWS = 128;                    // of W in a tile
constexpr int ST_TILE = ST_ROWS * 128;          // bytes of W in a stage: 64 bf16 or 256 codes a row
constexpr int ST_SCALES = ST_ROWS * 16;         // bytes of scales: of two stages, the least box of TMA
constexpr int ST_DEC0 = 6;                      // first decoding warp
constexpr int ST_SETS = 4;                      // of four warps that decode
constexpr int ST_SCALE_WARP = ST_DEC0 + 4 * ST_SETS;
constexpr int ST_X_WARP = ST_SCALE_WARP + 1;    // loads x, beside codes
constexpr int ST_MAX_BUFS = 3;                  // decoded stages in TMEM
constexpr int ST_MAX_STAGES = 12;
constexpr int ST_BINS = 257;                    // segments, where the kernel walks them itself
constexpr int ST_SEGMENTS = 5 * 1024;           // and their bytes
static_assert(seg_tab_bytes(ST_BINS) <= ST_SEGMENTS, "segments");
constexpr int ST_TABLE = 65536;                 // shared address of the wide table

// Where a kernel's rows of x come from: the copy, once it is complete, by its
// table of tiles; the copy, while weights are asked for, by the metadata's
// segments; gathers by TMA.  (Of a template: as values of the launch the same
// choices cost 3% of the time.)
constexpr int ST_COPY = 0, ST_EARLY = 1, ST_GATHER = 2;

template <bool FOUR, int NT>
struct StreamSizes {
    static constexpr int KC = FOUR ? 256 : 64;                  // elements of K in a stage
    static constexpr int PANELS = KC / 64;                      // of x: NT rows of 64
    static constexpr int X = PANELS * NT * 128;                 // their bytes
    // a stage of the ring: W and x, or the codes and the rows' scales, beside a
    // ring of XS stages of x
    static constexpr int STAGE = ST_TILE + (FOUR ? ST_SCALES : X);
    static constexpr int XS = !FOUR ? 0 : NT <= 16 ? 4 : 2;
    static constexpr int THREADS = 32 * (FOUR ? ST_X_WARP + 1 : ST_DEC0);
    static constexpr int BARS = 512;
    static constexpr int SUMS = NT * ST_ROWS * 4;               // bytes of one CTA's sums of a tile
    static constexpr int TABLE = FOUR ? 256 * 256 : 0;
    static constexpr int ALL = 232448;                          // shared memory of a CTA, from address 1024 on
    // stages of the ring beside that of x and the sums of parts - 1 other CTAs
    __host__ __device__ static constexpr int ring(int parts)
    {
        const int rest = XS * X + (parts - 1) * SUMS;
        const int n = FOUR ? (ST_TABLE - 1024) / STAGE + (1024 + ALL - ST_TABLE - TABLE - rest) / STAGE
                           : (ALL - 1024 - BARS - ST_SEGMENTS - rest) / STAGE;
        return n < ST_MAX_STAGES ? n : ST_MAX_STAGES;
    }
    static_assert(!FOUR || (ST_TABLE - 1024) % STAGE >= ST_SEGMENTS, "the segments lie between stages and table");
    static constexpr int COLS = FOUR ? 512 : 2 * NT < 32 ? 32 : 2 * NT;      // of TMEM
    static constexpr int DECODED = 2 * NT;                     // first TMEM column of the decoded stages
    static constexpr int BUFS = (512 - DECODED) / 128 < ST_MAX_BUFS ? (512 - DECODED) / 128 : ST_MAX_BUFS;
    static_assert(!FOUR || BUFS >= 2, "TMEM");
    // A decoding warp takes every other stage, and so waits on a barrier for
    // every other phase: the phase before has to be over by then, or its
    // parity says that the one two before is the one waited for.  A warp that
    // has decoded stage n - 2 knows that the products of n - 2 - BUFS have
    // run, so the stage that was in n's place before must be no later.
    static constexpr int LEAST = FOUR ? BUFS + 2 : 3;           // stages of the ring
    static_assert(ring(1) >= LEAST, "stages");
};

struct StreamItem {
    int row, valid, start, n0, expert;
};

// Item i: an expert's tiles of rows take 128 rows of its weights one after
// another, so that they are read from memory once.
template <int FROM, int NT>
__device__ __forceinline__ StreamItem stream_item(const ExpertArgs &p, const SegTab &tab, int i, int cols)
{
    if constexpr (FROM != ST_COPY) {
        const int k = find_segment(tab.tile, p.nbins, i / cols), first = tab.tile[k], tiles = tab.tile[k + 1] - first;
        const int j = i - first * cols, tile = j % tiles;
        const int at = tab.start[k] + tile * NT, none = tab.id[0] == -1 ? tab.count[0] : 0;
        return StreamItem{at - none, min(NT, tab.count[k] - tile * NT), at, j / tiles * ST_ROWS, tab.id[k]};
    }
    const int4 *at = reinterpret_cast<const int4 *>(p.table + i / cols);
    const int4 a = at[0], b = at[1];          // base, tiles, expert, start; count, row
    const int j = i - a.x * cols, tile = j % a.y;
    StreamItem it;
    it.row = b.y + tile * NT;
    it.valid = min(NT, b.x - tile * NT);
    it.start = a.w + tile * NT;
    it.n0 = j / a.y * ST_ROWS;
    it.expert = a.z;
    return it;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A block of 32 elements with scale byte c.  `table`: shared address of this
// lane's entries, a pair of bf16 for each byte; a byte's are 256 bytes apart
// and the table is aligned so that the byte is the address's second.  Each
// product with the scale is exact, also by 2^-127 (c = 0), which is subnormal;
// c = 255 is NaN.
__device__ __forceinline__ void decode_block(uint32_t table, const uint4 &w, uint32_t c, uint32_t *o)
{
    uint32_t f = c * 0x00800080u;                  // 2^(c - 127) twice
    if (c == 0u) f = 0x00400040u;
    if (c == 255u) f = 0x7FC07FC0u;
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t v;
            asm("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(__byte_perm(words[i], table, 0x7604 + (j << 4))));
            o[4 * i + j] = mul_bf16x2(v, f);
        }
    }
}

// The 4-bit element as bf16.
__device__ __forceinline__ uint32_t e2m1_bf16(uint32_t code)
{
    return (__float_as_uint(__uint_as_float((code & 8u) << 28 | (code & 7u) << 22) * 0x1p126f)) >> 16;
}

// One row's eight scale bytes of a stage, at any alignment, to `dst` (shared
// memory, 16 bytes): the words that they lie in, and in the fourth word which
// byte of the first is theirs.  In a row's last stage bytes that do not exist
// stand for 1 (their codes are zero).  (Bytes one by one, and waited for, took
// 128 rows of 16 experts 4096 x 2016 62 us; so 43.)
__device__ __forceinline__ void fetch_scales(const ExpertArgs &p, uint32_t dst, int expert, int n, int kb)
{
    const int per = p.K / 32, at = kb * 8;
    const int64_t off = (int64_t(expert) * p.N + min(n, p.N - 1)) * per + at;
    uint32_t first = 0;
    if (at + 8 <= per) {
        first = uint32_t(off) & 3u;
        const uint8_t *src = p.scales + (off - first);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n"
                     "cp.async.ca.shared.global [%0+4], [%1+4], 4;\n" :: "r"(dst), "l"(src) : "memory");
        if (first != 0) {
            // nothing is read behind the last expert's scales
            const int64_t left = int64_t(p.E) * p.N * per - (off - first) - 8;
            asm volatile("cp.async.ca.shared.global [%0+8], [%1+8], 4, %2;\n"
                         :: "r"(dst), "l"(src), "r"(int(min(int64_t(4), left))) : "memory");
        }
    } else {
        const uint8_t *src = p.scales + off;
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = at + i < per ? src[i] : 127u;
            if (i < 4) lo |= c << (8 * i);
            else hi |= c << (8 * i - 32);
        }
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" :: "r"(dst), "r"(lo), "r"(hi) : "memory");
    }
    asm volatile("st.shared.b32 [%0+12], %1;\n" :: "r"(dst), "r"(first) : "memory");
}

// D += A B over 64 of K, as four UMMAs: A decoded in TMEM, B K-major; one add
// to each descriptor.  `more` is 0 for a tile's first block.
__device__ __forceinline__ void umma_k64_tmem_a(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t more)
{
    const uint64_t db = umma_desc_sw128(b);
    const uint32_t b_lo = uint32_t(db), b_hi = uint32_t(db >> 32);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        asm volatile(
            "{\n.reg .pred p;\n.reg .b64 b;\n"
            "mov.b64 b, {%2, %3};\n"
            "setp.ne.b32 p, %5, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n"
            :: "r"(d_tmem), "r"(a + kk * 8), "r"(b_lo + kk * 2), "r"(b_hi), "r"(idesc),
               "r"(kk == 0 ? more : 1u) : "memory");
}

// The same with both operands K-major in shared memory.
__device__ __forceinline__ void umma_k64_smem(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t more)
{
    const uint64_t da = umma_desc_sw128(a), db = umma_desc_sw128(b);
    const uint32_t a_lo = uint32_t(da), b_lo = uint32_t(db), hi = uint32_t(da >> 32);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        asm volatile(
            "{\n.reg .pred p;\n.reg .b64 a, b;\n"
            "mov.b64 a, {%1, %3};\n"
            "mov.b64 b, {%2, %3};\n"
            "setp.ne.b32 p, %5, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n"
            :: "r"(d_tmem), "r"(a_lo + kk * 2), "r"(b_lo + kk * 2), "r"(hi), "r"(idesc),
               "r"(kk == 0 ? more : 1u) : "memory");
}

// No copy may be on its way to this CTA when it exits.
__device__ __forceinline__ void drain_ring(uint32_t full, uint32_t empty, int stages, int issued, volatile int *abort)
{
    const long long dd = clock64() + PG_TIMEOUT_CYCLES;
    for (int i = max(0, issued - stages); i < issued; ++i) {
        const uint32_t ph = uint32_t(i / stages) & 1u, b8 = 8u * uint32_t(i % stages);
        while (!mbar_try_wait(full + b8, ph) && clock64() < dd) {
        }
        while (!mbar_try_wait(empty + b8, ph) && !*abort && clock64() < dd) {
        }
    }
}

// One stage of x, by a whole warp: from the copy, or by gathers of four rows a
// lane (rows[0] < 0: none); PANELS boxes of 64 columns, `pitch` bytes apart.
template <bool DIRECT, int PANELS>
__device__ __forceinline__ void load_x(const StreamArgs &g, uint32_t to, int pitch, int col, int row, const int (&rows)[4],
                                       uint32_t bar)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < PANELS; ++j) {
        if constexpr (!DIRECT) {
            if (lane == 0) tma_load_2d(to + j * pitch, &g.x, col + j * 64, row, bar);
        } else if (rows[0] >= 0 && col + j * 64 < g.p.K) {
            tma_gather4(to + j * pitch + lane * 512, &g.x, col + j * 64, rows[0], rows[1], rows[2], rows[3], bar);
        }
    }
}

// The four rows of x that this lane gathers for a tile, outside the matrix
// behind the tile's last.
__device__ __forceinline__ void gathered_rows(const ExpertArgs &p, const StreamItem &it, int (&rows)[4])
{
    const int first = 4 * int(threadIdx.x & 31);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        int row = p.R;
        if (first + k < it.valid) {
            const int i = expert_row(p, it.start + first + k);
            row = i < 0 ? p.R : i / p.fan;
        }
        rows[k] = first < it.valid ? row : -1;
    }
}

template <bool FOUR, int NT, int FROM>
__global__ void __launch_bounds__(StreamSizes<FOUR, NT>::THREADS, 1)
expert_stream_kernel(const __grid_constant__ StreamArgs g)
{
    using Z = StreamSizes<FOUR, NT>;
    constexpr bool DIRECT = FROM == ST_GATHER, early = FROM == ST_EARLY;
    extern __shared__ uint8_t st_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(st_smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_addr(smem);
    // With 4-bit weights: stages, segments, the table, stages, x, the others'
    // sums; else stages, segments, the others' sums, barriers.
    const uint32_t end = smem_addr(st_smem_raw) + Z::ALL;
    const uint32_t lut = FOUR ? (base & 0xFF000000u) + ST_TABLE : (end - Z::BARS) & ~uint32_t(1023);
    uint32_t *table = reinterpret_cast<uint32_t *>(smem + (lut - base));
    const int below = FOUR ? int(lut - base) / Z::STAGE : ST_MAX_STAGES;
    auto stage_at = [&](int i) {
        return FOUR && i >= below ? lut + Z::TABLE + uint32_t(i - below) * Z::STAGE : base + uint32_t(i) * Z::STAGE;
    };
    // the others' sums, [parts - 1][NT][128], and x before them
    const ExpertArgs &p = g.p;
    const int cols = (p.N + ST_ROWS - 1) / ST_ROWS, nk = (p.K + Z::KC - 1) / Z::KC;
    // this CTA's share of a tile's K; parts that would have none are not counted
    const uint32_t rank = cluster_ctarank();
    const int cluster = int(cluster_nctarank()), per = (nk + cluster - 1) / cluster, parts = (nk + per - 1) / per;
    const int kb0 = int(rank) * per, kb1 = min(nk, kb0 + per);
    const uint32_t sums = (FOUR ? end : lut) - (cluster - 1) * Z::SUMS;
    const uint32_t x_at = sums - Z::XS * Z::X;
    const SegTab tab = seg_tab(reinterpret_cast<int *>(smem + ((FOUR ? lut : x_at) - ST_SEGMENTS - base)), p.nbins);
    const uint32_t bars = FOUR ? lut + 128 : end - Z::BARS;
    const uint32_t full = bars, empty = FOUR ? bars + 256 : full + 8 * ST_MAX_STAGES;
    const uint32_t accf = FOUR ? bars + 512 : empty + 8 * ST_MAX_STAGES, acce = accf + 16;       // [2] each
    const uint32_t decf = acce + 16, dece = decf + 8 * ST_MAX_BUFS, drain = dece + 8 * ST_MAX_BUFS;
    const uint32_t peers = drain + 16;                              // the others' sums are here
    const uint32_t xfull = FOUR ? bars + 768 : peers + 8, xempty = xfull + 8 * 4;
    static_assert(32 + 16 * ST_MAX_BUFS + 24 <= 128 && 8 * ST_MAX_STAGES <= 128, "barriers in a row's second half");
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + (drain + 8 - base));
    volatile int *abort = reinterpret_cast<volatile int *>(s_tmem + 1);
    // (the top byte of a shared address is the CTA's rank in its cluster)
    if (FOUR && (smem_addr(st_smem_raw) & 0xFFFFFFu) != 1024) {  // the ring was counted from there
        pdl_wait();
        if (threadIdx.x == 0) atomicOr(p.error_word, LORA_TIMEOUT_BIT);
        return;
    }
    // the warp as a value that the compiler knows to be the same in its lanes
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < g.stages; ++i) {
            mbar_init(full + 8 * i, FOUR && !g.boxed ? 33 : 1);      // the scales' 32 lanes
            mbar_init(empty + 8 * i, FOUR ? 8 : 1);                  // eight decoding warps; the UMMAs
        }
        for (int i = 0; i < Z::XS; ++i) {
            mbar_init(xfull + 8 * i, 1);
            mbar_init(xempty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf + 8 * i, 1);
            mbar_init(acce + 8 * i, 4);
        }
        for (int i = 0; FOUR && i < ST_MAX_BUFS; ++i) {
            mbar_init(decf + 8 * i, 8);
            mbar_init(dece + 8 * i, 1);
        }
        mbar_init(drain, 1);
        mbar_init(peers, parts > 1 ? 4 * (parts - 1) : 1);
        mbar_fence_init();
        *abort = 0;
        tma_prefetch_map(&g.w);
        tma_prefetch_map(&g.x);
        if (FOUR && g.boxed) tma_prefetch_map(&g.s);
    }
    if constexpr (FOUR) {
        for (int i = tid; i < 256 * 32; i += Z::THREADS) {
            const uint32_t byte = uint32_t(i) / 32;
            table[byte * 64 + i % 32] = e2m1_bf16(byte & 15u) | e2m1_bf16(byte >> 4) << 16;
        }
    }
    if (warp == 1) tmem_alloc(smem_addr(s_tmem), Z::COLS);
    tc_fence_before();
    if (cluster > 1) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
    // The copy of x is waited for by the warp that loads it, while weights are
    // on their way; the kernels before it are complete when it lets this one
    // begin.
    if (!early) pdl_wait();

    int total;
    if constexpr (FROM != ST_COPY) {
        total = load_segments(p.no_lora, p.active, p.counts, p.start_loc, p.nbins, NT, tab, false, 0, p.R, p.error_word,
                              true);
        total = __shfl_sync(0xffffffffu, total, 0);
    } else {
        total = *p.tiles;
    }
    total = kb0 < kb1 ? total * cols : 0;
    const int item0 = int(blockIdx.x) / cluster, items = int(gridDim.x) / cluster;
    // by a whole warp, whose lanes give up together
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) ||
                                           mbar_wait_bounded(bar, parity, abort, clock64() + PG_TIMEOUT_CYCLES));
    };
    // for warps that may be late: between polls they leave the issue slots to
    // the decoding warps
    auto lazy_wait = [&](uint32_t bar, uint32_t parity, uint32_t ns) {
        return mbar_try_wait(bar, parity) ||
               mbar_wait_backoff(bar, parity, abort, clock64() + PG_TIMEOUT_CYCLES, ns);
    };

    if (warp == 0) {
        // ---------------------------------------------------------- loads
        // One lane; where rows are gathered, all of them.
        if (lane == 0 || (!FOUR && DIRECT)) {
            // x was written by an ordinary kernel
            asm volatile("fence.proxy.async.global;\n" ::: "memory");
            TcPos pos;
            int issued = 0;
            bool ok = true, here = !early;
            // x of the first stages, whose weights were asked for before it was there
            [[maybe_unused]] auto first_x = [&] {
                pdl_wait();
                asm volatile("fence.proxy.async.global;\n" ::: "memory");
                const int none[4] = {};
                int n = 0;
                for (int i = item0; n < issued; i += items) {
                    const int row = stream_item<FROM, NT>(p, tab, i, cols).row;
                    for (int kb = kb0; kb < kb1 && n < issued; ++kb, ++n)
                        load_x<DIRECT, 1>(g, stage_at(n) + ST_TILE, 0, kb * 64, row, none, full + 8 * n);
                }
            };
            for (int i = item0; ok && i < total; i += items) {
                const StreamItem it = stream_item<FROM, NT>(p, tab, i, cols);
                int rows[4];
                if (!FOUR && DIRECT) gathered_rows(p, it, rows);
                const uint32_t bytes = FOUR ? ST_TILE + (g.boxed ? ST_SCALES : 0) : ST_TILE + (DIRECT ? uint32_t((it.valid + 3) / 4) * 512 : Z::X);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if constexpr (!FOUR && early) {
                        if (!here && issued == g.stages) {
                            first_x();
                            here = true;
                        }
                    }
                    ok = lazy_wait(empty + 8 * pos.stage, pos.phase ^ 1u, 40);
                    if (!FOUR && DIRECT) ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t at = stage_at(pos.stage), bar = full + 8 * pos.stage;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, bytes);
                        tma_load_3d(at, &g.w, kb * (FOUR ? 128 : 64), it.n0, it.expert, bar);
                        if (FOUR && g.boxed) tma_load_3d(at + ST_TILE, &g.s, (kb & ~1) * 8, it.n0, it.expert, bar);
                    }
                    if constexpr (!FOUR) {
                        if (DIRECT) __syncwarp();
                        if (!early || here) load_x<DIRECT, 1>(g, at + ST_TILE, 0, kb * 64, it.row, rows, bar);
                    }
                    pos.next(g.stages);
                    ++issued;
                }
            }
            if constexpr (!FOUR && early) {
                if (!here) first_x();
            }
            if (lane == 0) drain_ring(full, empty, g.stages, issued, abort);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- UMMAs
        // The whole warp walks the items and one lane issues, so that what
        // the products are addressed by is in uniform registers: from a
        // branch of one lane a product takes 75 clocks to issue.
        TcPos pos, dec;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        const bool leader = elect_one();
        for (int i = item0; ok && i < total; i += items) {
            const StreamItem it = stream_item<FROM, NT>(p, tab, i, cols);
            const uint32_t idesc = __shfl_sync(0xffffffffu, umma_idesc_bf16(ST_ROWS, (it.valid + 15) & ~15), 0);
            if (!wait(acce + 8 * acc, acc_phase ^ 1u)) break;
            tc_fence_after();
            const uint32_t d = tmem + uint32_t(acc * NT);
            for (int kb = kb0; ok && kb < kb1; ++kb) {
                if constexpr (FOUR) {
                    if (!wait(decf + 8 * dec.stage, dec.phase) || !wait(xfull + 8 * pos.stage, pos.phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = tmem + uint32_t(Z::DECODED + dec.stage * 128);
                    if (leader) {
                        const uint32_t at = x_at + pos.stage * Z::X;
#pragma unroll
                        for (int j = 0; j < Z::PANELS; ++j)
                            if (kb * Z::KC + j * 64 < p.K)
                                umma_k64_tmem_a(d, a + j * 32, at + j * NT * 128, idesc, kb != kb0 || j != 0);
                        umma_commit(xempty + 8 * pos.stage);
                        umma_commit(dece + 8 * dec.stage);
                    }
                    __syncwarp();
                    pos.next(Z::XS);
                    dec.next(Z::BUFS);
                } else {
                    if (!wait(full + 8 * pos.stage, pos.phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (leader) {
                        const uint32_t at = stage_at(pos.stage);
                        umma_k64_smem(d, at, at + ST_TILE, idesc, kb != kb0);
                        umma_commit(empty + 8 * pos.stage);
                    }
                    __syncwarp();
                    pos.next(g.stages);
                }
            }
            if (!ok) break;
            if (leader) umma_commit(accf + 8 * acc);
            __syncwarp();
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (leader && *abort) {                   // nothing in flight when TMEM is released
            umma_commit(drain);
            const long long dd = clock64() + PG_TIMEOUT_CYCLES;
            while (!mbar_try_wait(drain, 0) && clock64() < dd) {
            }
        }
        __syncwarp();
    } else if (warp < ST_DEC0) {
        // ------------------------------------------------------- epilogue
        const int q = warp & 3;                   // TMEM lane quarter of this warp
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int i = item0; i < total; i += items) {
            const StreamItem it = stream_item<FROM, NT>(p, tab, i, cols);
            if (!__all_sync(0xffffffffu, lazy_wait(accf + 8 * acc, acc_phase, 200))) break;
            tc_fence_after();
            const int n = it.n0 + q * 32 + lane;
            const uint32_t t = tmem + uint32_t(acc * NT) + (uint32_t(q * 32) << 16);
            const uint32_t mine = sums + uint32_t(q * 32 + lane) * 4;
            if (rank != 0) {
                const uint32_t to = cluster_map(mine, 0) + (rank - 1) * Z::SUMS;
                for (int c = 0; c < it.valid; c += 16) {
                    uint32_t v[16];
                    tmem_ld16_nowait(t + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        asm volatile("st.shared::cluster.b32 [%0], %1;\n" :: "r"(to + (c + j) * (ST_ROWS * 4)), "r"(v[j])
                                     : "memory");
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_map(peers, 0));
                continue;                         // a cluster has one tile at most (run_stream)
            }
            if (parts > 1) {
                if (!__all_sync(0xffffffffu, mbar_try_wait_cluster(peers, 0) ||
                                             mbar_wait_bounded_cluster(peers, 0, abort, clock64() + PG_TIMEOUT_CYCLES)))
                    break;
            }
            for (int c = 0; c < it.valid; c += 16) {
                uint32_t v[16];
                tmem_ld16_nowait(t + c, v);
                int row = -1;
                if (lane < 16 && c + lane < it.valid)
                    row = expert_row(p, it.start + c + lane);
                tmem_wait_ld();
                float old[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int r = __shfl_sync(0xffffffffu, row, j);
                    old[j] = p.add && r >= 0 && n < p.N ? bf16_to_f32(p.y[int64_t(r) * p.y_ld + n]) : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int r = __shfl_sync(0xffffffffu, row, j);
                    float s = __uint_as_float(v[j]);
                    for (int k = 1; k < parts; ++k) {
                        float more;
                        asm volatile("ld.shared.f32 %0, [%1];\n"
                                     : "=f"(more) : "r"(mine + (k - 1) * Z::SUMS + (c + j) * (ST_ROWS * 4)));
                        s += more;
                    }
                    if (p.add) s += old[j];
                    if (r >= 0 && n < p.N)
                        p.y[int64_t(r) * p.y_ld + n] = uint16_t(pack_bf16x2(s, 0.0f) & 0xFFFFu);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce + 8 * acc);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    } else if constexpr (FOUR) {
        if (warp == ST_SCALE_WARP) {
            // ---------------------------------------------------- scales
            TcPos pos;
            bool ok = !g.boxed;
            for (int i = item0; ok && i < total; i += items) {
                const StreamItem it = stream_item<FROM, NT>(p, tab, i, cols);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = __all_sync(0xffffffffu, lazy_wait(empty + 8 * pos.stage, pos.phase ^ 1u, 40));
                    if (!ok) break;
                    const uint32_t to = stage_at(pos.stage) + ST_TILE;
#pragma unroll
                    for (int r = lane; r < ST_ROWS; r += 32) fetch_scales(p, to + r * 16, it.expert, it.n0 + r, kb);
                    // stores before the arrival, which follows when the copies have landed
                    __threadfence_block();
                    cp_async_mbar_arrive_noinc(full + 8 * pos.stage);
                    pos.next(g.stages);
                }
            }
            cp_async_commit();
            cp_async_wait<0>();
        } else if (warp == ST_X_WARP) {
            // --------------------------------------------------------- x
            if (lane == 0 || DIRECT) {
                if (early) pdl_wait();
                asm volatile("fence.proxy.async.global;\n" ::: "memory");      // written by an ordinary kernel
                TcPos pos;
                int issued = 0;
                bool ok = true;
                for (int i = item0; ok && i < total; i += items) {
                    const StreamItem it = stream_item<FROM, NT>(p, tab, i, cols);
                    int rows[4];
                    if (DIRECT) gathered_rows(p, it, rows);
                    const uint32_t gathered = uint32_t((it.valid + 3) / 4) * 512;
                    for (int kb = kb0; kb < kb1; ++kb) {
                        const int k = kb * Z::KC;
                        const uint32_t bytes =
                            DIRECT ? gathered * uint32_t(min(Z::PANELS, (p.K - k + 63) / 64)) : uint32_t(Z::X);
                        ok = lazy_wait(xempty + 8 * pos.stage, pos.phase ^ 1u, 40);
                        if (DIRECT) ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        const uint32_t bar = xfull + 8 * pos.stage;
                        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                        if (DIRECT) __syncwarp();
                        load_x<DIRECT, Z::PANELS>(g, x_at + pos.stage * Z::X, NT * 128, k, it.row, rows, bar);
                        pos.next(Z::XS);
                        ++issued;
                    }
                }
                if (lane == 0) drain_ring(xfull, xempty, Z::XS, issued, abort);
            }
            __syncwarp();
        } else {
            // -------------------------------------------------- decoding
            // Two sets of four warps share a stage, the other two the next
            // one; a set has two of its four blocks of 64.
            const int set = (warp - ST_DEC0) >> 2, q = warp & 3, row = q * 32 + lane;
            const int half = set & 1;
            const uint32_t mine = smem_addr(table) + lane * 4;
            const uint32_t chunk = uint32_t(row * 128 + ((4 * half ^ row) & 7) * 16);      // chunk c of the half: ^ 16 c
            const uint32_t scale = ST_TILE + uint32_t(row * 16);
            const uint32_t tcol = tmem + uint32_t(Z::DECODED + half * 64) + (uint32_t(q * 32) << 16);
            // all stages of all tiles in one run: this warp's are every other
            // one, from its set's first
            const int tiles = total > item0 ? (total - item0 + items - 1) / items : 0;
            int left = tiles * (kb1 - kb0) - (set >> 1);
            int kb = kb0 + (set >> 1);            // its scales are half of a box
            int stage = set >> 1, buf = set >> 1;
            uint32_t phase = 0, buf_phase = 1;
            for (; left > 0; left -= 2) {
                const uint32_t bar = full + 8 * stage;
                while (kb >= kb1) kb -= kb1 - kb0;
                if (!__all_sync(0xffffffffu, mbar_try_wait(bar, phase)) &&
                    !__all_sync(0xffffffffu, lazy_wait(bar, phase, 20)))
                    break;
                const uint32_t at = stage_at(stage);
                uint32_t sc;
                if (g.boxed) {
                    asm volatile("ld.shared.b32 %0, [%1];\n"
                                 : "=r"(sc) : "r"(at + scale + (kb & 1) * 8 + half * 4) : "memory");
                } else {
                    uint32_t a, b, c, first;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                                 : "=r"(a), "=r"(b), "=r"(c), "=r"(first) : "r"(at + scale) : "memory");
                    sc = __funnelshift_r(half ? b : a, half ? c : b, 8 * first);
                }
                uint4 w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                                 : "=r"(w[c].x), "=r"(w[c].y), "=r"(w[c].z), "=r"(w[c].w)
                                 : "r"(at + (chunk ^ uint32_t(16 * c))) : "memory");
                if (!__all_sync(0xffffffffu, mbar_try_wait(dece + 8 * buf, buf_phase)) &&
                    !__all_sync(0xffffffffu, lazy_wait(dece + 8 * buf, buf_phase, 20)))
                    break;
                tc_fence_after();
                const uint32_t to = tcol + uint32_t(buf * 128);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[16];
                    decode_block(mine, w[c], sc >> (8 * c) & 255u, o);
                    tmem_st<16>(to + 16 * c, o);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                // the stage is given back only now: nothing orders an arrival
                // behind loads whose values have not been used
                if (lane == 0) {
                    mbar_arrive(decf + 8 * buf);
                    mbar_arrive(empty + 8 * stage);
                }
                kb += 2;
                stage += 2;
                if (stage >= g.stages) {
                    stage -= g.stages;
                    phase ^= 1u;
                }
                buf += 2;
                if (buf >= Z::BUFS) {
                    buf -= Z::BUFS;
                    buf_phase ^= 1u;
                }
            }
        }
    }

    // not over before the copy: what waits for this kernel may write there
    if (early) pdl_wait();
    tc_fence_before();
    if (cluster > 1) cluster_sync_all();          // nobody writes to a CTA that is gone
    else __syncthreads();
    tc_fence_after();
    if (tid == 0 && *abort && p.error_word != nullptr) atomicOr(p.error_word, LORA_TIMEOUT_BIT);
    if (warp == 1) tmem_dealloc(tmem, Z::COLS);
}

// ---------------------------------------------------------------- host

template <bool FOUR, int NT, int FROM>
static int run_stream(StreamArgs &g, cudaStream_t st)
{
    using Z = StreamSizes<FOUR, NT>;
    static std::atomic<uint64_t> done{0};
    const auto kernel = expert_stream_kernel<FOUR, NT, FROM>;
    if (int e = expert_shared_memory((const void *)kernel, Z::ALL, done)) return e;
    // Tiles at most: an expert may end in one that is not full.  The segments
    // are those of the call's rows (load_segments: clamp), so a cluster that
    // shares a tile has one, and its barriers' first phases are all it needs.
    // Up to half the SMs, two CTAs share each, up to a quarter four (us with
    // one, two and four, in a graph: 64 tiles of 4096 x 4096 for one token in
    // bf16 30.3, 28.8, 29.8, in 4 bits 24.6, 23.6, 23.0; 32 tiles, 16 rows: 35.3,
    // 26.2, 22.5 and 29.0, 28.9, 28.5).
    const int64_t rows = g.p.R, experts = rows < g.p.E ? rows : g.p.E;
    const int64_t most = (rows / NT + experts) * ((g.p.N + ST_ROWS - 1) / ST_ROWS), sms = device_sm_count();
    int parts = most * 4 <= sms ? 4 : most * 2 <= sms ? 2 : 1;
    while (parts > 1 && Z::ring(parts) < Z::LEAST) parts /= 2;
    g.stages = Z::ring(parts);
    if (parts == 1)
        return int(launch_kernel(kernel, dim3(unsigned(sms)), dim3(Z::THREADS), Z::ALL, st, g));
    return int(launch_clusters(kernel, parts, int(most), st, g, Z::THREADS, Z::ALL));
}

// Weights are asked for while x is copied, where they are few: this saves a
// part of the copy's time, and costs a walk of the segments for every tile
// (us in a graph, after the copy and beside it: 4 bits, 128 rows of 16 experts
// 4096 x 4096, 143 MB: 57 and 52; 32 rows of one of 8192 x 8192: 40 and 37; bf16, 32
// rows of one of 4096 x 4096: 29.5 and 27.6; 128 rows of 8, 268 MB: 71.5 and 69.8; of
// 16, 537 MB: 117 and 118; 4 bits, 767 MB: 171 and 175).
bool expert_stream_early(const ExpertArgs &p)
{
    const int64_t experts = p.R < p.E ? p.R : p.E, row = p.scales != nullptr ? p.K / 2 + p.K / 32 : 2 * p.K;
    return p.nbins <= ST_BINS && experts * p.N * row <= int64_t(256) << 20;
}

bool expert_stream_gathers(const ExpertArgs &p)
{
    // Gathers of a stage, 90 clocks each, in the time of its 16 KB of W (about
    // 740; 1100 with the decoding of four panels' codes).  Measured with a
    // copy and with gathers (us, experts of 4096 x 4096, in a graph): bf16, two
    // rows of 8 experts 33.7 and 28.9, 24 rows of one expert 31 and 25, 32 rows
    // 31 and 32 (width 11008: 40 and 44); 4 bits, two rows 29 and 23, 12 rows
    // of one expert 27 and 21, 64 rows of 16 experts 60 and 62.
    return p.x_vec && p.nbins <= ST_BINS && p.R <= (p.scales != nullptr ? 12 : 24);
}

int launch_expert_stream(const ExpertArgs &p, cudaStream_t st)
{
    StreamArgs g;
    g.p = p;
    const bool four = p.scales != nullptr, direct = expert_stream_gathers(p);
    // Boxes of 16 bytes on rows of whole ones; else 32 lanes fetch eight bytes
    // a row, whose writes to shared memory are in the way of the decoding's
    // table (128 rows of 32 experts, 4096 to 11008, in a graph:
    // 184 us, boxed 176).
    g.boxed = four && p.K % 512 == 0;
    if (g.boxed && !encode_stack_map_u8(&g.s, p.scales, uint64_t(p.E), uint64_t(p.N), uint64_t(p.K / 32), 16, ST_ROWS))
        return LORA_ERR_DEVICE;
    if (!(direct ? encode_tile_map(&g.x, p.x, uint64_t(p.R / p.fan), uint64_t(p.K), uint64_t(p.x_ld), 64, 1,
                                   CU_TENSOR_MAP_SWIZZLE_128B)
                 : encode_tile_map(&g.x, p.xs, uint64_t(p.rows), uint64_t(p.K), uint64_t(p.K), 64, uint32_t(p.tile_rows),
                                   CU_TENSOR_MAP_SWIZZLE_128B)) ||
        !(four ? encode_stack_map_u8(&g.w, p.codes, uint64_t(p.E), uint64_t(p.N), uint64_t(p.K / 2), 128, ST_ROWS)
               : encode_stack_map(&g.w, p.w, uint64_t(p.E), uint64_t(p.N), uint64_t(p.K), 64, ST_ROWS)))
        return LORA_ERR_DEVICE;
    // tiles are of 16 rows (4 bits) or 32 where rows are gathered
    if (direct) return four ? run_stream<true, 16, ST_GATHER>(g, st) : run_stream<false, 32, ST_GATHER>(g, st);
    if (four && p.tile_rows == 16)
        return p.early ? run_stream<true, 16, ST_EARLY>(g, st) : run_stream<true, 16, ST_COPY>(g, st);
    if (four) return p.early ? run_stream<true, 64, ST_EARLY>(g, st) : run_stream<true, 64, ST_COPY>(g, st);
    return p.early ? run_stream<false, 32, ST_EARLY>(g, st) : run_stream<false, 32, ST_COPY>(g, st);
}

}  // namespace lora
