// lora_ortho_tc.cu -- lora_orthogonalize for ranks 65 to 128 on tcgen05; see
// lora_ortho.cu for the mathematics.  Short sides are padded to 128 by the
// loads (zeros).
//
// gram_tc_kernel   U U^T: both operands of a UMMA are the same tile.
// iterate_tc_kernel  the steps on 128 x 128 matrices.  An fp32 value is a sum
//     of three bf16 terms (24 bits), a product the six pairs of terms down
//     to 2^-16.  (Two terms in the later steps would save 20 of the about
//     110 us at 192 matrices; a matrix of rank one then comes out 1% off.)
//     A UMMA contracts rows with rows, X Y^T, so symmetric matrices need no
//     transposing; the products are ordered so that R stays symmetric: Q R
//     Q^T.  As (R Q^T) Q^T its rounding errors do not commute with R and
//     grow sixfold a step.
// apply_tc_kernel  P U with P as two bf16 terms.
//
// fp32 entries of U are split into two bf16 terms by four warps on the way
// to shared memory; bf16 tiles come by TMA.
#include <math.h>

#include "lora_ortho.cuh"
#include "lora_tc.cuh"

namespace lora {

constexpr int OT_R = 128;
constexpr int OT_PANEL = OT_R * 128;             // 128 rows of 64 bf16, 16 KB
constexpr int OT_GRAM_RING = 80 * 1024;          // two CTAs an SM
constexpr int OT_GRAM_SMEM = OT_GRAM_RING + TC_STAGE_ROWS + TC_BAR_BYTES + 1024;
constexpr int OT_APPLY_RING = 128 * 1024;
constexpr int OT_APPLY_SMEM = OT_APPLY_RING + 4 * OT_PANEL + TC_STAGE_ROWS + TC_BAR_BYTES + 1024;
constexpr int OT_ITER_THREADS = 256;
constexpr int OT_TERM = 2 * OT_PANEL;            // one bf16 term of a matrix
constexpr int OT_ITER_SMEM = 6 * OT_TERM + 64 + 1024;

struct OrthoTcArgs {
    OrthoArgs o;
    CUtensorMap u;        // U in boxes of 64 columns x 128 rows (bf16 only)
    CUtensorMap u64;      // a tall U in boxes of 64 columns x 64 rows
    CUtensorMap p;        // [count * 2 * 128][128]: P's terms, boxes 64 x 128
};

// A thread's share of a tile of fp32 entries: chunks of eight, as two bf16
// terms into the swizzled panels at dst (second term `lo` bytes behind).
template <int ROWS, int CPR, int THREADS>
struct Converter {
    static constexpr int PER = ROWS * CPR / THREADS;
    Chunk<true> c[PER];
    __device__ __forceinline__ void fetch(const OrthoArgs &p, int m, int row0, int col0, int thread)
    {
        const int64_t mat = int64_t(m) * p.rows * p.cols;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int k = thread + i * THREADS, row = row0 + k / CPR, col = col0 + k % CPR * 8;
            c[i] = load_chunk<true>(p.u, mat + int64_t(row) * p.cols + col, row < p.rows && col < p.cols);
        }
    }
    __device__ __forceinline__ void put(uint8_t *dst, int lo, int thread) const
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int k = thread + i * THREADS;
            uint8_t *at = dst + tile_at<CPR, ROWS>(k / CPR, k % CPR);
            *reinterpret_cast<uint4 *>(at) = c[i].hi;
            *reinterpret_cast<uint4 *>(at + lo) = c[i].lo;
        }
    }
};

// ---------------------------------------------------------------- gram

// A CTA's run of units (64 of the long side each): one accumulator a matrix.
template <bool TALL, bool F32>
__global__ void __launch_bounds__(TC_THREADS, 2) gram_tc_kernel(const __grid_constant__ OrthoTcArgs q)
{
    constexpr int STAGE = OT_PANEL * (F32 ? 2 : 1), STAGES = OT_GRAM_RING / STAGE;
    constexpr int ROWS = TALL ? 64 : OT_R, CPR = TALL ? 16 : 8;
    constexpr uint32_t IDESC = umma_idesc_bf16(OT_R, OT_R) | (TALL ? (1u << 15) | (1u << 16) : 0u);
    const OrthoArgs &p = q.o;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const TcRing ring = tc_setup<256>(smem, OT_GRAM_RING, STAGE, STAGES, F32 ? 4 : 1);
    pdl_wait();
    pdl_launch_dependents();
    const int64_t first = unit_begin(p, blockIdx.x), end = unit_begin(p, blockIdx.x + 1);

    if (warp == 0 && !F32) {
        if (lane == 0) {
            TcPos pos;
            int issued = 0;
            for (int64_t u = first; u < end; ++u) {
                if (!pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort)) break;
                const uint32_t full = ring.full + 8 * pos.stage, at = ring.ring + pos.stage * STAGE;
                const int m = int(u / p.units), k = int(u % p.units) * OR_TC_UNIT;
                mbar_arrive_expect_tx(full, OT_PANEL);
                if constexpr (TALL) {
                    tma_load_3d(at, &q.u64, 0, k, m, full);
                    tma_load_3d(at + OT_PANEL / 2, &q.u64, 64, k, m, full);
                } else {
                    tma_load_3d(at, &q.u, k, 0, m, full);
                }
                ++issued;
                pos.next(STAGES);
            }
            tc_drain_loads(ring, issued);
        }
    } else if (warp == 2) {
        if (lane == 0) {
            TcPos pos;
            int buf = 0;
            uint32_t bphase = 0;
            bool start = true;
            for (int64_t u = first; u < end; ++u) {
                if (start && !pg_wait(ring.acce + 8 * buf, bphase ^ 1u, ring.abort)) break;
                if (!pg_wait(ring.full + 8 * pos.stage, pos.phase, ring.abort)) break;
                tc_fence_after();
                const uint32_t d = ring.tmem + uint32_t(buf * OT_R), t = ring.ring + pos.stage * STAGE;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t hi = TALL ? umma_desc_mn(t + kk * 2048) : umma_desc_sw128(t + kk * 32);
                    if constexpr (F32) {
                        const uint32_t tl = t + OT_PANEL;
                        const uint64_t lo = TALL ? umma_desc_mn(tl + kk * 2048) : umma_desc_sw128(tl + kk * 32);
                        umma_bf16(d, hi, lo, IDESC, !start || kk != 0);
                        umma_bf16(d, lo, hi, IDESC, 1);
                        umma_bf16(d, hi, hi, IDESC, 1);
                    } else {
                        umma_bf16(d, hi, hi, IDESC, !start || kk != 0);
                    }
                }
                umma_commit(ring.empty + 8 * pos.stage);
                pos.next(STAGES);
                start = u + 1 == end || (u + 1) % p.units == 0;
                if (start) {
                    umma_commit(ring.accf + 8 * buf);
                    buf ^= 1;
                    if (buf == 0) bphase ^= 1u;
                }
            }
        }
    } else if (warp >= 4) {
        const int row = (warp - 4) * 32 + lane;
        TcPos pos;
        int buf = 0;
        uint32_t bphase = 0;
        Converter<ROWS, CPR, 128> conv;
        auto fetch = [&](int64_t u) {
            const int k = int(u % p.units) * OR_TC_UNIT;
            conv.fetch(p, int(u / p.units), TALL ? k : 0, TALL ? 0 : k, row);
        };
        if (F32 && first < end) fetch(first);
        bool ok = true;
        for (int64_t u = first; ok && u < end; ++u) {
            if constexpr (F32) {
                const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
                if (__all_sync(0xffffffffu, got) == 0) break;
                conv.put(smem + pos.stage * STAGE, OT_PANEL, row);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(ring.full + 8 * pos.stage);
                if (u + 1 < end) fetch(u + 1);
                pos.next(STAGES);
            }
            if (u + 1 < end && (u + 1) % p.units != 0) continue;
            const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
            ok = __all_sync(0xffffffffu, got) != 0;
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = ring.tmem + uint32_t(buf * OT_R) + (uint32_t((warp - 4) * 32) << 16);
            float *out = p.gram + ((blockIdx.x + u / p.units) * OT_R + row) * OT_R;
            for (int c = 0; c < OT_R; c += 32) {
                uint32_t v[32];
                tmem_ld32_nowait(d + uint32_t(c), v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4 *>(out + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.acce + 8 * buf);
            buf ^= 1;
            if (buf == 0) bphase ^= 1u;
        }
        // the last commits have arrived before the CTA exits
        if (F32 && lane == 0 && warp == 4) {
            const long long dd = clock64() + PG_TIMEOUT_CYCLES;
            const int issued = int(end - first);
            for (int i = max(0, issued - STAGES); ok && i < issued; ++i)
                while (!mbar_try_wait(ring.empty + 8 * (i % STAGES), uint32_t(i / STAGES) & 1u) &&
                       !*ring.abort && clock64() < dd) {
                }
        }
    }
    tc_finish<256>(ring, p.error_word);
}

// ---------------------------------------------------------------- iterate

// D[128 x 128] = X Y^T for operands of three bf16 terms in shared memory (X
// also in TMEM: columns of 64 words a term), by pairs of terms (i, j) with
// i + j <= 2, the small ones first.
template <bool X_TMEM>
__device__ __forceinline__ void mul_terms(uint32_t d, uint32_t x, uint32_t y)
{
    constexpr uint32_t IDESC = umma_idesc_bf16(OT_R, OT_R);
    uint32_t acc = 0;
    for (int sum = 2; sum >= 0; --sum)
        for (int i = 0; i <= sum; ++i) {
            const uint32_t xt = x + uint32_t(i) * (X_TMEM ? 64u : uint32_t(OT_TERM));
            const uint32_t yt = y + uint32_t(sum - i) * uint32_t(OT_TERM);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint32_t off = uint32_t((kk >> 2) * OT_PANEL + (kk & 3) * 32);
                if constexpr (X_TMEM)
                    umma_bf16_tmem_a(d, xt + uint32_t(kk * 8), umma_desc_sw128(yt + off), IDESC, acc);
                else
                    umma_bf16(d, umma_desc_sw128(xt + off), umma_desc_sw128(yt + off), IDESC, acc);
                acc = 1;
            }
        }
}

// Eight values as three terms of bf16 (four words each).
__device__ __forceinline__ void split8(const float *v, uint32_t (&t0)[4], uint32_t (&t1)[4], uint32_t (&t2)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = v[2 * j], b = v[2 * j + 1];
        t0[j] = pack_bf16x2(a, b);
        a -= bf16_lo(t0[j]);
        b -= bf16_hi(t0[j]);
        t1[j] = pack_bf16x2(a, b);
        t2[j] = pack_bf16x2(a - bf16_lo(t1[j]), b - bf16_hi(t1[j]));
    }
}

// One matrix a CTA.  Thread (warp w, lane) holds row 32 (w % 4) + lane,
// columns 64 (w / 4) to + 63: R in registers.  Shared memory: R (then S = Q
// R, then R again) and Q as three terms; TMEM: two accumulators and P's
// terms.  A step: R^2 -> Q; then P Q and Q R together; then (Q R) Q.
__global__ void __launch_bounds__(OT_ITER_THREADS, 1) iterate_tc_kernel(const OrthoArgs p)
{
    uint8_t *smem = tc_smem();
    const uint32_t sr = smem_addr(smem), sq = sr + 3 * OT_TERM, bar = sq + 3 * OT_TERM;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + 6 * OT_TERM + 8);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + 6 * OT_TERM + 12);
    float *s_trace = reinterpret_cast<float *>(smem + 6 * OT_TERM + 16);      // a warp's each
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, m = blockIdx.x;
    const int quarter = warp & 3, half = warp >> 2;
    const int row = quarter * 32 + lane, col0 = half * 64;
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_fence_init();
        *s_abort = 0;
    }
    if (warp == 0) tmem_alloc(smem_addr(s_tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem, lanes = uint32_t(quarter * 32) << 16;
    const uint32_t d0 = tmem, d1 = tmem + 128, tp = tmem + 256;
    pdl_wait();
    pdl_launch_dependents();

    float rv[64];                                     // this thread's part of R
    {
        const int lo = unit_cta(p, int64_t(m) * p.units), hi = unit_cta(p, int64_t(m + 1) * p.units - 1);
#pragma unroll
        for (int j = 0; j < 64; ++j) rv[j] = 0.0f;
        for (int c = lo; c <= hi; ++c) {
            const float4 *src = reinterpret_cast<const float4 *>(
                p.gram + (int64_t(c + m) * OT_R + row) * OT_R + col0);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float4 x = src[j];
                rv[4 * j] += x.x;
                rv[4 * j + 1] += x.y;
                rv[4 * j + 2] += x.z;
                rv[4 * j + 3] += x.w;
            }
        }
    }
    float trace = 0.0f;
#pragma unroll
    for (int j = 0; j < 64; ++j) trace += col0 + j == row ? rv[j] : 0.0f;
    for (int o = 16; o > 0; o >>= 1) trace += __shfl_xor_sync(0xffffffffu, trace, o);
    if (lane == 0) s_trace[warp] = trace;
    __syncthreads();
    trace = 0.0f;
    for (int w = 0; w < 8; ++w) trace += s_trace[w];
    const float f = 1.0f / (sqrtf(trace) + p.eps);
#pragma unroll
    for (int j = 0; j < 64; ++j) rv[j] = rv[j] * f * f;

    // eight values of this thread's row from column col0 + 8 c, as terms
    auto to_smem = [&](uint8_t *at, const float *v, int c) {
        uint32_t t0[4], t1[4], t2[4];
        split8(v, t0, t1, t2);
        uint8_t *dst = at + half * OT_PANEL + row * 128 + ((c ^ row) & 7) * 16;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
        *reinterpret_cast<uint4 *>(dst + OT_TERM) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
        *reinterpret_cast<uint4 *>(dst + 2 * OT_TERM) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
    };
    auto p_to_tmem = [&](const float *v, int c) {
        uint32_t t0[4], t1[4], t2[4];
        split8(v, t0, t1, t2);
        const uint32_t at = tp + lanes + uint32_t(half * 32 + c * 4);
        tmem_st<4>(at, t0);
        tmem_st<4>(at + 64, t1);
        tmem_st<4>(at + 128, t2);
    };
    uint16_t *out = p.p + int64_t(m) * 2 * OT_R * OT_R + row * OT_R + col0;
    auto p_out = [&](const float *v, int c) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = v[2 * j] * f * p.scale, b = v[2 * j + 1] * f * p.scale;
            h[j] = pack_bf16x2(a, b);
            l[j] = pack_bf16x2(a - bf16_lo(h[j]), b - bf16_hi(h[j]));
        }
        *reinterpret_cast<uint4 *>(out + 8 * c) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(out + OT_R * OT_R + 8 * c) = make_uint4(l[0], l[1], l[2], l[3]);
    };
    // Every thread's writes of operands are done before, and the UMMAs that
    // `issue` starts are done after (false: the wait ran out).
    uint32_t phase = 0;
    auto products = [&](auto issue) {
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            issue();
            umma_commit(bar);
        }
        __syncwarp();
        const bool got = pg_wait(bar, phase, s_abort);
        phase ^= 1u;
        tc_fence_after();
        return __syncthreads_and(int(got)) != 0;
    };
    auto load32 = [&](uint32_t d, int c, float *v) {
        uint32_t w[32];
        tmem_ld32_nowait(d + lanes + uint32_t(col0 + c), w);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]);
    };

#pragma unroll
    for (int c = 0; c < 8; ++c) to_smem(smem, rv + 8 * c, c);
    for (int step = 0; step < p.steps; ++step) {
        const bool last = step + 1 == p.steps;
        if (!products([&] { mul_terms<false>(d0, sr, sr); })) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[32];
            load32(d0, 32 * h, v);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] = fmaf(p.c, v[j], fmaf(p.b, rv[32 * h + j], col0 + 32 * h + j == row ? p.a : 0.0f));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (!last || step > 0) to_smem(smem + 3 * OT_TERM, v + 8 * c, 4 * h + c);
                if (step == 0) {                       // P was the identity
                    if (last) p_out(v + 8 * c, 4 * h + c);
                    else p_to_tmem(v + 8 * c, 4 * h + c);
                }
            }
        }
        if (step == 0 && last) break;
        if (!products([&] {
                if (step > 0) mul_terms<true>(d0, tp, sq);
                if (!last) mul_terms<false>(d1, sq, sr);
            }))
            break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[32];
            if (step > 0) {
                load32(d0, 32 * h, v);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (last) p_out(v + 8 * c, 4 * h + c);
                    else p_to_tmem(v + 8 * c, 4 * h + c);
                }
            }
            if (!last) {
                load32(d1, 32 * h, v);
#pragma unroll
                for (int c = 0; c < 4; ++c) to_smem(smem, v + 8 * c, 4 * h + c);
            }
        }
        if (last) break;
        if (!products([&] { mul_terms<false>(d1, sr, sq); })) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            load32(d1, 32 * h, rv + 32 * h);
#pragma unroll
            for (int c = 0; c < 4; ++c) to_smem(smem, rv + 32 * h + 8 * c, 4 * h + c);
        }
    }
    if (*s_abort) {
        // the UMMAs of the wait that ran out: one more bounded wait for them
        if (tid == 0) {
            if (p.error_word != nullptr) atomicOr(p.error_word, LORA_TIMEOUT_BIT);
            const long long dd = clock64() + PG_TIMEOUT_CYCLES;
            while (!mbar_try_wait(bar, phase ^ 1u) && clock64() < dd) {
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- apply

// A CTA's run of tiles (128 of the long side each) of the stacked matrices;
// P's terms of the current matrix stay in shared memory.  F32: warps 8 to 11
// convert.
template <bool TALL, bool F32>
__global__ void __launch_bounds__(F32 ? TC_THREADS + 128 : TC_THREADS, 1)
apply_tc_kernel(const __grid_constant__ OrthoTcArgs q)
{
    constexpr int STAGE = 2 * OT_PANEL * (F32 ? 2 : 1), STAGES = OT_APPLY_RING / STAGE;
    constexpr uint32_t IDESC = umma_idesc_bf16(OT_R, OT_R) | (TALL ? 0u : 1u << 16);
    const OrthoArgs &p = q.o;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // ring, then P's four panels
    const TcRing ring = tc_setup<256>(smem, OT_APPLY_RING + 4 * OT_PANEL, STAGE, STAGES, F32 ? 4 : 1);
    const uint32_t sp = ring.ring + OT_APPLY_RING;
    const uint32_t p_full = ring.drain + 24, p_empty = p_full + 8;
    if (threadIdx.x == 0) {
        mbar_init(p_full, 1);
        mbar_init(p_empty, 1);
        mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const int tiles = (p.n + OT_R - 1) / OT_R;
    const int64_t total = int64_t(p.count) * tiles;
    const int64_t first = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;

    if (warp == 0) {
        if (lane == 0 && !F32) {
            TcPos pos;
            int issued = 0;
            for (int64_t i = first; i < end; ++i) {
                if (!pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort)) break;
                const uint32_t full = ring.full + 8 * pos.stage, at = ring.ring + pos.stage * STAGE;
                const int m = int(i / tiles), n0 = int(i % tiles) * OT_R;
                mbar_arrive_expect_tx(full, 2 * OT_PANEL);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    tma_load_3d(at + j * OT_PANEL, &q.u, TALL ? 64 * j : n0 + 64 * j, TALL ? n0 : 0, m, full);
                ++issued;
                pos.next(STAGES);
            }
            tc_drain_loads(ring, issued);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // P was written by the stream's previous kernel with ordinary stores
            asm volatile("fence.proxy.async.global;\n" ::: "memory");
            int held = -1;
            uint32_t phase = 0;
            for (int64_t i = first; i < end; ++i) {
                const int m = int(i / tiles);
                if (m == held) continue;
                if (!pg_wait(p_empty, phase ^ 1u, ring.abort)) break;
                mbar_arrive_expect_tx(p_full, 4 * OT_PANEL);
                for (int k = 0; k < 4; ++k)
                    tma_load_2d(sp + k * OT_PANEL, &q.p, (k & 1) * 64, (2 * m + (k >> 1)) * OT_R, p_full);
                phase ^= 1u;
                held = m;
            }
            if (held >= 0) {
                const long long dd = clock64() + PG_TIMEOUT_CYCLES;
                while (!mbar_try_wait(p_full, phase ^ 1u) && clock64() < dd) {
                }
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            TcPos pos;
            int buf = 0, held = -1;
            uint32_t bphase = 0, pphase = 0;
            for (int64_t i = first; i < end; ++i) {
                if (!pg_wait(ring.acce + 8 * buf, bphase ^ 1u, ring.abort)) break;
                const int m = int(i / tiles);
                if (m != held) {
                    if (!pg_wait(p_full, pphase, ring.abort)) break;
                    pphase ^= 1u;
                    held = m;
                }
                if (!pg_wait(ring.full + 8 * pos.stage, pos.phase, ring.abort)) break;
                tc_fence_after();
                const uint32_t d = ring.tmem + uint32_t(buf * OT_R), t = ring.ring + pos.stage * STAGE;
                uint32_t acc = 0;
                auto product = [&](uint32_t pt, uint32_t ut) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = uint32_t((kk >> 2) * OT_PANEL + (kk & 3) * 32);
                        if constexpr (TALL)
                            umma_bf16(d, umma_desc_sw128(ut + off), umma_desc_sw128(pt + off), IDESC, acc);
                        else
                            umma_bf16(d, umma_desc_sw128(pt + off), umma_desc_mn(ut + kk * 2048, OT_PANEL), IDESC, acc);
                        acc = 1;
                    }
                };
                if constexpr (F32) product(sp, t + 2 * OT_PANEL);
                product(sp + 2 * OT_PANEL, t);
                product(sp, t);
                umma_commit(ring.empty + 8 * pos.stage);
                umma_commit(ring.accf + 8 * buf);
                if (i + 1 < end && int((i + 1) / tiles) != m) umma_commit(p_empty);
                pos.next(STAGES);
                buf ^= 1;
                if (buf == 0) bphase ^= 1u;
            }
        }
    } else if (warp >= 4 && warp < 8) {
        const int row = (warp - 4) * 32 + lane;
        uint8_t *stage = smem + OT_APPLY_RING + 4 * OT_PANEL + (warp - 4) * (TC_STAGE_ROWS / 4);
        int buf = 0;
        uint32_t bphase = 0;
        for (int64_t i = first; i < end; ++i) {
            const bool got = pg_wait(ring.accf + 8 * buf, bphase, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            tc_fence_after();
            const uint32_t d = ring.tmem + uint32_t(buf * OT_R) + (uint32_t((warp - 4) * 32) << 16);
            const int n0 = int(i % tiles) * OT_R;
            const int gr = TALL ? n0 + row : row, gc = TALL ? 0 : n0;
            uint16_t *dst = gr < p.rows ? p.out + (i / tiles * p.rows + gr) * p.cols + gc : nullptr;
#pragma unroll
            for (int c = 0; c < OT_R; c += 64) {
                uint32_t o[32];
                load64(d + uint32_t(c), 1.0f, o);
                store_rows(stage, o, dst != nullptr ? dst + c : nullptr, p.cols - gc - c);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.acce + 8 * buf);
            buf ^= 1;
            if (buf == 0) bphase ^= 1u;
        }
    } else if (F32 && warp >= 8) {
        const int thread = (warp - 8) * 32 + lane;
        TcPos pos;
        // half a tile at a time: 64 rows
        Converter<64, 16, 128> conv;
        auto fetch = [&](int64_t i, int h) {
            const int n0 = int(i % tiles) * OT_R;
            conv.fetch(p, int(i / tiles), (TALL ? n0 : 0) + 64 * h, TALL ? 0 : n0, thread);
        };
        auto put = [&](uint8_t *at, int h) {
#pragma unroll
            for (int k = 0; k < conv.PER; ++k) {
                const int c = thread + k * 128;
                uint8_t *to = at + tile_at<16, OT_R>(64 * h + c / 16, c % 16);
                *reinterpret_cast<uint4 *>(to) = conv.c[k].hi;
                *reinterpret_cast<uint4 *>(to + 2 * OT_PANEL) = conv.c[k].lo;
            }
        };
        int issued = 0;
        if (first < end) fetch(first, 0);
        for (int64_t i = first; i < end; ++i) {
            const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            uint8_t *at = smem + pos.stage * STAGE;
            put(at, 0);
            fetch(i, 1);
            put(at, 1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.full + 8 * pos.stage);
            if (i + 1 < end) fetch(i + 1, 0);
            ++issued;
            pos.next(STAGES);
        }
        if (thread == 0) {
            const long long dd = clock64() + PG_TIMEOUT_CYCLES;
            for (int i = max(0, issued - STAGES); i < issued; ++i)
                while (!mbar_try_wait(ring.empty + 8 * (i % STAGES), uint32_t(i / STAGES) & 1u) &&
                       !*ring.abort && clock64() < dd) {
                }
        }
    }
    tc_finish<256>(ring, p.error_word);
}

// ---------------------------------------------------------------- host

template <bool TALL, bool F32>
static int run_tc(const OrthoTcArgs &q, cudaStream_t st)
{
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    if (dev >= 64 || !configured[dev]) {
        if ((e = cudaFuncSetAttribute(gram_tc_kernel<TALL, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      OT_GRAM_SMEM)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(iterate_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      OT_ITER_SMEM)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(apply_tc_kernel<TALL, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      OT_APPLY_SMEM)) != cudaSuccess)
            return int(e);
        if (dev < 64) configured[dev] = 1;
    }
    e = launch_kernel(gram_tc_kernel<TALL, F32>, dim3(unsigned(q.o.ctas)), dim3(TC_THREADS), OT_GRAM_SMEM, st, q);
    if (e != cudaSuccess) return int(e);
    e = launch_kernel(iterate_tc_kernel, dim3(unsigned(q.o.count)), dim3(OT_ITER_THREADS), OT_ITER_SMEM, st, q.o);
    if (e != cudaSuccess) return int(e);
    const int64_t tiles = int64_t(q.o.count) * ((q.o.n + OT_R - 1) / OT_R);
    const int sms = device_sm_count();
    e = launch_kernel(apply_tc_kernel<TALL, F32>, dim3(unsigned(tiles < sms ? tiles : sms)),
                      dim3(F32 ? TC_THREADS + 128 : TC_THREADS), OT_APPLY_SMEM, st, q);
    return e == cudaSuccess ? LORA_OK : int(e);
}

int run_ortho_tc(OrthoArgs p, bool f32, cudaStream_t st)
{
    const bool tall = p.rows > p.cols;
    static thread_local OrthoTcArgs q;
    q.o = p;
    if (!encode_tile_map(&q.p, p.p, uint64_t(p.count) * 2 * OT_R, OT_R, OT_R, 64, OT_R,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return LORA_ERR_DEVICE;
    const uint64_t n = uint64_t(p.count), rows = uint64_t(p.rows), cols = uint64_t(p.cols);
    if (!f32 && (!encode_stack_map(&q.u, p.u, n, rows, cols, 64, OT_R) ||
                 !encode_stack_map(&q.u64, p.u, n, rows, cols, 64, 64)))
        return LORA_ERR_DEVICE;
    if (f32) return tall ? run_tc<true, true>(q, st) : run_tc<false, true>(q, st);
    return tall ? run_tc<true, false>(q, st) : run_tc<false, false>(q, st);
}

}  // namespace lora
