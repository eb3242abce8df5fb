// lora_ortho_tc.cu -- lora_orthogonalize for ranks 33 to 128 on tcgen05; see
// lora_ortho.cu for the mathematics.  Short sides are padded to 64 or 128 by
// the loads (zeros).
//
// gram_tc_kernel   U U^T: both operands of a UMMA are the same tile.
// iterate_tc_kernel  the steps on 128 x 128 matrices, or (ranks 33 to 64) on
//     two of 64 x 64 at once.  An fp32 value is a sum of three bf16 terms
//     (24 bits), a product the six pairs of terms down to 2^-16.  Two terms
//     do for P, whose result is rounded to two; in R's last three steps they
//     would leave a matrix of rank one 1% off.
//     A UMMA contracts rows with rows, X Y^T, so symmetric matrices need no
//     transposing; the products are ordered so that R stays symmetric: Q R
//     Q^T.  As (R Q^T) Q^T its rounding errors do not commute with R and
//     grow sixfold a step.
// apply_tc_kernel  P U with P as two bf16 terms.
//
// fp32 entries of U are split into two bf16 terms by four warps on the way
// to shared memory; bf16 tiles come by TMA.
//
// 192 matrices of 128 x 8192 (bf16, 805 MB): gram 80 us (5.0 TB/s), iterate
// 106 us (two rounds of 53 on 152 SMs, 60% of it UMMAs), apply 138 us (5.8
// TB/s).
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

struct OrthoTcArgs {
    OrthoArgs o;
    // bf16 U, boxes of 64 columns: 64 rows of a tall U, else RP, for the sum
    // U U^T; 128 rows of a tall U, else RP, for P U
    CUtensorMap gram_u, apply_u;
    CUtensorMap p;        // [count * 2 * RP][RP]: P's terms, boxes 64 x RP
};

// A thread's share of a tile of fp32 entries: chunks of eight, as two bf16
// terms into the swizzled panels at dst (second term `lo` bytes behind).
template <int ROWS, int CPR, int THREADS>
struct Converter {
    static constexpr int PER = ROWS * CPR / THREADS;
    float4 c[PER][2];
    __device__ __forceinline__ void fetch(const OrthoArgs &p, int m, int row0, int col0, int thread)
    {
        const int64_t mat = int64_t(m) * p.rows * p.cols;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int k = thread + i * THREADS, row = row0 + k / CPR, col = col0 + k % CPR * 8;
            c[i][0] = c[i][1] = make_float4(0, 0, 0, 0);
            if (row < p.rows && col < p.cols) {
                const float4 *src = reinterpret_cast<const float4 *>(
                    static_cast<const float *>(p.u) + mat + int64_t(row) * p.cols + col);
                c[i][0] = src[0];
                c[i][1] = src[1];
            }
        }
    }
    __device__ __forceinline__ void put(uint8_t *dst, int lo, int thread) const
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int k = thread + i * THREADS;
            uint8_t *at = dst + tile_at<CPR, ROWS>(k / CPR, k % CPR);
            const Chunk v = split_chunk(c[i][0], c[i][1]);
            *reinterpret_cast<uint4 *>(at) = v.hi;
            *reinterpret_cast<uint4 *>(at + lo) = v.lo;
        }
    }
};

// ---------------------------------------------------------------- gram

// A CTA's run of units (64 of the long side each): one accumulator a matrix.
// At rank 64 the UMMAs read 64 rows past the tile: they reach only rows and
// columns of the result that are not stored.
template <int RP, bool TALL, bool F32>
__global__ void __launch_bounds__(TC_THREADS, 2) gram_tc_kernel(const __grid_constant__ OrthoTcArgs q)
{
    constexpr int TERM = RP * 128, STAGE = TERM * (F32 ? 2 : 1);
    constexpr int STAGES = OT_GRAM_RING / STAGE < TC_MAX_STAGES ? OT_GRAM_RING / STAGE : TC_MAX_STAGES;
    constexpr int ROWS = TALL ? 64 : RP, CPR = TALL ? RP / 8 : 8;
    constexpr uint32_t IDESC = umma_idesc_bf16(OT_R, OT_R) | (TALL ? (1u << 15) | (1u << 16) : 0u);
    const OrthoArgs &p = q.o;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const TcRing ring = tc_setup<256>(smem, OT_GRAM_RING, STAGE, STAGES, F32 ? 4 : 1);
    pdl_wait();
    const int64_t first = unit_begin(p, blockIdx.x), end = unit_begin(p, blockIdx.x + 1);

    if (warp == 0 && !F32) {
        if (lane == 0) {
            TcPos pos;
            int issued = 0;
            for (int64_t u = first; u < end; ++u) {
                if (!pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort)) break;
                const uint32_t full = ring.full + 8 * pos.stage, at = ring.ring + pos.stage * STAGE;
                const int m = int(u / p.units), k = int(u % p.units) * OR_TC_UNIT;
                mbar_arrive_expect_tx(full, TERM);
#pragma unroll
                for (int j = 0; j < (TALL ? RP / 64 : 1); ++j)
                    tma_load_3d(at + j * TC_PANEL, &q.gram_u, TALL ? 64 * j : k, TALL ? k : 0, m, full);
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
                        const uint32_t tl = t + TERM;
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
                conv.put(smem + pos.stage * STAGE, TERM, row);
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
            float *out = p.gram + ((blockIdx.x + u / p.units) * RP + row) * RP;
            for (int c = 0; c < RP; c += 32) {
                uint32_t v[32];
                tmem_ld32_nowait(d + uint32_t(c), v);
                tmem_wait_ld();
                if (row >= RP) continue;
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

constexpr int OT_ITER_THREADS = 512 + 32;       // and the warp that issues UMMAs

// The shared memory of one CTA's R and Q as three terms, panels of 64 K.
template <int K>
constexpr int iter_smem() { return 6 * (K / 64) * OT_PANEL + 128 + 1024; }

// D[128 x 128] = X Y^T over K for operands of three bf16 terms in shared
// memory (X also in TMEM: K / 2 columns a term), by pairs of terms (i, j)
// with i + j < terms, the small ones first.
template <int K, bool X_TMEM>
__device__ __forceinline__ void mul_terms(uint32_t d, uint32_t x, uint32_t y, int terms)
{
    constexpr uint32_t IDESC = umma_idesc_bf16(OT_R, OT_R);
    constexpr uint32_t TERM = uint32_t(K / 64 * OT_PANEL);
    uint32_t acc = 0;
    for (int sum = terms - 1; sum >= 0; --sum)
        for (int i = 0; i <= sum; ++i) {
            const uint32_t xt = x + uint32_t(i) * (X_TMEM ? uint32_t(K / 2) : TERM);
            const uint32_t yt = y + uint32_t(sum - i) * TERM;
#pragma unroll
            for (int kk = 0; kk < K / 16; ++kk) {
                const uint32_t off = uint32_t((kk >> 2) * OT_PANEL + (kk & 3) * 32);
                if constexpr (X_TMEM)
                    umma_bf16_tmem_a(d, xt + uint32_t(kk * 8), umma_desc_sw128(yt + off), IDESC, acc);
                else
                    umma_bf16(d, umma_desc_sw128(xt + off), umma_desc_sw128(yt + off), IDESC, acc);
                acc = 1;
            }
        }
}

// Eight values as three terms of bf16 (four words each), by truncation: the
// terms hold eight bits each, 24 together, so nothing is lost; and masks and
// byte permutes are cheaper than conversions.
__device__ __forceinline__ void split8(const float *v, uint32_t (&t0)[4], uint32_t (&t1)[4], uint32_t (&t2)[4])
{
    auto high = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); };
    auto both = [](float lo, float hi) {
        return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = v[2 * j], b = v[2 * j + 1];
        t0[j] = both(a, b);
        a -= high(a);
        b -= high(b);
        t1[j] = both(a, b);
        t2[j] = both(a - high(a), b - high(b));
    }
}

// Eight values as two terms, rounded (relative 2^-18).
__device__ __forceinline__ void round8(const float *v, float f, uint32_t (&h)[4], uint32_t (&l)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j] * f, b = v[2 * j + 1] * f;
        h[j] = pack_bf16x2(a, b);
        l[j] = pack_bf16x2(a - bf16_lo(h[j]), b - bf16_hi(h[j]));
    }
}

// 128 / K matrices a CTA, one under the other: of D = X Y^T the diagonal
// blocks are their products.  Thread (warp w < 16, lane) holds row 32 (w %
// 4) + lane, a quarter of its matrix's columns (w / 4): R in registers.
// Shared memory: R (then S = Q R, then R again) and Q as three terms; TMEM:
// two accumulators and P's two terms.  A step: R^2 -> Q; then Q R -> S, then
// S Q -> R, each after the last one's epilogue; P Q runs on the tensor cores
// during the epilogue of S, and its own epilogue during S Q.  The last warp
// issues all UMMAs: a product's issue takes as long as the product (66
// clocks a UMMA; 120 with X in TMEM), so no other thread waits in it.
template <int K>
__global__ void __launch_bounds__(OT_ITER_THREADS, 1) iterate_tc_kernel(const OrthoArgs p)
{
    constexpr int C = K / 4;                          // columns of a thread
    constexpr int TERM = K / 64 * OT_PANEL;
    uint8_t *smem = tc_smem();
    const uint32_t sr = smem_addr(smem), sq = sr + 3 * TERM;
    const uint32_t bar = sq + 3 * TERM, bar_p = bar + 8, bar_ready = bar + 16, bar_end = bar + 24;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + 6 * TERM + 32);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + 6 * TERM + 36);
    float *s_trace = reinterpret_cast<float *>(smem + 6 * TERM + 40);         // a warp's each
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3, part = warp >> 2;
    const int row = quarter * 32 + lane, block = quarter * 32 / K;            // of the stack
    const int m = blockIdx.x * (OT_R / K) + block, mrow = row % K, col0 = part * C;
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar_p, 1);
        mbar_init(bar_ready, 16);
        mbar_init(bar_end, 1);
        mbar_fence_init();
        *s_abort = 0;
    }
    if (warp == 16) tmem_alloc(smem_addr(s_tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem, lanes = uint32_t(quarter * 32) << 16;
    const uint32_t d0 = tmem, d1 = tmem + 128, tp = tmem + 256;
    pdl_wait();

    if (warp == 16) {
        if (lane == 0) {
            uint32_t phase = 0;
            bool ok = true;
            // every thread's writes of operands and reads of accumulators are done
            auto ready = [&] {
                ok = ok && pg_wait(bar_ready, phase, s_abort);
                phase ^= 1u;
                tc_fence_after();
                return ok;
            };
            for (int step = 0; step < p.steps; ++step) {
                const bool last = step + 1 == p.steps;
                if (!ready()) break;
                mul_terms<K, false>(d0, sr, sr, 3);
                umma_commit(bar);
                if (step == 0 && last) break;
                if (!ready()) break;
                if (!last) {
                    mul_terms<K, false>(d1, sq, sr, 3);
                    umma_commit(bar);
                }
                if (step > 0) {
                    mul_terms<K, true>(d0, tp, sq, 2);
                    umma_commit(bar_p);
                }
                if (last || !ready()) break;
                mul_terms<K, false>(d1, sr, sq, 3);
                umma_commit(bar);
            }
            if (!ok) {
                // nothing in flight when TMEM is released
                if (p.error_word != nullptr) atomicOr(p.error_word, LORA_TIMEOUT_BIT);
                umma_commit(bar_end);
                const long long dd = clock64() + PG_TIMEOUT_CYCLES;
                while (!mbar_try_wait(bar_end, 0) && clock64() < dd) {
                }
            }
        }
        __syncwarp();
    } else {
        // The matrices' sums over their slots, read along the rows and left
        // where Q will be; a thread's row is then read back (a chunk of four
        // at its place ^ row, against bank conflicts).
        float *sum = reinterpret_cast<float *>(smem + 3 * TERM);
        for (int b = 0; b < OT_R / K; ++b) {
            const int mm = blockIdx.x * (OT_R / K) + b;
            const bool in = mm < p.count;
            const int lo = in ? unit_cta(p, int64_t(mm) * p.units) : 0;
            const int hi = in ? unit_cta(p, int64_t(mm + 1) * p.units - 1) : -1;
            for (int i = tid; i < K * K / 4; i += 512) {
                const int r = i / (K / 4), ch = i % (K / 4);
                float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
                for (int c = lo; c <= hi; ++c) {
                    const float4 x = reinterpret_cast<const float4 *>(p.gram + int64_t(c + mm) * K * K)[i];
                    v.x += x.x;
                    v.y += x.y;
                    v.z += x.z;
                    v.w += x.w;
                }
                reinterpret_cast<float4 *>(sum)[(b * K + r) * (K / 4) + (ch ^ (r & 7))] = v;
            }
        }
        asm volatile("bar.sync 1, 512;\n" ::: "memory");
        float rv[C];                                  // this thread's part of R
#pragma unroll
        for (int j = 0; j < C / 4; ++j)
            *reinterpret_cast<float4 *>(rv + 4 * j) =
                reinterpret_cast<const float4 *>(sum)[row * (K / 4) + ((col0 / 4 + j) ^ (row & 7))];
        float trace = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) trace += col0 + j == mrow ? rv[j] : 0.0f;
        for (int o = 16; o > 0; o >>= 1) trace += __shfl_xor_sync(0xffffffffu, trace, o);
        if (lane == 0) s_trace[warp] = trace;
        asm volatile("bar.sync 1, 512;\n" ::: "memory");
        trace = 0.0f;
        for (int w = 0; w < 16; ++w)
            if ((w & 3) * 32 / K == block) trace += s_trace[w];
        const float f = 1.0f / (sqrtf(trace) + p.eps);
#pragma unroll
        for (int j = 0; j < C; ++j) rv[j] = rv[j] * f * f;

        // this thread's values as three terms, into an operand in shared memory
        auto to_smem = [&](uint8_t *at, const float *v) {
#pragma unroll
            for (int c = 0; c < C / 8; ++c) {
                uint32_t t0[4], t1[4], t2[4];
                split8(v + 8 * c, t0, t1, t2);
                const int col = col0 + 8 * c;
                uint8_t *dst = at + (col >> 6) * OT_PANEL + row * 128 + (((col >> 3) ^ row) & 7) * 16;
                *reinterpret_cast<uint4 *>(dst) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
                *reinterpret_cast<uint4 *>(dst + TERM) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                *reinterpret_cast<uint4 *>(dst + 2 * TERM) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
            }
        };
        auto p_to_tmem = [&](const float *v) {
#pragma unroll
            for (int c = 0; c < C / 8; ++c) {
                uint32_t h[4], l[4];
                round8(v + 8 * c, 1.0f, h, l);
                const uint32_t at = tp + lanes + uint32_t(col0 / 2 + c * 4);
                tmem_st<4>(at, h);
                tmem_st<4>(at + K / 2, l);
            }
        };
        uint16_t *out = p.p + (int64_t(m) * 2 * K + mrow) * K + col0;
        auto p_out = [&](const float *v) {
            if (m >= p.count) return;
#pragma unroll
            for (int c = 0; c < C / 8; ++c) {
                uint32_t h[4], l[4];
                round8(v + 8 * c, f * p.scale, h, l);
                *reinterpret_cast<uint4 *>(out + 8 * c) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(out + K * K + 8 * c) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        };
        auto ready = [&] {
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_ready);
        };
        uint32_t phase = 0, phase_p = 0;
        auto done = [&](uint32_t b, uint32_t &ph) {       // false: the wait ran out
            const bool got = pg_wait(b, ph, s_abort);
            ph ^= 1u;
            tc_fence_after();
            return __all_sync(0xffffffffu, got) != 0;
        };
        auto load = [&](uint32_t d, float *v) {
            const uint32_t at = d + lanes + uint32_t(block * K + col0);
            uint32_t w[C];
            if constexpr (C == 32) tmem_ld32_nowait(at, w);
            else tmem_ld16_nowait(at, w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] = __uint_as_float(w[j]);
        };

        to_smem(smem, rv);
        for (int step = 0; step < p.steps; ++step) {
            const bool last = step + 1 == p.steps;
            float v[C];
            ready();
            if (!done(bar, phase)) break;
            load(d0, v);
#pragma unroll
            for (int j = 0; j < C; ++j)
                v[j] = fmaf(p.c, v[j], fmaf(p.b, rv[j], col0 + j == mrow ? p.a : 0.0f));
            if (step == 0 && last) {
                p_out(v);
                break;
            }
            to_smem(smem + 3 * TERM, v);
            if (step == 0) p_to_tmem(v);                   // P was the identity
            ready();
            if (!last) {
                if (!done(bar, phase)) break;
                load(d1, v);
                to_smem(smem, v);
                ready();
            }
            if (step > 0) {
                if (!done(bar_p, phase_p)) break;
                load(d0, v);
                if (last) p_out(v);
                else p_to_tmem(v);
            }
            if (last) break;
            if (!done(bar, phase)) break;
            load(d1, rv);
            to_smem(smem, rv);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 16) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- apply

// A CTA's run of tiles (128 of the long side each) of the stacked matrices;
// P's terms of the current matrix stay in shared memory.  F32: warps 8 to 11
// convert.  (Rank 64: the UMMAs read past P's and a wide tile's 64 rows, as
// in gram_tc_kernel.)
template <int RP, bool TALL, bool F32>
__global__ void __launch_bounds__(F32 ? TC_THREADS + 128 : TC_THREADS, 1)
apply_tc_kernel(const __grid_constant__ OrthoTcArgs q)
{
    constexpr int TERM = RP * OT_R * 2, STAGE = TERM * (F32 ? 2 : 1);
    constexpr int STAGES = OT_APPLY_RING / STAGE < TC_MAX_STAGES ? OT_APPLY_RING / STAGE : TC_MAX_STAGES;
    constexpr int U_PANEL = (TALL ? OT_R : RP) * 128, P_PANEL = RP * 128, P_TERM = RP * RP * 2;
    constexpr uint32_t IDESC = umma_idesc_bf16(OT_R, OT_R) | (TALL ? 0u : 1u << 16);
    const OrthoArgs &p = q.o;
    uint8_t *smem = tc_smem();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // ring, then P's terms
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
                mbar_arrive_expect_tx(full, TERM);
#pragma unroll
                for (int j = 0; j < (TALL ? RP / 64 : 2); ++j)
                    tma_load_3d(at + j * U_PANEL, &q.apply_u, TALL ? 64 * j : n0 + 64 * j, TALL ? n0 : 0, m, full);
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
                mbar_arrive_expect_tx(p_full, 2 * P_TERM);
                for (int t = 0; t < 2; ++t)
                    for (int j = 0; j < RP / 64; ++j)
                        tma_load_2d(sp + t * P_TERM + j * P_PANEL, &q.p, j * 64, (2 * m + t) * RP, p_full);
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
                    for (int kk = 0; kk < RP / 16; ++kk) {
                        const uint64_t dp = umma_desc_sw128(pt + uint32_t((kk >> 2) * P_PANEL + (kk & 3) * 32));
                        if constexpr (TALL)
                            umma_bf16(d, umma_desc_sw128(ut + uint32_t((kk >> 2) * U_PANEL + (kk & 3) * 32)), dp,
                                      IDESC, acc);
                        else
                            umma_bf16(d, dp, umma_desc_mn(ut + kk * 2048, U_PANEL), IDESC, acc);
                        acc = 1;
                    }
                };
                if constexpr (F32) product(sp, t + TERM);
                product(sp + P_TERM, t);
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
            if (TALL || (warp - 4) * 32 < RP) {
#pragma unroll
                for (int c = 0; c < (TALL ? RP : OT_R); c += 64) {
                    uint32_t o[32];
                    load64(d + uint32_t(c), 1.0f, o);
                    store_rows(stage, o, dst != nullptr ? dst + c : nullptr, p.cols - gc - c);
                }
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
        // 1024 chunks at a time: a tile of rank 64, half a tile of rank 128
        constexpr int CPR = TALL ? RP / 8 : 16, ROWS = 1024 / CPR, PARTS = RP / 64;
        Converter<ROWS, CPR, 128> conv;
        auto fetch = [&](int64_t i, int h) {
            const int n0 = int(i % tiles) * OT_R;
            conv.fetch(p, int(i / tiles), (TALL ? n0 : 0) + ROWS * h, TALL ? 0 : n0, thread);
        };
        auto put = [&](uint8_t *at, int h) {
#pragma unroll
            for (int k = 0; k < conv.PER; ++k) {
                const int c = thread + k * 128;
                uint8_t *to = at + tile_at<CPR, (TALL ? OT_R : RP)>(ROWS * h + c / CPR, c % CPR);
                const Chunk v = split_chunk(conv.c[k][0], conv.c[k][1]);
                *reinterpret_cast<uint4 *>(to) = v.hi;
                *reinterpret_cast<uint4 *>(to + TERM) = v.lo;
            }
        };
        int issued = 0;
        if (first < end) fetch(first, 0);
        for (int64_t i = first; i < end; ++i) {
            const bool got = pg_wait(ring.empty + 8 * pos.stage, pos.phase ^ 1u, ring.abort);
            if (__all_sync(0xffffffffu, got) == 0) break;
            uint8_t *at = smem + pos.stage * STAGE;
            put(at, 0);
            if constexpr (PARTS == 2) {
                fetch(i, 1);
                put(at, 1);
            }
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

template <int RP, bool TALL, bool F32>
static int run_tc(const OrthoTcArgs &q, cudaStream_t st)
{
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    if (dev >= 64 || !configured[dev]) {
        if ((e = cudaFuncSetAttribute(gram_tc_kernel<RP, TALL, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      OT_GRAM_SMEM)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(iterate_tc_kernel<RP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      iter_smem<RP>())) != cudaSuccess ||
            (e = cudaFuncSetAttribute(apply_tc_kernel<RP, TALL, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      OT_APPLY_SMEM)) != cudaSuccess)
            return int(e);
        if (dev < 64) configured[dev] = 1;
    }
    e = launch_kernel(gram_tc_kernel<RP, TALL, F32>, dim3(unsigned(q.o.ctas)), dim3(TC_THREADS), OT_GRAM_SMEM, st, q);
    if (e != cudaSuccess) return int(e);
    e = launch_kernel(iterate_tc_kernel<RP>, dim3(unsigned((q.o.count + OT_R / RP - 1) / (OT_R / RP))),
                      dim3(OT_ITER_THREADS), iter_smem<RP>(), st, q.o);
    if (e != cudaSuccess) return int(e);
    const int64_t tiles = int64_t(q.o.count) * ((q.o.n + OT_R - 1) / OT_R);
    const int sms = device_sm_count();
    e = launch_kernel(apply_tc_kernel<RP, TALL, F32>, dim3(unsigned(tiles < sms ? tiles : sms)),
                      dim3(F32 ? TC_THREADS + 128 : TC_THREADS), OT_APPLY_SMEM, st, q);
    return e == cudaSuccess ? LORA_OK : int(e);
}

template <int RP>
static int run_rank(const OrthoTcArgs &q, bool f32, cudaStream_t st)
{
    const bool tall = q.o.rows > q.o.cols;
    if (f32) return tall ? run_tc<RP, true, true>(q, st) : run_tc<RP, false, true>(q, st);
    return tall ? run_tc<RP, true, false>(q, st) : run_tc<RP, false, false>(q, st);
}

int run_ortho_tc(OrthoArgs p, int rp, bool f32, cudaStream_t st)
{
    const bool tall = p.rows > p.cols;
    static thread_local OrthoTcArgs q;
    q.o = p;
    const uint64_t n = uint64_t(p.count), rows = uint64_t(p.rows), cols = uint64_t(p.cols);
    if (!encode_tile_map(&q.p, p.p, n * 2 * uint64_t(rp), uint64_t(rp), uint64_t(rp), 64, uint32_t(rp),
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        (!f32 && (!encode_stack_map(&q.gram_u, p.u, n, rows, cols, 64, tall ? 64u : uint32_t(rp)) ||
                  !encode_stack_map(&q.apply_u, p.u, n, rows, cols, 64, tall ? uint32_t(OT_R) : uint32_t(rp)))))
        return LORA_ERR_DEVICE;
    return rp == 64 ? run_rank<64>(q, f32, st) : run_rank<128>(q, f32, st);
}

}  // namespace lora
