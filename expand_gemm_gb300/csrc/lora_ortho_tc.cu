// lora_ortho_tc.cu -- lora_orthogonalize on tcgen05: ranks 65 to 128, and the
// steps of ranks 33 to 64; see lora_ortho.cu for the mathematics.  Short sides are padded to 128 by the
// loads (zeros).
//
// gram_tc_kernel   U U^T: both operands of a UMMA are the same tile.
// iterate_tc_kernel  the steps on 128 x 128 matrices, or (ranks 33 to 64) on
//     two of 64 x 64 at once.  An fp32 value is a sum
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

constexpr int OT_ITER_THREADS = 512;

// The shared memory of one CTA's R and Q as three terms, panels of 64 K.
template <int K>
constexpr int iter_smem() { return 6 * (K / 64) * OT_PANEL + 128 + 1024; }

// D[128 x 128] = X Y^T over K for operands of three bf16 terms in shared
// memory (X also in TMEM: K / 2 columns a term), by pairs of terms (i, j)
// with i + j <= 2, the small ones first.
template <int K, bool X_TMEM>
__device__ __forceinline__ void mul_terms(uint32_t d, uint32_t x, uint32_t y)
{
    constexpr uint32_t IDESC = umma_idesc_bf16(OT_R, OT_R);
    constexpr uint32_t TERM = uint32_t(K / 64 * OT_PANEL);
    uint32_t acc = 0;
    for (int sum = 2; sum >= 0; --sum)
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

// 128 / K matrices a CTA, one under the other: of D = X Y^T the diagonal
// blocks are their products.  Thread (warp w, lane) holds row 32 (w % 4) +
// lane, a quarter of its matrix's columns (w / 4): R in registers.  Shared
// memory: R (then S = Q R, then R again) and Q as three terms; TMEM: two
// accumulators and P's terms.  A step: R^2 -> Q; then Q R -> S, then S Q ->
// R, each after the last one's epilogue; P Q runs on the tensor cores
// during the epilogue of S, and its own epilogue during S Q.
template <int K>
__global__ void __launch_bounds__(OT_ITER_THREADS, 1) iterate_tc_kernel(const OrthoArgs p)
{
    constexpr int C = K / 4;                          // columns of a thread
    constexpr int TERM = K / 64 * OT_PANEL;
    uint8_t *smem = tc_smem();
    const uint32_t sr = smem_addr(smem), sq = sr + 3 * TERM, bar = sq + 3 * TERM, bar_p = bar + 8;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + 6 * TERM + 16);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + 6 * TERM + 20);
    float *s_trace = reinterpret_cast<float *>(smem + 6 * TERM + 24);         // a warp's each
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3, part = warp >> 2;
    const int row = quarter * 32 + lane, block = quarter * 32 / K;            // of the stack
    const int m = blockIdx.x * (OT_R / K) + block, mrow = row % K, col0 = part * C;
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar_p, 1);
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

    float rv[C];                                      // this thread's part of R
#pragma unroll
    for (int j = 0; j < C; ++j) rv[j] = 0.0f;
    if (m < p.count) {
        const int lo = unit_cta(p, int64_t(m) * p.units), hi = unit_cta(p, int64_t(m + 1) * p.units - 1);
        for (int c = lo; c <= hi; ++c) {
            const float4 *src = reinterpret_cast<const float4 *>(
                p.gram + (int64_t(c + m) * K + mrow) * K + col0);
#pragma unroll
            for (int j = 0; j < C / 4; ++j) {
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
    for (int j = 0; j < C; ++j) trace += col0 + j == mrow ? rv[j] : 0.0f;
    for (int o = 16; o > 0; o >>= 1) trace += __shfl_xor_sync(0xffffffffu, trace, o);
    if (lane == 0) s_trace[warp] = trace;
    __syncthreads();
    trace = 0.0f;
    for (int w = 0; w < 16; ++w)
        if ((w & 3) * 32 / K == block) trace += s_trace[w];
    const float f = 1.0f / (sqrtf(trace) + p.eps);
#pragma unroll
    for (int j = 0; j < C; ++j) rv[j] = rv[j] * f * f;

    // this thread's values as terms, into an operand in shared memory
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
            uint32_t t0[4], t1[4], t2[4];
            split8(v + 8 * c, t0, t1, t2);
            const uint32_t at = tp + lanes + uint32_t(col0 / 2 + c * 4);
            tmem_st<4>(at, t0);
            tmem_st<4>(at + K / 2, t1);
            tmem_st<4>(at + K, t2);
        }
    };
    uint16_t *out = p.p + (int64_t(m) * 2 * K + mrow) * K + col0;
    auto p_out = [&](const float *v) {
        if (m >= p.count) return;
#pragma unroll
        for (int c = 0; c < C / 8; ++c) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = v[8 * c + 2 * j] * f * p.scale, b = v[8 * c + 2 * j + 1] * f * p.scale;
                h[j] = pack_bf16x2(a, b);
                l[j] = pack_bf16x2(a - bf16_lo(h[j]), b - bf16_hi(h[j]));
            }
            *reinterpret_cast<uint4 *>(out + 8 * c) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(out + K * K + 8 * c) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    };
    // Every thread's writes of operands and reads of accumulators are done
    // before the UMMAs that thread 0 starts.
    auto products = [&](auto issue) {
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            issue();
        }
        __syncwarp();
    };
    // ... and the wait for them (false: it ran out, for the whole CTA).
    uint32_t phase = 0, phase_p = 0;
    auto done = [&](uint32_t b, uint32_t &ph) {
        const bool got = pg_wait(b, ph, s_abort);
        ph ^= 1u;
        tc_fence_after();
        return __syncthreads_and(int(got)) != 0;
    };
    auto load = [&](uint32_t d, float *v) {
        const uint32_t at = d + lanes + uint32_t(block * K + col0);
        if constexpr (C == 32) {
            uint32_t w[32];
            tmem_ld32_nowait(at, w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]);
        } else {
            uint32_t w[16];
            tmem_ld16_nowait(at, w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(w[j]);
        }
    };

    to_smem(smem, rv);
    bool ok = true;
    for (int step = 0; ok && step < p.steps; ++step) {
        const bool last = step + 1 == p.steps;
        float v[C];
        products([&] {
            mul_terms<K, false>(d0, sr, sr);
            umma_commit(bar);
        });
        if (!(ok = done(bar, phase))) break;
        load(d0, v);
#pragma unroll
        for (int j = 0; j < C; ++j)
            v[j] = fmaf(p.c, v[j], fmaf(p.b, rv[j], col0 + j == mrow ? p.a : 0.0f));
        to_smem(smem + 3 * TERM, v);
        if (step == 0) {                               // P was the identity
            if (last) {
                p_out(v);
                break;
            }
            p_to_tmem(v);
        }
        products([&] {
            if (!last) {
                mul_terms<K, false>(d1, sq, sr);
                umma_commit(bar);
            }
            if (step > 0) {
                mul_terms<K, true>(d0, tp, sq);
                umma_commit(bar_p);
            }
        });
        if (!last) {
            if (!(ok = done(bar, phase))) break;
            load(d1, v);
            to_smem(smem, v);
            products([&] {
                mul_terms<K, false>(d1, sr, sq);
                umma_commit(bar);
            });
        }
        if (step > 0) {
            if (!(ok = done(bar_p, phase_p))) break;
            load(d0, v);
            if (last) p_out(v);
            else p_to_tmem(v);
        }
        if (last) break;
        if (!(ok = done(bar, phase))) break;
        load(d1, rv);
        to_smem(smem, rv);
    }
    if (!ok && tid == 0) {
        // nothing in flight when TMEM is released: a bounded wait for all
        // products so far
        if (p.error_word != nullptr) atomicOr(p.error_word, LORA_TIMEOUT_BIT);
        const uint32_t bar_end = bar + 120;
        mbar_init(bar_end, 1);
        mbar_fence_init();
        umma_commit(bar_end);
        const long long dd = clock64() + PG_TIMEOUT_CYCLES;
        while (!mbar_try_wait(bar_end, 0) && clock64() < dd) {
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

int launch_iterate_tc(const OrthoArgs &p, int rp, cudaStream_t st)
{
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    if (dev >= 64 || !configured[dev]) {
        if ((e = cudaFuncSetAttribute(iterate_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      iter_smem<64>())) != cudaSuccess ||
            (e = cudaFuncSetAttribute(iterate_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      iter_smem<128>())) != cudaSuccess)
            return int(e);
        if (dev < 64) configured[dev] = 1;
    }
    if (rp == 64)
        return int(launch_kernel(iterate_tc_kernel<64>, dim3(unsigned((p.count + 1) / 2)), dim3(OT_ITER_THREADS),
                                 iter_smem<64>(), st, p));
    return int(launch_kernel(iterate_tc_kernel<128>, dim3(unsigned(p.count)), dim3(OT_ITER_THREADS),
                             iter_smem<128>(), st, p));
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
                const Chunk v = split_chunk(conv.c[k][0], conv.c[k][1]);
                *reinterpret_cast<uint4 *>(to) = v.hi;
                *reinterpret_cast<uint4 *>(to + 2 * OT_PANEL) = v.lo;
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
            (e = cudaFuncSetAttribute(apply_tc_kernel<TALL, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      OT_APPLY_SMEM)) != cudaSuccess)
            return int(e);
        if (dev < 64) configured[dev] = 1;
    }
    e = launch_kernel(gram_tc_kernel<TALL, F32>, dim3(unsigned(q.o.ctas)), dim3(TC_THREADS), OT_GRAM_SMEM, st, q);
    if (e != cudaSuccess) return int(e);
    if (int r = launch_iterate_tc(q.o, OT_R, st)) return r;
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
