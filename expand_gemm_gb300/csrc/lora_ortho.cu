// lora_ortho.cu -- orthogonalises stacked matrices by Newton-Schulz steps:
//   X = U / (|U|_F + eps);  X <- a X + (b G + c G^2) X, G = X X^T, n times.
//
// Every iterate is X_k = P_k X_0 with P_k a polynomial in G_0 = X_0 X_0^T,
// and everything that multiplies X commutes.  So the iteration runs on
// r x r matrices (r, the short side, is an adapter's rank, at most 128):
//   R_0 = G_0, P_0 = I;  Q = a I + b R + c R^2;  P <- Q P;  R <- Q R Q
// and U is read twice (G_0; P U) instead of twice a step.  |U|_F^2 is the
// trace of U U^T.
//
// Three kernels: gram_kernel sums U U^T over even runs of the long sides of
// all matrices, iterate_kernel runs the steps on one matrix a block in fp32,
// apply_kernel writes P U.  The products with U run on the tensor cores with
// U exact: bf16 as it is, fp32 as a sum of two bf16 values (relative 2^-17),
// P as a sum of two bf16 values -- P holds factors up to a^n = 485 for
// directions that U has little of, which cancel where U is large, so one
// bf16 would show in the result.
//
// This file: ranks up to 64, on mma.sync and FFMA.  lora_ortho_tc.cu: ranks
// to 128, on tcgen05.
#include <math.h>

#include "lora_ortho.cuh"

namespace lora {

// ---------------------------------------------------------------- gram

// Warps of gram_kernel: WM x WN over the RP x RP result, WK over the K step.
template <int RP> struct GramShape;
template <> struct GramShape<16> { static constexpr int WM = 1, WN = 1, WK = 8; };
template <> struct GramShape<32> { static constexpr int WM = 1, WN = 1, WK = 8; };
template <> struct GramShape<64> { static constexpr int WM = 2, WN = 1, WK = 4; };

template <int RP>
constexpr int gram_step() { return RP == 64 ? 128 : 256; }

template <int RP, bool F32>
constexpr int gram_smem()
{
    constexpr int tile = RP * gram_step<RP>() * 2 * (F32 ? 2 : 1);
    constexpr int join = GramShape<RP>::WK > 1 ? GramShape<RP>::WK * RP * RP * 4 : 0;
    return 2 * tile > join ? 2 * tile : join;
}

// Each block sums over its run of units.  TALL: U is [n][r] (its rows are
// K), else [r][n].
template <int RP, bool TALL, bool F32>
__global__ void __launch_bounds__(OR_THREADS) gram_kernel(const OrthoArgs p)
{
    constexpr int WM = GramShape<RP>::WM, WN = GramShape<RP>::WN, WK = GramShape<RP>::WK;
    constexpr int KS = gram_step<RP>();
    constexpr int ROWS = TALL ? KS : RP, COLS = TALL ? RP : KS;     // of the tile
    constexpr int CPR = COLS / 8;
    constexpr int TILE = RP * KS * 2;                               // bytes of one term
    constexpr int TERMS = F32 ? 2 : 1;
    constexpr int PER = ROWS * CPR / OR_THREADS;                    // chunks a thread loads
    constexpr int MI = RP / WM / 16, NI = RP / WN / 8;
    static_assert(PER >= 1 && MI >= 1 && NI >= 2 && WK > 1, "shape");
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int wk = warp / (WM * WN), wm = warp % WM, wn = warp / WM % WN;
    const int m0 = wm * (RP / WM), n0 = wn * (RP / WN);
    pdl_wait();
    pdl_launch_dependents();
    const int64_t first = unit_begin(p, blockIdx.x), end = unit_begin(p, blockIdx.x + 1);

    Chunk<F32> next[PER];
    auto fetch = [&](int64_t unit) {
        const int64_t mat = unit / p.units * p.rows * p.cols;
        const int k = int(unit % p.units) * KS;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = tid + i * OR_THREADS, row = c / CPR, ch = c % CPR;
            const int gr = TALL ? k + row : row, gc = (TALL ? 0 : k) + ch * 8;
            next[i] = load_chunk<F32>(p.u, mat + int64_t(gr) * p.cols + gc, gr < p.rows && gc < p.cols);
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = tid + i * OR_THREADS;
            uint8_t *at = smem + buf * TILE * TERMS + tile_at<CPR, ROWS>(c / CPR, c % CPR);
            *reinterpret_cast<uint4 *>(at) = next[i].hi;
            if constexpr (F32) *reinterpret_cast<uint4 *>(at + TILE) = next[i].lo;
        }
    };
    float acc[MI][NI][4] = {};
    int buf = 0;
    if (first < end) fetch(first);
    for (int64_t unit = first; unit < end; ++unit) {
        put(buf);
        __syncthreads();
        if (unit + 1 < end) fetch(unit + 1);
        const uint32_t hi = base + buf * TILE * TERMS;
#pragma unroll 2
        for (int kk = wk * (KS / WK); kk < (wk + 1) * (KS / WK); kk += 16) {
            uint32_t a[MI][4], al[MI][4];
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                frag_a<CPR, ROWS, !TALL>(hi, m0 + 16 * i, kk, a[i]);
                if constexpr (F32) frag_a<CPR, ROWS, !TALL>(hi + TILE, m0 + 16 * i, kk, al[i]);
            }
#pragma unroll
            for (int j = 0; j < NI; j += 2) {
                uint32_t b[4], bl[4];
                frag_b<CPR, ROWS, !TALL>(hi, kk, n0 + 8 * j, b);
                if constexpr (F32) frag_b<CPR, ROWS, !TALL>(hi + TILE, kk, n0 + 8 * j, bl);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    mma_bf16_16816(acc[i][j], a[i], b[0], b[1]);
                    mma_bf16_16816(acc[i][j + 1], a[i], b[2], b[3]);
                    if constexpr (F32) {
                        mma_bf16_16816(acc[i][j], al[i], b[0], b[1]);
                        mma_bf16_16816(acc[i][j + 1], al[i], b[2], b[3]);
                        mma_bf16_16816(acc[i][j], a[i], bl[0], bl[1]);
                        mma_bf16_16816(acc[i][j + 1], a[i], bl[2], bl[3]);
                    }
                }
            }
        }
        buf ^= 1;
        if (unit + 1 < end && (unit + 1) % p.units != 0) continue;
        // the matrix or the run ends: the warps' sums over K, joined
        float *out = p.gram + (blockIdx.x + unit / p.units) * RP * RP;
        const int g = (tid & 31) >> 2, t = tid & 3;
        __syncthreads();
        float *part = reinterpret_cast<float *>(smem) + wk * RP * RP;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                float *at = part + (m0 + 16 * i + g) * RP + n0 + 8 * j + 2 * t;
                at[0] = acc[i][j][0];
                at[1] = acc[i][j][1];
                at[8 * RP] = acc[i][j][2];
                at[8 * RP + 1] = acc[i][j][3];
                acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;
            }
        __syncthreads();
        for (int i = tid; i < RP * RP; i += OR_THREADS) {
            float s = 0.0f;
            for (int w = 0; w < WK; ++w) s += reinterpret_cast<float *>(smem)[w * RP * RP + i];
            out[i] = s;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- iterate

// C = A B where A, B and C are symmetric (polynomials in one matrix): one
// E x E block (ty, tx) on or above the diagonal a thread, the sum over k of
// rows k of A and B.
template <int RP, int E>
__device__ __forceinline__ void mul(const float *A, const float *B, int ty, int tx, float (&c)[E][E])
{
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) c[i][j] = 0.0f;
#pragma unroll 8
    for (int k = 0; k < RP; ++k) {
        float a[E], b[E];
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] = A[k * RP + ty * E + i];
#pragma unroll
        for (int j = 0; j < E; ++j) b[j] = B[k * RP + tx * E + j];
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) c[i][j] = fmaf(a[i], b[j], c[i][j]);
    }
}

// One block per matrix; R, P, Q in shared memory, in fp32.  The 136 blocks
// on or above the diagonal of a 16 x 16 grid are a thread's each; the rest
// is their mirror image.  (All 256 blocks by 256 threads: 49 us at rank 64.)
template <int RP>
__global__ void __launch_bounds__(OR_THREADS) iterate_kernel(const OrthoArgs p)
{
    constexpr int E = RP / 16;
    extern __shared__ __align__(128) float sm[];
    float *R = sm, *P = R + RP * RP, *Q = P + RP * RP;
    __shared__ float s_norm;
    const int tid = threadIdx.x, m = blockIdx.x;
    int ty = 0, tx = tid;                     // the tid-th block, row by row
    while (ty < 16 && tx >= 16 - ty) tx -= 16 - ty++;
    const bool mine = ty < 16;
    tx += ty;
    pdl_wait();
    pdl_launch_dependents();
    const int lo = unit_cta(p, int64_t(m) * p.units), hi = unit_cta(p, int64_t(m + 1) * p.units - 1);
    for (int i = tid; i < RP * RP; i += OR_THREADS) {
        R[i] = gram_sum<RP>(p, m, lo, hi, i);
    }
    __syncthreads();
    if (tid < 32) {
        float s = 0.0f;
        for (int i = tid; i < RP; i += 32) s += R[i * RP + i];
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid == 0) s_norm = 1.0f / (sqrtf(s) + p.eps);
    }
    __syncthreads();
    const float f = s_norm;
    for (int i = tid; i < RP * RP; i += OR_THREADS) R[i] = R[i] * f * f;
    __syncthreads();
    float c[E][E];
    auto store = [&](float *to) {
        __syncthreads();                      // every read of `to` is done
        if (mine) {
#pragma unroll
            for (int i = 0; i < E; ++i)
#pragma unroll
                for (int j = 0; j < E; ++j) to[(ty * E + i) * RP + tx * E + j] = c[i][j];
            if (tx != ty)
#pragma unroll
                for (int i = 0; i < E; ++i)
#pragma unroll
                    for (int j = 0; j < E; ++j) to[(tx * E + j) * RP + ty * E + i] = c[i][j];
        }
        __syncthreads();
    };
    for (int step = 0; step < p.steps; ++step) {
        if (mine) {
            mul<RP, E>(R, R, ty, tx, c);
#pragma unroll
            for (int i = 0; i < E; ++i)
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const int y = ty * E + i, x = tx * E + j;
                    c[i][j] = fmaf(p.c, c[i][j], fmaf(p.b, R[y * RP + x], y == x ? p.a : 0.0f));
                }
        }
        store(Q);
        if (step == 0) {                      // P was the identity
            for (int i = tid; i < RP * RP; i += OR_THREADS) P[i] = Q[i];
        } else {
            if (mine) mul<RP, E>(Q, P, ty, tx, c);
            store(P);
        }
        if (step + 1 < p.steps) {
            if (mine) mul<RP, E>(Q, R, ty, tx, c);
            store(R);
            if (mine) mul<RP, E>(R, Q, ty, tx, c);
            store(R);
        }
    }
    __syncthreads();
    uint16_t *out = p.p + int64_t(m) * 2 * RP * RP;
    const float s = f * p.scale;
    for (int i = tid; i < RP * RP / 2; i += OR_THREADS) {
        const float v0 = P[2 * i] * s, v1 = P[2 * i + 1] * s;
        const uint32_t h = pack_bf16x2(v0, v1);
        reinterpret_cast<uint32_t *>(out)[i] = h;
        reinterpret_cast<uint32_t *>(out + RP * RP)[i] = pack_bf16x2(v0 - bf16_lo(h), v1 - bf16_hi(h));
    }
}

// ---------------------------------------------------------------- apply

constexpr int OR_LONG = 128;              // long-side elements of a tile of apply_kernel

template <int RP, bool F32>
constexpr int apply_smem()
{
    return 2 * RP * RP * 2 + RP * OR_LONG * 2 * (F32 ? 2 : 1) ;
}

// Each block takes a run of tiles of the stacked matrices, P of the current
// one in shared memory: out = P U (or U P, TALL; P is symmetric).
template <int RP, bool TALL, bool F32>
__global__ void __launch_bounds__(OR_THREADS) apply_kernel(const OrthoArgs p)
{
    constexpr int ROWS = TALL ? OR_LONG : RP, COLS = TALL ? RP : OR_LONG;
    constexpr int CPR = COLS / 8, PCPR = RP / 8;
    constexpr int TILE = RP * OR_LONG * 2;
    constexpr int PER = ROWS * CPR / OR_THREADS;
    // warps over the [ROWS x COLS] output
    constexpr int WM = TALL ? 8 : RP / 16, WN = 8 / WM;
    constexpr int MI = ROWS / WM / 16, NI = COLS / WN / 8;
    static_assert(PER >= 1 && MI >= 1 && NI >= 2, "shape");
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *s_u = smem + 2 * RP * RP * 2;
    const uint32_t sp = smem_addr(smem), su = smem_addr(s_u);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int m0 = warp % WM * (ROWS / WM), n0 = warp / WM * (COLS / WN);
    pdl_wait();
    pdl_launch_dependents();
    const int tiles = (p.n + OR_LONG - 1) / OR_LONG;
    const int64_t total = int64_t(p.count) * tiles;
    const int64_t first = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
    int held = -1;
    Chunk<F32> next[PER];
    auto fetch = [&](int64_t item) {
        const int64_t mat = item / tiles * p.rows * p.cols;
        const int tile = int(item % tiles);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = tid + i * OR_THREADS, row = c / CPR, ch = c % CPR;
            const int gr = TALL ? tile * OR_LONG + row : row;
            const int gc = (TALL ? 0 : tile * OR_LONG) + ch * 8;
            next[i] = load_chunk<F32>(p.u, mat + int64_t(gr) * p.cols + gc, gr < p.rows && gc < p.cols);
        }
    };
    if (first < end) fetch(first);
    for (int64_t item = first; item < end; ++item) {
        const int m = int(item / tiles), tile = int(item % tiles);
        const int64_t mat = int64_t(m) * p.rows * p.cols;
        __syncthreads();
        if (m != held) {
            const uint4 *gp = reinterpret_cast<const uint4 *>(p.p + int64_t(m) * 2 * RP * RP);
            for (int i = tid; i < 2 * RP * PCPR; i += OR_THREADS) {
                const int term = i / (RP * PCPR), c = i % (RP * PCPR);
                *reinterpret_cast<uint4 *>(smem + term * RP * RP * 2 +
                                           tile_at<PCPR, RP>(c / PCPR, c % PCPR)) = gp[i];
            }
            held = m;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = tid + i * OR_THREADS;
            uint8_t *at = s_u + tile_at<CPR, ROWS>(c / CPR, c % CPR);
            *reinterpret_cast<uint4 *>(at) = next[i].hi;
            if constexpr (F32) *reinterpret_cast<uint4 *>(at + TILE) = next[i].lo;
        }
        __syncthreads();
        if (item + 1 < end) fetch(item + 1);
        float acc[MI][NI][4] = {};
#pragma unroll 2
        for (int kk = 0; kk < RP; kk += 16) {
            uint32_t a[MI][4], al[MI][4];
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if constexpr (TALL) {
                    frag_a<CPR, ROWS, true>(su, m0 + 16 * i, kk, a[i]);
                    if constexpr (F32) frag_a<CPR, ROWS, true>(su + TILE, m0 + 16 * i, kk, al[i]);
                } else {
                    frag_a<PCPR, RP, true>(sp, m0 + 16 * i, kk, a[i]);
                    frag_a<PCPR, RP, true>(sp + RP * RP * 2, m0 + 16 * i, kk, al[i]);
                }
            }
#pragma unroll
            for (int j = 0; j < NI; j += 2) {
                uint32_t b[4], bl[4];
                if constexpr (TALL) {
                    frag_b<PCPR, RP, true>(sp, kk, n0 + 8 * j, b);
                    frag_b<PCPR, RP, true>(sp + RP * RP * 2, kk, n0 + 8 * j, bl);
                } else {
                    frag_b<CPR, ROWS, false>(su, kk, n0 + 8 * j, b);
                    if constexpr (F32) frag_b<CPR, ROWS, false>(su + TILE, kk, n0 + 8 * j, bl);
                }
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    mma_bf16_16816(acc[i][j], a[i], b[0], b[1]);
                    mma_bf16_16816(acc[i][j + 1], a[i], b[2], b[3]);
                    if constexpr (F32 || !TALL) {
                        mma_bf16_16816(acc[i][j], al[i], b[0], b[1]);
                        mma_bf16_16816(acc[i][j + 1], al[i], b[2], b[3]);
                    }
                    if constexpr (F32 || TALL) {
                        mma_bf16_16816(acc[i][j], a[i], bl[0], bl[1]);
                        mma_bf16_16816(acc[i][j + 1], a[i], bl[2], bl[3]);
                    }
                }
            }
        }
        // through shared memory, so that rows are written 16 bytes at a time
        __syncthreads();
        const int g = (tid & 31) >> 2, t = tid & 3;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int row = m0 + 16 * i + g, col = n0 + 8 * j + 2 * t;
                *reinterpret_cast<uint32_t *>(s_u + tile_at<CPR, ROWS>(row, col / 8) + col % 8 * 2) =
                    pack_bf16x2(acc[i][j][0], acc[i][j][1]);
                *reinterpret_cast<uint32_t *>(s_u + tile_at<CPR, ROWS>(row + 8, col / 8) + col % 8 * 2) =
                    pack_bf16x2(acc[i][j][2], acc[i][j][3]);
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = tid + i * OR_THREADS, row = c / CPR, ch = c % CPR;
            const int gr = TALL ? tile * OR_LONG + row : row;
            const int gc = (TALL ? 0 : tile * OR_LONG) + ch * 8;
            if (gr < p.rows && gc < p.cols)
                *reinterpret_cast<uint4 *>(p.out + mat + int64_t(gr) * p.cols + gc) =
                    *reinterpret_cast<const uint4 *>(s_u + tile_at<CPR, ROWS>(row, ch));
        }
    }
}

// ---------------------------------------------------------------- host

struct OrthoLayout {
    int r, n, rp, unit, units, ctas;
    int64_t p, bytes;
};

// Blocks of a kernel on an SM by its shared memory, at most four.
static int blocks_per_sm(int smem)
{
    const int n = 227 * 1024 / (smem + 1024);
    return n > 4 ? 4 : n;
}

template <bool F32>
static int gram_blocks(int rp)
{
    return rp == 16 ? blocks_per_sm(gram_smem<16, F32>())
                    : rp == 32 ? blocks_per_sm(gram_smem<32, F32>()) : blocks_per_sm(gram_smem<64, F32>());
}

// The sum U U^T is cut into units of one tile each and those into as many
// runs as blocks fit the GPU at once (or as there are units).
static OrthoLayout ortho_layout(int32_t count, int32_t rows, int32_t cols, bool f32, int sms)
{
    OrthoLayout l;
    l.r = rows <= cols ? rows : cols;
    l.n = rows <= cols ? cols : rows;
    l.rp = 16;
    while (l.rp < l.r) l.rp *= 2;
    l.unit = l.rp == 128 ? OR_TC_UNIT : l.rp == 64 ? gram_step<64>() : gram_step<32>();
    l.units = (l.n + l.unit - 1) / l.unit;
    const int64_t most = int64_t(sms) * (l.rp == 128 ? OR_TC_CTAS
                                                     : f32 ? gram_blocks<true>(l.rp) : gram_blocks<false>(l.rp));
    const int64_t total = int64_t(count) * l.units;
    l.ctas = int(total < most ? total : most);
    l.p = (int64_t(l.ctas) + count) * l.rp * l.rp * 4;
    l.bytes = l.p + int64_t(count) * 2 * l.rp * l.rp * 2;
    return l;
}

template <typename Kern>
static cudaError_t allow_smem(Kern k, int bytes)
{
    return bytes > 40 * 1024      // 48 KB hold static shared memory too
               ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
               : cudaSuccess;
}

template <int RP, bool TALL, bool F32>
static int run_ortho(const OrthoArgs &p, cudaStream_t st)
{
    constexpr int gs = gram_smem<RP, F32>(), is = 3 * RP * RP * 4, as = apply_smem<RP, F32>();
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    if (dev >= 64 || !configured[dev]) {
        if ((e = allow_smem(gram_kernel<RP, TALL, F32>, gs)) != cudaSuccess ||
            (e = allow_smem(iterate_kernel<RP>, is)) != cudaSuccess ||
            (e = allow_smem(apply_kernel<RP, TALL, F32>, as)) != cudaSuccess)
            return int(e);
        if (dev < 64) configured[dev] = 1;
    }
    e = launch_kernel(gram_kernel<RP, TALL, F32>, dim3(p.ctas), dim3(OR_THREADS), gs, st, p);
    if (e != cudaSuccess) return int(e);
    e = launch_kernel(iterate_kernel<RP>, dim3(p.count), dim3(OR_THREADS), is, st, p);
    if (e != cudaSuccess) return int(e);
    const int64_t tiles = int64_t(p.count) * ((p.n + OR_LONG - 1) / OR_LONG);
    const int64_t most = int64_t(device_sm_count()) * blocks_per_sm(as);
    e = launch_kernel(apply_kernel<RP, TALL, F32>, dim3(unsigned(tiles < most ? tiles : most)),
                      dim3(OR_THREADS), as, st, p);
    return e == cudaSuccess ? LORA_OK : int(e);
}

template <bool TALL, bool F32>
static int run_ortho_rank(const OrthoArgs &p, int rp, cudaStream_t st)
{
    switch (rp) {
    case 16: return run_ortho<16, TALL, F32>(p, st);
    case 32: return run_ortho<32, TALL, F32>(p, st);
    default: return run_ortho<64, TALL, F32>(p, st);
    }
}

static bool ortho_sizes_ok(int32_t count, int32_t rows, int32_t cols)
{
    // count is a grid's dimension
    return count >= 0 && count <= 65535 && rows >= 1 && cols >= 8 && cols % 8 == 0 &&
           (rows <= OR_MAX_RANK || cols <= OR_MAX_RANK);
}

}  // namespace lora

LORA_API int64_t lora_orthogonalize_workspace(int32_t count, int32_t rows, int32_t cols)
{
    if (!lora::ortho_sizes_ok(count, rows, cols)) return LORA_ERR_SIZE;
    const int sms = lora::device_sm_count();
    const int64_t a = lora::ortho_layout(count > 0 ? count : 1, rows, cols, false, sms).bytes;
    const int64_t b = lora::ortho_layout(count > 0 ? count : 1, rows, cols, true, sms).bytes;
    return a > b ? a : b;
}

LORA_API int lora_orthogonalize(const void *update, int32_t update_f32, int32_t count, int32_t rows,
                                int32_t cols, int32_t steps, float coef_a, float coef_b,
                                float coef_c, float eps, float scale, lora_bf16_t *out,
                                int32_t *error_word, void *workspace, int64_t workspace_bytes, void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_orthogonalize");
    if (!ortho_sizes_ok(count, rows, cols) || steps < 1) return LORA_ERR_SIZE;
    if (count == 0) return LORA_OK;
    if (update == nullptr || out == nullptr || workspace == nullptr) return LORA_ERR_NULL;
    auto bits = [](const void *ptr) { return reinterpret_cast<uintptr_t>(ptr); };
    if ((bits(update) | bits(out)) & 15u || bits(workspace) & 255u) return LORA_ERR_ALIGN;
    const OrthoLayout l = ortho_layout(count, rows, cols, update_f32 != 0, device_sm_count());
    if (workspace_bytes < l.bytes) return LORA_ERR_WORKSPACE;
    OrthoArgs p;
    p.u = update;
    p.out = out;
    p.count = count;
    p.rows = rows;
    p.cols = cols;
    p.r = l.r;
    p.n = l.n;
    p.units = l.units;
    p.unit = l.unit;
    p.ctas = l.ctas;
    p.error_word = error_word;
    p.steps = steps;
    p.a = coef_a;
    p.b = coef_b;
    p.c = coef_c;
    p.eps = eps;
    p.scale = scale;
    p.gram = reinterpret_cast<float *>(workspace);
    p.p = reinterpret_cast<uint16_t *>(static_cast<char *>(workspace) + l.p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool tall = rows > cols;
    if (l.rp == 128) return run_ortho_tc(p, update_f32 != 0, st);
    if (update_f32)
        return tall ? run_ortho_rank<true, true>(p, l.rp, st) : run_ortho_rank<false, true>(p, l.rp, st);
    return tall ? run_ortho_rank<true, false>(p, l.rp, st) : run_ortho_rank<false, false>(p, l.rp, st);
}
