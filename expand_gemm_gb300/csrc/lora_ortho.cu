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
// Three kernels: gram_kernel sums U U^T over shares of the long side (the
// shares are joined in a fixed order), iterate_kernel runs the steps on one
// matrix a block in fp32, apply_kernel writes P U.  The products with U run
// on the tensor cores with U exact: bf16 as it is, fp32 as a sum of two
// bf16 values (relative 2^-17), P as a sum of two bf16 values -- P holds
// factors up to a^n = 485 for directions that U has little of, which cancel
// where U is large, so one bf16 would show in the result.
#include <math.h>

#include "lora_frag.cuh"

namespace lora {

constexpr int OR_THREADS = 256;
constexpr int OR_MAX_RANK = 128;

struct OrthoArgs {
    const void *u;
    uint16_t *out;
    int32_t count, rows, cols;    // matrices, each [rows, cols]
    int32_t r, n;                 // short and long side
    int32_t shares;               // of the long side in gram_kernel
    int32_t share;                // its length, a multiple of the K step
    int32_t steps;
    float a, b, c, eps, scale;
    float *gram;                  // [count][shares][RP][RP]
    uint16_t *p;                  // [count][2][RP][RP]: P as two bf16 terms
};

// Eight consecutive elements of U as bf16 terms: hi, and (fp32) what hi
// leaves over.
template <bool F32>
struct Chunk {
    uint4 hi, lo;
};

template <bool F32>
__device__ __forceinline__ Chunk<F32> load_chunk(const void *u, int64_t at, bool valid)
{
    Chunk<F32> c;
    c.hi = c.lo = make_uint4(0, 0, 0, 0);
    if (!valid) return c;
    if constexpr (F32) {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(u) + at);
        const float4 x = src[0], y = src[1];
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            l[i] = pack_bf16x2(v[2 * i] - bf16_lo(h[i]), v[2 * i + 1] - bf16_hi(h[i]));
        }
        c.hi = make_uint4(h[0], h[1], h[2], h[3]);
        c.lo = make_uint4(l[0], l[1], l[2], l[3]);
    } else {
        c.hi = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(u) + at);
    }
    return c;
}

// ---------------------------------------------------------------- gram

// Warps of gram_kernel: WM x WN over the RP x RP result, WK over the K step.
template <int RP> struct GramShape;
template <> struct GramShape<16> { static constexpr int WM = 1, WN = 1, WK = 8; };
template <> struct GramShape<32> { static constexpr int WM = 1, WN = 1, WK = 8; };
template <> struct GramShape<64> { static constexpr int WM = 2, WN = 1, WK = 4; };
template <> struct GramShape<128> { static constexpr int WM = 4, WN = 2, WK = 1; };

template <int RP>
constexpr int gram_step() { return RP == 128 ? 64 : RP == 64 ? 128 : 256; }

template <int RP, bool F32>
constexpr int gram_smem()
{
    constexpr int tile = RP * gram_step<RP>() * 2 * (F32 ? 2 : 1);
    constexpr int join = GramShape<RP>::WK > 1 ? GramShape<RP>::WK * RP * RP * 4 : 0;
    return 2 * tile > join ? 2 * tile : join;
}

// Block (share, matrix): the sum over its share of the long side.  TALL: U
// is [n][r] (its rows are K), else [r][n].
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
    static_assert(PER >= 1 && MI >= 1 && NI >= 2, "shape");
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int wk = warp / (WM * WN), wm = warp % WM, wn = warp / WM % WN;
    const int m0 = wm * (RP / WM), n0 = wn * (RP / WN);
    pdl_wait();
    pdl_launch_dependents();
    const int64_t mat = int64_t(blockIdx.y) * p.rows * p.cols;
    const int k_lo = blockIdx.x * p.share, k_hi = min(p.n, k_lo + p.share);

    Chunk<F32> next[PER];
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = tid + i * OR_THREADS, row = c / CPR, ch = c % CPR;
            const int gr = TALL ? k + row : row, gc = (TALL ? 0 : k) + ch * 8;
            const bool ok = TALL ? (gr < k_hi && gc < p.r) : (gr < p.r && gc < k_hi);
            next[i] = load_chunk<F32>(p.u, mat + int64_t(gr) * p.cols + gc, ok);
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
    if (k_lo < k_hi) fetch(k_lo);
    for (int k = k_lo; k < k_hi; k += KS) {
        put(buf);
        __syncthreads();
        if (k + KS < k_hi) fetch(k + KS);
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
    }
    float *out = p.gram + (int64_t(blockIdx.y) * p.shares + blockIdx.x) * RP * RP;
    const int g = (tid & 31) >> 2, t = tid & 3;
    if constexpr (WK > 1) {
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
            }
        __syncthreads();
        for (int i = tid; i < RP * RP; i += OR_THREADS) {
            float s = 0.0f;
            for (int w = 0; w < WK; ++w) s += reinterpret_cast<float *>(smem)[w * RP * RP + i];
            out[i] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                float *at = out + (m0 + 16 * i + g) * RP + n0 + 8 * j + 2 * t;
                *reinterpret_cast<float2 *>(at) = make_float2(acc[i][j][0], acc[i][j][1]);
                *reinterpret_cast<float2 *>(at + 8 * RP) = make_float2(acc[i][j][2], acc[i][j][3]);
            }
    }
}

// ---------------------------------------------------------------- iterate

// C = A B for symmetric A, each thread an E x E block: sum over k of rows k
// of A and B.
template <int RP, int E>
__device__ __forceinline__ void mul(const float *A, const float *B, int ty, int tx, float (&c)[E][E])
{
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) c[i][j] = 0.0f;
#pragma unroll 4
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

// One block per matrix; R, P, Q in shared memory.
template <int RP>
__global__ void __launch_bounds__(OR_THREADS) iterate_kernel(const OrthoArgs p)
{
    constexpr int E = RP / 16;
    extern __shared__ __align__(128) float sm[];
    float *R = sm, *P = R + RP * RP, *Q = P + RP * RP;
    __shared__ float s_norm;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    pdl_wait();
    pdl_launch_dependents();
    const float *gram = p.gram + int64_t(blockIdx.x) * p.shares * RP * RP;
    for (int i = tid; i < RP * RP; i += OR_THREADS) {
        float s = 0.0f;
        for (int q = 0; q < p.shares; ++q) s += gram[int64_t(q) * RP * RP + i];
        R[i] = s;
        P[i] = i / RP == i % RP ? 1.0f : 0.0f;
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
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) to[(ty * E + i) * RP + tx * E + j] = c[i][j];
        __syncthreads();
    };
    for (int step = 0; step < p.steps; ++step) {
        mul<RP, E>(R, R, ty, tx, c);
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int y = ty * E + i, x = tx * E + j;
                c[i][j] = fmaf(p.c, c[i][j], fmaf(p.b, R[y * RP + x], y == x ? p.a : 0.0f));
            }
        store(Q);
        mul<RP, E>(Q, P, ty, tx, c);
        store(P);
        if (step + 1 < p.steps) {
            mul<RP, E>(Q, R, ty, tx, c);
            store(R);
            mul<RP, E>(R, Q, ty, tx, c);
            store(R);
        }
    }
    uint16_t *out = p.p + int64_t(blockIdx.x) * 2 * RP * RP;
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

// Block (tile group, matrix): P in shared memory, then tiles of U: out = P U
// (or U P, TALL; P is symmetric).
template <int RP, bool TALL, bool F32>
__global__ void __launch_bounds__(OR_THREADS) apply_kernel(const OrthoArgs p)
{
    constexpr int ROWS = TALL ? OR_LONG : RP, COLS = TALL ? RP : OR_LONG;
    constexpr int CPR = COLS / 8, PCPR = RP / 8;
    constexpr int TILE = RP * OR_LONG * 2;
    constexpr int PER = ROWS * CPR / OR_THREADS;
    // warps over the [ROWS x COLS] output
    constexpr int WM = TALL ? 8 : (RP >= 64 ? 4 : RP / 16), WN = 8 / WM;
    constexpr int MI = ROWS / WM / 16, NI = COLS / WN / 8;
    static_assert(PER >= 1 && MI >= 1 && NI >= 2, "shape");
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *s_u = smem + 2 * RP * RP * 2;
    const uint32_t sp = smem_addr(smem), su = smem_addr(s_u);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int m0 = warp % WM * (ROWS / WM), n0 = warp / WM * (COLS / WN);
    pdl_wait();
    pdl_launch_dependents();
    const uint4 *gp = reinterpret_cast<const uint4 *>(p.p + int64_t(blockIdx.y) * 2 * RP * RP);
    for (int i = tid; i < 2 * RP * PCPR; i += OR_THREADS) {
        const int term = i / (RP * PCPR), c = i % (RP * PCPR);
        *reinterpret_cast<uint4 *>(smem + term * RP * RP * 2 + tile_at<PCPR, RP>(c / PCPR, c % PCPR)) = gp[i];
    }
    const int64_t mat = int64_t(blockIdx.y) * p.rows * p.cols;
    const int tiles = (p.n + OR_LONG - 1) / OR_LONG;
    Chunk<F32> next[PER];
    auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = tid + i * OR_THREADS, row = c / CPR, ch = c % CPR;
            const int gr = TALL ? tile * OR_LONG + row : row;
            const int gc = (TALL ? 0 : tile * OR_LONG) + ch * 8;
            next[i] = load_chunk<F32>(p.u, mat + int64_t(gr) * p.cols + gc, gr < p.rows && gc < p.cols);
        }
    };
    if (blockIdx.x < unsigned(tiles)) fetch(blockIdx.x);
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = tid + i * OR_THREADS;
            uint8_t *at = s_u + tile_at<CPR, ROWS>(c / CPR, c % CPR);
            *reinterpret_cast<uint4 *>(at) = next[i].hi;
            if constexpr (F32) *reinterpret_cast<uint4 *>(at + TILE) = next[i].lo;
        }
        __syncthreads();
        if (tile + int(gridDim.x) < tiles) fetch(tile + gridDim.x);
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
    int r, n, rp, shares, share;
    int64_t gram, p, bytes;
};

static OrthoLayout ortho_layout(int32_t count, int32_t rows, int32_t cols, int sms)
{
    OrthoLayout l;
    l.r = rows <= cols ? rows : cols;
    l.n = rows <= cols ? cols : rows;
    l.rp = 16;
    while (l.rp < l.r) l.rp *= 2;
    const int step = l.rp == 128 ? gram_step<128>() : l.rp == 64 ? gram_step<64>() : gram_step<32>();
    // About four blocks an SM over all matrices, but no share shorter than
    // 16 rp elements: its RP x RP partial sum is written and read again.
    int64_t shares = (int64_t(4) * sms + count - 1) / count;
    const int64_t most = (l.n + 16 * l.rp - 1) / (16 * l.rp);
    if (shares > most) shares = most;
    if (shares < 1) shares = 1;
    int64_t share = (l.n + shares - 1) / shares;
    share = (share + step - 1) / step * step;
    l.share = int(share);
    l.shares = int((l.n + share - 1) / share);
    l.gram = 0;
    l.p = int64_t(count) * l.shares * l.rp * l.rp * 4;
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
    e = launch_kernel(gram_kernel<RP, TALL, F32>, dim3(p.shares, p.count), dim3(OR_THREADS), gs, st, p);
    if (e != cudaSuccess) return int(e);
    e = launch_kernel(iterate_kernel<RP>, dim3(p.count), dim3(OR_THREADS), is, st, p);
    if (e != cudaSuccess) return int(e);
    // each block loads P once: two tiles or more a block where there are enough
    const int tiles = (p.n + OR_LONG - 1) / OR_LONG;
    int groups = (8 * device_sm_count() + p.count - 1) / p.count;
    if (groups > tiles) groups = tiles;
    e = launch_kernel(apply_kernel<RP, TALL, F32>, dim3(groups, p.count), dim3(OR_THREADS), as, st, p);
    return e == cudaSuccess ? LORA_OK : int(e);
}

template <bool TALL, bool F32>
static int run_ortho_rank(const OrthoArgs &p, int rp, cudaStream_t st)
{
    switch (rp) {
    case 16: return run_ortho<16, TALL, F32>(p, st);
    case 32: return run_ortho<32, TALL, F32>(p, st);
    case 64: return run_ortho<64, TALL, F32>(p, st);
    default: return run_ortho<128, TALL, F32>(p, st);
    }
}

static bool ortho_sizes_ok(int32_t count, int32_t rows, int32_t cols)
{
    // count is a grid's second dimension
    return count >= 0 && count <= 65535 && rows >= 1 && cols >= 8 && cols % 8 == 0 &&
           (rows <= OR_MAX_RANK || cols <= OR_MAX_RANK);
}

}  // namespace lora

LORA_API int64_t lora_orthogonalize_workspace(int32_t count, int32_t rows, int32_t cols)
{
    if (!lora::ortho_sizes_ok(count, rows, cols)) return LORA_ERR_SIZE;
    return lora::ortho_layout(count > 0 ? count : 1, rows, cols, lora::device_sm_count()).bytes;
}

LORA_API int lora_orthogonalize(const void *update, int32_t update_f32, int32_t count, int32_t rows,
                                int32_t cols, int32_t steps, float coef_a, float coef_b,
                                float coef_c, float eps, float scale, lora_bf16_t *out,
                                void *workspace, int64_t workspace_bytes, void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_orthogonalize");
    if (!ortho_sizes_ok(count, rows, cols) || steps < 1) return LORA_ERR_SIZE;
    if (count == 0) return LORA_OK;
    if (update == nullptr || out == nullptr || workspace == nullptr) return LORA_ERR_NULL;
    auto bits = [](const void *ptr) { return reinterpret_cast<uintptr_t>(ptr); };
    if ((bits(update) | bits(out)) & 15u || bits(workspace) & 255u) return LORA_ERR_ALIGN;
    const OrthoLayout l = ortho_layout(count, rows, cols, device_sm_count());
    if (workspace_bytes < l.bytes) return LORA_ERR_WORKSPACE;
    OrthoArgs p;
    p.u = update;
    p.out = out;
    p.count = count;
    p.rows = rows;
    p.cols = cols;
    p.r = l.r;
    p.n = l.n;
    p.shares = l.shares;
    p.share = l.share;
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
    if (update_f32)
        return tall ? run_ortho_rank<true, true>(p, l.rp, st) : run_ortho_rank<false, true>(p, l.rp, st);
    return tall ? run_ortho_rank<true, false>(p, l.rp, st) : run_ortho_rank<false, false>(p, l.rp, st);
}
