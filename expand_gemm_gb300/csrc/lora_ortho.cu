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
// The errors of R grow by a^2 a step in directions that U lacks, so where
// |a|^steps is above 512 the sum is taken afresh every few steps
// (lora_ortho_long.cu).
//
// This file: ranks up to 32, on mma.sync, the steps in FFMA.
// lora_ortho_tc.cu: ranks 33 to 128, on tcgen05 (whose tiles of 64 cost rank
// 32 twice the time: 64 matrices of 11008 x 32 58 us here, 137 there; 8 of
// 16 x 4096 13 and 46).
//
// Bound by HBM above a few MB: 64 matrices of 11008 x 32 in fp32 (135 MB)
// take 24 us in gram_kernel (3.7 TB/s), 12 in iterate_kernel, 22 in
// apply_kernel (6.2 TB/s); below, by three launches in a row.
#include <math.h>

#include <type_traits>

#include "lora_ortho.cuh"

namespace lora {

// ---------------------------------------------------------------- rings
//
// Every warp works by itself on its part of a tile of U, so that no barrier
// of the block stands in the loops.  Its 16-byte pieces come by cp.async,
// several tiles ahead, neighbouring lanes copying neighbouring pieces (a
// lane copying both halves of its eight fp32 entries halved the rate: every
// 32-byte sector was asked for twice).  A bf16 tile lands swizzled, ready
// for ldmatrix.  SPLIT_ROWS: a warp's part is an eighth of the tile's rows,
// else of its columns.

// A walk over the tiles of the stacked matrices, without divisions in the
// loop (64-bit ones took half of its instructions).
struct TileWalk {
    int64_t left;             // tiles still to come
    int64_t mat;              // first element of the matrix
    int m, k;                 // matrix, tile in it
    __device__ __forceinline__ TileWalk(int64_t first, int64_t end, int per, int64_t size)
        : left(end - first), m(int(first / per)), k(int(first % per))
    {
        mat = m * size;
    }
    __device__ __forceinline__ void next(int per, int64_t size)
    {
        --left;
        if (++k == per) {
            k = 0;
            ++m;
            mat += size;
        }
    }
};

template <int ROWS, int CPR, bool SPLIT_ROWS>
struct TileRing {
    static constexpr int PER = ROWS * CPR / OR_THREADS;            // chunks of a lane
    static constexpr int BYTES = ROWS * CPR * 16;
    static_assert(PER >= 1 && (SPLIT_ROWS ? ROWS : CPR) % 8 == 0, "an eighth a warp");

    __device__ __forceinline__ static void place(int i, int &row, int &ch)
    {
        const int warp = threadIdx.x >> 5, at = (threadIdx.x & 31) + 32 * i;
        if constexpr (SPLIT_ROWS) {
            row = warp * (ROWS / 8) + at / CPR;
            ch = at % CPR;
        } else {
            row = at / (CPR / 8);
            ch = warp * (CPR / 8) + at % (CPR / 8);
        }
    }
    __device__ __forceinline__ static void issue(const OrthoArgs &p, uint8_t *stage, int64_t mat, int row0,
                                                 int col0)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            int r, ch;
            place(i, r, ch);
            const int row = row0 + r, col = col0 + ch * 8;
            const bool ok = row < p.rows && col < p.cols;
            cp_async16(smem_addr(stage + tile_at<CPR, ROWS>(r, ch)),
                       static_cast<const uint16_t *>(p.u) + (ok ? mat + int64_t(row) * p.cols + col : 0), ok);
        }
    }
};

// An fp32 tile; a warp's part of it has ROWS rows of PPR 16-byte pieces.
// Fragments are read from it as they are and split in registers: split in
// shared memory and read with ldmatrix, a 16 x 32 block took 64 passes over
// the banks in place of 16 (64 matrices of 11008 x 32: gram 38 us in place
// of 24, apply 30 in place of 22).  K_ROWS: the rows are K.  The pieces lie
// so that the lanes of one load meet no bank twice.
template <int ROWS, int PPR, bool SPLIT_ROWS, bool K_ROWS>
struct FloatRing {
    static constexpr int PART = ROWS * PPR * 16, BYTES = 8 * PART;
    static constexpr int PER = ROWS * PPR / 32;                    // pieces of a lane
    __device__ __forceinline__ static int spot(int row, int ch)
    {
        if constexpr (K_ROWS && PPR == 8) return row * 8 + (ch ^ (row & 6));
        else if constexpr (K_ROWS) return ((row >> 1) + (row & 1) * (ROWS / 2)) * 4 + (ch ^ (row >> 1 & 2));
        else if constexpr (PPR == 8) return row * 8 + (ch ^ (row & 3) << 1);
        else return row * 4 + (ch ^ (row & 2));
    }
    __device__ __forceinline__ static void issue(const OrthoArgs &p, uint8_t *stage, int64_t mat, int row0,
                                                 int col0)
    {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = (lane + 32 * i) / PPR, ch = (lane + 32 * i) % PPR;
            const int row = row0 + (SPLIT_ROWS ? warp * ROWS : 0) + r;
            const int col = col0 + (SPLIT_ROWS ? 0 : warp * PPR * 4) + ch * 4;
            const bool ok = row < p.rows && col < p.cols;
            cp_async16(smem_addr(stage + warp * PART + spot(r, ch) * 16),
                       static_cast<const float *>(p.u) + (ok ? mat + int64_t(row) * p.cols + col : 0), ok);
        }
    }
    // The 16 x 16 block at (m0, k0) of the warp's part as an A fragment, two
    // terms.  As B it is the same registers: [h], [h + 2] for columns 8 h on.
    __device__ __forceinline__ static void frag(const uint8_t *part, int m0, int k0, uint32_t (&hi)[4],
                                                uint32_t (&lo)[4])
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = m0 + g + 8 * (q & 1), k = k0 + 2 * t + 8 * (q >> 1);
            float x, y;
            if constexpr (K_ROWS) {
                x = *reinterpret_cast<const float *>(part + spot(k, m >> 2) * 16 + (m & 3) * 4);
                y = *reinterpret_cast<const float *>(part + spot(k + 1, m >> 2) * 16 + (m & 3) * 4);
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(part + spot(m, k >> 2) * 16 + (k & 3) * 4);
                x = v.x;
                y = v.y;
            }
            hi[q] = pack_bf16x2(x, y);
            lo[q] = pack_bf16x2(x - bf16_lo(hi[q]), y - bf16_hi(hi[q]));
        }
    }
};

// ---------------------------------------------------------------- gram

template <int RP>
constexpr int gram_step() { return 4096 / RP; }     // of the long side, a tile of 4096 entries

template <bool F32>
constexpr int gram_stages() { return F32 ? 4 : 5; }

template <int RP, bool F32>
constexpr int gram_smem() { return 4096 * gram_stages<F32>() * (F32 ? 4 : 2) + RP * RP * 4; }

// Each block sums over its run of units; a warp takes an eighth of a unit's
// K, the 8-column blocks on and right of the diagonal.  TALL: U is [n][r]
// (its rows are K), else [r][n].
template <int RP, bool TALL, bool F32>
__global__ void __launch_bounds__(OR_THREADS, 3) gram_kernel(const OrthoArgs p)
{
    constexpr int KS = gram_step<RP>(), ST = gram_stages<F32>();
    constexpr int ROWS = TALL ? KS : RP, CPR = (TALL ? RP : KS) / 8;     // of the tile
    constexpr int MI = RP / 16, NI = RP / 8;
    using Ring = std::conditional_t<F32, FloatRing<TALL ? KS / 8 : RP, (TALL ? RP : KS / 8) / 4, TALL, TALL>,
                                    TileRing<ROWS, CPR, TALL>>;
    extern __shared__ __align__(128) uint8_t smem[];
    float *sum = reinterpret_cast<float *>(smem + ST * Ring::BYTES);
    const int tid = threadIdx.x, warp = tid >> 5;
    pdl_wait();
    const int64_t first = unit_begin(p, blockIdx.x), end = unit_begin(p, blockIdx.x + 1);
    const int64_t size = int64_t(p.rows) * p.cols;
    TileWalk in(first, end, p.units, size), run(first, end, p.units, size);
    auto issue = [&](int stage) {
        if (in.left > 0) {
            Ring::issue(p, smem + stage * Ring::BYTES, in.mat, TALL ? in.k * KS : 0, TALL ? 0 : in.k * KS);
            in.next(p.units, size);
        }
        cp_async_commit();
    };
    float acc[MI][NI][4] = {};
    for (int i = 0; i < ST - 1; ++i) issue(i);
    int stage = 0;
    for (; run.left > 0; run.next(p.units, size)) {
        cp_async_wait<ST - 2>();
        const uint8_t *tile = smem + stage * Ring::BYTES;
        __syncwarp();
        issue(stage == 0 ? ST - 1 : stage - 1);
        stage = stage + 1 == ST ? 0 : stage + 1;
        // the rows of B are those of A, so its fragments are A's registers
#pragma unroll
        for (int kk = 0; kk < KS / 8; kk += 16) {
            uint32_t a[MI][4], al[MI][4];
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if constexpr (F32) Ring::frag(tile + warp * Ring::PART, 16 * i, kk, a[i], al[i]);
                else frag_a<CPR, ROWS, !TALL>(smem_addr(tile), 16 * i, warp * (KS / 8) + kk, a[i]);
            }
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = i; j < MI; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float(&d)[4] = acc[i][2 * j + h];
                        mma_bf16_16816(d, a[i], a[j][h], a[j][h + 2]);
                        if constexpr (F32) {
                            mma_bf16_16816(d, al[i], a[j][h], a[j][h + 2]);
                            mma_bf16_16816(d, a[i], al[j][h], al[j][h + 2]);
                        }
                    }
        }
        if (run.left > 1 && run.k + 1 != p.units) continue;
        // the matrix or the run ends: the warps' sums over K, one after the
        // other; what lies left of the diagonal is the mirror image
        const int g = (tid & 31) >> 2, t = tid & 3;
        for (int w = 0; w < 8; ++w) {
            if (warp == w) {
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int j = 2 * i; j < NI; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float2 *at = reinterpret_cast<float2 *>(sum + (16 * i + g + 8 * h) * RP + 8 * j + 2 * t);
                            const float2 was = w > 0 ? *at : make_float2(0.0f, 0.0f);
                            *at = make_float2(was.x + acc[i][j][2 * h], was.y + acc[i][j][2 * h + 1]);
                            acc[i][j][2 * h] = acc[i][j][2 * h + 1] = 0.0f;
                        }
            }
            __syncthreads();
        }
        float *out = p.gram + (int64_t(blockIdx.x) + run.m) * RP * RP;
        for (int i = tid; i < RP * RP; i += OR_THREADS) {
            const int y = i / RP, x = i % RP;
            out[i] = sum[x / 16 < y / 16 ? x * RP + y : i];
        }
        __syncthreads();
    }
    cp_async_wait<0>();
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
#pragma unroll
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
// is their mirror image.  Ranks up to 32; above, the products are long
// enough for the tensor cores: five steps at rank 32 take 12 us here and 29
// in lora_ortho_tc.cu, at rank 40 59 here and 27 there.
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
    const int lo = unit_cta(p, int64_t(m) * p.units), hi = unit_cta(p, int64_t(m + 1) * p.units - 1);
    // a matrix's slots, all of a thread's loads under way at once
    if (tid < RP * RP / 4) {
        float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 8
        for (int c = lo; c <= hi; ++c) {
            const float4 x = reinterpret_cast<const float4 *>(p.gram + int64_t(c + m) * RP * RP)[tid];
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
        }
        reinterpret_cast<float4 *>(R)[tid] = v;
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

template <bool F32>
constexpr int apply_stages() { return F32 ? 3 : 4; }

// P's terms, the ring, and a tile that holds the converted terms (fp32) and
// then the output.
template <int RP, bool F32>
constexpr int apply_smem()
{
    return 2 * RP * RP * 2 + RP * OR_LONG * (apply_stages<F32>() * (F32 ? 4 : 2) + 2);
}

// Each block takes a run of tiles of the stacked matrices: out = P U (or U
// P, TALL; P is symmetric).  A warp takes 16 of a tile's 128 long-side
// elements, from load to store; P's fragments stay in its registers.
template <int RP, bool TALL, bool F32>
__global__ void __launch_bounds__(OR_THREADS, 3) apply_kernel(const OrthoArgs p)
{
    constexpr int ROWS = TALL ? OR_LONG : RP, COLS = TALL ? RP : OR_LONG;
    constexpr int CPR = COLS / 8, PCPR = RP / 8, ST = apply_stages<F32>();
    constexpr int MI = TALL ? 1 : RP / 16, NI = TALL ? RP / 8 : 2, KK = RP / 16;
    using Out = TileRing<ROWS, CPR, TALL>;
    using Ring = std::conditional_t<F32, FloatRing<TALL ? 16 : RP, TALL ? RP / 4 : 4, TALL, !TALL>, Out>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *ring = smem + 2 * RP * RP * 2, *tile_buf = ring + ST * Ring::BYTES;
    const uint32_t sp = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int m0 = TALL ? warp * 16 : 0, n0 = TALL ? 0 : warp * 16;
    pdl_wait();
    const int tiles = (p.n + OR_LONG - 1) / OR_LONG;
    const int64_t total = int64_t(p.count) * tiles;
    const int64_t first = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
    const int64_t size = int64_t(p.rows) * p.cols;
    TileWalk in(first, end, tiles, size), run(first, end, tiles, size);
    auto issue = [&](int stage) {
        if (in.left > 0) {
            const int n = in.k * OR_LONG;
            Ring::issue(p, ring + stage * Ring::BYTES, in.mat, TALL ? n : 0, TALL ? 0 : n);
            in.next(tiles, size);
        }
        cp_async_commit();
    };
    for (int i = 0; i < ST - 1; ++i) issue(i);
    int held = -1, stage = 0;
    uint32_t pf[2][KK][RP / 16][4];        // P: terms, K steps, 16 rows (or columns) each
    for (; run.left > 0; run.next(tiles, size)) {
        const int m = run.m, tile = run.k;
        if (m != held) {
            __syncthreads();
            const uint4 *gp = reinterpret_cast<const uint4 *>(p.p + int64_t(m) * 2 * RP * RP);
            for (int i = tid; i < 2 * RP * PCPR; i += OR_THREADS) {
                const int term = i / (RP * PCPR), c = i % (RP * PCPR);
                *reinterpret_cast<uint4 *>(smem + term * RP * RP * 2 +
                                           tile_at<PCPR, RP>(c / PCPR, c % PCPR)) = gp[i];
            }
            __syncthreads();
            held = m;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < RP / 16; ++i) {
                        if constexpr (TALL) frag_b<PCPR, RP, true>(sp + t * RP * RP * 2, 16 * k, 16 * i, pf[t][k][i]);
                        else frag_a<PCPR, RP, true>(sp + t * RP * RP * 2, 16 * i, 16 * k, pf[t][k][i]);
                    }
        }
        cp_async_wait<ST - 2>();
        __syncwarp();                          // and the last tile's output has left
        const uint8_t *u_tile = ring + stage * Ring::BYTES;
        issue(stage == 0 ? ST - 1 : stage - 1);
        stage = stage + 1 == ST ? 0 : stage + 1;
        float acc[MI][NI][4] = {};
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            uint32_t u[2][4];                  // U's terms
            if constexpr (F32) {
                Ring::frag(u_tile + warp * Ring::PART, 0, 16 * k, u[0], u[1]);
            } else if constexpr (TALL) {
                frag_a<CPR, ROWS, true>(smem_addr(u_tile), m0, 16 * k, u[0]);
            } else {
                uint32_t b[4];
                frag_b<CPR, ROWS, false>(smem_addr(u_tile), 16 * k, n0, b);
                u[0][0] = b[0];
                u[0][2] = b[1];
                u[0][1] = b[2];
                u[0][3] = b[3];
            }
#pragma unroll
            for (int ut = 0; ut < (F32 ? 2 : 1); ++ut)
#pragma unroll
                for (int t = 0; t < (ut == 0 ? 2 : 1); ++t)
#pragma unroll
                    for (int i = 0; i < RP / 16; ++i) {
                        const uint32_t(&q)[4] = pf[t][k][i];
                        if constexpr (TALL) {
                            mma_bf16_16816(acc[0][2 * i], u[ut], q[0], q[1]);
                            mma_bf16_16816(acc[0][2 * i + 1], u[ut], q[2], q[3]);
                        } else {
                            mma_bf16_16816(acc[i][0], q, u[ut][0], u[ut][2]);
                            mma_bf16_16816(acc[i][1], q, u[ut][1], u[ut][3]);
                        }
                    }
        }
        // through the warp's part of the tile, so that rows are written 16
        // bytes at a time
        __syncwarp();
        const int g = (tid & 31) >> 2, t = tid & 3;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int row = m0 + 16 * i + g, col = n0 + 8 * j + 2 * t;
                *reinterpret_cast<uint32_t *>(tile_buf + tile_at<CPR, ROWS>(row, col / 8) + col % 8 * 2) =
                    pack_bf16x2(acc[i][j][0], acc[i][j][1]);
                *reinterpret_cast<uint32_t *>(tile_buf + tile_at<CPR, ROWS>(row + 8, col / 8) + col % 8 * 2) =
                    pack_bf16x2(acc[i][j][2], acc[i][j][3]);
            }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < Out::PER; ++i) {
            int row, ch;
            Out::place(i, row, ch);
            const int gr = TALL ? tile * OR_LONG + row : row;
            const int gc = (TALL ? 0 : tile * OR_LONG) + ch * 8;
            if (gr < p.rows && gc < p.cols)
                *reinterpret_cast<uint4 *>(p.out + run.mat + int64_t(gr) * p.cols + gc) =
                    *reinterpret_cast<const uint4 *>(tile_buf + tile_at<CPR, ROWS>(row, ch));
        }
    }
    cp_async_wait<0>();
}

// ---------------------------------------------------------------- host

struct OrthoLayout {
    int r, n, rp, unit, units, ctas;
    int64_t p, bytes;
};

constexpr int OR_BLOCKS = 3;              // of gram_kernel and apply_kernel on an SM

// The sum U U^T is cut into units of one tile each and those into as many
// runs as blocks fit the GPU at once, but not so many that a matrix has more
// parts than about the root of its units (at least four): the next kernel's
// one block a matrix reads them all.
static OrthoLayout ortho_layout(int32_t count, int32_t rows, int32_t cols, int sms)
{
    OrthoLayout l;
    l.r = rows <= cols ? rows : cols;
    l.n = rows <= cols ? cols : rows;
    l.rp = 16;
    while (l.rp < l.r) l.rp *= 2;
    l.unit = l.rp >= 64 ? OR_TC_UNIT : l.rp == 32 ? gram_step<32>() : gram_step<16>();
    l.units = (l.n + l.unit - 1) / l.unit;
    int parts = 4;
    while (int64_t(parts) * parts < l.units) ++parts;
    int64_t most = int64_t(sms) * (l.rp >= 64 ? OR_TC_CTAS : OR_BLOCKS);
    if (int64_t(count) * parts < most) most = int64_t(count) * parts;
    const int64_t total = int64_t(count) * l.units;
    l.ctas = int(total < most ? total : most);
    l.p = (int64_t(l.ctas) + count) * l.rp * l.rp * 4;
    l.bytes = l.p + int64_t(count) * 2 * l.rp * l.rp * 2;
    // a long run of steps takes its matrices by groups: one must fit
    const int64_t one = ortho_long_bytes(l.r, l.n, l.rp);
    if (l.bytes < one) l.bytes = one;
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
    constexpr int gs = gram_smem<RP, F32>(), as = apply_smem<RP, F32>();
    constexpr int is = 3 * RP * RP * 4;
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    if (dev >= 64 || !configured[dev]) {
        if ((e = allow_smem(gram_kernel<RP, TALL, F32>, gs)) != cudaSuccess ||
            (e = allow_smem(apply_kernel<RP, TALL, F32>, as)) != cudaSuccess)
            return int(e);
        if (dev < 64) configured[dev] = 1;
    }
    e = launch_kernel(gram_kernel<RP, TALL, F32>, dim3(p.ctas), dim3(OR_THREADS), gs, st, p);
    if (e != cudaSuccess) return int(e);
    e = launch_kernel(iterate_kernel<RP>, dim3(p.count), dim3(OR_THREADS), is, st, p);
    if (e != cudaSuccess) return int(e);
    const int64_t tiles = int64_t(p.count) * ((p.n + OR_LONG - 1) / OR_LONG);
    const int64_t most = int64_t(device_sm_count()) * OR_BLOCKS;
    e = launch_kernel(apply_kernel<RP, TALL, F32>, dim3(unsigned(tiles < most ? tiles : most)),
                      dim3(OR_THREADS), as, st, p);
    return e == cudaSuccess ? LORA_OK : int(e);
}

static bool ortho_sizes_ok(int32_t count, int32_t rows, int32_t cols)
{
    return count >= 0 && rows >= 1 && cols >= 8 && cols % 8 == 0 && (rows <= OR_MAX_RANK || cols <= OR_MAX_RANK);
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
                                int32_t *error_word, void *workspace, int64_t workspace_bytes, void *stream)
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
    if (pow(fabs(double(coef_a)), double(steps)) > OR_LONG_GROWTH)
        return run_ortho_long(p, l.rp, update_f32 != 0, workspace, workspace_bytes, st);
    if (l.rp >= 64) return run_ortho_tc(p, l.rp, update_f32 != 0, st);
    if (l.rp == 16) {
        if (update_f32) return tall ? run_ortho<16, true, true>(p, st) : run_ortho<16, false, true>(p, st);
        return tall ? run_ortho<16, true, false>(p, st) : run_ortho<16, false, false>(p, st);
    }
    if (update_f32) return tall ? run_ortho<32, true, true>(p, st) : run_ortho<32, false, true>(p, st);
    return tall ? run_ortho<32, true, false>(p, st) : run_ortho<32, false, false>(p, st);
}
