// lora_ortho_long.cu -- lora_orthogonalize for long runs of steps.
//
// The r x r iteration of lora_ortho.cu holds R = X X^T with errors of about
// 2^-24 of its largest eigenvalue.  In directions that U lacks R's eigenvalue
// is that error alone, of either sign, and a step multiplies it by a^2: with
// a = 3.4445 it is 0.01 after five steps and above 1 after seven, where a
// negative one grows without bound (updates of rank 8 in 32 x 1024, fp32:
// off by 0.0007 of the norm after five steps, 0.012 after seven, 6 times the
// norm after eight).  A sum X X^T taken afresh has no such eigenvalue.
//
// So where |a|^steps passes OR_LONG_GROWTH the steps are cut into short runs
// (growth up to OL_RUN_GROWTH: three steps of 3.4445, whose error stays below
// 1e-5), and after each run X = P X is formed and X X^T summed again, in fp32
// throughout (FFMA): what errors of X grow by is then a a step, as they do in
// the iteration on X itself.  A group of matrices at a time, as many as the
// workspace holds in fp32, one at least:
//   gram_long_kernel   partial sums of X X^T over chunks of the long side;
//   steps_long_kernel  the run's steps on r x r matrices, a block a matrix;
//   apply_long_kernel  X <- P X, 64 of the long side a block, in place.
// A form for being right: bound by FFMA and loads that nothing overlaps.  Six
// steps, all matrices in one group: 192 matrices of 128 x 8192 12.7 ms (16
// TFLOP/s), 64 of 11008 x 32 430 us, 8 of 16 x 4096 40 us (five steps on r x r
// matrices alone: 326, 57 and 13 us).
#include <math.h>

#include "lora_ortho.cuh"

namespace lora {

constexpr double OL_RUN_GROWTH = 64.0;    // |a|^steps of a run
constexpr int OL_K = 32;                  // of the long side, a tile of gram_long_kernel
constexpr int OL_COLS = 64;               // of the long side, a tile of apply_long_kernel
constexpr int OL_LD = OL_COLS + 4;        // floats of a row of that tile
constexpr int OL_MAX_CHUNKS = 32;

struct LongArgs {
    OrthoArgs o;
    const void *src;                      // U in the first run, then x
    int32_t src_f32;
    float *x;                             // [group][rows][cols]
    float *part;                          // [group][chunks][RP][RP]
    float *p;                             // [group][RP][RP]: the run's polynomial
    int32_t chunks, chunk;                // of the long side; a chunk's length, a multiple of OL_K
    int32_t steps, first, last;           // of this run; whether it is the first, the last
    uint16_t *out;                        // of the group
};

__device__ __forceinline__ float long_entry(const LongArgs &p, int64_t at)
{
    return p.src_f32 ? static_cast<const float *>(p.src)[at] : bf16_to_f32(static_cast<const uint16_t *>(p.src)[at]);
}

// Where entry (i of the short side, j of the long one) lies.
__device__ __forceinline__ int64_t long_at(const OrthoArgs &o, int64_t mat, int i, int64_t j)
{
    return o.rows > o.cols ? mat + j * o.cols + i : mat + int64_t(i) * o.cols + j;
}

// E consecutive floats.
template <int E>
__device__ __forceinline__ void load_e(const float *at, float (&v)[E])
{
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(at + i);
            v[i] = x.x;
            v[i + 1] = x.y;
            v[i + 2] = x.z;
            v[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = at[i];
    }
}

// Thread's block of A^T B over rows [0, K): rows k of A from column i0, of B
// from column j0.
template <int K, int EI, int EJ>
__device__ __forceinline__ void outer(const float *A, int lda, int i0, const float *B, int ldb, int j0,
                                      float (&acc)[EI][EJ])
{
#pragma unroll
    for (int i = 0; i < EI; ++i)
#pragma unroll
        for (int j = 0; j < EJ; ++j) acc[i][j] = 0.0f;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float a[EI], b[EJ];
        load_e(A + k * lda + i0, a);
        load_e(B + k * ldb + j0, b);
#pragma unroll
        for (int i = 0; i < EI; ++i)
#pragma unroll
            for (int j = 0; j < EJ; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
}

// Block (chunk, matrix); thread (ty, tx) holds an E x E block of X X^T.  A
// tile's sum is added to the chunk's, so that few terms meet a long sum.
template <int RP>
__global__ void __launch_bounds__(OR_THREADS) gram_long_kernel(const LongArgs p)
{
    constexpr int E = RP / 16, LD = RP + 4;
    __shared__ __align__(16) float tile[OL_K * LD];
    const OrthoArgs &o = p.o;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const bool tall = o.rows > o.cols;
    pdl_wait();
    const int64_t mat = int64_t(blockIdx.y) * o.rows * o.cols;
    const int64_t j_end = min(int64_t(o.n), (int64_t(blockIdx.x) + 1) * p.chunk);
    float sum[E][E] = {};
    for (int64_t j0 = int64_t(blockIdx.x) * p.chunk; j0 < j_end; j0 += OL_K) {
#pragma unroll
        for (int e = tid; e < OL_K * RP; e += OR_THREADS) {
            const int i = tall ? e % RP : e / OL_K, k = tall ? e / RP : e % OL_K;
            tile[k * LD + i] = i < o.r && j0 + k < j_end ? long_entry(p, long_at(o, mat, i, j0 + k)) : 0.0f;
        }
        __syncthreads();
        float acc[E][E];
        outer<OL_K>(tile, LD, ty * E, tile, LD, tx * E, acc);
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) sum[i][j] += acc[i][j];
        __syncthreads();
    }
    float *out = p.part + (int64_t(blockIdx.y) * p.chunks + blockIdx.x) * RP * RP;
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) out[(ty * E + i) * RP + tx * E + j] = sum[i][j];
}

template <int RP>
constexpr int steps_long_smem() { return 3 * RP * RP * 4; }

// R = X X^T (of the first run f^2 U U^T, f = 1 / (|U|_F + eps)), then the
// run's steps Q = a I + b R + c R^2, P <- Q P, R <- Q R Q.  f enters P in the
// first run, the scale in the last.  R, P and Q stay symmetric: what lies
// below the diagonal is the mirror image.
template <int RP>
__global__ void __launch_bounds__(OR_THREADS) steps_long_kernel(const LongArgs p)
{
    constexpr int E = RP / 16;
    extern __shared__ __align__(16) float sm[];
    float *R = sm, *P = R + RP * RP, *Q = P + RP * RP;
    __shared__ float s_f;
    const OrthoArgs &o = p.o;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    pdl_wait();
    const float *part = p.part + int64_t(blockIdx.x) * p.chunks * RP * RP;
    for (int i = tid; i < RP * RP; i += OR_THREADS) {
        float s = 0.0f;
        for (int c = 0; c < p.chunks; ++c) s += part[int64_t(c) * RP * RP + i];
        R[i] = s;
    }
    if (tid == 0) s_f = 1.0f;
    __syncthreads();
    if (p.first) {
        if (tid < 32) {
            float s = 0.0f;
            for (int i = tid; i < RP; i += 32) s += R[i * RP + i];
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (tid == 0) s_f = 1.0f / (sqrtf(s) + o.eps);
        }
        __syncthreads();
        for (int i = tid; i < RP * RP; i += OR_THREADS) R[i] = R[i] * s_f * s_f;
        __syncthreads();
    }
    float acc[E][E];
    auto store = [&](float *to) {
        __syncthreads();                      // every read of `to` is done
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int y = ty * E + i, x = tx * E + j;
                if (y <= x) to[y * RP + x] = to[x * RP + y] = acc[i][j];
            }
        __syncthreads();
    };
    for (int step = 0; step < p.steps; ++step) {
        outer<RP>(R, RP, ty * E, R, RP, tx * E, acc);
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int y = ty * E + i, x = tx * E + j;
                acc[i][j] = fmaf(o.c, acc[i][j], fmaf(o.b, R[y * RP + x], y == x ? o.a : 0.0f));
            }
        store(Q);
        if (step == 0) {                      // P was the identity
            for (int i = tid; i < RP * RP; i += OR_THREADS) P[i] = Q[i];
            __syncthreads();
        } else {
            outer<RP>(Q, RP, ty * E, P, RP, tx * E, acc);
            store(P);
        }
        if (step + 1 < p.steps) {
            outer<RP>(Q, RP, ty * E, R, RP, tx * E, acc);
            store(R);
            outer<RP>(R, RP, ty * E, Q, RP, tx * E, acc);
            store(R);
        }
    }
    const float f = s_f * (p.last ? o.scale : 1.0f);
    float *out = p.p + int64_t(blockIdx.x) * RP * RP;
    for (int i = tid; i < RP * RP; i += OR_THREADS) out[i] = f * P[i];
}

template <int RP>
constexpr int apply_long_smem() { return (RP * RP + RP * OL_LD) * 4; }

// Block (64 of the long side, matrix): the tile is read whole before any of it
// is written, and is no other block's.
template <int RP>
__global__ void __launch_bounds__(OR_THREADS) apply_long_kernel(const LongArgs p)
{
    constexpr int E = RP / 16, C = OL_COLS / 16;
    extern __shared__ __align__(16) float sm[];
    float *P = sm, *tile = P + RP * RP;       // [RP][RP], [RP][OL_LD]
    const OrthoArgs &o = p.o;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const bool tall = o.rows > o.cols;
    pdl_wait();
    const int64_t mat = int64_t(blockIdx.y) * o.rows * o.cols;
    const int64_t j0 = int64_t(blockIdx.x) * OL_COLS;
#pragma unroll
    for (int e = tid; e < RP * OL_COLS; e += OR_THREADS) {
        const int i = tall ? e % RP : e / OL_COLS, j = tall ? e / RP : e % OL_COLS;
        tile[i * OL_LD + j] = i < o.r && j0 + j < o.n ? long_entry(p, long_at(o, mat, i, j0 + j)) : 0.0f;
    }
    for (int i = tid; i < RP * RP; i += OR_THREADS) P[i] = p.p[int64_t(blockIdx.y) * RP * RP + i];
    __syncthreads();
    float acc[E][C];
    outer<RP>(P, RP, ty * E, tile, OL_LD, tx * C, acc);       // P is symmetric
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
        for (int j = 0; j < C; ++j) tile[(ty * E + i) * OL_LD + tx * C + j] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int e = tid; e < RP * OL_COLS; e += OR_THREADS) {
        const int i = tall ? e % RP : e / OL_COLS, j = tall ? e / RP : e % OL_COLS;
        if (i >= o.r || j0 + j >= o.n) continue;
        const int64_t at = long_at(o, mat, i, j0 + j);
        const float v = tile[i * OL_LD + j];
        if (p.last) p.out[at] = uint16_t(pack_bf16x2(v, 0.0f) & 0xFFFFu);
        else p.x[at] = v;
    }
}

// What one matrix takes of the workspace: X, partial sums, P.
struct LongLayout {
    int chunk, chunks;
    int64_t bytes;
};
static LongLayout long_layout(int r, int n, int rp)
{
    LongLayout l;
    const int most = n / 512 < 1 ? 1 : n / 512 < OL_MAX_CHUNKS ? n / 512 : OL_MAX_CHUNKS;
    l.chunk = ((n - 1) / most / OL_K + 1) * OL_K;
    l.chunks = (n - 1) / l.chunk + 1;
    l.bytes = (int64_t(r) * n + int64_t(l.chunks + 1) * rp * rp) * 4;
    return l;
}

int64_t ortho_long_bytes(int r, int n, int rp) { return long_layout(r, n, rp).bytes; }

template <int RP>
static int run_long(const OrthoArgs &o, bool f32, void *workspace, int64_t bytes, cudaStream_t st)
{
    constexpr int ss = steps_long_smem<RP>(), as = apply_long_smem<RP>();
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    if (dev >= 64 || !configured[dev]) {
        if ((e = cudaFuncSetAttribute(steps_long_kernel<RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, ss)) !=
                cudaSuccess ||
            (e = cudaFuncSetAttribute(apply_long_kernel<RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, as)) !=
                cudaSuccess)
            return int(e);
        if (dev < 64) configured[dev] = 1;
    }
    const LongLayout l = long_layout(o.r, o.n, RP);
    int64_t group = bytes / l.bytes;
    if (group > 65535) group = 65535;         // a grid's y dimension
    if (group > o.count) group = o.count;
    const int64_t size = int64_t(o.rows) * o.cols;
    LongArgs p;
    p.o = o;
    p.chunks = l.chunks;
    p.chunk = l.chunk;
    p.x = static_cast<float *>(workspace);
    p.part = p.x + group * size;
    p.p = p.part + group * l.chunks * RP * RP;
    // even runs of steps, each of growth OL_RUN_GROWTH at most (one at least)
    const double each = log(OL_RUN_GROWTH) / log(fabs(double(o.a)));
    const int run = each < 1.0 ? 1 : each < double(o.steps) ? int(each) : o.steps;
    const int runs = (o.steps - 1) / run + 1;
    for (int64_t m0 = 0; m0 < o.count; m0 += group) {
        const unsigned many = unsigned(group < o.count - m0 ? group : o.count - m0);
        p.out = o.out + m0 * size;
        for (int k = 0; k < runs; ++k) {
            p.steps = int(int64_t(o.steps) * (k + 1) / runs - int64_t(o.steps) * k / runs);
            p.first = k == 0;
            p.last = k + 1 == runs;
            p.src = k > 0 ? static_cast<const void *>(p.x)
                          : static_cast<const char *>(o.u) + m0 * size * (f32 ? 4 : 2);
            p.src_f32 = k > 0 || f32;
            e = launch_kernel(gram_long_kernel<RP>, dim3(unsigned(l.chunks), many), dim3(OR_THREADS), 0, st, p);
            if (e == cudaSuccess)
                e = launch_kernel(steps_long_kernel<RP>, dim3(many), dim3(OR_THREADS), ss, st, p);
            if (e == cudaSuccess)
                e = launch_kernel(apply_long_kernel<RP>, dim3(unsigned((o.n - 1) / OL_COLS + 1), many),
                                  dim3(OR_THREADS), as, st, p);
            if (e != cudaSuccess) return int(e);
        }
    }
    return LORA_OK;
}

int run_ortho_long(const OrthoArgs &o, int rp, bool f32, void *workspace, int64_t bytes, cudaStream_t st)
{
    switch (rp) {
    case 16: return run_long<16>(o, f32, workspace, bytes, st);
    case 32: return run_long<32>(o, f32, workspace, bytes, st);
    case 64: return run_long<64>(o, f32, workspace, bytes, st);
    default: return run_long<128>(o, f32, workspace, bytes, st);
    }
}

}  // namespace lora
