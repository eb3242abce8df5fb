// lora_expert_gemm.cu -- the three products of a mixture of experts on CTA
// pairs (lora_pair_gemm.cuh), over rows copied into the order of experts:
//   y^T  = W[e] x^T     A: rows of W, B: rows of x (both K-major)
//   dx^T = W[e]^T dy^T  A: W with its rows as the K dimension, B: rows of dy
//   dW[e] = dy^T x      both with the rows as the K dimension; a segment is
//                       padded with zeros to whole K blocks
// The first two have the tokens as the UMMA's N, so that the last tile of an
// expert costs what its rows need (in steps of 32) and not 256 of them.  W is
// mapped with a dimension of its own for the expert: what lies behind an
// expert's last row or column arrives as zeros, never as its neighbour's
// values.
//
// Bound by the tensor cores.  One GB300, each kernel's launch alone on a cool
// machine: 8192 tokens, 2 of 16 experts 4096 to 11008: 895 us, 1.65 PFLOP/s of
// what the result needs (a dense library product of the same operations: 767
// in a burst, 825 sustained); gradients of 4096 tokens, 2 of 8 experts 4096 x
// 4096: dx 174, dW 168 (1.58, 1.64).  Whole calls, one after another: 990 to
// 1040 and 420 to 430.
#include "lora_expert.cuh"
#include "lora_tc.cuh"

namespace lora {

struct ExpertGemm {
    ExpertArgs p;
    CUtensorMap a, b;
};

constexpr int EX_STAGE = 32 * 128;                               // a warp's rows on their way out
constexpr int EX_SMEM = PG_SMEM + 8 * EX_STAGE;                   // of dW
static_assert(EX_SMEM <= 232448, "shared memory of a CTA");
constexpr int EX_SIDE = 4;                                       // warps that copy or join beside a product
constexpr int EX_GROUP = 16;                                     // token tiles that share a sweep over the columns

// Item i of an expert's tiles: the tile and the column block.  Up to
// EX_GROUP tiles of tokens take a column block one after another, so that
// the pairs at work share its weights, and x's rows stay in L2.
struct ExpertItem {
    int row, valid, start, col, expert;
};
__device__ __forceinline__ ExpertItem expert_item(const ExpertArgs &p, int i, int cols)
{
    const int4 *at = reinterpret_cast<const int4 *>(p.table + i / cols);
    const int4 a = at[0], b = at[1];          // base, tiles, expert, start; count, row
    const int j = i - a.x * cols;
    const int g = j / (EX_GROUP * cols) * EX_GROUP, many = min(EX_GROUP, a.y - g), k = j - g * cols;
    const int tile = g + k % many;
    ExpertItem it;
    it.row = b.y + tile * p.tile_rows;
    it.valid = min(p.tile_rows, b.x - tile * p.tile_rows);
    it.start = a.w + tile * p.tile_rows;
    it.col = k / many * EX_TILE;
    it.expert = a.z;
    return it;
}

// Sixteen tokens' values of this thread's column, rounded once (added to what
// is there in fp32 first): a warp writes 64 bytes of a token's row at a time.
__device__ __forceinline__ void put_tokens(const uint32_t (&v)[16], const int (&row)[16], uint16_t *y, int64_t ld,
                                           int col, bool in, bool add)
{
    float old[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        old[j] = add && in && row[j] >= 0 ? bf16_to_f32(y[int64_t(row[j]) * ld + col]) : 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float s = __uint_as_float(v[j]);
        if (add) s += old[j];
        if (in && row[j] >= 0) y[int64_t(row[j]) * ld + col] = uint16_t(pack_bf16x2(s, 0.0f) & 0xFFFFu);
    }
}

__device__ __forceinline__ uint8_t *warp_stage()
{
    extern __shared__ uint8_t pg_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(pg_smem_raw) + 1023) & ~uintptr_t(1023));
    return smem + PG_STAGES * PG_STAGE_BYTES + 256 + (int(threadIdx.x >> 5) - PG_EPI_WARP0) * EX_STAGE;
}

// y or dx: `width` columns of the result, `depth` of the sum.
template <bool DX>
__device__ __forceinline__ void expert_product(const ExpertGemm &g)
{
    const ExpertArgs &p = g.p;
    const int width = DX ? p.K : p.N, depth = DX ? p.N : p.K;
    const int cols = (width + EX_TILE - 1) / EX_TILE, kb = (depth + PG_BK - 1) / PG_BK;
    const int total = *p.tiles * cols;
    auto item = [&](int i) {
        const ExpertItem it = expert_item(p, i, cols);
        return PairItem{it.col, it.row, 0, kb, it.expert, (it.valid + 31) & ~31};
    };
    auto epilogue = [&](int i, const PairItem &, uint32_t tmem, int r, int c0, int rank, bool) {
        const ExpertItem it = expert_item(p, i, cols);
        const int col = it.col + rank * PG_HALF + r, lane = threadIdx.x & 31;
        const bool in = col < width;
        for (int c = c0; c < min(c0 + PG_HALF, it.valid); c += 16) {
            uint32_t v[16];
            tmem_ld16_nowait(tmem + c, v);
            int mine = -1, row[16];
            if (lane < 16 && c + lane < it.valid)
                mine = expert_row(p, it.start + c + lane);
#pragma unroll
            for (int j = 0; j < 16; ++j) row[j] = __shfl_sync(0xffffffffu, mine, j);
            tmem_wait_ld();
            if (!DX) {
                put_tokens(v, row, p.y, p.y_ld, col, in, p.add);
            } else if (p.part == nullptr) {
                put_tokens(v, row, p.dx, p.dx_ld, col, in, p.add);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (in && row[j] >= 0) p.part[int64_t(row[j]) * p.K + col] = __uint_as_float(v[j]);
            }
        }
    };
    // x into the order of experts, for dW's product
    auto copy_x = [&](int warp) {
        if (!DX || !p.later) return;
        const int64_t rows = int64_t(*p.copied) * EX_PAD, warps = int64_t(gridDim.x) * EX_SIDE;
        for (int64_t q = int64_t(blockIdx.x) * EX_SIDE + warp; q < rows; q += warps) {
            const int row = p.from[q];
            uint16_t *to = p.xs + q * p.K;
            if (row >= 0) copy_row(to, p.x + int64_t(row / p.fan) * p.x_ld, p.K, p.x_vec);
            else clear_row(to, p.K);
        }
    };
    pair_gemm<DX, false, true>(&g.a, &g.b, total, p.error_word, item, epilogue, copy_x);
}

__global__ void __launch_bounds__(PG_THREADS, 1) expert_forward_kernel(const __grid_constant__ ExpertGemm g)
{
    pdl_wait();
    expert_product<false>(g);
}

__global__ void __launch_bounds__(PG_THREADS + EX_SIDE * 32, 1) expert_dx_kernel(const __grid_constant__ ExpertGemm g)
{
    pdl_wait();
    expert_product<true>(g);
}

__global__ void __launch_bounds__(PG_THREADS + EX_SIDE * 32, 1) expert_dw_kernel(const __grid_constant__ ExpertGemm g)
{
    pdl_wait();
    const ExpertArgs &p = g.p;
    const int nt = (p.N + EX_TILE - 1) / EX_TILE, kt = (p.K + EX_TILE - 1) / EX_TILE;
    auto item = [&](int i) {
        const int e = i / (nt * kt), j = i % (nt * kt);
        const int2 b = p.blocks[e];
        return PairItem{j / kt * EX_TILE, j % kt * EX_TILE, b.x, b.x + b.y, e};
    };
    auto epilogue = [&](int, const PairItem &it, uint32_t tmem, int r, int c0, int rank, bool empty) {
        const int n = it.row_a + rank * PG_HALF + r;
        uint16_t *dst = n < p.N ? p.dw + (int64_t(it.mat) * p.N + n) * p.K + it.row_b : nullptr;
        const int lim = min(c0 + PG_HALF, p.K - it.row_b);
        for (int c = c0; c < lim; c += 64) {
            uint32_t o[32];
            if (empty) {
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = 0u;
            } else {
                load64(tmem + c, 1.0f, o);
            }
            store_rows(warp_stage(), o, dst == nullptr ? nullptr : dst + c, lim - c);
        }
    };
    auto join = [&](int warp) {
        if (p.later && p.part != nullptr)
            join_rows(p, int64_t(blockIdx.x) * EX_SIDE + warp, int64_t(gridDim.x) * EX_SIDE);
    };
    pair_gemm<true, true>(&g.a, &g.b, p.E * nt * kt, p.error_word, item, epilogue, join);
}

// ---------------------------------------------------------------- host

template <typename Kern>
static int run_pairs(Kern kernel, std::atomic<uint64_t> &done, const ExpertGemm &g, int smem, int threads,
                     cudaStream_t st)
{
    if (int e = expert_shared_memory((const void *)kernel, smem, done)) return e;
    const int pairs = device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1;
    return int(launch_pair_kernel(kernel, pairs, st, g, threads, smem));
}

int launch_expert_forward(const ExpertArgs &p, cudaStream_t st)
{
    ExpertGemm g;
    g.p = p;
    if (!encode_stack_map(&g.a, p.w, uint64_t(p.E), uint64_t(p.N), uint64_t(p.K), PG_BK, PG_HALF) ||
        !encode_tile_map(&g.b, p.xs, uint64_t(p.rows), uint64_t(p.K), uint64_t(p.K), PG_BK, PG_HALF,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return LORA_ERR_DEVICE;
    static std::atomic<uint64_t> done{0};
    return run_pairs(expert_forward_kernel, done, g, PG_SMEM, PG_THREADS, st);
}

int launch_expert_dx(const ExpertArgs &p, cudaStream_t st)
{
    ExpertGemm g;
    g.p = p;
    if (!encode_stack_map(&g.a, p.w, uint64_t(p.E), uint64_t(p.N), uint64_t(p.K), PG_BK, PG_BK) ||
        !encode_tile_map(&g.b, p.dys, uint64_t(p.rows), uint64_t(p.N), uint64_t(p.dys_ld), PG_BK, PG_HALF,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return LORA_ERR_DEVICE;
    static std::atomic<uint64_t> done{0};
    return run_pairs(expert_dx_kernel, done, g, PG_SMEM, PG_THREADS + EX_SIDE * 32, st);
}

int launch_expert_dw(const ExpertArgs &p, cudaStream_t st)
{
    ExpertGemm g;
    g.p = p;
    if (!encode_tile_map(&g.a, p.dys, uint64_t(p.rows), uint64_t(p.N), uint64_t(p.dys_ld), PG_BK, PG_BK,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&g.b, p.xs, uint64_t(p.rows), uint64_t(p.K), uint64_t(p.K), PG_BK, PG_BK,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return LORA_ERR_DEVICE;
    static std::atomic<uint64_t> done{0};
    return run_pairs(expert_dw_kernel, done, g, EX_SMEM, PG_THREADS + EX_SIDE * 32, st);
}

}  // namespace lora
