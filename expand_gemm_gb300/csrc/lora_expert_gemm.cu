// lora_expert_gemm.cu -- the three products of a mixture of experts on CTA
// pairs (lora_pair_gemm.cuh), over rows copied into the order of experts:
//   y  = x W[e]^T      A: rows of x, B: rows of W (both K-major)
//   dx = dy W[e]       A: rows of dy, B: W with its rows as the K dimension
//   dW[e] = dy^T x     both with the rows as the K dimension; a segment is
//                      padded with zeros to whole K blocks
// W is mapped with a dimension of its own for the expert: what lies behind an
// expert's last row or column arrives as zeros, never as its neighbour's
// values.
#include "lora_expert.cuh"
#include "lora_tc.cuh"

namespace lora {

struct ExpertGemm {
    ExpertArgs p;
    CUtensorMap a, b;
};

constexpr int EX_STAGE = 32 * 128;                               // a warp's rows on their way out
constexpr int EX_SMEM = PG_SMEM + 8 * EX_STAGE;
static_assert(EX_SMEM <= 232448, "shared memory of a CTA");
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
    it.row = b.y + tile * EX_TILE;
    it.valid = b.x - tile * EX_TILE;
    it.start = a.w + tile * EX_TILE;
    it.col = k / many * EX_TILE;
    it.expert = a.z;
    return it;
}

// 32 columns of a warp's 32 rows, element by element: rows that begin off a
// 16-byte boundary.
__device__ __forceinline__ void put_rows_unaligned(uint8_t *stage, const uint32_t (&v)[32], uint16_t *dst, int many,
                                                   bool add)
{
    const int lane = threadIdx.x & 31;
    float *at = reinterpret_cast<float *>(stage);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j) at[lane * 32 + ((j + lane) & 31)] = __uint_as_float(v[j]);
    __syncwarp();
    for (int r = 0; r < 32; ++r) {
        uint16_t *to = reinterpret_cast<uint16_t *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
        if (to == nullptr || lane >= many) continue;
        float s = at[r * 32 + ((lane + r) & 31)];
        if (add) s += bf16_to_f32(to[lane]);
        to[lane] = uint16_t(pack_bf16x2(s, 0.0f) & 0xFFFFu);
    }
}

// 32 fp32 columns of a warp's 32 rows, 128 bytes of a row at a time.
__device__ __forceinline__ void put_rows_f32(uint8_t *stage, const uint32_t (&v)[32], float *dst, int many)
{
    const int lane = threadIdx.x & 31, c = lane & 7;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((k ^ lane) & 7) * 16) =
            make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + (lane >> 3);
        float *to = reinterpret_cast<float *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
        if (to != nullptr && 4 * c < many)
            *reinterpret_cast<uint4 *>(to + 4 * c) =
                *reinterpret_cast<const uint4 *>(stage + row * 128 + ((c ^ row) & 7) * 16);
    }
}

// The columns [c0, lim) of a warp's 32 rows from TMEM to dst (null: nowhere),
// rounded once, or added to what is there in fp32 first.
__device__ __forceinline__ void put_tile(uint8_t *stage, uint32_t tmem, bool empty, uint16_t *dst, int c0, int lim,
                                         bool vec, bool add)
{
    if (vec && !add) {
        for (int c = c0; c < lim; c += 64) {
            uint32_t o[32];
            if (empty) {
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = 0u;
            } else {
                load64(tmem + c, 1.0f, o);
            }
            store_rows(stage, o, dst == nullptr ? nullptr : dst + c, lim - c);
        }
        return;
    }
    for (int c = c0; c < lim; c += 32) {
        uint32_t v[32];
        if (empty) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
        } else {
            tmem_ld32_nowait(tmem + c, v);
            tmem_wait_ld();
        }
        uint16_t *to = dst == nullptr ? nullptr : dst + c;
        if (vec) add_rows(stage, v, 1.0f, to, lim - c);
        else put_rows_unaligned(stage, v, to, min(32, lim - c), add);
    }
}

__device__ __forceinline__ uint8_t *warp_stage()
{
    extern __shared__ uint8_t pg_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(pg_smem_raw) + 1023) & ~uintptr_t(1023));
    return smem + PG_STAGES * PG_STAGE_BYTES + 256 + (int(threadIdx.x >> 5) - PG_EPI_WARP0) * EX_STAGE;
}

__global__ void __launch_bounds__(PG_THREADS, 1) expert_forward_kernel(const __grid_constant__ ExpertGemm g)
{
    pdl_wait();
    const ExpertArgs &p = g.p;
    const int cols = (p.N + EX_TILE - 1) / EX_TILE, kb = (p.K + PG_BK - 1) / PG_BK;
    const int total = *p.tiles * cols;
    auto item = [&](int i) {
        const ExpertItem it = expert_item(p, i, cols);
        return PairItem{it.row, it.col, 0, kb, it.expert};
    };
    auto epilogue = [&](int i, const PairItem &, uint32_t tmem, int r, int c0, int rank, bool empty) {
        const ExpertItem it = expert_item(p, i, cols);
        const int local = rank * PG_HALF + r;
        uint16_t *dst = nullptr;
        if (local < it.valid) {
            const int row = checked_token(p.sorted[it.start + local], p.R, p.error_word);
            if (row >= 0) dst = p.y + int64_t(row) * p.y_ld + it.col;
        }
        put_tile(warp_stage(), tmem, empty, dst, c0, min(c0 + PG_HALF, p.N - it.col), p.y_vec, p.add);
    };
    pair_gemm<false, false, true>(&g.a, &g.b, total, p.error_word, item, epilogue);
}

__global__ void __launch_bounds__(PG_THREADS, 1) expert_dx_kernel(const __grid_constant__ ExpertGemm g)
{
    pdl_wait();
    const ExpertArgs &p = g.p;
    const int cols = (p.K + EX_TILE - 1) / EX_TILE, kb = (p.N + PG_BK - 1) / PG_BK;
    const int total = *p.tiles * cols;
    auto item = [&](int i) {
        const ExpertItem it = expert_item(p, i, cols);
        return PairItem{it.row, it.col, 0, kb, it.expert};
    };
    auto epilogue = [&](int i, const PairItem &, uint32_t tmem, int r, int c0, int rank, bool empty) {
        const ExpertItem it = expert_item(p, i, cols);
        const int local = rank * PG_HALF + r, lim = min(c0 + PG_HALF, p.K - it.col);
        int row = -1;
        if (local < it.valid) row = checked_token(p.sorted[it.start + local], p.R, p.error_word);
        if (p.part != nullptr) {
            float *dst = row >= 0 ? p.part + int64_t(row) * p.K + it.col : nullptr;
            for (int c = c0; c < lim; c += 32) {
                uint32_t v[32];
                tmem_ld32_nowait(tmem + c, v);
                tmem_wait_ld();
                put_rows_f32(warp_stage(), v, dst == nullptr ? nullptr : dst + c, lim - c);
            }
            return;
        }
        uint16_t *dst = row >= 0 ? p.dx + int64_t(row) * p.dx_ld + it.col : nullptr;
        put_tile(warp_stage(), tmem, empty, dst, c0, lim, p.dx_vec, p.add);
    };
    pair_gemm<false, true, true>(&g.a, &g.b, total, p.error_word, item, epilogue);
}

__global__ void __launch_bounds__(PG_THREADS, 1) expert_dw_kernel(const __grid_constant__ ExpertGemm g)
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
        put_tile(warp_stage(), tmem, empty, dst, c0, min(c0 + PG_HALF, p.K - it.row_b), true, false);
    };
    pair_gemm<true, true>(&g.a, &g.b, p.E * nt * kt, p.error_word, item, epilogue);
}

// ---------------------------------------------------------------- host

template <typename Kern>
static int run_pairs(Kern kernel, std::atomic<uint64_t> &done, const ExpertGemm &g, cudaStream_t st)
{
    if (int e = expert_shared_memory((const void *)kernel, EX_SMEM, done)) return e;
    const int pairs = device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1;
    return int(launch_pair_kernel(kernel, pairs, st, g, PG_THREADS, EX_SMEM));
}

int launch_expert_forward(const ExpertArgs &p, int64_t rows, cudaStream_t st)
{
    ExpertGemm g;
    g.p = p;
    if (!encode_tile_map(&g.a, p.xs, uint64_t(rows), uint64_t(p.K), uint64_t(p.K), PG_BK, PG_HALF,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_stack_map(&g.b, p.w, uint64_t(p.E), uint64_t(p.N), uint64_t(p.K), PG_BK, PG_HALF))
        return LORA_ERR_DEVICE;
    static std::atomic<uint64_t> done{0};
    return run_pairs(expert_forward_kernel, done, g, st);
}

int launch_expert_dx(const ExpertArgs &p, int64_t rows, cudaStream_t st)
{
    ExpertGemm g;
    g.p = p;
    if (!encode_tile_map(&g.a, p.dys, uint64_t(rows), uint64_t(p.N), uint64_t(p.dys_ld), PG_BK, PG_HALF,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_stack_map(&g.b, p.w, uint64_t(p.E), uint64_t(p.N), uint64_t(p.K), PG_BK, PG_BK))
        return LORA_ERR_DEVICE;
    static std::atomic<uint64_t> done{0};
    return run_pairs(expert_dx_kernel, done, g, st);
}

int launch_expert_dw(const ExpertArgs &p, int64_t rows, cudaStream_t st)
{
    ExpertGemm g;
    g.p = p;
    if (!encode_tile_map(&g.a, p.dys, uint64_t(rows), uint64_t(p.N), uint64_t(p.dys_ld), PG_BK, PG_BK,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&g.b, p.xs, uint64_t(rows), uint64_t(p.K), uint64_t(p.K), PG_BK, PG_BK,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return LORA_ERR_DEVICE;
    static std::atomic<uint64_t> done{0};
    return run_pairs(expert_dw_kernel, done, g, st);
}

}  // namespace lora
