// lora_expert.cu -- lora_expert_linear and lora_expert_linear_backward: the
// products of a mixture of experts (or, with one expert, of one frozen
// layer), grouped by the ids that LoRAKernelMeta sorts:
//   y[i]  (+)= W[id(i)] x[i / fan]
//   dx[t] (+)= sum_{j < fan} W[id]^T dy[t fan + j]
//   dW[e]  = sum_{i: id(i) = e} dy[i] x[i / fan]^T
// This file: the copies in the order of experts, the table of tiles, the join
// of a token's rows, and the C entries.
#include <stdint.h>

#include "lora_expert.cuh"

namespace lora {

constexpr int EX_PACK_THREADS = 256;

// The table of tiles and, for dW, each expert's K blocks: one block.
__device__ __forceinline__ void expert_tables(const ExpertArgs &p, const SegTab &tab, int units, int *first_row)
{
    const int pad = p.pad ? EX_PAD : 1;
    if (p.copied != nullptr && threadIdx.x == 0) *p.copied = int(min(int64_t(units), p.rows / pad));
    if (p.blocks != nullptr) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.blocks[e] = make_int2(0, 0);
        __syncthreads();
        for (int k = threadIdx.x; units > 0 && k < p.nbins; k += blockDim.x)
            if (tab.id[k] >= 0 && tab.count[k] > 0)
                p.blocks[tab.id[k]] = make_int2(tab.tile[k], tab.tile[k + 1] - tab.tile[k]);
    }
    if (p.table == nullptr) return;
    // the segments' rows in the copy, kept while the same memory takes the tiles'
    for (int k = threadIdx.x; units > 0 && k < p.nbins; k += blockDim.x) first_row[k] = tab.tile[k] * pad;
    __syncthreads();
    const int tiles = min(p.entries, load_segments(p.no_lora, p.active, p.counts, p.start_loc, p.nbins, p.tile_rows, tab,
                                                   false, 0, p.R, p.error_word, true));
    if (threadIdx.x == 0) *p.tiles = tiles;
    for (int t = threadIdx.x; t < tiles; t += blockDim.x) {
        const int k = find_segment(tab.tile, p.nbins, t);
        ExpertTile e;
        e.base = tab.tile[k];
        e.tiles = tab.tile[k + 1] - tab.tile[k];
        e.expert = tab.id[k];
        e.start = tab.start[k];
        e.count = tab.count[k];
        e.row = first_row[k];
        e.pad0 = e.pad1 = 0;
        p.table[t] = e;
    }
}

// The first block writes the tables; the others copy x (blockIdx.y == 0) and
// dy (1) into the order of experts, a warp a row, and clear the rows of dx
// that no expert adds to (dx overwritten, one row a token).  Bound by memory:
// 16384 rows of 4096 from 8192 of x 36 us, 5.6 TB/s read and written.  Gathers by
// TMA would take 2900 clocks a stage of 512 in the product.
__global__ void __launch_bounds__(EX_PACK_THREADS) expert_pack_kernel(const __grid_constant__ ExpertArgs p)
{
    extern __shared__ int ex_tab[];
    pdl_wait();
    // the next kernel may begin: the metadata are complete, and what it needs
    // of this one it waits for
    pdl_launch_dependents();
    const bool tables = blockIdx.x == 0;
    if (tables && blockIdx.y != 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = int64_t(blockIdx.x - 1) * (EX_PACK_THREADS / 32) + warp;
    const int64_t step = int64_t(gridDim.x - 1) * (EX_PACK_THREADS / 32);
    const SegTab tab = seg_tab(ex_tab, p.nbins);
    const int pad = p.pad ? EX_PAD : 1;
    const int units = load_segments(p.no_lora, p.active, p.counts, p.start_loc, p.nbins, pad, tab, false, 0,
                                    p.R, p.error_word, true);
    if (tables) {
        expert_tables(p, tab, units, ex_tab + 4 * p.nbins + 2);
        return;
    }
    const bool dy = blockIdx.y == 1 || p.later;      // later: dy alone
    const uint16_t *src = dy ? p.dy : p.x;
    uint16_t *dst = dy ? p.dys : p.xs;
    const int64_t src_ld = dy ? p.dy_ld : p.x_ld, dst_ld = dy ? p.dys_ld : p.K;
    const int cols = dy ? p.N : p.K, fan = dy ? 1 : p.fan;
    const bool vec = dy ? p.dy_vec : p.x_vec;
    if (dst != nullptr) {
        const int64_t rows = min(int64_t(units) * pad, p.rows);
        for (int64_t q = first; q < rows; q += step) {
            const int k = find_segment(tab.tile, p.nbins, int(q / pad));
            const int local = int(q - int64_t(tab.tile[k]) * pad);
            uint16_t *to = dst + q * dst_ld;
            int row = -1;
            if (local < tab.count[k]) row = expert_row(p, tab.start[k] + local);
            if (row >= 0) copy_row(to, src + int64_t(row / fan) * src_ld, cols, vec);
            else clear_row(to, dst_ld);
            if (dy && p.from != nullptr && lane == 0) p.from[q] = row;
        }
    }
    if (blockIdx.y == 0 && p.dx != nullptr && p.fan == 1 && !p.add) {
        const bool none = *p.no_lora != 0;
        const int rest = none ? p.R : (tab.id[0] == -1 ? tab.count[0] : 0);
        for (int64_t i = first; i < rest; i += step) {
            const int row = none ? int(i) : expert_row(p, int(i));
            if (row < 0) continue;
            uint16_t *to = p.dx + int64_t(row) * p.dx_ld;
            if (p.dx_vec) {
                clear_row(to, p.K);
            } else {
                for (int c = lane; c < p.K; c += 32) to[c] = 0;
            }
        }
    }
}

__global__ void __launch_bounds__(256) expert_join_kernel(const __grid_constant__ ExpertArgs p)
{
    pdl_wait();
    const int64_t per = blockDim.x / 32;
    join_rows(p, blockIdx.x * per + threadIdx.x / 32, gridDim.x * per);
}

// ---------------------------------------------------------------- host

int expert_shared_memory(const void *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return 0;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return int(e);
    done.fetch_or(bit, std::memory_order_relaxed);
    return 0;
}

static int64_t up256(int64_t v) { return (v + 255) & ~int64_t(255); }

// Offsets in the workspace, in bytes.
struct ExpertLayout {
    int64_t tiles, table, blocks, from, xs, dys, part, w, bytes;
    int64_t rows, entries;            // of the copies and of the table
};

// Rows of a tile of the forward product, by how many rows an expert has on
// average; EX_TILE: the product on CTA pairs, where 4-bit weights are decoded
// first.  The host knows neither the rows' shares nor which have an id: every
// row and every expert counts.  Both sides measured, with equal shares and an id
// for every row (us; 16 experts of 4096 x 4096 if nothing else is
// said, in a graph).  bf16, tiles of 32 rows and pairs: 32 rows: 115 and 119;
// 40 rows: 124 and 120; 64 rows: 138 and 121; one expert, 16 rows: 23 and 34;
// one of width 11008, 64 rows: 51 and 44.  4 bits, tiles of 16 and of 64 rows:
// 12 rows: 60 and 62; 16 rows: 68 and 63; 32 rows: 100 and 66.  4 bits, 64 and
// pairs: 256 rows: 221 and 274; 375 rows: 293 and 298; 512 rows: 394 and 330;
// one expert, 512 rows: 46 and 45; one of width 11008, 384 rows: 68 and 78,
// 1024 rows: 136 and 107.
// Where the average is far from the shares (experts of 4096 x 4096, and the same
// rows by metadata of the experts in use): bf16, 2048 rows of 64 experts, all on
// one 200 and 67, on eight 200 and 81; 512 rows of 16, on one 69 and 38, on four
// 71 and 50; 4 bits, 2048 rows of 64, on one 92 and 73; 512 of 16, on one 42 and
// 44.  Rows without an id cost little: half of 1024 rows of 16 experts, on pairs
// 116, the other half alone, in tiles of 32, 120; in 4 bits 61 and 62.
static int forward_tile(int64_t R, int64_t E, bool quantized)
{
    const int64_t mean = R / E;
    if (!quantized) return mean <= 32 ? 32 : EX_TILE;
    return mean <= 12 ? 16 : mean <= 384 ? 64 : EX_TILE;
}

// Rows of a tile of the products on CTA pairs.  One expert: what takes the
// pairs the least time in whole rounds, where each tile costs about 16 rows
// more than it has (4096 rows, 4096 to 4096: 98 us with tiles of 224 rows, 104
// with 256, 107 with 192).  Rows without an id count too (a tenth of the 4096:
// 93, as those with one alone; half: 73, those alone 68).  Several have shares that vary, and a tile costs
// what its rows need, so that short tiles only split experts that one tile
// would have held (16 experts of 4096 x 4096, 128 rows on average: 139 with
// 128, 125 with 256; 256 rows: 155 with 192, 151 with 256; 1024 rows of 8: 196
// with 224, 195 with 256).
static int pair_tile(int64_t R, int64_t E, int64_t cols)
{
    if (E > 1) return EX_TILE;
    const int64_t pairs = device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1;
    const int64_t blocks = (cols + EX_TILE - 1) / EX_TILE;
    int best = EX_TILE;
    int64_t least = INT64_MAX;
    for (int t = EX_TILE; t >= 64; t -= 32) {
        const int64_t tiles = (R + t - 1) / t * blocks;
        const int64_t cost = (tiles + pairs - 1) / pairs * (t + 16);
        if (cost < least) {
            least = cost;
            best = t;
        }
    }
    return best;
}

// A batch of R rows; every size grows with R, so that a workspace for a batch
// holds each smaller one.
static ExpertLayout expert_layout(int64_t R, int fan, int64_t K, int64_t N, int64_t E, bool x_copy, bool dx, bool dw,
                                  bool decode)
{
    ExpertLayout l;
    const int64_t active = R < E ? R : E;
    l.rows = R + (dw ? (EX_PAD - 1) * active : 0);
    int64_t at = 256;
    l.tiles = 0;
    l.table = at;
    l.entries = R / EX_LEAST_TILE + active;
    at += up256(l.entries * int64_t(sizeof(ExpertTile)));
    l.blocks = at;
    at += dw ? up256(E * 8) : 0;
    l.from = at;
    at += dx && dw ? up256(l.rows * 4) : 0;
    l.xs = at;
    at += x_copy ? up256(l.rows * K * 2) : 0;
    l.dys = at;
    at += dx || dw ? up256(l.rows * ((N + 7) / 8 * 8) * 2) : 0;
    l.part = at;
    at += dx && fan > 1 ? up256(R * K * 4) : 0;
    l.w = at;
    at += decode ? up256(E * N * K * 2) : 0;
    l.bytes = at;
    return l;
}

static uintptr_t bits(const void *ptr) { return reinterpret_cast<uintptr_t>(ptr); }

static int check_sizes(int32_t R, int32_t fan, int32_t K, int32_t N, int32_t E, bool quantized)
{
    if (R < 0 || fan < 1 || R % fan != 0 || K < 8 || N < 1 || E < 1 || E > LORA_MAX_LORAS) return LORA_ERR_SIZE;
    if (K % (quantized ? 32 : 8) != 0) return LORA_ERR_ALIGN;
    return LORA_OK;
}

static int fill(ExpertArgs &p, int32_t R, int32_t fan, int32_t K, int32_t N, const lora_bf16_t *x, int64_t x_ld,
                const void *weight, const uint8_t *scale, const lora_meta_t *meta)
{
    if (meta == nullptr || meta->token_lora_mapping == nullptr || meta->token_indices_sorted_by_lora_ids == nullptr ||
        meta->num_tokens_per_lora == nullptr || meta->lora_token_start_loc == nullptr ||
        meta->active_lora_ids == nullptr || meta->no_lora_flag == nullptr || meta->error_word == nullptr)
        return LORA_ERR_NULL;
    if (int e = check_sizes(R, fan, K, N, meta->max_loras, scale != nullptr)) return e;
    if (R > meta->max_num_tokens) return LORA_ERR_TOKENS;
    if (weight == nullptr || (R > 0 && x == nullptr)) return LORA_ERR_NULL;
    if (x_ld < K) return LORA_ERR_SIZE;
    if ((bits(weight) | bits(scale)) & 15u) return LORA_ERR_ALIGN;
    p = ExpertArgs{};
    p.x = x;
    p.x_ld = x_ld;
    p.x_vec = (bits(x) & 15u) == 0 && x_ld % 8 == 0;
    if (scale != nullptr) {
        p.codes = static_cast<const uint8_t *>(weight);
        p.scales = scale;
    } else {
        p.w = static_cast<const uint16_t *>(weight);
    }
    p.R = R;
    p.fan = fan;
    p.K = K;
    p.N = N;
    p.E = meta->max_loras;
    p.nbins = meta->max_loras + 1;
    p.tile_rows = EX_TILE;
    p.ids = meta->token_lora_mapping;
    p.sorted = meta->token_indices_sorted_by_lora_ids;
    p.counts = meta->num_tokens_per_lora;
    p.start_loc = meta->lora_token_start_loc;
    p.active = meta->active_lora_ids;
    p.no_lora = meta->no_lora_flag;
    p.error_word = meta->error_word;
    return LORA_OK;
}

static int launch_pack(const ExpertArgs &p, cudaStream_t st)
{
    const int64_t want = (p.rows + EX_PACK_THREADS / 32 - 1) / (EX_PACK_THREADS / 32);
    const int64_t most = 6ll * device_sm_count();
    const dim3 grid(unsigned(1 + (want < most ? (want > 0 ? want : 1) : most)), p.dys != nullptr && !p.later ? 2 : 1);
    return int(launch_kernel(expert_pack_kernel, grid, dim3(EX_PACK_THREADS),
                             seg_tab_bytes(p.nbins) + p.nbins * sizeof(int), st, p));
}

}  // namespace lora

LORA_API int64_t lora_expert_linear_workspace(int32_t num_rows, int32_t hidden, int32_t out_features,
                                              int32_t max_loras, int32_t quantized)
{
    using namespace lora;
    if (int e = check_sizes(num_rows, 1, hidden, out_features, max_loras, quantized != 0)) return e;
    return expert_layout(num_rows, 1, hidden, out_features, max_loras, true, false, false,
                         quantized != 0 && forward_tile(num_rows, max_loras, true) == EX_TILE).bytes;
}

LORA_API int lora_expert_linear(const lora_bf16_t *x, int64_t x_ld, int32_t num_rows, int32_t fan_out,
                                int32_t hidden, const void *weight, const uint8_t *weight_scale,
                                int32_t out_features, lora_bf16_t *y, int64_t y_ld, int32_t add_inputs,
                                const lora_meta_t *meta, void *workspace, int64_t workspace_bytes, void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_expert_linear");
    ExpertArgs p;
    if (int e = fill(p, num_rows, fan_out, hidden, out_features, x, x_ld, weight, weight_scale, meta)) return e;
    if (workspace == nullptr || (num_rows > 0 && y == nullptr)) return LORA_ERR_NULL;
    if (y_ld < out_features) return LORA_ERR_SIZE;
    if (bits(workspace) & 255u) return LORA_ERR_ALIGN;
    const bool quantized = weight_scale != nullptr;
    p.tile_rows = forward_tile(num_rows, p.E, quantized);
    const bool decode = quantized && p.tile_rows == EX_TILE;
    const ExpertLayout lay = expert_layout(num_rows, 1, hidden, out_features, p.E, true, false, false, decode);
    if (workspace_bytes < lay.bytes) return LORA_ERR_WORKSPACE;
    if (num_rows == 0) return LORA_OK;
    const bool pairs = p.tile_rows == EX_TILE;
    if (pairs) p.tile_rows = pair_tile(num_rows, p.E, out_features);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    p.y = y;
    p.y_ld = y_ld;
    p.add = add_inputs != 0;
    p.rows = lay.rows;
    p.entries = int32_t(lay.entries);
    p.tiles = reinterpret_cast<int32_t *>(ws + lay.tiles);
    p.table = reinterpret_cast<ExpertTile *>(ws + lay.table);
    p.xs = reinterpret_cast<uint16_t *>(ws + lay.xs);
    if (!pairs) {
        p.early = expert_stream_early(p);
        const bool gathers = expert_stream_gathers(p);
        if (p.early || gathers) p.table = nullptr;
        if (gathers) return launch_expert_stream(p, st);
    }
    if (int e = launch_pack(p, st)) return e;
    if (!pairs) return launch_expert_stream(p, st);
    if (decode) {
        uint16_t *w = reinterpret_cast<uint16_t *>(ws + lay.w);
        if (int e = launch_expert_decode(p, w, st)) return e;
        p.w = w;
    }
    return launch_expert_forward(p, st);
}

LORA_API int64_t lora_expert_linear_backward_workspace(int32_t num_rows, int32_t fan_out, int32_t hidden,
                                                       int32_t out_features, int32_t max_loras, int32_t hidden_grad,
                                                       int32_t weight_grad, int32_t quantized)
{
    using namespace lora;
    if (int e = check_sizes(num_rows, fan_out, hidden, out_features, max_loras, quantized != 0)) return e;
    return expert_layout(num_rows, fan_out, hidden, out_features, max_loras, weight_grad != 0, hidden_grad != 0,
                         weight_grad != 0, hidden_grad != 0 && quantized != 0).bytes;
}

LORA_API int lora_expert_linear_backward(const lora_bf16_t *dy, int64_t dy_ld, int32_t num_rows, int32_t fan_out,
                                         const lora_bf16_t *x, int64_t x_ld, int32_t hidden, const void *weight,
                                         const uint8_t *weight_scale, int32_t out_features, lora_bf16_t *dx,
                                         int64_t dx_ld, int32_t add_inputs, lora_bf16_t *d_weight,
                                         const lora_meta_t *meta, void *workspace, int64_t workspace_bytes,
                                         void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_expert_linear_backward");
    ExpertArgs p;
    if (int e = fill(p, num_rows, fan_out, hidden, out_features, x, x_ld, weight, weight_scale, meta)) return e;
    if (workspace == nullptr || (num_rows > 0 && dy == nullptr)) return LORA_ERR_NULL;
    if (dy_ld < out_features || (dx != nullptr && dx_ld < hidden)) return LORA_ERR_SIZE;
    if ((bits(workspace) & 255u) || (bits(d_weight) & 15u)) return LORA_ERR_ALIGN;
    const bool hx = dx != nullptr, hw = d_weight != nullptr, decode = hx && weight_scale != nullptr;
    const ExpertLayout lay = expert_layout(num_rows, fan_out, hidden, out_features, p.E, hw, hx, hw, decode);
    if (workspace_bytes < lay.bytes) return LORA_ERR_WORKSPACE;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!hx && !hw) return LORA_OK;
    if (num_rows == 0) {
        if (!hw) return LORA_OK;
        return int(cudaMemsetAsync(d_weight, 0, size_t(p.E) * out_features * hidden * 2, st));
    }
    char *ws = static_cast<char *>(workspace);
    p.dy = dy;
    p.dy_ld = dy_ld;
    p.dy_vec = (bits(dy) & 15u) == 0 && dy_ld % 8 == 0;
    p.dys = reinterpret_cast<uint16_t *>(ws + lay.dys);
    p.dys_ld = (out_features + 7) / 8 * 8;
    p.xs = hw ? reinterpret_cast<uint16_t *>(ws + lay.xs) : nullptr;
    p.pad = hw;
    p.dx = dx;
    p.dx_ld = dx_ld;
    p.dx_vec = (bits(dx) & 15u) == 0 && dx_ld % 8 == 0;
    p.dw = d_weight;
    p.add = add_inputs != 0;
    p.rows = lay.rows;
    p.entries = int32_t(lay.entries);
    p.tiles = reinterpret_cast<int32_t *>(ws + lay.tiles);
    p.tile_rows = pair_tile(num_rows, p.E, hidden);
    p.table = hx ? reinterpret_cast<ExpertTile *>(ws + lay.table) : nullptr;
    p.blocks = hw ? reinterpret_cast<int2 *>(ws + lay.blocks) : nullptr;
    p.part = hx && fan_out > 1 ? reinterpret_cast<float *>(ws + lay.part) : nullptr;
    // With both gradients, what memory has to do for one product runs beside
    // the other: x is copied under dx's, and the rows of dx are joined under
    // dW's (4096 tokens, 2 of 8 experts 4096 x 4096: 441 us apart, 419 so).
    p.later = hx && hw;
    p.copied = p.later ? p.tiles + 1 : nullptr;
    p.from = p.later ? reinterpret_cast<int32_t *>(ws + lay.from) : nullptr;
    if (int e = launch_pack(p, st)) return e;
    if (hx) {
        if (decode) {
            uint16_t *w = reinterpret_cast<uint16_t *>(ws + lay.w);
            if (int e = launch_expert_decode(p, w, st)) return e;
            p.w = w;
        }
        if (int e = launch_expert_dx(p, st)) return e;
    }
    if (hw) return launch_expert_dw(p, st);
    if (fan_out == 1) return LORA_OK;
    const int64_t tokens = num_rows / fan_out, want = (tokens + 7) / 8, most = 8ll * device_sm_count();
    return int(launch_kernel(expert_join_kernel, dim3(unsigned(want < most ? want : most)), dim3(256), 0, st, p));
}
