// lora_expert.cuh -- what the kernels of lora_expert_linear and
// lora_expert_linear_backward share: the call's arguments, the rows laid out
// by expert, and the table of their tiles.
//
// Rows (a token's fan_out of them follow one another) have an expert id each;
// the metadata sorts them by it.  expert_pack_kernel copies x (and dy) into
// that order, so that a tile of one expert's rows is a box that TMA loads, at
// any alignment and stride of the caller's.
#pragma once

#include <atomic>

#include "lora_common.cuh"
#include "lora_umma.cuh"

namespace lora {

// One tile of the table: what segment it belongs to.  Items are numbered by
// tile, so i / columns is a tile of item i's expert whatever the order
// within the expert.
struct ExpertTile {
    int32_t base, tiles;      // the segment's first tile and how many it has
    int32_t expert;
    int32_t start, count;     // in the metadata's order
    int32_t row;              // first row of the segment's copy
    int32_t pad0, pad1;
};
static_assert(sizeof(ExpertTile) == 32, "two 16-byte loads");

constexpr int EX_TILE = 256;          // rows of a pair's tile
constexpr int EX_LEAST_TILE = 16;     // the smallest tile_rows
constexpr int EX_PAD = 64;            // rows that a segment is padded to for dW (a K block)

struct ExpertArgs {
    const uint16_t *x, *dy;
    int64_t x_ld, dy_ld;
    const uint16_t *w;                // bf16 [E, N, K]: the caller's, or the decoded copy
    const uint8_t *codes, *scales;    // MXFP4 instead
    uint16_t *y;                      // [R, y_ld]
    int64_t y_ld;
    uint16_t *dx;                     // [R / fan, dx_ld]
    int64_t dx_ld;
    uint16_t *dw;                     // [E, N, K]
    float *part;                      // dx by row, where tokens have several
    uint16_t *xs, *dys;               // copies in the metadata's order
    int64_t dys_ld;
    ExpertTile *table;
    int32_t *tiles;                   // [1]: entries of the table
    int2 *blocks;                     // [E]: first K block and K blocks of dW
    int32_t R, fan, K, N, E, nbins;
    int32_t add, pad, tile_rows;
    int32_t x_vec, dy_vec, dx_vec;
    const int32_t *ids, *sorted, *counts, *start_loc, *active, *no_lora;
    int32_t *error_word;
};

// Allows a kernel `bytes` of dynamic shared memory on the current device
// (lora_expert.cu); `done` holds the devices where it was.
int expert_shared_memory(const void *kernel, int bytes, std::atomic<uint64_t> &done);

// lora_expert_gemm.cu: products on CTA pairs over the copies.
int launch_expert_forward(const ExpertArgs &p, int64_t rows, cudaStream_t st);
int launch_expert_dx(const ExpertArgs &p, int64_t rows, cudaStream_t st);
int launch_expert_dw(const ExpertArgs &p, int64_t rows, cudaStream_t st);

// lora_expert_stream.cu: few rows an expert, weights in either form.
int launch_expert_stream(const ExpertArgs &p, int64_t rows, cudaStream_t st);

// lora_mxfp4.cu: the weights of the experts that have rows, decoded to bf16.
int launch_expert_decode(const ExpertArgs &p, uint16_t *out, cudaStream_t st);

}  // namespace lora
