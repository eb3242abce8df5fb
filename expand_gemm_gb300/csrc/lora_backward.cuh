// lora_backward.cuh -- what the kernels of lora_linear_backward share: the
// call's arguments, the layout of g and u, and the walk over the metadata.
#pragma once

#include "lora_frag.cuh"

namespace lora {

constexpr int BW_THREADS = 256;
constexpr int BW_TOK = 64;                 // tokens of a tile
constexpr int BW_COLS = 128;               // columns of a tile of dx, dA, dB
constexpr int BW_TERMS_TOKENS = BW_TOK;    // tokens up to which g and u are two bf16 terms

struct BackwardArgs {
    const uint16_t *dy, *x;
    int64_t dy_ld, x_ld;
    const float *buf;
    const uint16_t *a[LORA_MAX_SLICES], *b[LORA_MAX_SLICES];
    uint16_t *da[LORA_MAX_SLICES], *db[LORA_MAX_SLICES], *dbias[LORA_MAX_SLICES];
    uint16_t *dx;
    int64_t dx_ld;
    int32_t n[LORA_MAX_SLICES], off[LORA_MAX_SLICES];      // widths, first columns in dy
    // grad_w_kernel's column blocks of one adapter: dB of slice s ends
    // before block_end[s], dA of slice s before block_end[S + s]
    int32_t block_end[2 * LORA_MAX_SLICES];
    int32_t T, H, S, r, L, width;
    int32_t add, dy_vec, x_vec, dx_vec;
    float scale;
    uint16_t *g, *u;                       // [S][rows][RP]
    // for grad_w_tc_kernel, in the place of u, and beside g: the tiles
    // transposed, [S][rows / BW_TOK][RP][BW_TOK]; else null
    uint16_t *gt, *ut;
    int64_t rows;
    // elements from g to its second terms, and likewise from u, gt and ut; 0
    // where each is one bf16 value
    int64_t low;
    float *part;                           // grad_u_kernel's partial sums, [BW_TOK][RP] each
    int32_t step_end[LORA_MAX_SLICES];     // its 64-column steps of one tile, by slice
    int32_t u_ctas;
    const int32_t *sorted, *counts, *start_loc, *active, *no_lora;
    int32_t *error_word;
    int32_t nbins;
};

constexpr int backward_tab_words(int nbins, int loras) { return 4 * nbins + 2 + loras; }

__device__ __forceinline__ SegTab load_tab(const BackwardArgs &p, int *mem, int &tiles)
{
    const SegTab tab = seg_tab(mem, p.nbins);
    tiles = load_segments(p.no_lora, p.active, p.counts, p.start_loc, p.nbins, BW_TOK, tab, false, 0,
                          p.T, p.error_word);
    return tab;
}

// Tokens without an adapter: the metadata's first segment, or every token
// when the batch has no adapter at all (the order is then unset).  Their
// rows of dx are cleared (dx is overwritten, not added to).
__device__ __forceinline__ void clear_rest(const BackwardArgs &p, const SegTab &tab, int warp, int warps)
{
    const int lane = threadIdx.x & 31;
    const bool none = *p.no_lora != 0;
    const int rest = none ? p.T : (tab.id[0] == -1 ? tab.count[0] : 0);
    for (int64_t i = int64_t(blockIdx.x) * warps + warp; i < rest; i += int64_t(gridDim.x) * warps) {
        const int tok = none ? int(i) : checked_token(p.sorted[i], p.T, p.error_word);
        if (tok < 0) continue;
        uint16_t *dst = p.dx + int64_t(tok) * p.dx_ld;
        if (p.dx_vec) {
            for (int c = lane * 8; c < p.H; c += 256)
                *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
        } else {
            for (int c = lane; c < p.H; c += 32) dst[c] = 0;
        }
    }
}

// The segment of each adapter (-1: no tokens), in the words behind the table.
__device__ __forceinline__ const int *load_seg_of(const BackwardArgs &p, const SegTab &tab, int tiles,
                                                  int *mem)
{
    int *seg_of = mem + 4 * p.nbins + 2;
    for (int i = threadIdx.x; i < p.L; i += blockDim.x) seg_of[i] = -1;
    __syncthreads();
    if (tiles > 0)
        for (int k = threadIdx.x; k < p.nbins; k += blockDim.x)
            if (tab.id[k] >= 0 && tab.count[k] > 0) seg_of[tab.id[k]] = k;
    __syncthreads();
    return seg_of;
}

// The kernels on the tensor cores (lora_backward_tc.cu), for padded ranks 64
// and 128.  Each returns 0 when launched, -1 when the call does not fit it,
// or a cudaError_t.
int launch_grad_u_tc(const BackwardArgs &p, int rp, cudaStream_t st);
int launch_grad_x_tc(const BackwardArgs &p, int rp, cudaStream_t st);
// grad_w_tc takes the transposed g and u, so whether it fits is known before.
bool grad_w_tc_fits(const BackwardArgs &p, int rp);
int launch_grad_w_tc(const BackwardArgs &p, int rp, cudaStream_t st);

}  // namespace lora
