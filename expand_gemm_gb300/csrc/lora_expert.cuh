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
    int32_t *from;                    // the row that each row of the copies holds, -1: padding
    int32_t later;                    // x is copied beside the product of dx, not before it
    int32_t early;                    // weights are asked for while x is copied
    int64_t dys_ld;
    ExpertTile *table;
    int32_t *tiles;                   // [1]: entries of the table
    int32_t *copied;                  // [1]: padded blocks of the copies, beside it
    int2 *blocks;                     // [E]: first K block and K blocks of dW
    int32_t R, fan, K, N, E, nbins;
    int64_t rows;                     // that the copies have room for
    int32_t entries;                  // that the table has room for
    int32_t add, pad, tile_rows;
    int32_t x_vec, dy_vec, dx_vec;
    const int32_t *ids, *sorted, *counts, *start_loc, *active, *no_lora;
    int32_t *error_word;
};

// The row that the metadata names at `at` < R, -1 where that is none of the
// batch's (metadata that were prepared for more rows than the call has).
__device__ __forceinline__ int expert_row(const ExpertArgs &p, int at)
{
    const int row = checked_token(p.sorted[at], p.R, p.error_word);
    return row < p.R ? row : -1;
}

// One row of `cols` bf16, by a warp.  Whole 16-byte pieces where both ends
// allow it.
__device__ __forceinline__ void copy_row(uint16_t *dst, const uint16_t *src, int cols, bool vec)
{
    const int lane = threadIdx.x & 31;
    if (vec) {
        const int n = cols / 8;
        const uint4 *from = reinterpret_cast<const uint4 *>(src);
        uint4 *to = reinterpret_cast<uint4 *>(dst);
        int c = lane;
        for (; c + 96 < n; c += 128) {
            const uint4 a = from[c], b = from[c + 32], d = from[c + 64], e = from[c + 96];
            to[c] = a;
            to[c + 32] = b;
            to[c + 64] = d;
            to[c + 96] = e;
        }
        for (; c < n; c += 32) to[c] = from[c];
        for (int i = n * 8 + lane; i < cols; i += 32) dst[i] = src[i];
    } else {
        // eight loads before their stores: one after another they wait for
        // each other's way through memory
        for (int i0 = lane; i0 < cols; i0 += 256) {
            uint16_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i0 + 32 * k < cols ? src[i0 + 32 * k] : uint16_t(0);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i0 + 32 * k < cols) dst[i0 + 32 * k] = v[k];
        }
    }
}

__device__ __forceinline__ void clear_row(uint16_t *dst, int64_t cols)
{
    for (int c = threadIdx.x & 31; c < int(cols / 8); c += 32)
        reinterpret_cast<uint4 *>(dst)[c] = make_uint4(0, 0, 0, 0);
}

// dx[t] (+)= the sum of the token's rows, in fp32 and in their order, rounded
// once.  Rows without an expert have no part.  Warp `warp` of `warps`, a token
// at a time, 512 columns of it: with 128 the loads of four warps an SM took
// longer than the product they run beside.
__device__ __forceinline__ void join_rows(const ExpertArgs &p, int64_t warp, int64_t warps)
{
    constexpr int MANY = 4;
    const int lane = threadIdx.x & 31;
    const bool none = *p.no_lora != 0;
    const int64_t T = p.R / p.fan;
    for (int64_t t = warp; t < T; t += warps) {
        const int32_t *ids = p.ids + t * p.fan;
        const float *part = p.part + t * p.fan * p.K;
        uint16_t *out = p.dx + t * p.dx_ld;
        bool any = false;
        for (int j = 0; !none && j < p.fan; ++j) any = any || (ids[j] >= 0 && ids[j] < p.E);
        if (p.add && !any) continue;
        for (int c0 = lane * 4; c0 < p.K; c0 += 128 * MANY) {
            float4 s[MANY];
            bool first = true;
#pragma unroll
            for (int k = 0; k < MANY; ++k) s[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (any) {
#pragma unroll 2
                for (int j = 0; j < p.fan; ++j) {
                    const int id = ids[j];
                    if (id < 0 || id >= p.E) continue;
                    float4 v[MANY];
#pragma unroll
                    for (int k = 0; k < MANY; ++k) {
                        const int c = c0 + 128 * k;
                        v[k] = c < p.K ? *reinterpret_cast<const float4 *>(part + int64_t(j) * p.K + c)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
#pragma unroll
                    for (int k = 0; k < MANY; ++k)
                        // the first part as it is: 0 + -0 would lose its sign
                        s[k] = first ? v[k] : make_float4(s[k].x + v[k].x, s[k].y + v[k].y, s[k].z + v[k].z, s[k].w + v[k].w);
                    first = false;
                }
            }
#pragma unroll
            for (int k = 0; k < MANY; ++k) {
                const int c = c0 + 128 * k;
                if (c >= p.K) break;
                if (p.dx_vec) {
                    uint2 *to = reinterpret_cast<uint2 *>(out + c);
                    if (p.add) {
                        const uint2 was = *to;
                        s[k] = make_float4(s[k].x + bf16_lo(was.x), s[k].y + bf16_hi(was.x), s[k].z + bf16_lo(was.y),
                                           s[k].w + bf16_hi(was.y));
                    }
                    *to = make_uint2(pack_bf16x2(s[k].x, s[k].y), pack_bf16x2(s[k].z, s[k].w));
                } else {
                    const float v[4] = {s[k].x, s[k].y, s[k].z, s[k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        out[c + i] = uint16_t(pack_bf16x2(v[i] + (p.add ? bf16_to_f32(out[c + i]) : 0.0f), 0.0f) & 0xFFFFu);
                }
            }
        }
    }
}

// Allows a kernel `bytes` of dynamic shared memory on the current device
// (lora_expert.cu); `done` holds the devices where it was.
int expert_shared_memory(const void *kernel, int bytes, std::atomic<uint64_t> &done);

// lora_expert_gemm.cu: products on CTA pairs over the copies.
int launch_expert_forward(const ExpertArgs &p, cudaStream_t st);
int launch_expert_dx(const ExpertArgs &p, cudaStream_t st);
int launch_expert_dw(const ExpertArgs &p, cudaStream_t st);

// lora_expert_stream.cu: few rows an expert, weights in either form.  Where it
// walks the metadata's segments itself it needs no table (p.table is null): to
// ask for weights while x is copied, and where it gathers, without a copy.
bool expert_stream_early(const ExpertArgs &p);
bool expert_stream_gathers(const ExpertArgs &p);
int launch_expert_stream(const ExpertArgs &p, cudaStream_t st);

// lora_mxfp4.cu: the weights of the experts that have rows, decoded to bf16.
int launch_expert_decode(const ExpertArgs &p, uint16_t *out, cudaStream_t st);

}  // namespace lora
