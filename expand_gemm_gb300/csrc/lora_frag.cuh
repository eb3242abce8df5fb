// lora_frag.cuh -- mma.sync fragments from swizzled bf16 tiles in shared
// memory, with either operand stored along K or across it.
#pragma once

#include "lora_common.cuh"

namespace lora {

__device__ __forceinline__ void ldmatrix_x4_t(uint32_t addr, uint32_t &r0, uint32_t &r1,
                                              uint32_t &r2, uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr));
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a bf16 tile with
// CPR chunks a row; tiles wider than 64 elements are panels of 64.
template <int CPR, int ROWS>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk)
{
    if constexpr (CPR > 8)
        return uint32_t((chunk >> 3) * ROWS * 128) + swz<8>(row, chunk & 7);
    else
        return swz<CPR>(row, chunk);
}

// A fragment (16 x 16) at (m0, k0).  KM: the tile's rows are M; otherwise
// its rows are K.
template <int CPR, int ROWS, bool KM>
__device__ __forceinline__ void frag_a(uint32_t tile, int m0, int k0, uint32_t (&a)[4])
{
    const int lane = threadIdx.x & 31;
    if constexpr (KM) {
        const int row = m0 + (lane & 15), ch = k0 / 8 + (lane >> 4);
        ldmatrix_x4(tile + tile_at<CPR, ROWS>(row, ch), a[0], a[1], a[2], a[3]);
    } else {
        const int row = k0 + (lane & 7) + ((lane >> 4) << 3), ch = m0 / 8 + ((lane >> 3) & 1);
        ldmatrix_x4_t(tile + tile_at<CPR, ROWS>(row, ch), a[0], a[1], a[2], a[3]);
    }
}

// Two B fragments (16 K x 8 N each) at (k0, n0) and (k0, n0 + 8).  KN: the
// tile's rows are N; otherwise its rows are K.
template <int CPR, int ROWS, bool KN>
__device__ __forceinline__ void frag_b(uint32_t tile, int k0, int n0, uint32_t (&b)[4])
{
    const int lane = threadIdx.x & 31;
    if constexpr (KN) {
        const int row = n0 + (lane & 7) + ((lane >> 4) << 3), ch = k0 / 8 + ((lane >> 3) & 1);
        ldmatrix_x4(tile + tile_at<CPR, ROWS>(row, ch), b[0], b[1], b[2], b[3]);
    } else {
        const int row = k0 + (lane & 15), ch = n0 / 8 + (lane >> 4);
        ldmatrix_x4_t(tile + tile_at<CPR, ROWS>(row, ch), b[0], b[1], b[2], b[3]);
    }
}

// One B fragment (16 K x 8 N) at (k0, n0) of a tile whose rows are K.
template <int CPR, int ROWS>
__device__ __forceinline__ void frag_b1(uint32_t tile, int k0, int n0, uint32_t (&b)[2])
{
    const int lane = threadIdx.x & 15;         // lanes 16 to 31 name rows too, unused
    const uint32_t addr = tile + tile_at<CPR, ROWS>(k0 + lane, n0 / 8);
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];\n"
                 : "=r"(b[0]), "=r"(b[1]) : "r"(addr));
}

}  // namespace lora
