// lora_tc.cuh -- what the single-CTA tcgen05 kernels share: a ring of operand
// stages with its barriers, TMEM, and epilogues that write whole 128-byte
// pieces of rows.  Warps: 0 and 1 load, 2 issues UMMAs, 3 owns TMEM, 4..7 run
// the epilogue (thread = TMEM lane).
#pragma once

#include "lora_pair_gemm.cuh"

namespace lora {

constexpr int TC_THREADS = 256;
constexpr int TC_PANEL = 64 * 64 * 2;            // 64 rows of 64 bf16
constexpr int TC_SMEM = 227 * 1024;              // of a CTA
constexpr int TC_STAGE_ROWS = 4 * 32 * 128;      // the epilogue's staging: 32 rows x 128 bytes a warp
constexpr int TC_MAX_STAGES = 8;
constexpr int TC_BAR_BYTES = 256;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                            int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];\n"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// The ring of operand stages and the accumulators' barriers of one CTA.
struct TcRing {
    uint32_t ring, full, empty, accf, acce, drain, stage_bytes;
    int stages;
    volatile int *abort;
    uint32_t tmem;
};

// D += A B over 64 of K, as four UMMAs (K = 16): A K-major, B MN-major with
// panels of 64 x 64, both with the 128-byte swizzle.  The descriptors differ
// in their low words only, one add each: with 64-bit descriptors built for
// every UMMA, one thread issued M = 128, N = 128 every 108 clocks instead of
// every 75.  `more` is 0 for the accumulator's first product.
__device__ __forceinline__ void umma_k64(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t more)
{
    const uint64_t da = umma_desc_sw128(a), db = umma_desc_mn(b);
    const uint32_t a_hi = uint32_t(da >> 32), b_hi = uint32_t(db >> 32);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        asm volatile(
            "{\n.reg .pred p;\n.reg .b64 a, b;\n"
            "mov.b64 a, {%1, %2};\n"
            "mov.b64 b, {%3, %4};\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n"
            :: "r"(d_tmem), "r"(uint32_t(da) + kk * 2), "r"(a_hi), "r"(uint32_t(db) + kk * 128), "r"(b_hi),
               "r"(idesc), "r"(kk == 0 ? more : 1u) : "memory");
}

// Position in the ring.
struct TcPos {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// Shared memory: `ring` bytes (the stages, and what the kernel keeps behind
// them), the epilogue's staging, barriers; then the kernel's tables.
// COLS: TMEM columns of the CTA.
template <int COLS = 512>
__device__ __forceinline__ TcRing tc_setup(uint8_t *smem, int ring, int stage_bytes, int stages,
                                           int loaders)
{
    TcRing r;
    r.ring = smem_addr(smem);
    r.full = r.ring + ring + TC_STAGE_ROWS;
    r.empty = r.full + 8 * TC_MAX_STAGES;
    r.accf = r.empty + 8 * TC_MAX_STAGES;
    r.acce = r.accf + 16;
    r.drain = r.acce + 16;
    r.stage_bytes = uint32_t(stage_bytes);
    r.stages = stages;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + ring + TC_STAGE_ROWS + 16 * TC_MAX_STAGES + 40);
    r.abort = reinterpret_cast<volatile int *>(misc + 1);
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(r.full + 8 * i, uint32_t(loaders));
            mbar_init(r.empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(r.accf + 8 * i, 1);
            mbar_init(r.acce + 8 * i, 4);
        }
        mbar_init(r.drain, 1);
        mbar_fence_init();
        *r.abort = 0;
    }
    if (threadIdx.x / 32 == 3) tmem_alloc(smem_addr(misc), COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    r.tmem = *misc;
    return r;
}

// One thread of a loading warp, after its last fill: the fills of the last
// stages have landed and been consumed before the CTA may exit.
__device__ __forceinline__ void tc_drain_loads(const TcRing &r, int issued)
{
    const long long dd = clock64() + PG_TIMEOUT_CYCLES;
    for (int i = max(0, issued - r.stages); i < issued; ++i) {
        const uint32_t ph = uint32_t(i / r.stages) & 1u, b8 = 8u * uint32_t(i % r.stages);
        while (!mbar_try_wait(r.full + b8, ph) && clock64() < dd) {
        }
        while (!mbar_try_wait(r.empty + b8, ph) && !*r.abort && clock64() < dd) {
        }
    }
}

template <int COLS = 512>
__device__ __forceinline__ void tc_finish(const TcRing &r, int32_t *error_word)
{
    __syncwarp();
    if (threadIdx.x == 64 && *r.abort) {              // the thread that issues UMMAs
        umma_commit(r.drain);
        const long long dd = clock64() + PG_TIMEOUT_CYCLES;
        while (!mbar_try_wait(r.drain, 0) && clock64() < dd) {
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && *r.abort && error_word != nullptr) atomicOr(error_word, LORA_TIMEOUT_BIT);
    if (threadIdx.x / 32 == 3) tmem_dealloc(r.tmem, COLS);
}

// 32 accumulators of this thread's row as 32 bf16, times f.
__device__ __forceinline__ void pack32(const uint32_t (&v)[32], float f, uint32_t *o)
{
#pragma unroll
    for (int j = 0; j < 16; ++j)
        o[j] = pack_bf16x2(f * __uint_as_float(v[2 * j]), f * __uint_as_float(v[2 * j + 1]));
}

// 64 accumulators from `tmem` on, rounded: 32 words.
__device__ __forceinline__ void load64(uint32_t tmem, float f, uint32_t (&o)[32])
{
    uint32_t v0[32], v1[32];
    tmem_ld32_nowait(tmem, v0);
    tmem_ld32_nowait(tmem + 32, v1);
    tmem_wait_ld();
    pack32(v0, f, o);
    pack32(v1, f, o + 16);
}

// Writes a warp's 32 rows of 64 bf16: lane l holds row l (32 words) and where
// it goes (null: nowhere); the first `many` columns (a multiple of 8) are
// written.  Through 4 KB of the warp's shared memory, so that eight lanes
// write 128 bytes of one row: a store of 16 bytes a lane into 32 rows takes
// the load/store unit eight times as long.
__device__ __forceinline__ void store_rows(uint8_t *stage, const uint32_t (&o)[32], uint16_t *dst, int many)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((c ^ lane) & 7) * 16) =
            make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
    __syncwarp();
    const int c = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + (lane >> 3);
        uint16_t *to = reinterpret_cast<uint16_t *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
        if (to != nullptr && 8 * c < many)
            *reinterpret_cast<uint4 *>(to + 8 * c) =
                *reinterpret_cast<const uint4 *>(stage + row * 128 + ((c ^ row) & 7) * 16);
    }
}

// The same for 32 columns that are added to what is there, in fp32 with one
// rounding: lane l holds row l's 32 sums.
__device__ __forceinline__ void add_rows(uint8_t *stage, const uint32_t (&v)[32], float f, uint16_t *dst,
                                         int many)
{
    const int lane = threadIdx.x & 31, c = lane & 7;
    uint16_t *to[8];
    uint2 was[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        to[i] = reinterpret_cast<uint16_t *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), 4 * i + (lane >> 3)));
        was[i] = make_uint2(0u, 0u);
        if (to[i] != nullptr && 4 * c < many) was[i] = *reinterpret_cast<const uint2 *>(to[i] + 4 * c);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((k ^ lane) & 7) * 16) =
            make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + (lane >> 3);
        if (to[i] == nullptr || 4 * c >= many) continue;
        const float4 x = *reinterpret_cast<const float4 *>(stage + row * 128 + ((c ^ row) & 7) * 16);
        *reinterpret_cast<uint2 *>(to[i] + 4 * c) =
            make_uint2(pack_bf16x2(fmaf(f, x.x, bf16_lo(was[i].x)), fmaf(f, x.y, bf16_hi(was[i].x))),
                       pack_bf16x2(fmaf(f, x.z, bf16_lo(was[i].y)), fmaf(f, x.w, bf16_hi(was[i].y))));
    }
}

// Writes a warp's 32 columns of 64 rows of a row-major matrix: lane l holds
// column l (64 values, 32 words from the first row down); row r goes to dst
// + r * ld where first <= r < rows.  `many`: columns that exist (a multiple
// of 8).
__device__ __forceinline__ void store_columns(uint8_t *stage, const uint32_t (&o)[32], uint16_t *dst,
                                              int64_t ld, int first, int rows, int many)
{
    const int lane = threadIdx.x & 31;
    uint16_t *at = reinterpret_cast<uint16_t *>(stage);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        at[(2 * j) * 32 + lane] = uint16_t(o[j] & 0xFFFFu);
        at[(2 * j + 1) * 32 + lane] = uint16_t(o[j] >> 16);
    }
    __syncwarp();
    const int c = (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * i + (lane >> 2);
        if (r >= first && r < rows && c < many)
            *reinterpret_cast<uint4 *>(dst + r * ld + c) = *reinterpret_cast<const uint4 *>(at + r * 32 + c);
    }
}

__device__ __forceinline__ uint8_t *tc_smem()
{
    extern __shared__ uint8_t tc_smem_raw[];
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tc_smem_raw) + 1023) & ~uintptr_t(1023));
}

// What the ring may take beside `tables` words, in whole KB.
inline int tc_ring_bytes(int64_t words)
{
    return int((TC_SMEM - 1024 - TC_STAGE_ROWS - TC_BAR_BYTES - words * 4) / 1024 * 1024);
}

inline int tc_stages(int ring, int stage_bytes)
{
    return ring / stage_bytes < TC_MAX_STAGES ? ring / stage_bytes : TC_MAX_STAGES;
}

}  // namespace lora
