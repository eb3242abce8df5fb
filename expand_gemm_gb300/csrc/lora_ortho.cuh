// lora_ortho.cuh -- what the kernels of lora_orthogonalize share.
#pragma once

#include "lora_frag.cuh"

namespace lora {

constexpr int OR_THREADS = 256;
constexpr int OR_MAX_RANK = 128;

struct OrthoArgs {
    const void *u;
    uint16_t *out;
    int32_t count, rows, cols;    // matrices, each [rows, cols]
    int32_t r, n;                 // short and long side
    int32_t units, unit;          // of the long side in the sum U U^T; a unit's length
    int32_t ctas;                 // that share the units of all matrices
    int32_t steps;
    float a, b, c, eps, scale;
    float *gram;                  // partial sums, [ctas + count][RP][RP]
    uint16_t *p;                  // [count][2][RP][RP]: P as two bf16 terms
    int32_t *error_word;
};

// The units of all matrices, in order, are cut into p.ctas even runs.  CTA c
// takes units [unit_begin(c), unit_begin(c + 1)); its part of matrix m's sum
// goes to slot c + m (a new slot whenever the CTA or the matrix changes), so
// matrix m is the sum of slots c + m over the CTAs that hold its units, in
// that order.
__device__ __forceinline__ int64_t unit_begin(const OrthoArgs &p, int c)
{
    return int64_t(p.count) * p.units * c / p.ctas;
}
__device__ __forceinline__ int unit_cta(const OrthoArgs &p, int64_t unit)
{
    return int(((unit + 1) * p.ctas - 1) / (int64_t(p.count) * p.units));
}

// Eight consecutive fp32 entries as bf16 terms: hi, and what hi leaves over.
struct Chunk {
    uint4 hi, lo;
};

__device__ __forceinline__ Chunk split_chunk(const float4 &x, const float4 &y)
{
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        l[i] = pack_bf16x2(v[2 * i] - bf16_lo(h[i]), v[2 * i + 1] - bf16_hi(h[i]));
    }
    return Chunk{make_uint4(h[0], h[1], h[2], h[3]), make_uint4(l[0], l[1], l[2], l[3])};
}

// Padded ranks 64 and 128 (lora_ortho_tc.cu).  Returns 0 or an error.
int run_ortho_tc(OrthoArgs p, int rp, bool f32, cudaStream_t st);
constexpr int OR_TC_UNIT = 64;
constexpr int OR_TC_CTAS = 2;         // of the sum U U^T on an SM

// Runs of steps that the r x r iteration does not hold (lora_ortho_long.cu):
// |a|^steps above this.  Five steps of 3.4445 are 485, fifteen of 1.5 are 438.
constexpr double OR_LONG_GROWTH = 512.0;
int64_t ortho_long_bytes(int r, int n, int rp);       // of workspace, for one matrix
int run_ortho_long(const OrthoArgs &o, int rp, bool f32, void *workspace, int64_t bytes, cudaStream_t st);

}  // namespace lora
