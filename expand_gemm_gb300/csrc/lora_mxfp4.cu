// lora_mxfp4.cu -- weights in microscaled 4 bits (OCP MXFP4): blocks of 32
// elements along a row share a scale of eight bits, a power of two,
//   s = max(floor(log2 max|v|) - 2, -127)     stored as s + 127, 255 = NaN
//   element = v / 2^s rounded to {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even
//             code, beyond 6 to 6; two to a byte, the even one in the low half
// A block that holds a NaN or an infinity becomes NaN as a whole.  Every
// element times its scale is a bf16 value, so decoding rounds nothing.
//
// Bound by memory: 2 or 4 bytes in and 0.53 out an element, and the reverse.
// 134 M elements from and to bf16: 57 and 55 us, 5.9 and 6.2 TB/s.  The loads
// of several eights go out together (one at a time: 124 us for both).
#include "lora_expert.cuh"

namespace lora {

constexpr int MX_THREADS = 256;

// 2^e for -127 <= e <= 127.
__device__ __forceinline__ float power2(int e)
{
    return __uint_as_float(e > -127 ? uint32_t(e + 127) << 23 : 0x00400000u);
}

// Two elements: a in the low half of the byte.
__device__ __forceinline__ uint32_t to_e2m1x2(float a, float b)
{
    uint32_t r;
    asm("{\n.reg .b8 t;\n"
        "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n"
        "cvt.u32.u8 %0, t;\n}\n"
        : "=r"(r) : "f"(a), "f"(b));
    return r;
}

// The value of a 4-bit element (s e e m).
__device__ __forceinline__ float e2m1_value(uint32_t code)
{
    // e and m where a float has its last exponent bits and first mantissa
    // bit: 2^-126 times the value, also for the subnormal 0.5
    return __uint_as_float((code & 8u) << 28 | (code & 7u) << 22) * 0x1p126f;
}

struct MxArgs {
    const void *weight;
    uint8_t *codes, *scales;
    void *out;
    int64_t eighths;              // elements / 8
};

constexpr int MX_MANY = 4;             // eights of a thread whose loads go out together

// A thread takes eight elements, four threads a block.
template <bool F32>
__global__ void __launch_bounds__(MX_THREADS) quantize_kernel(const MxArgs a)
{
    constexpr int MANY = F32 ? MX_MANY / 2 : MX_MANY;
    pdl_wait();
    const int64_t step = int64_t(gridDim.x) * MX_THREADS;
    // whole warps: the block's threads exchange their maxima
    const int64_t end = (a.eighths + 31) / 32 * 32;
    for (int64_t i0 = int64_t(blockIdx.x) * MX_THREADS + threadIdx.x; i0 < end; i0 += MANY * step) {
        uint4 raw[MANY][F32 ? 2 : 1];
#pragma unroll
        for (int m = 0; m < MANY; ++m) {
            const int64_t i = i0 + m * step;
#pragma unroll
            for (int h = 0; h < (F32 ? 2 : 1); ++h)
                raw[m][h] = i < a.eighths ? static_cast<const uint4 *>(a.weight)[F32 ? 2 * i + h : i] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MANY; ++m) {
            const int64_t i = i0 + m * step;
            if (i >= end) break;               // whole warps
            float v[8];
            if constexpr (F32) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[4 * h] = __uint_as_float(raw[m][h].x);
                    v[4 * h + 1] = __uint_as_float(raw[m][h].y);
                    v[4 * h + 2] = __uint_as_float(raw[m][h].z);
                    v[4 * h + 3] = __uint_as_float(raw[m][h].w);
                }
            } else {
                const uint32_t w[4] = {raw[m][0].x, raw[m][0].y, raw[m][0].z, raw[m][0].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = bf16_lo(w[j]);
                    v[2 * j + 1] = bf16_hi(w[j]);
                }
            }
            // magnitudes as integers: their order is the values', and a NaN
            // or an infinity is the largest
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // below 2^-126 the exponent field says less than it is, and the
            // scale is 2^-127 all the same
            const int s = max(int(top >> 23) - 129, -127);
            const bool bad = top >= 0x7F800000u;
            const float f = power2(-s);
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) word |= to_e2m1x2(v[2 * j] * f, v[2 * j + 1] * f) << (8 * j);
            if (i < a.eighths) {
                reinterpret_cast<uint32_t *>(a.codes)[i] = bad ? 0u : word;
                if ((threadIdx.x & 3) == 0) a.scales[i / 4] = uint8_t(bad ? 255 : s + 127);
            }
        }
    }
}

// Eight elements of a block with scale byte c, as fp32.
__device__ __forceinline__ void decode8(uint32_t word, uint32_t c, float (&v)[8])
{
    const float f = c == 255u ? __uint_as_float(0x7FC00000u) : power2(int(c) - 127);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e2m1_value(word >> (4 * j) & 15u) * f;
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

template <bool F32>
__global__ void __launch_bounds__(MX_THREADS) dequantize_kernel(const MxArgs a)
{
    pdl_wait();
    const int64_t step = int64_t(gridDim.x) * MX_THREADS;
    for (int64_t i0 = int64_t(blockIdx.x) * MX_THREADS + threadIdx.x; i0 < a.eighths; i0 += MX_MANY * step) {
        uint32_t word[MX_MANY], c[MX_MANY];
#pragma unroll
        for (int m = 0; m < MX_MANY; ++m) {
            const int64_t i = i0 + m * step;
            word[m] = i < a.eighths ? reinterpret_cast<const uint32_t *>(a.codes)[i] : 0u;
            c[m] = i < a.eighths ? a.scales[i / 4] : 0u;
        }
#pragma unroll
        for (int m = 0; m < MX_MANY; ++m) {
            const int64_t i = i0 + m * step;
            if (i >= a.eighths) break;
            float v[8];
            decode8(word[m], c[m], v);
            if constexpr (F32) {
                float4 *to = static_cast<float4 *>(a.out) + 2 * i;
                to[0] = make_float4(v[0], v[1], v[2], v[3]);
                to[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                static_cast<uint4 *>(a.out)[i] = pack8(v);
            }
        }
    }
}

struct DecodeArgs {
    ExpertArgs p;
    uint16_t *out;
};

// The same for the experts of the metadata's segments only: blockIdx.y takes
// every gridDim.y-th segment.
// Runs beside the copy of x, which it needs nothing of: the kernels before that
// are complete when it lets this one begin.  It ends after it, for the product
// waits for this one alone.
__global__ void __launch_bounds__(MX_THREADS) expert_decode_kernel(const __grid_constant__ DecodeArgs a)
{
    const ExpertArgs &p = a.p;
    const int bins = *p.no_lora ? 0 : p.nbins;
    const int64_t per = int64_t(p.N) * p.K / 8, step = int64_t(gridDim.x) * MX_THREADS;
    for (int k = blockIdx.y; k < bins; k += gridDim.y) {
        const int e = p.active[k];
        if (e < 0 || e >= p.E || p.counts[k] <= 0) continue;
        const uint32_t *codes = reinterpret_cast<const uint32_t *>(p.codes) + e * per;
        const uint8_t *scales = p.scales + e * (per / 4);
        uint4 *out = reinterpret_cast<uint4 *>(a.out) + e * per;
        for (int64_t i = int64_t(blockIdx.x) * MX_THREADS + threadIdx.x; i < per; i += step) {
            float v[8];
            decode8(codes[i], scales[i / 4], v);
            out[i] = pack8(v);
        }
    }
    pdl_wait();
}

static unsigned grid_for(int64_t eighths)
{
    const int64_t want = (eighths + MX_THREADS - 1) / MX_THREADS, most = 8ll * device_sm_count();
    return unsigned(want < most ? want : most);
}

int launch_expert_decode(const ExpertArgs &p, uint16_t *out, cudaStream_t st)
{
    DecodeArgs a{p, out};
    // every segment's blocks could fill the GPU alone; those of segments
    // without rows return at once
    const int y = p.nbins < 64 ? p.nbins : 64;
    const unsigned x = grid_for(int64_t(p.N) * p.K / 8);
    return int(launch_kernel(expert_decode_kernel, dim3(x, unsigned(y)), dim3(MX_THREADS), 0, st, a));
}

static bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace lora

LORA_API int lora_quantize_mxfp4(const void *weight, int32_t weight_f32, int64_t elements, uint8_t *codes,
                                 uint8_t *scales, void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_quantize_mxfp4");
    if (elements < 0 || elements % 32 != 0) return LORA_ERR_SIZE;
    if (elements == 0) return LORA_OK;
    if (weight == nullptr || codes == nullptr || scales == nullptr) return LORA_ERR_NULL;
    if (off16(weight) || off16(codes)) return LORA_ERR_ALIGN;
    const MxArgs a{weight, codes, scales, nullptr, elements / 8};
    const auto kernel = weight_f32 ? quantize_kernel<true> : quantize_kernel<false>;
    return int(launch_kernel(kernel, dim3(grid_for(a.eighths)), dim3(MX_THREADS), 0,
                             static_cast<cudaStream_t>(stream), a));
}

LORA_API int lora_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t elements, void *out,
                                   int32_t out_f32, void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_dequantize_mxfp4");
    if (elements < 0 || elements % 32 != 0) return LORA_ERR_SIZE;
    if (elements == 0) return LORA_OK;
    if (out == nullptr || codes == nullptr || scales == nullptr) return LORA_ERR_NULL;
    if (off16(out) || off16(codes)) return LORA_ERR_ALIGN;
    const MxArgs a{nullptr, const_cast<uint8_t *>(codes), const_cast<uint8_t *>(scales), out, elements / 8};
    const auto kernel = out_f32 ? dequantize_kernel<true> : dequantize_kernel<false>;
    return int(launch_kernel(kernel, dim3(grid_for(a.eighths)), dim3(MX_THREADS), 0,
                             static_cast<cudaStream_t>(stream), a));
}
