// lora_clip.cu -- lora_clip_gradients: the norm of many tensors' gradients,
// together or for every adapter of their stacks, and the gradients scaled
// down to a largest norm:
//   norms[g] = sqrt(sum over tensors and elements of slice g of v^2)
//   out      = v min(1, max_norm / (norms[g] + eps))
//
// Bound by memory: the gradients are read for the norm and once more to be
// scaled.  Every slice is cut into units of 2^unit_log elements; CTAs take
// even runs of units, group by group, so that a CTA leaves one partial sum for
// each group that it meets, in an order that depends on the sizes alone: equal
// inputs give equal bits.  940 MB of gradients: norm 138 us (6.8 TB/s), scaling
// 285 (6.6 TB/s read and written); 6 MB: 9 us in all, two launches.
//
// Squares are summed in fp32 over up to 33 elements of a thread and in fp64
// from there on.  Eight values whose squares would overflow fp32 or lose
// digits to underflow (magnitudes above 2^60, or all below 2^-50) are squared
// in fp64.
#include <math.h>

#include "lora_common.cuh"

namespace lora {

constexpr int CL_THREADS = 512;
constexpr int CL_UNIT_LOG = 14;                // units of 2^14 elements, or of
constexpr int CL_LONG_LOG = 17;                // 2^17 where there are many
constexpr int CL_FEW = 64;                     // tensors of a launch: with so many
constexpr int CL_MANY = 1024;                  // or so many, 28 bytes of arguments each

// What a group's gradients are multiplied by, mantissa * 2^exponent: a norm of
// 2^126 largest norms leaves a factor that 32 bits hold with few digits or as
// zero, and its largest gradients still count.  The exponent is 0 where the
// mantissa alone, a normal number or zero, is the factor.
struct ClipFactor {
    float mantissa;
    int32_t exponent;
};

struct ClipShared {
    int32_t tensors, groups;
    int32_t unit_log;
    int32_t units;                             // of one slice of all tensors of the launch
    int64_t run;                               // units of a CTA
    int32_t add;                               // the sums are added to those of earlier tensors
    double *part;                              // [CTAs + groups]: CTA c's sum for group g at c + g
    double *sum;                               // [groups]
    ClipFactor *factor;                        // [groups]
    float *norms;                              // [groups]
    float max_norm, eps;
    int32_t scale;                             // 0: norms only (out then receives copies)
};

template <int MAX>
struct ClipArgs {
    ClipShared s;
    const void *in[MAX];
    void *out[MAX];
    int64_t n[MAX];                            // elements of a slice; bit 62: fp32
    int32_t end[MAX];                          // units of a slice up to and with this tensor
};
constexpr int64_t CL_F32 = int64_t(1) << 62;
static_assert(sizeof(ClipArgs<CL_MANY>) <= 32764, "kernel arguments");

// A CTA's place among the units: the group, the unit in its slice, and the
// tensor that the unit belongs to.
template <int MAX>
struct ClipWalk {
    int64_t left;                              // units to go, this one among them
    int group, unit, tensor;

    __device__ __forceinline__ ClipWalk(const ClipArgs<MAX> &a, bool back)
    {
        const int64_t total = int64_t(a.s.units) * a.s.groups, first = blockIdx.x * a.s.run;
        const int64_t last = min(total, first + a.s.run) - 1, at = back ? last : first;
        left = last - first + 1;
        group = int(at / a.s.units);
        unit = int(at - int64_t(group) * a.s.units);
        int lo = 0, hi = a.s.tensors - 1;      // the first tensor that ends behind the unit
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.end[mid] > unit) hi = mid; else lo = mid + 1;
        }
        tensor = lo;
    }
    __device__ __forceinline__ void next(const ClipArgs<MAX> &a)
    {
        --left;
        if (++unit == a.s.units) {
            unit = tensor = 0;
            ++group;
        }
        while (tensor < a.s.tensors - 1 && a.end[tensor] <= unit) ++tensor;
    }
    __device__ __forceinline__ void back(const ClipArgs<MAX> &a)
    {
        --left;
        if (--unit < 0) {
            unit = a.s.units - 1;
            tensor = a.s.tensors - 1;
            --group;
        }
        while (tensor > 0 && a.end[tensor - 1] > unit) --tensor;
    }
};

__device__ __forceinline__ void clip_unpack(const uint4 &w, bool f32, float (&v)[8])
{
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = f32 ? __uint_as_float(r[j]) : bf16_lo(r[j]);
        v[2 * j + 1] = f32 ? 0.0f : bf16_hi(r[j]);
    }
}

// The squares of eight values (of four where they are fp32).
__device__ __forceinline__ void clip_add(const float (&v)[8], float &acc, double &far)
{
    float s = 0.0f, top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        s = fmaf(v[j], v[j], s);
        top = fmaxf(top, fabsf(v[j]));
    }
    if ((top <= 0x1p60f && top >= 0x1p-50f) || top == 0.0f) {
        acc += s;                              // NaN among zeros ends here too
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) far += double(v[j]) * double(v[j]);
    }
}

// The block's sum in thread 0.  One warp adds: fp64 runs at two additions a
// clock on an SM, and 512 threads' shuffles are 2560 of them.
__device__ __forceinline__ double block_sum(double v, double *all)
{
    __syncthreads();
    all[threadIdx.x] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x < 32) {
        for (int i = threadIdx.x; i < CL_THREADS; i += 32) s += all[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    return s;
}

// Where unit `unit` of slice `group` lies: its first element and how many.
struct ClipUnit {
    const char *in;
    char *out;
    int count;
    bool f32;
};
template <int MAX>
__device__ __forceinline__ ClipUnit clip_unit(const ClipArgs<MAX> &a, const ClipWalk<MAX> &w)
{
    const int t = w.tensor;
    const int64_t n = a.n[t] & ~CL_F32;
    ClipUnit u;
    u.f32 = (a.n[t] & CL_F32) != 0;
    const int64_t at = int64_t(w.unit - (t > 0 ? a.end[t - 1] : 0)) << a.s.unit_log;
    const int64_t first = (w.group * n + at) * (u.f32 ? 4 : 2);
    u.in = static_cast<const char *>(a.in[t]) + first;
    u.out = static_cast<char *>(a.out[t]) + first;
    u.count = int(min(n - at, int64_t(1) << a.s.unit_log));
    return u;
}

__device__ __forceinline__ float clip_load(const char *p, bool f32, int i)
{
    return f32 ? reinterpret_cast<const float *>(p)[i] : bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
}

template <int MAX>
__global__ void __launch_bounds__(CL_THREADS, 3) clip_sum_kernel(const __grid_constant__ ClipArgs<MAX> a)
{
    __shared__ double s_all[CL_THREADS];
    pdl_wait();
    double far = 0.0;
    for (ClipWalk<MAX> w(a, false); w.left > 0;) {
        const ClipUnit c = clip_unit(a, w);
        const int per = c.f32 ? 4 : 8;
        float acc = 0.0f;
        // elements before the first 16-byte boundary and behind the last
        const int head = min(c.count, int((16 - (reinterpret_cast<uintptr_t>(c.in) & 15u)) & 15u) / (c.f32 ? 4 : 2));
        const int whole = (c.count - head) / per;
        const uint4 *src = reinterpret_cast<const uint4 *>(c.in + head * (c.f32 ? 4 : 2));
        const int rest = c.count - whole * per;              // single elements: head, then tail
        if (int(threadIdx.x) < rest) {
            const int i = int(threadIdx.x) < head ? int(threadIdx.x) : int(threadIdx.x) + whole * per;
            const float v[8] = {clip_load(c.in, c.f32, i), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            clip_add(v, acc, far);
        }
        int i = threadIdx.x;
        for (; i + 3 * CL_THREADS < whole; i += 4 * CL_THREADS) {
            uint4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = src[i + k * CL_THREADS];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float v[8];
                clip_unpack(w[k], c.f32, v);
                clip_add(v, acc, far);
            }
            far += double(acc);                // of up to 33 squares
            acc = 0.0f;
        }
        for (; i < whole; i += CL_THREADS) {
            float v[8];
            clip_unpack(src[i], c.f32, v);
            clip_add(v, acc, far);
        }
        far += double(acc);
        const int group = w.group;
        w.next(a);
        if (w.left == 0 || w.group != group) {
            const double s = block_sum(far, s_all);
            if (threadIdx.x == 0) a.s.part[blockIdx.x + group] = s;
            far = 0.0;
        }
    }
}

// The factor of a group with this norm, which is in 64 bits: it may lie beyond
// fp32.  A zero gradient stays one; NaN stays NaN.
__device__ __forceinline__ ClipFactor clip_factor(const ClipShared &a, double norm)
{
    if (!a.scale) return {1.0f, 0};
    const double f = double(a.max_norm) / (norm + double(a.eps));
    if (f >= 1.0 || norm == 0.0) return {1.0f, 0};
    if (f > 0.0 && f < 0x1p-126) {
        int e;
        const double m = frexp(f, &e);
        return {float(m), e};
    }
    return {float(f), 0};
}

// The partial sums of a group, by a warp, in an order that depends on their
// number alone.
__device__ __forceinline__ double clip_group_sum(const ClipShared &a, int g, int from, int to)
{
    double s = 0.0;
    for (int c = from + int(threadIdx.x & 31); c <= to; c += 32) s += a.part[c + g];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The partial sums of a group, in order; its norm and factor.  One warp a
// group.  (Where one launch holds all tensors and the gradients are written,
// clip_scale_kernel does this itself.)
__global__ void __launch_bounds__(256) clip_join_kernel(const ClipShared a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    for (int g = blockIdx.x * 8 + (threadIdx.x >> 5); g < a.groups; g += gridDim.x * 8) {
        const int64_t first = int64_t(g) * a.units, last = first + a.units;
        const int from = int(first / a.run), to = int((last - 1) / a.run);
        double s = clip_group_sum(a, g, from, to);
        if (lane == 0) {
            if (a.add) s += a.sum[g];
            const double norm = sqrt(s);
            a.sum[g] = s;
            a.norms[g] = float(norm);
            a.factor[g] = clip_factor(a, norm);
        }
    }
}

// out = v * factor.  Units are taken from the last one back: the end of what
// the norm read may still lie in L2.  JOIN: every CTA adds up the partial sums
// of its groups, which saves a launch (one layer's adapters: 12 -> 9 us); the
// one with a group's first unit writes its norm.
template <int MAX, bool JOIN>
__global__ void __launch_bounds__(CL_THREADS, 3) clip_scale_kernel(const __grid_constant__ ClipArgs<MAX> a)
{
    __shared__ ClipFactor s_factor;
    pdl_wait();
    int known = -1;
    ClipFactor by{1.0f, 0};
    for (ClipWalk<MAX> w(a, true); w.left > 0; w.back(a)) {
        const ClipUnit c = clip_unit(a, w);
        if (w.group != known) {
            known = w.group;
            if constexpr (JOIN) {
                const int64_t first = int64_t(known) * a.s.units;
                const int from = int(first / a.s.run), to = int((first + a.s.units - 1) / a.s.run);
                __syncthreads();
                if (threadIdx.x < 32) {
                    const double norm = sqrt(clip_group_sum(a.s, known, from, to));
                    if (threadIdx.x == 0) {
                        if (int(blockIdx.x) == from) a.s.norms[known] = float(norm);
                        s_factor = clip_factor(a.s, norm);
                    }
                }
                __syncthreads();
                by = s_factor;
            } else {
                by = a.s.factor[known];
            }
        }
        const float f = by.mantissa;
        if (f == 1.0f && by.exponent == 0 && c.in == c.out) continue;
        if (by.exponent != 0) {                // rare
            for (int i = threadIdx.x; i < c.count; i += CL_THREADS) {
                const float v = scalbnf(clip_load(c.in, c.f32, i) * f, by.exponent);
                if (c.f32) reinterpret_cast<float *>(c.out)[i] = v;
                else reinterpret_cast<uint16_t *>(c.out)[i] = uint16_t(pack_bf16x2(v, 0.0f) & 0xFFFFu);
            }
            continue;
        }
        const int size = c.f32 ? 4 : 2, per = 16 / size;
        const bool same = ((reinterpret_cast<uintptr_t>(c.in) ^ reinterpret_cast<uintptr_t>(c.out)) & 15u) == 0;
        const int head = same ? min(c.count, int((16 - (reinterpret_cast<uintptr_t>(c.in) & 15u)) & 15u) / size)
                              : c.count;
        const int whole = (c.count - head) / per;
        for (int j = threadIdx.x; j < c.count - whole * per; j += CL_THREADS) {
            const int i = j < head ? j : j + whole * per;
            const float v = clip_load(c.in, c.f32, i) * f;
            if (c.f32) reinterpret_cast<float *>(c.out)[i] = v;
            else reinterpret_cast<uint16_t *>(c.out)[i] = uint16_t(pack_bf16x2(v, 0.0f) & 0xFFFFu);
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(c.in + head * size);
        uint4 *dst = reinterpret_cast<uint4 *>(c.out + head * size);
        auto scaled = [&](const uint4 &w) {
            if (c.f32)
                return make_uint4(__float_as_uint(__uint_as_float(w.x) * f), __float_as_uint(__uint_as_float(w.y) * f),
                                  __float_as_uint(__uint_as_float(w.z) * f), __float_as_uint(__uint_as_float(w.w) * f));
            return make_uint4(pack_bf16x2(bf16_lo(w.x) * f, bf16_hi(w.x) * f),
                              pack_bf16x2(bf16_lo(w.y) * f, bf16_hi(w.y) * f),
                              pack_bf16x2(bf16_lo(w.z) * f, bf16_hi(w.z) * f),
                              pack_bf16x2(bf16_lo(w.w) * f, bf16_hi(w.w) * f));
        };
        int i = threadIdx.x;
        for (; i + 3 * CL_THREADS < whole; i += 4 * CL_THREADS) {
            uint4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = src[i + k * CL_THREADS];
#pragma unroll
            for (int k = 0; k < 4; ++k) dst[i + k * CL_THREADS] = scaled(w[k]);
        }
        for (; i < whole; i += CL_THREADS) dst[i] = scaled(src[i]);
    }
}

// ---------------------------------------------------------------- host

struct ClipPlan {
    int32_t groups;
    int ctas;                                  // most CTAs of a launch
    int64_t sum, factor, bytes;
};

static ClipPlan clip_plan(int32_t groups)
{
    ClipPlan p;
    p.groups = groups;
    p.ctas = 3 * device_sm_count();            // as many as fit
    const int64_t part = (int64_t(p.ctas) + groups) * 8;
    p.sum = (part + 255) / 256 * 256;
    p.factor = p.sum + (int64_t(groups) * 8 + 255) / 256 * 256;
    p.bytes = p.factor + (int64_t(groups) * 8 + 255) / 256 * 256;
    return p;
}

static int64_t clip_units(int64_t n, int log) { return (n + (int64_t(1) << log) - 1) >> log; }

struct ClipCall {
    const void *const *grads;
    void *const *out;
    const int64_t *sizes;
    const int32_t *f32;
    int32_t tensors;
    ClipShared s;
};

// Returns the CTAs, 0 where there is nothing to do.
template <int MAX>
static int clip_args(ClipArgs<MAX> &a, const ClipCall &c, int first, int most)
{
    a.s = c.s;
    a.s.tensors = c.tensors - first < MAX ? c.tensors - first : MAX;
    int64_t units = 0;
    for (int i = 0; i < a.s.tensors; ++i) {
        const int64_t n = c.sizes[first + i];
        a.in[i] = c.grads[first + i];
        a.out[i] = c.out != nullptr ? c.out[first + i] : const_cast<void *>(c.grads[first + i]);
        a.n[i] = n | (c.f32[first + i] ? CL_F32 : 0);
        units += clip_units(n, a.s.unit_log);
        a.end[i] = int32_t(units);
    }
    a.s.units = int32_t(units);
    const int64_t total = units * a.s.groups;
    a.s.run = (total + most - 1) / most;
    return total > 0 ? int((total + a.s.run - 1) / a.s.run) : 0;
}

template <int MAX>
static int run_clip(const ClipCall &c, int most, cudaStream_t st)
{
    const bool write = c.s.scale || c.out != nullptr, join = !write || c.tensors > MAX;
    bool any = false;
    ClipArgs<MAX> a;
    for (int first = 0; first < c.tensors; first += MAX) {
        const int ctas = clip_args(a, c, first, most);
        if (ctas == 0) continue;
        a.s.add = any;
        any = true;
        cudaError_t e = launch_kernel(clip_sum_kernel<MAX>, dim3(unsigned(ctas)), dim3(CL_THREADS), 0, st, a);
        if (e != cudaSuccess) return int(e);
        if (!join) continue;
        const int joins = (c.s.groups + 7) / 8 < 64 ? (c.s.groups + 7) / 8 : 64;
        e = launch_kernel(clip_join_kernel, dim3(unsigned(joins)), dim3(256), 0, st, a.s);
        if (e != cudaSuccess) return int(e);
    }
    if (!any) return int(cudaMemsetAsync(c.s.norms, 0, size_t(c.s.groups) * sizeof(float), st));
    if (!write) return LORA_OK;
    const auto scale = join ? clip_scale_kernel<MAX, false> : clip_scale_kernel<MAX, true>;
    for (int first = 0; first < c.tensors; first += MAX) {
        const int ctas = clip_args(a, c, first, most);
        if (ctas == 0) continue;
        const cudaError_t e = launch_kernel(scale, dim3(unsigned(ctas)), dim3(CL_THREADS), 0, st, a);
        if (e != cudaSuccess) return int(e);
    }
    return LORA_OK;
}

}  // namespace lora

LORA_API int64_t lora_clip_gradients_workspace(int32_t groups)
{
    if (groups < 1) return LORA_ERR_SIZE;
    return lora::clip_plan(groups).bytes;
}

LORA_API int lora_clip_gradients(const void *const *grads, void *const *out, const int64_t *slice_sizes,
                                 const int32_t *grads_f32, int32_t num_tensors, int32_t groups, float max_norm,
                                 float eps, float *norms, void *workspace, int64_t workspace_bytes, void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_clip_gradients");
    if (num_tensors < 0 || groups < 1 || !(max_norm >= 0.0f) || !(eps >= 0.0f)) return LORA_ERR_SIZE;
    if (norms == nullptr || workspace == nullptr ||
        (num_tensors > 0 && (grads == nullptr || slice_sizes == nullptr || grads_f32 == nullptr)))
        return LORA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return LORA_ERR_ALIGN;
    int64_t elements = 0;
    for (int i = 0; i < num_tensors; ++i) {
        if (slice_sizes[i] < 0 || slice_sizes[i] > INT64_MAX / 16) return LORA_ERR_SIZE;
        elements += slice_sizes[i];
        if (elements > INT64_MAX / 8 / groups || clip_units(elements, CL_UNIT_LOG) + num_tensors > INT32_MAX)
            return LORA_ERR_SIZE;
        if (slice_sizes[i] == 0) continue;
        if (grads[i] == nullptr || (out != nullptr && out[i] == nullptr)) return LORA_ERR_NULL;
        const uintptr_t at = reinterpret_cast<uintptr_t>(grads[i]) |
                             (out != nullptr ? reinterpret_cast<uintptr_t>(out[i]) : 0);
        if (at & (grads_f32[i] ? 3u : 1u)) return LORA_ERR_ALIGN;
    }
    const ClipPlan plan = clip_plan(groups);
    if (workspace_bytes < plan.bytes) return LORA_ERR_WORKSPACE;
    ClipCall c;
    c.grads = grads;
    c.out = out;
    c.sizes = slice_sizes;
    c.f32 = grads_f32;
    c.tensors = num_tensors;
    char *ws = static_cast<char *>(workspace);
    c.s = ClipShared{};
    c.s.groups = groups;
    // long units where every CTA gets one or more: finding the next unit and
    // the round of sums then cost little beside its loads (bf16, norms alone,
    // short and long: 67 M elements 45.4 and 42.4 us, 537 M 200 and 190; 67 M
    // in stacks of half a million each 44.8 and 45.6)
    c.s.unit_log = elements * groups >= (int64_t(plan.ctas) << CL_LONG_LOG) ? CL_LONG_LOG : CL_UNIT_LOG;
    c.s.part = reinterpret_cast<double *>(ws);
    c.s.sum = reinterpret_cast<double *>(ws + plan.sum);
    c.s.factor = reinterpret_cast<ClipFactor *>(ws + plan.factor);
    c.s.norms = norms;
    c.s.max_norm = max_norm;
    c.s.eps = eps;
    c.s.scale = max_norm < INFINITY;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return num_tensors <= CL_FEW ? run_clip<CL_FEW>(c, plan.ctas, st) : run_clip<CL_MANY>(c, plan.ctas, st);
}
