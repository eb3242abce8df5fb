// lora_loss_row.cu -- lora_cross_entropy for one or two tokens (see
// lora_loss.cu for the formulas): one pass over the head.
//
// With so few tokens the time is the reading of W.  The products on the
// tensor cores read it twice (the softmax's sum lies between them); here a
// row of W that has given its logit is still in registers and is added,
// times its softmax term, to the running gradient, as an attention over one
// query does with its values.  The reference of the terms is a whole power
// of two that moves only when a logit lies 60 exponents above it.
//
// Bound by HBM: vocabulary 32000 x hidden 4096 is 262 MB, 39 us at the
// measured copy rate.  Rows come by cp.async, 96 KB ahead in each of two
// blocks an SM; a thread copies the columns that it reads.  One token takes
// 53 us, 46 for the pass (5.7 TB/s; 51 with the next four rows in registers)
// and the join of the blocks' sums; two tokens take 62.
#include "lora_loss.cuh"

namespace lora {

constexpr int LR_THREADS = 256;
constexpr int LR_WINDOW = 60;

// CH: 16-byte chunks of a row a thread; NT: tokens.
template <int CH, int NT>
struct RowShape {
    static constexpr int RB = 4 / NT;                             // rows at a time
    static constexpr int BLOCKS = CH >= 4 ? 1 : 2;                // on an SM
    static constexpr int STAGE = RB * CH * LR_THREADS * 16;
    static constexpr int ST = 192 * 1024 / BLOCKS / STAGE;        // of the ring
};

template <int CH, int NT>
__global__ void __launch_bounds__(LR_THREADS, RowShape<CH, NT>::BLOCKS) loss_row_kernel(const LossRowArgs p)
{
    constexpr int RB = RowShape<CH, NT>::RB, ST = RowShape<CH, NT>::ST, STAGE = RowShape<CH, NT>::STAGE;
    extern __shared__ __align__(16) uint8_t lr_ring[];
    __shared__ float s_dot[2][8][RB * NT];                        // parity, warp
    const int part = threadIdx.x, lane = part & 31, warp = part >> 5;
    pdl_wait();
    int y[NT];
    bool any = false;
    float h[NT][CH][8];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        y[t] = t < p.T ? p.targets[t] : -1;
        const bool valid = y[t] >= 0 && y[t] < p.V;
        any = any || valid;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * LR_THREADS + part) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[t][c][j] = valid && col < p.H ? bf16_to_f32(p.hidden[t * p.hidden_ld + col + j]) * LOSS_LOG2E : 0.0f;
        }
    }
    if (!any) return;                     // the next kernel reads nothing of this one then
    float acc[NT][CH][8], ref[NT], sum[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        ref[t] = -INFINITY;
        sum[t] = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[t][c][j] = 0.0f;
    }
    const int batches = (p.V + RB - 1) / RB;
    int parity = 0;
    // a thread reads only what it copied itself, so the ring needs no barrier
    uint8_t *ring = lr_ring + part * 16;
    int in = blockIdx.x, in_stage = 0, stage = 0;
    auto fetch = [&]() {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int col = (c * LR_THREADS + part) * 8;
                const bool ok = in < batches && in * RB + r < p.V && col < p.H;
                cp_async16(smem_addr(ring + in_stage * STAGE + (r * CH + c) * LR_THREADS * 16),
                           ok ? p.weight + int64_t(in * RB + r) * p.H + col : p.weight, ok);
            }
        cp_async_commit();
        in += gridDim.x;
        in_stage = in_stage + 1 == ST ? 0 : in_stage + 1;
    };
    for (int i = 0; i < ST; ++i) fetch();
    for (int b = blockIdx.x; b < batches; b += gridDim.x, parity ^= 1) {
        cp_async_wait<ST - 1>();
        uint4 w[RB][CH];
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                w[r][c] = *reinterpret_cast<const uint4 *>(ring + stage * STAGE + (r * CH + c) * LR_THREADS * 16);
        stage = stage + 1 == ST ? 0 : stage + 1;
        float dot[RB * NT];
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float d = 0.0f;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint32_t x[4] = {w[r][c].x, w[r][c].y, w[r][c].z, w[r][c].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        d = fmaf(bf16_lo(x[j]), h[t][c][2 * j], d);
                        d = fmaf(bf16_hi(x[j]), h[t][c][2 * j + 1], d);
                    }
                }
                dot[r * NT + t] = d;
            }
        fetch();                                // into the stage that was just read
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < RB * NT; ++i) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < RB * NT; ++i) s_dot[parity][warp][i] = dot[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RB * NT; ++i) {
            dot[i] = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) dot[i] += s_dot[parity][q][i];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float top = -INFINITY;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                float &d = dot[r * NT + t];
                const int row = b * RB + r;
                if (row == y[t]) {
                    if (part == 0) p.logit[t] = d;
                    d = -INFINITY;                       // the target enters at the end, in fp32
                }
                if (row >= p.V) d = -INFINITY;
                top = fmaxf(top, d);
            }
            if (top > ref[t] + float(LR_WINDOW)) {       // and the first time
                const float to = ceilf(fminf(top, LOSS_MAX_REF));
                const float f = exp2f(ref[t] - to);      // 0 from -infinity
                ref[t] = to;
                sum[t] *= f;
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[t][c][j] *= f;
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                // rows of -infinity before any other keep the reference unset
                const float e = dot[r * NT + t] == -INFINITY ? 0.0f : exp2f(dot[r * NT + t] - ref[t]);
                sum[t] += e;
                if (p.acc != nullptr) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const uint32_t x[4] = {w[r][c].x, w[r][c].y, w[r][c].z, w[r][c].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[t][c][2 * j] = fmaf(e, bf16_lo(x[j]), acc[t][c][2 * j]);
                            acc[t][c][2 * j + 1] = fmaf(e, bf16_hi(x[j]), acc[t][c][2 * j + 1]);
                        }
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (part == 0) p.stat[blockIdx.x * NT + t] = make_float2(ref[t], sum[t]);
        if (p.acc != nullptr) {
            float *out = p.acc + (int64_t(blockIdx.x) * NT + t) * p.H;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int col = (c * LR_THREADS + part) * 8;
                if (col >= p.H) continue;
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    *reinterpret_cast<float4 *>(out + col + j) =
                        make_float4(acc[t][c][j], acc[t][c][j + 1], acc[t][c][j + 2], acc[t][c][j + 3]);
            }
        }
    }
}

constexpr int LR_JOIN_THREADS = 512;
constexpr int LR_JOIN_COLS = 64;
constexpr int LR_JOIN_AHEAD = 20;         // slots of a warp loaded at once: 320 in all

// Block (64 columns, token): the blocks' partial sums in a fixed order, the
// loss, and dh.
__global__ void __launch_bounds__(LR_JOIN_THREADS) loss_row_join_kernel(const LossRowArgs p)
{
    __shared__ float s_part[16][LR_JOIN_COLS];
    __shared__ float s_red[16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = blockIdx.y;
    pdl_wait();
    const int y = p.targets[t];
    const bool valid = y >= 0 && y < p.V;
    const int col = blockIdx.x * LR_JOIN_COLS + lane * 2;
    // a warp's slots are warp, warp + 16, ...: their values are asked for
    // before the sums are known
    const bool read = valid && p.dh != nullptr && col < p.H;
    float2 v[LR_JOIN_AHEAD];
#pragma unroll
    for (int i = 0; i < LR_JOIN_AHEAD; ++i) {
        const int s = warp + 16 * i;
        v[i] = make_float2(0.0f, 0.0f);
        if (read && s < p.slots)
            v[i] = *reinterpret_cast<const float2 *>(p.acc + (int64_t(s) * p.nt + t) * p.H + col);
    }
    if (blockIdx.x == 0 && t == 0 && tid == 0 && p.error_word != nullptr) {
        int bad = 0;
        for (int i = 0; i < p.T; ++i) bad += p.targets[i] >= p.V;
        *p.error_word = bad;
    }
    float top = -INFINITY, sum = 0.0f;
    if (valid) {
        for (int s = tid; s < p.slots; s += LR_JOIN_THREADS) top = fmaxf(top, p.stat[s * p.nt + t].x);
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) s_red[warp] = top;
        __syncthreads();
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s_red[i]);
        __syncthreads();
        for (int s = tid; s < p.slots; s += LR_JOIN_THREADS) {
            const float2 x = p.stat[s * p.nt + t];
            // a block without a reference has a sum of 0, or NaN if that is
            // all that its logits were: the row's loss is then NaN too
            sum += x.x > -INFINITY ? x.y * exp2f(x.x - top) : x.y;
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_red[warp] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int i = 0; i < 16; ++i) sum += s_red[i];
    }
    LossRow row = {0.0f, 0.0f, 0.0f, 0.0f};
    float w = 0.0f;
    if (valid) {
        row = loss_row(sum, top, p.logit[t]);
        w = p.token_weight != nullptr ? p.token_weight[t] : 1.0f;
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.loss[t] = valid ? w * row.loss : 0.0f;
        if (p.logsumexp != nullptr) p.logsumexp[t] = row.lse2 * LOSS_LN2;
    }
    if (p.dh == nullptr) return;
    float a = 0.0f, b = 0.0f;
    auto add = [&](int s, const float2 &x) {
        const float ref = p.stat[s * p.nt + t].x;
        const float f = ref > -INFINITY ? exp2f(ref - top) : 0.0f;
        a = fmaf(f, x.x, a);
        b = fmaf(f, x.y, b);
    };
    if (read) {
#pragma unroll
        for (int i = 0; i < LR_JOIN_AHEAD; ++i)
            if (warp + 16 * i < p.slots) add(warp + 16 * i, v[i]);
        for (int s = warp + 16 * LR_JOIN_AHEAD; s < p.slots; s += 16)
            add(s, *reinterpret_cast<const float2 *>(p.acc + (int64_t(s) * p.nt + t) * p.H + col));
    }
    s_part[warp][lane * 2] = a;
    s_part[warp][lane * 2 + 1] = b;
    __syncthreads();
    if (tid < LR_JOIN_COLS && blockIdx.x * LR_JOIN_COLS + tid < p.H) {
        const int c = blockIdx.x * LR_JOIN_COLS + tid;
        float g = 0.0f;
        if (valid) {
            for (int i = 0; i < 16; ++i) g += s_part[i][tid];
            g = w * (row.inv * g - row.share * bf16_to_f32(p.weight[int64_t(y) * p.H + c]));
        }
        p.dh[t * p.dh_ld + c] = uint16_t(pack_bf16x2(g, 0.0f) & 0xFFFFu);
    }
}

bool loss_row_fits(int32_t T, int32_t H) { return T >= 1 && T <= LOSS_ROW_TOKENS && H <= 4 * 8 * LR_THREADS; }

int loss_row_slots() { return 2 * device_sm_count(); }

template <int CH, int NT>
static cudaError_t launch_row(const LossRowArgs &p, cudaStream_t st)
{
    constexpr int smem = RowShape<CH, NT>::ST * RowShape<CH, NT>::STAGE;
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(loss_row_kernel<CH, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = 1;
    }
    return launch_kernel(loss_row_kernel<CH, NT>, dim3(unsigned(p.slots)), dim3(LR_THREADS), size_t(smem), st, p);
}

template <int NT>
static cudaError_t launch_row_width(const LossRowArgs &p, cudaStream_t st)
{
    const int chunks = (p.H + 8 * LR_THREADS - 1) / (8 * LR_THREADS);
    if (chunks <= 1) return launch_row<1, NT>(p, st);
    if (chunks <= 2) return launch_row<2, NT>(p, st);
    return launch_row<4, NT>(p, st);
}

int run_loss_row(LossRowArgs p, cudaStream_t st)
{
    p.nt = p.T;
    p.slots = loss_row_slots();
    cudaError_t e = p.T == 1 ? launch_row_width<1>(p, st) : launch_row_width<2>(p, st);
    if (e != cudaSuccess) return int(e);
    const int blocks = p.dh != nullptr ? (p.H + LR_JOIN_COLS - 1) / LR_JOIN_COLS : 1;
    e = launch_kernel(loss_row_join_kernel, dim3(unsigned(blocks), unsigned(p.T)), dim3(LR_JOIN_THREADS), 0, st, p);
    return e == cudaSuccess ? LORA_OK : int(e);
}

}  // namespace lora
