// lora_loss.cu -- softmax cross entropy over a vocabulary whose logits are
// never kept, with the gradients of the hidden states and of the head.
//
//   S = h W^T,  loss_t = w_t (log sum_v exp S_tv - S_ty)
//   dh_t = w_t (sum_{v != y} p_tv W_v - (1 - p_ty) W_y),  p = softmax(S)
//   dW_v = sum_t w_t (p_tv - [v = y_t]) h_t
//
// The vocabulary is walked in pieces.  For each piece one product gives its
// logits in TMEM, the epilogue turns them into powers of two relative to a
// whole-number reference of the row and writes those as bf16 (the piece's
// scratch), and a second product adds scratch x W to the fp32 rows of dh.
// The softmax's sum is known only after the last piece, so dh is divided by
// it at the end.  The target's column stays zero in the scratch and enters
// as -(1 - p_y) W_y in fp32: 1 - p_y is the sum over the other columns, so
// nothing cancels when the model is sure of the target.
//
// References.  A bf16 power of two keeps its 8 bits anywhere between 2^-126
// and 2^127, so a reference need not be the row's maximum: it starts at 0
// and a tile whose largest exponent lies within 60 of it uses it.  A tile
// outside that window takes its own maximum, and join_kernel then brings
// the row's scratch to one reference (multiplications by powers of two,
// exact).
//
// dW needs the finished sums, so with a head gradient the pieces are walked
// a second time: the same product, the epilogue writes w (p - [y]) and a
// third product contracts it with h over the tokens.  Those terms as one bf16
// each leave dW 1.4 times the error of its own rounding over many tokens, up
// to 1.8 times over few.  With up to 128 tokens, which fill half a tile's rows,
// the other half holds the same tokens again and takes what the rounding left
// over (1.0 times; 16 tokens, hidden 4096, vocabulary 32000: 304 us in place
// of 295).
//
// Tokens without a target (outside [0, V)) are left out from the start:
// pack_kernel copies the others' rows next to each other, so a prompt's
// masked tokens cost nothing, and what their rows hold is never read.
//
// What bounds it: the tensor cores.  8192 tokens (5489 with a target), hidden
// 4096, vocabulary 32000: 1900 us for 2.88e12 operations, 1515 TFLOP/s, on a
// GPU that has warmed up (1740 us, 1655 TFLOP/s, before the power cap); 256
// tokens: 127 us, where each of the two products reads the 262 MB of W in 55
// us (4.8 TB/s; 125 tiles on 76 pairs are two rounds, the second two thirds
// full).
//
// One or two tokens without a head gradient take lora_loss_row.cu (hidden
// 4096, vocabulary 32000: 53 and 62 us there, 122 here).
#include "lora_loss.cuh"
#include "lora_pair_gemm.cuh"

namespace lora {

constexpr int LS_PIECE_ELEMS = 128 << 20;     // tokens x columns of one piece's scratch
constexpr int LS_MIN_PIECE = 1024;            // columns
constexpr int LS_WINDOW = 60;                 // exponents a tile may be off the reference
constexpr float LS_FAR = 1048576.0f;          // references whose rounding is no longer small beside 1
constexpr int LS_MAX_SPLIT = 8;
constexpr int LS_PACK_TOKENS = 4;             // tokens of one block of pack_kernel
constexpr int LS_PACK_THREADS = 256;
constexpr int LS_PAD_BLOCKS = 32;
constexpr int LS_JOIN_ROWS = 8;               // rows of a block of join_kernel, a warp each

// What a call's workspace holds; every part begins on a 256-byte boundary.
struct LossLayout {
    int64_t tokens;        // T rounded up to whole tiles
    int64_t piece;         // columns of a piece, a multiple of PG_TILE
    int pieces, split;
    int64_t count, row, target, weight, ref, sum, logit, factor, inv, share, stat, h, p, acc;
    int64_t bytes;
    bool rows;             // one or two tokens: logit, stat and acc of lora_loss_row.cu alone
};

// Row stride of the packed hidden states: whole 128-byte lines, whatever the
// caller's stride (a TMA box of rows that straddle lines loads at less than
// half the rate).
__host__ __device__ constexpr int64_t packed_ld(int64_t H) { return (H + 63) / 64 * 64; }

static LossLayout loss_layout(int64_t T, int64_t H, int64_t V, bool hidden_grad, bool weight_grad,
                              int pairs)
{
    LossLayout l;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b * b; };
    l.tokens = up(T, PG_TILE);
    int64_t most = LS_PIECE_ELEMS / l.tokens / PG_TILE * PG_TILE;
    if (most < LS_MIN_PIECE) most = LS_MIN_PIECE;
    l.pieces = int((V + most - 1) / most);
    l.piece = up((V + l.pieces - 1) / l.pieces, PG_TILE);
    l.pieces = int((V + l.piece - 1) / l.piece);
    // The product of the scratch and W has few tiles when there are few
    // tokens: its K (the piece) is then split over up to LS_MAX_SPLIT
    // partial sums, joined in a fixed order by finish_kernel.
    const int64_t tiles = l.tokens / PG_TILE * ((H + PG_TILE - 1) / PG_TILE);
    int64_t split = pairs / tiles;
    if (split > LS_MAX_SPLIT) split = LS_MAX_SPLIT;
    if (split > l.piece / PG_BK / 8) split = l.piece / PG_BK / 8;
    l.split = split < 1 ? 1 : int(split);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    l.rows = !weight_grad && loss_row_fits(int32_t(T), int32_t(H));
    if (l.rows) {
        l.count = l.row = l.target = l.weight = l.ref = l.sum = l.factor = l.inv = l.share = l.h = l.p = 0;
        l.logit = take(T * 4);
        l.stat = take(loss_row_slots() * T * 8);
        l.acc = take(hidden_grad ? loss_row_slots() * T * H * 4 : 0);
        l.bytes = at;
        return l;
    }
    l.count = take(4);
    l.row = take(l.tokens * 4);
    l.target = take(l.tokens * 4);
    l.weight = take(l.tokens * 4);
    l.ref = take(l.tokens * 4);
    l.sum = take(l.tokens * 4);
    l.logit = take(l.tokens * 4);
    l.factor = take(l.tokens * 4);
    l.inv = take(l.tokens * 4);
    l.share = take(l.tokens * 4);
    l.stat = take(l.tokens * (l.piece / PG_HALF) * 8);
    l.h = take(l.tokens * packed_ld(H) * 2);
    l.p = take(hidden_grad || weight_grad ? l.tokens * l.piece * 2 : 0);
    l.acc = take(hidden_grad && (l.split > 1 || l.pieces > 1) ? l.split * l.tokens * H * 4 : 0);
    l.bytes = at;
    return l;
}

// What a call may need at up to T tokens, with the gradients asked for or
// without: a training loop sizes its workspace for its largest batch, and
// smaller ones can take more (larger pieces, more partial sums).
static int64_t loss_bytes(int64_t T, int64_t H, int64_t V, bool hidden_grad, bool weight_grad, int pairs)
{
    if (T == 0) return 256;                   // nothing but clearing outputs
    int64_t most = loss_layout(T, H, V, hidden_grad, weight_grad, pairs).bytes;
    auto also = [&](int64_t tokens, bool head) {
        const int64_t bytes = loss_layout(tokens, H, V, hidden_grad, head, pairs).bytes;
        if (bytes > most) most = bytes;
    };
    for (int64_t t = PG_TILE; t < T; t += PG_TILE) also(t, weight_grad);
    also(T < LOSS_ROW_TOKENS ? T : LOSS_ROW_TOKENS, false);
    return most;
}

struct LossArgs {
    const uint16_t *hidden;
    int64_t hidden_ld;
    const uint16_t *weight;
    const int32_t *targets;
    const float *token_weight;
    float *loss, *logsumexp;
    uint16_t *dh;
    int64_t dh_ld;
    int32_t T, H, V;
    int32_t hidden_vec, dh_vec;        // rows allow 16-byte accesses
    int32_t *error_word;
    // workspace
    int32_t *count;                    // tokens with a target
    int32_t *row, *target;
    float *ref, *wt, *sum, *logit, *factor, *inv, *share;
    float2 *stat;                      // [128 columns each][tokens]: reference, sum
    uint16_t *h, *p;
    float *acc;
    int64_t tokens, piece;
    int32_t split;
    int32_t two;                       // dW's terms as two bf16 values: rows from PG_HALF on are the tokens again
};

// ---------------------------------------------------------------- pack

// Block b copies tokens [4 b, 4 b + 4) that have a target to their place
// among those that have one (the count of targets before them, which every
// block takes itself), and clears the outputs of the others.  Behind them,
// for a head gradient, LS_PAD_BLOCKS blocks fill the last tile with zeros
// (other products never use what rows past the last give).  The target's logit is
// summed here, in ordinary fp32: the loss is a difference with it, and the
// tensor cores' sums truncate (over 4096 products they leave the loss 4
// times further off).  Two warps a token with their loads unrolled: at 256
// tokens x 4096 one warp for four tokens, one load after another, took 64 us.
__global__ void __launch_bounds__(LS_PACK_THREADS) pack_kernel(const LossArgs p)
{
    constexpr int WARPS = LS_PACK_THREADS / 32, TEAM = LS_PACK_THREADS / LS_PACK_TOKENS;
    __shared__ int s_part[2][WARPS];
    __shared__ float s_dot[WARPS];
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c0 = blockIdx.x * LS_PACK_TOKENS;
    const int blocks = (p.T + LS_PACK_TOKENS - 1) / LS_PACK_TOKENS;
    const bool last = int(blockIdx.x) == blocks - 1, pad = int(blockIdx.x) >= blocks;
    int before = 0, bad = 0;
#pragma unroll 8
    for (int t = tid; t < min(c0, p.T); t += LS_PACK_THREADS) {
        const int y = p.targets[t];
        before += y >= 0 && y < p.V;
        bad += y >= p.V;
    }
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        bad += __shfl_xor_sync(0xffffffffu, bad, o);
    }
    if (lane == 0) {
        s_part[0][warp] = before;
        s_part[1][warp] = bad;
    }
    __syncthreads();
    before = bad = 0;
    for (int i = 0; i < WARPS; ++i) {
        before += s_part[0][i];
        bad += s_part[1][i];
    }
    if (pad) {
        const int n_up = (before + PG_TILE - 1) / PG_TILE * PG_TILE;
        auto clear = [&](int first, int end) {
            uint4 *rows = reinterpret_cast<uint4 *>(p.h + int64_t(first) * packed_ld(p.H));
            const int64_t all = int64_t(end - first) * (packed_ld(p.H) / 8);
            for (int64_t i = int64_t(blockIdx.x - blocks) * LS_PACK_THREADS + tid; i < all;
                 i += LS_PAD_BLOCKS * LS_PACK_THREADS)
                rows[i] = make_uint4(0, 0, 0, 0);
        };
        if (p.two) {
            clear(before, PG_HALF);
            clear(PG_HALF + before, PG_TILE);
        } else {
            clear(before, n_up);
        }
        return;
    }
    // lane i < LS_PACK_TOKENS of every warp: the block's token i
    const int y = lane < LS_PACK_TOKENS && c0 + lane < p.T ? p.targets[c0 + lane] : -1;
    const uint32_t mask = __ballot_sync(0xffffffffu, y >= 0 && y < p.V);
    bad += __popc(__ballot_sync(0xffffffffu, y >= p.V));
    const int n = before + __popc(mask);
    if (last) {
        const int n_up = (n + PG_TILE - 1) / PG_TILE * PG_TILE;
        if (tid == 0) {
            *p.count = n;
            if (p.error_word != nullptr) *p.error_word = bad;
        }
        for (int r = n + tid; r < n_up; r += LS_PACK_THREADS) {
            p.row[r] = -1;
            p.target[r] = -1;
            p.wt[r] = 0.0f;
            p.ref[r] = 0.0f;
            p.sum[r] = 0.0f;
            p.logit[r] = 0.0f;
        }
    }
    const int mine = tid / TEAM, part = tid % TEAM, t = c0 + mine;     // this thread's token
    const int target = __shfl_sync(0xffffffffu, y, mine);
    const bool valid = mask >> mine & 1u;
    const int to = before + __popc(mask & ((1u << mine) - 1u));
    float dot = 0.0f;
    if (valid) {
        const uint16_t *src = p.hidden + int64_t(t) * p.hidden_ld;
        uint16_t *dst = p.h + int64_t(to) * packed_ld(p.H);
        const uint16_t *w = p.weight + int64_t(target) * p.H;
        auto one = [&](int c, const uint4 &v, const uint4 &u) {
            *reinterpret_cast<uint4 *>(dst + c) = v;
            if (p.two) *reinterpret_cast<uint4 *>(dst + PG_HALF * packed_ld(p.H) + c) = v;
            const uint32_t a[4] = {v.x, v.y, v.z, v.w}, b[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dot = fmaf(bf16_lo(a[j]), bf16_lo(b[j]), dot);
                dot = fmaf(bf16_hi(a[j]), bf16_hi(b[j]), dot);
            }
        };
        if (p.hidden_vec) {
            for (int c = part * 8; c < p.H; c += TEAM * 32) {
                uint4 v[4], u[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + k * TEAM * 8 < p.H) {
                        v[k] = *reinterpret_cast<const uint4 *>(src + c + k * TEAM * 8);
                        u[k] = *reinterpret_cast<const uint4 *>(w + c + k * TEAM * 8);
                    }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + k * TEAM * 8 < p.H) one(c + k * TEAM * 8, v[k], u[k]);
            }
        } else {
            for (int c = part * 8; c < p.H; c += TEAM * 8) {
                uint32_t v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = src[c + 2 * j] | uint32_t(src[c + 2 * j + 1]) << 16;
                one(c, make_uint4(v[0], v[1], v[2], v[3]), *reinterpret_cast<const uint4 *>(w + c));
            }
        }
    } else if (t < p.T && p.dh != nullptr) {
        uint16_t *dst = p.dh + int64_t(t) * p.dh_ld;
        if (p.dh_vec) {
            for (int c = part * 8; c < p.H; c += TEAM * 8)
                *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
        } else {
            for (int c = part; c < p.H; c += TEAM) dst[c] = 0;
        }
    }
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_dot[warp] = dot;
    __syncthreads();
    if (part == 0) {
        if (valid) {
            float d = 0.0f;
            for (int i = 0; i < TEAM / 32; ++i) d += s_dot[warp + i];
            p.row[to] = t;
            p.target[to] = target;
            p.wt[to] = p.token_weight != nullptr ? p.token_weight[t] : 1.0f;
            p.ref[to] = 0.0f;
            p.sum[to] = 0.0f;
            p.logit[to] = d * LOSS_LOG2E;
        } else if (t < p.T) {
            p.loss[t] = 0.0f;
            if (p.logsumexp != nullptr) p.logsumexp[t] = 0.0f;
        }
    }
}

// ---------------------------------------------------------------- products

struct LossGemm {
    CUtensorMap a, b;
    LossArgs l;
    int32_t col0, cols;       // this piece of the vocabulary
    int32_t store;            // logits: write the scratch
    int32_t first;            // scratch x W: the rows of dh start here
    int32_t last;             // ... and are finished here (no split)
    uint16_t *dw;             // head gradient
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// Logits of a piece: 256 tokens x 256 columns a tile, tokens innermost (the
// packed rows stay in L2 while a few tiles of W pass).
// GRAD: the sums are known, the scratch becomes w (p - [y]); p is the term
// relative to the row's reference times 1 / sum (relative to the logarithm of
// the sum it would lose that logarithm's rounding).
template <bool GRAD>
__global__ void __launch_bounds__(PG_THREADS, 1)
logits_kernel(const __grid_constant__ LossGemm g)
{
    pdl_wait();
    const LossArgs &l = g.l;
    const int mt = (*l.count + PG_TILE - 1) / PG_TILE;
    const int nt = (g.cols + PG_TILE - 1) / PG_TILE;
    const int kb = (l.H + PG_BK - 1) / PG_BK;
    auto item = [&](int i) {
        return PairItem{(i % mt) * PG_TILE, g.col0 + (i / mt) * PG_TILE, 0, kb};
    };
    auto epilogue = [&](int i, const PairItem &it, uint32_t tmem, int r, int c0, int rank, bool) {
        const int row = it.row_a + rank * PG_HALF + r;
        const int tile = i / mt;
        const int c_end = c0 + PG_HALF;
        const int lim = min(c_end, g.col0 + g.cols - it.row_b);         // columns end here
        // row of the token's sums and target
        const bool second = GRAD && l.two && row >= PG_HALF;
        const int of = second ? row - PG_HALF : row;
        const int y = l.target[of] - it.row_b;                          // column of the target
        uint16_t *dst = l.p + int64_t(row) * l.piece + tile * PG_TILE;
        uint32_t v[32];
        float ref, scale = 1.0f, q = 0.0f, sum = 0.0f;
        if constexpr (GRAD) {
            ref = l.ref[of];
            scale = l.inv[of];
            q = -l.share[of];
        } else {
            float top = -INFINITY;
            for (int c = c0; c < lim; c += 32) {
                tmem_ld32_nowait(tmem + c, v);
                tmem_wait_ld();
                if (__any_sync(0xffffffffu, y >= c && y < c + 32)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j == y) v[j] = 0xff800000u;             // -inf
                }
                if (c + 32 <= lim) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, __uint_as_float(v[j]));
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < lim) top = fmaxf(top, __uint_as_float(v[j]));
                }
            }
            top *= LOSS_LOG2E;
            ref = l.ref[row];
            if (top > -INFINITY && !(fabsf(top - ref) <= float(LS_WINDOW)))
                ref = ceilf(fminf(fmaxf(top, -LOSS_MAX_REF), LOSS_MAX_REF));
        }
        // Near zero the exponent and its difference to the reference are one
        // operation, rounded once.  Far out it has to be rounded as the
        // reference and the target's were, or the three do not match.
        const bool far = fabsf(ref) >= LS_FAR;
        const float pre = far ? LOSS_LOG2E : 1.0f, mul = far ? 1.0f : LOSS_LOG2E;
        for (int c = c0; c < c_end; c += 32) {
            if (GRAD ? c >= lim : (c >= lim && !g.store)) break;
            uint32_t pk[16];
            if (c < lim) {
                tmem_ld32_nowait(tmem + c, v);
                tmem_wait_ld();
                float e[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    e[j] = exp2_fast(fmaf(__uint_as_float(v[j]) * pre, mul, -ref));
                if (c + 32 > lim) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j >= lim) e[j] = 0.0f;
                }
                if constexpr (GRAD) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) e[j] *= scale;
                }
                if (__any_sync(0xffffffffu, y >= c && y < c + 32)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j == y) e[j] = q;
                }
                if constexpr (!GRAD) {
                    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        s0 += e[j];
                        s1 += e[j + 1];
                    }
                    sum += s0 + s1;
                }
                // rounded to bf16 for the second product: relative 2^-9 of
                // each term on average, the size of the output's own rounding
#pragma unroll
                for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(e[2 * j], e[2 * j + 1]);
                if constexpr (GRAD) {
                    if (second) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            pk[j] = pack_bf16x2(e[2 * j] - bf16_lo(pk[j]), e[2 * j + 1] - bf16_hi(pk[j]));
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) pk[j] = 0u;
            }
            if (GRAD || g.store) {
                const uint32_t lo[8] = {pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]};
                const uint32_t hi[8] = {pk[8], pk[9], pk[10], pk[11], pk[12], pk[13], pk[14], pk[15]};
                st_global_v8(dst + c, lo);
                st_global_v8(dst + c + 16, hi);
            }
        }
        if constexpr (!GRAD) l.stat[int64_t(tile * 2 + c0 / PG_HALF) * l.tokens + row] = make_float2(ref, sum);
    };
    pair_gemm<false, false>(&g.a, &g.b, mt * nt, l.error_word, item, epilogue);
}

// Eight values of dh: inv * sum - share * W[y], their only rounding.
__device__ __forceinline__ void finish8(uint16_t *dst, const uint16_t *w, const uint32_t *sum,
                                        float inv, float share, int vec)
{
    const uint4 wv = *reinterpret_cast<const uint4 *>(w);
    const uint32_t wr[4] = {wv.x, wv.y, wv.z, wv.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = pack_bf16x2(fmaf(-share, bf16_lo(wr[j]), inv * __uint_as_float(sum[2 * j])),
                           fmaf(-share, bf16_hi(wr[j]), inv * __uint_as_float(sum[2 * j + 1])));
    if (vec) {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dst[2 * j] = uint16_t(o[j] & 0xFFFFu);
            dst[2 * j + 1] = uint16_t(o[j] >> 16);
        }
    }
}

// acc[split][token][h] (+)= scratch x W over a share of the piece's columns
// (W's rows are the K dimension: its rows are contiguous along N).
__global__ void __launch_bounds__(PG_THREADS, 1)
hidden_grad_kernel(const __grid_constant__ LossGemm g)
{
    pdl_wait();
    const LossArgs &l = g.l;
    const int mt = (*l.count + PG_TILE - 1) / PG_TILE;
    const int nt = (l.H + PG_TILE - 1) / PG_TILE;
    const int kb = (g.cols + PG_BK - 1) / PG_BK;
    const int per = (kb + l.split - 1) / l.split;
    auto item = [&](int i) {
        const int s = i / (mt * nt), j = i % (mt * nt);
        return PairItem{(j % mt) * PG_TILE, (j / mt) * PG_TILE, min(kb, s * per),
                        min(kb, (s + 1) * per)};
    };
    auto epilogue = [&](int i, const PairItem &it, uint32_t tmem, int r, int c0, int rank, bool empty) {
        const int row = it.row_a + rank * PG_HALF + r;
        const int s = i / (mt * nt);
        float *dst = l.acc + (int64_t(s) * l.tokens + row) * l.H + it.row_b;
        const float f = g.first ? 0.0f : l.factor[row];
        const int lim = min(c0 + PG_HALF, l.H - it.row_b);
        float inv = 0.0f, share = 0.0f;
        const uint16_t *w = l.weight;
        uint16_t *out = nullptr;
        if (g.last) {
            const int t = l.row[row];
            if (t >= 0) {
                inv = l.inv[row];
                share = l.share[row];
                w += int64_t(l.target[row]) * l.H + it.row_b;
                out = l.dh + int64_t(t) * l.dh_ld + it.row_b;
            }
        }
        for (int c = c0; c < lim; c += 32) {
            const int many = min(32, lim - c);                 // a multiple of 8
            uint32_t v[32];
            if (empty) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0u;
            } else {
                tmem_ld32_nowait(tmem + c, v);
            }
            // all of a chunk's loads before its first store: one after
            // another they took longer than the tile's product
            float4 was[8];
            if (!g.first) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (4 * j < many) was[j] = *reinterpret_cast<const float4 *>(dst + c + 4 * j);
            }
            if (!empty) tmem_wait_ld();
            if (!g.first) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[4 * j] = __float_as_uint(fmaf(was[j].x, f, __uint_as_float(v[4 * j])));
                    v[4 * j + 1] = __float_as_uint(fmaf(was[j].y, f, __uint_as_float(v[4 * j + 1])));
                    v[4 * j + 2] = __float_as_uint(fmaf(was[j].z, f, __uint_as_float(v[4 * j + 2])));
                    v[4 * j + 3] = __float_as_uint(fmaf(was[j].w, f, __uint_as_float(v[4 * j + 3])));
                }
            }
            if (!g.last) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (4 * j < many)
                        *reinterpret_cast<uint4 *>(dst + c + 4 * j) =
                            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            } else if (out != nullptr) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (8 * j < many) finish8(out + c + 8 * j, w + c + 8 * j, v + 8 * j, inv, share, l.dh_vec);
            }
        }
    };
    pair_gemm<false, true>(&g.a, &g.b, mt * nt * l.split, l.error_word, item, epilogue);
}

// dW[v] = sum over tokens of scratch[t][v] h[t]: both operands have their
// rows contiguous.
__global__ void __launch_bounds__(PG_THREADS, 1)
head_grad_kernel(const __grid_constant__ LossGemm g)
{
    pdl_wait();
    const LossArgs &l = g.l;
    const int mt = (g.cols + PG_TILE - 1) / PG_TILE;
    const int nt = (l.H + PG_TILE - 1) / PG_TILE;
    const int kb = l.two && *l.count > 0 ? PG_TILE / PG_BK : (*l.count + PG_BK - 1) / PG_BK;
    auto item = [&](int i) {
        return PairItem{(i / nt) * PG_TILE, (i % nt) * PG_TILE, 0, kb};
    };
    auto epilogue = [&](int, const PairItem &it, uint32_t tmem, int r, int c0, int rank, bool empty) {
        const int v0 = it.row_a + rank * PG_HALF + r;
        const int lim = min(c0 + PG_HALF, l.H - it.row_b);
        uint16_t *dst = g.dw + int64_t(g.col0 + v0) * l.H + it.row_b;
        for (int c = c0; c < lim; c += 32) {
            uint32_t v[32];
            if (empty) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0u;
            } else {
                tmem_ld32_nowait(tmem + c, v);
                tmem_wait_ld();
            }
            if (v0 >= g.cols) continue;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                if (c + j >= lim) break;
                uint4 o;
                o.x = pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                o.y = pack_bf16x2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
                o.z = pack_bf16x2(__uint_as_float(v[j + 4]), __uint_as_float(v[j + 5]));
                o.w = pack_bf16x2(__uint_as_float(v[j + 6]), __uint_as_float(v[j + 7]));
                *reinterpret_cast<uint4 *>(dst + c + j) = o;
            }
        }
    };
    pair_gemm<true, true>(&g.a, &g.b, mt * nt, l.error_word, item, epilogue);
}

// ---------------------------------------------------------------- join

struct JoinArgs {
    LossArgs l;
    int32_t tiles;       // of the piece, 128 columns each
    int32_t last;        // no piece follows: also the loss and the row factors
    int32_t store;
};

// After a piece's logits: a warp a row adds the tiles' sums to the row's (a
// fixed order) and, where a tile fell outside the window, brings the row to
// a common reference (the block then rescales the row's scratch).
__global__ void __launch_bounds__(LS_JOIN_ROWS * 32) join_kernel(const JoinArgs a)
{
    constexpr int THREADS = LS_JOIN_ROWS * 32;
    __shared__ int s_off[LS_JOIN_ROWS];
    __shared__ float s_new[LS_JOIN_ROWS];
    pdl_wait();
    const LossArgs &l = a.l;
    const int k = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * LS_JOIN_ROWS + k;
    const bool in = row < *l.count;
    if (lane == 0) s_off[k] = 0;
    if (in) {
        const float2 *stat = l.stat + row;
        const float have = l.ref[row], old = l.sum[row];
        float sum = 0.0f, own = -INFINITY;
        bool used = old != 0.0f;                    // something took the row's reference (or was NaN)
#pragma unroll 4
        for (int j = lane; j < a.tiles; j += 32) {
            const float2 s = stat[int64_t(j) * l.tokens];
            if (s.x == have) {
                sum += s.y;
                used = used || s.y != 0.0f;
            } else {
                own = fmaxf(own, s.x);
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            own = fmaxf(own, __shfl_xor_sync(0xffffffffu, own, o));
        }
        used = __any_sync(0xffffffffu, used);
        float ref = have, f = 1.0f, total = old + sum;
        if (own > -INFINITY) {                      // a tile has a reference of its own
            ref = used ? fmaxf(have, own) : own;
            f = used ? exp2f(have - ref) : 0.0f;
            float more = 0.0f;
            for (int j = lane; j < a.tiles; j += 32) {
                const float2 s = stat[int64_t(j) * l.tokens];
                if (s.x != have) more += s.y * exp2f(s.x - ref);
            }
            for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
            total = (used ? total * f : 0.0f) + more;
        }
        if (lane == 0) {
            if (ref != have || own > -INFINITY) {
                s_off[k] = a.store;
                s_new[k] = ref;
                l.ref[row] = ref;
            }
            l.sum[row] = total;
            l.factor[row] = f;
            if (a.last) {
                const float w = l.wt[row];
                const LossRow r = loss_row(total, ref, l.logit[row]);
                const int t = l.row[row];
                l.loss[t] = w * r.loss;
                if (l.logsumexp != nullptr) l.logsumexp[t] = r.lse2 * LOSS_LN2;
                l.inv[row] = w * r.inv;
                l.share[row] = w * r.share;
            }
        }
    } else if (a.last && lane == 0 && row < l.tokens) {
        l.inv[row] = l.share[row] = 0.0f;
    }
    __syncthreads();
    for (int q = 0; q < LS_JOIN_ROWS; ++q) {
        if (!s_off[q]) continue;
        const int r = blockIdx.x * LS_JOIN_ROWS + q;
        for (int j = 0; j < a.tiles; ++j) {
            const float2 was = l.stat[int64_t(j) * l.tokens + r];
            // a tile of zeros (nothing but the target, say) may have kept a
            // reference far above the new one: 0 * inf
            if (was.x == s_new[q] || was.y == 0.0f) continue;
            const float f = exp2f(was.x - s_new[q]);
            uint32_t *at = reinterpret_cast<uint32_t *>(l.p + int64_t(r) * l.piece + j * PG_HALF);
            for (int i = threadIdx.x; i < PG_HALF / 2; i += THREADS)
                at[i] = pack_bf16x2(bf16_lo(at[i]) * f, bf16_hi(at[i]) * f);
        }
    }
}

// dh where the pieces were split: the partial rows summed in order.  One
// block per row (a stride of the grid apart).
__global__ void __launch_bounds__(256) finish_kernel(const LossArgs l)
{
    pdl_wait();
    const int n = *l.count;
    for (int row = blockIdx.x; row < n; row += gridDim.x) {
        const float inv = l.inv[row], share = l.share[row];
        const uint16_t *w = l.weight + int64_t(l.target[row]) * l.H;
        uint16_t *dst = l.dh + int64_t(l.row[row]) * l.dh_ld;
        for (int c = threadIdx.x * 8; c < l.H; c += 256 * 8) {
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
            for (int s = 0; s < l.split; ++s) {
                const float4 *a = reinterpret_cast<const float4 *>(
                    l.acc + (int64_t(s) * l.tokens + row) * l.H + c);
                const float4 x = a[0], y = a[1];
                v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
                v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
            }
            uint32_t bits[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) bits[j] = __float_as_uint(v[j]);
            finish8(dst + c, w + c, bits, inv, share, l.dh_vec);
        }
    }
}

// ---------------------------------------------------------------- host

static int prepare_kernels()
{
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return int(e);
    if (dev < 64 && configured[dev]) return 0;
    const void *fns[] = {(const void *)logits_kernel<false>, (const void *)logits_kernel<true>,
                         (const void *)hidden_grad_kernel, (const void *)head_grad_kernel};
    for (const void *f : fns) {
        e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, PG_SMEM);
        if (e != cudaSuccess) return int(e);
    }
    if (dev < 64) configured[dev] = 1;
    return 0;
}

// Tensor map of a bf16 matrix: an operand with K contiguous is loaded in
// boxes of 64 K x 128 rows, one with its rows contiguous in 64 x 64.
static bool operand_map(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols, int64_t ld,
                        bool rows_contiguous)
{
    return encode_tile_map(m, ptr, uint64_t(rows), uint64_t(cols), uint64_t(ld), PG_BK,
                           rows_contiguous ? PG_BK : PG_HALF, CU_TENSOR_MAP_SWIZZLE_128B);
}

static int run_loss(LossArgs l, const LossLayout &lay, uint16_t *dw, cudaStream_t st)
{
    if (int e = prepare_kernels()) return e;
    const int pairs = device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1;
    LossGemm logits, dhid, grad, head;
    logits.l = dhid.l = grad.l = head.l = l;
    const bool store = l.dh != nullptr;
    if (!operand_map(&logits.a, l.h, lay.tokens, l.H, packed_ld(l.H), false) ||
        !operand_map(&logits.b, l.weight, l.V, l.H, l.H, false) ||
        ((store || dw != nullptr) &&
         (!operand_map(&dhid.a, l.p, lay.tokens, lay.piece, lay.piece, false) ||
          !operand_map(&head.a, l.p, lay.tokens, lay.piece, lay.piece, true))) ||
        !operand_map(&head.b, l.h, lay.tokens, l.H, packed_ld(l.H), true))
        return LORA_ERR_DEVICE;
    const int blocks = (l.T + LS_PACK_TOKENS - 1) / LS_PACK_TOKENS;
    cudaError_t e = launch_kernel(pack_kernel, dim3(unsigned(blocks + (dw != nullptr ? LS_PAD_BLOCKS : 0))),
                                  dim3(LS_PACK_THREADS), 0, st, l);
    if (e != cudaSuccess) return int(e);
    for (int i = 0; i < lay.pieces; ++i) {
        const int32_t col0 = int32_t(i * lay.piece);
        const int32_t cols = int32_t(lay.piece < l.V - col0 ? lay.piece : l.V - col0);
        logits.col0 = dhid.col0 = col0;
        logits.cols = dhid.cols = cols;
        logits.store = store;
        e = launch_pair_kernel(logits_kernel<false>, pairs, st, logits);
        if (e != cudaSuccess) return int(e);
        JoinArgs j;
        j.l = l;
        j.tiles = (cols + PG_HALF - 1) / PG_HALF;
        j.last = i + 1 == lay.pieces;
        j.store = store;
        e = launch_kernel(join_kernel, dim3(unsigned(lay.tokens / LS_JOIN_ROWS)),
                          dim3(LS_JOIN_ROWS * 32), 0, st, j);
        if (e != cudaSuccess) return int(e);
        if (store) {
            dhid.first = i == 0;
            dhid.last = i + 1 == lay.pieces && lay.split == 1;
            // W's rows of this piece are the K dimension
            if (!operand_map(&dhid.b, l.weight + int64_t(col0) * l.H, cols, l.H, l.H, true))
                return LORA_ERR_DEVICE;
            e = launch_pair_kernel(hidden_grad_kernel, pairs, st, dhid);
            if (e != cudaSuccess) return int(e);
        }
    }
    if (store && lay.split > 1) {
        const int grid = l.T < 4 * 2 * pairs ? l.T : 4 * 2 * pairs;
        e = launch_kernel(finish_kernel, dim3(grid), dim3(256), 0, st, l);
        if (e != cudaSuccess) return int(e);
    }
    if (dw != nullptr) {
        grad.a = logits.a;
        grad.b = logits.b;
        grad.store = 1;
        head.dw = dw;
        for (int i = 0; i < lay.pieces; ++i) {
            const int32_t col0 = int32_t(i * lay.piece);
            const int32_t cols = int32_t(lay.piece < l.V - col0 ? lay.piece : l.V - col0);
            grad.col0 = head.col0 = col0;
            grad.cols = head.cols = cols;
            e = launch_pair_kernel(logits_kernel<true>, pairs, st, grad);
            if (e != cudaSuccess) return int(e);
            e = launch_pair_kernel(head_grad_kernel, pairs, st, head);
            if (e != cudaSuccess) return int(e);
        }
    }
    return LORA_OK;
}

}  // namespace lora

LORA_API int64_t lora_cross_entropy_workspace(int32_t num_tokens, int32_t hidden, int32_t vocab,
                                              int32_t hidden_grad, int32_t weight_grad)
{
    if (num_tokens < 0 || hidden < 8 || hidden % 8 != 0 || vocab < 1) return LORA_ERR_SIZE;
    const int pairs = lora::device_sm_count() / 2 > 0 ? lora::device_sm_count() / 2 : 1;
    return lora::loss_bytes(num_tokens, hidden, vocab, hidden_grad != 0, weight_grad != 0, pairs);
}

LORA_API int lora_cross_entropy(const lora_bf16_t *hidden, int32_t num_tokens, int32_t hidden_size,
                                int64_t hidden_ld, const lora_bf16_t *weight, int32_t vocab,
                                const int32_t *targets, const float *token_weight, float *loss,
                                float *logsumexp, lora_bf16_t *hidden_grad, int64_t hidden_grad_ld,
                                lora_bf16_t *weight_grad, int32_t *error_word, void *workspace,
                                int64_t workspace_bytes, void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_cross_entropy");
    if (num_tokens < 0 || hidden_size < 8 || vocab < 1 || hidden_ld < hidden_size ||
        (hidden_grad != nullptr && hidden_grad_ld < hidden_size))
        return LORA_ERR_SIZE;
    if (hidden_size % 8 != 0) return LORA_ERR_ALIGN;
    if (weight == nullptr || workspace == nullptr ||
        (num_tokens > 0 && (hidden == nullptr || targets == nullptr || loss == nullptr)))
        return LORA_ERR_NULL;
    auto bits = [](const void *ptr) { return reinterpret_cast<uintptr_t>(ptr); };
    if ((bits(weight) | bits(weight_grad)) & 15u || bits(workspace) & 255u) return LORA_ERR_ALIGN;
    const int pairs = device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1;
    if (workspace_bytes < loss_bytes(num_tokens, hidden_size, vocab, hidden_grad != nullptr, weight_grad != nullptr,
                                     pairs))
        return LORA_ERR_WORKSPACE;
    if (num_tokens == 0) {
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        cudaError_t e = cudaSuccess;
        if (weight_grad != nullptr) e = cudaMemsetAsync(weight_grad, 0, size_t(vocab) * hidden_size * 2, st);
        if (error_word != nullptr && e == cudaSuccess) e = cudaMemsetAsync(error_word, 0, sizeof(int32_t), st);
        return e == cudaSuccess ? LORA_OK : int(e);
    }
    const LossLayout lay = loss_layout(num_tokens, hidden_size, vocab, hidden_grad != nullptr,
                                       weight_grad != nullptr, pairs);
    if (lay.rows) {
        char *at = static_cast<char *>(workspace);
        LossRowArgs r;
        r.hidden = hidden;
        r.weight = weight;
        r.hidden_ld = hidden_ld;
        r.dh_ld = hidden_grad_ld;
        r.targets = targets;
        r.token_weight = token_weight;
        r.loss = loss;
        r.logsumexp = logsumexp;
        r.dh = hidden_grad;
        r.T = num_tokens;
        r.H = hidden_size;
        r.V = vocab;
        r.error_word = error_word;
        r.logit = reinterpret_cast<float *>(at + lay.logit);
        r.stat = reinterpret_cast<float2 *>(at + lay.stat);
        r.acc = hidden_grad != nullptr ? reinterpret_cast<float *>(at + lay.acc) : nullptr;
        return run_loss_row(r, static_cast<cudaStream_t>(stream));
    }
    LossArgs l;
    l.hidden = hidden;
    l.hidden_ld = hidden_ld;
    l.weight = weight;
    l.targets = targets;
    l.token_weight = token_weight;
    l.loss = loss;
    l.logsumexp = logsumexp;
    l.dh = hidden_grad;
    l.dh_ld = hidden_grad_ld;
    l.T = num_tokens;
    l.H = hidden_size;
    l.V = vocab;
    l.hidden_vec = (bits(hidden) & 15u) == 0 && hidden_ld % 8 == 0;
    l.dh_vec = (bits(hidden_grad) & 15u) == 0 && hidden_grad_ld % 8 == 0;
    l.error_word = error_word;
    char *ws = static_cast<char *>(workspace);
    l.count = reinterpret_cast<int32_t *>(ws + lay.count);
    l.row = reinterpret_cast<int32_t *>(ws + lay.row);
    l.target = reinterpret_cast<int32_t *>(ws + lay.target);
    l.wt = reinterpret_cast<float *>(ws + lay.weight);
    l.ref = reinterpret_cast<float *>(ws + lay.ref);
    l.sum = reinterpret_cast<float *>(ws + lay.sum);
    l.logit = reinterpret_cast<float *>(ws + lay.logit);
    l.factor = reinterpret_cast<float *>(ws + lay.factor);
    l.inv = reinterpret_cast<float *>(ws + lay.inv);
    l.share = reinterpret_cast<float *>(ws + lay.share);
    l.stat = reinterpret_cast<float2 *>(ws + lay.stat);
    l.h = reinterpret_cast<uint16_t *>(ws + lay.h);
    l.p = reinterpret_cast<uint16_t *>(ws + lay.p);
    l.acc = reinterpret_cast<float *>(ws + lay.acc);
    l.tokens = lay.tokens;
    l.piece = lay.piece;
    l.split = lay.split;
    l.two = weight_grad != nullptr && num_tokens <= PG_HALF;
    return run_loss(l, lay, weight_grad, static_cast<cudaStream_t>(stream));
}
