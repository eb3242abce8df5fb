// lora_backward.cu -- the gradients of a linear layer's adapters, for a
// batch whose tokens use many adapters:
//   forward   u_t = scale A_a x_t (the fp32 buffer),  y_t += B_a u_t + bias_a
//   g_t = B_a^T dy_t                  dx_t (+)= scale sum_s A_a^T g_t
//   dB_a = sum_t dy_t u_t^T           dA_a = scale sum_t g_t x_t^T
//   dbias_a = sum_t dy_t              (a = id(t); -1: nothing)
//
// Tokens are taken in the metadata's order (sorted by adapter), in tiles of
// 64 tokens of one adapter.  The kernels:
//   grad_u_kernel, join_u_kernel
//                  g of a tile, and u, rounded to bf16 for the products
//                  that follow and laid out by tile with the rows behind an
//                  adapter's last token zero (the products over tokens then
//                  need no masks on them);
//   grad_x_kernel  dx of a tile x 128 hidden columns, all slices summed;
//   grad_w_kernel  dB and dA of an adapter x 128 columns, summed over the
//                  adapter's tokens in a fixed order (no atomics).
// They run on mma.sync; lora_backward_tc.cu holds their forms for ranks above
// 32 on tcgen05.  g and u in bf16 cost about 2^-9 a term, like the
// rounding of the outputs (and u enters as lora_expand took it); all sums are
// fp32.  The two roundings together leave 1.41 times the error of one, evenly
// over many terms, but up to 1.9 times over the few of a small batch.  Calls
// of up to BW_TERMS_TOKENS tokens therefore keep g and u as two bf16 terms
// (2^-16): the second ones are further steps of the products, on the same rows
// of A, x and dy.  64 tokens of rank 8, hidden 256: 10.5 us in place of 9.5;
// 64 of rank 32, 8 adapters, 4096 to 2 x 11008: 36 in place of 30; 16 of rank
// 128, 8192 to 8192, 1024, 1024, 4 adapters: 55 in place of 45 (64 tokens over
// 64 adapters: 340 in place of 265).
//
// 2048 tokens by token over 32 adapters, rank 32, 4096 to 2 x 11008: grad_u
// 32 us (126 MB of dy and B, 4.3 TB/s with its ring a third of an SM's
// memory), join 6, grad_x 16, grad_w 45 (96 MB read and 62 MB written, bound
// by instructions: 59% of the issue slots for tiles of 58 tokens on average).
#include "lora_backward.cuh"

namespace lora {

// Eight elements of a row from column c; columns outside [lo, hi) give zero
// and are not read.
__device__ __forceinline__ uint4 load8(const uint16_t *row, int c, int lo, int hi, bool vec)
{
    if (vec && c >= lo && c + 8 <= hi) return *reinterpret_cast<const uint4 *>(row + c);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j >= lo && c + j < hi) w[j >> 1] |= uint32_t(row[c + j]) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One 16-byte chunk of a row into shared memory: asynchronously where all of
// it lies in [lo, hi) and is aligned, else element by element.
__device__ __forceinline__ void copy8(uint8_t *dst, const uint16_t *row, int c, int lo, int hi, bool vec)
{
    if (vec && c >= lo && c + 8 <= hi)
        cp_async16(smem_addr(dst), row + c, true);
    else
        *reinterpret_cast<uint4 *>(dst) = load8(row, c, lo, hi, false);
}

// ---------------------------------------------------------------- g and u

__device__ __forceinline__ uint2 round4(const float4 &v)
{
    return make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
// What rounding v to h left over, as bf16.
__device__ __forceinline__ uint2 rest4(const float4 &v, const uint2 &h)
{
    return make_uint2(pack_bf16x2(v.x - bf16_lo(h.x), v.y - bf16_hi(h.x)),
                      pack_bf16x2(v.z - bf16_lo(h.y), v.w - bf16_hi(h.y)));
}

template <int RP> struct UShape { static constexpr int WM = 4, WN = 2; };
constexpr int BW_U_STAGES = 4;
constexpr int BW_U_WHOLE = 16;

template <int RP>
constexpr int grad_u_smem() { return BW_U_STAGES * (BW_TOK * 64 * 2 + 64 * RP * 2); }

// The 64-column steps of all (tile, slice) items, in order, cut into even
// runs, one a CTA, whatever the number and the widths of the items: CTA c
// takes steps [step_begin(c), step_begin(c + 1)).
__device__ __forceinline__ int64_t step_begin(int64_t total, int c, int ctas) { return total * c / ctas; }
__device__ __forceinline__ int step_cta(int64_t total, int64_t step, int ctas)
{
    return int(((step + 1) * ctas - 1) / total);
}

// Each CTA walks its run of steps; its part of an item's sum goes to slot
// (CTA + item), a new one whenever the CTA or the item changes.  Bound by
// the reads of dy: a ring of four steps by cp.async.
//
// WHOLE: a CTA takes whole items and writes g and u itself; the join is not
// launched.  For slices of up to BW_U_WHOLE steps: 512 tokens, rank 32, 16
// steps 10.1 us, split and joined 10.3 and a launch more; 4 steps 6.1 and
// 9.5; 24 steps 12.8 and 10.7.
template <int RP, bool WHOLE>
__global__ void __launch_bounds__(BW_THREADS) grad_u_kernel(const __grid_constant__ BackwardArgs p)
{
    constexpr int WM = UShape<RP>::WM, WN = UShape<RP>::WN;
    constexpr int NI = RP / WN / 8, CPR = RP / 8;
    constexpr int SD = BW_TOK * 64 * 2, SB = 64 * RP * 2, ST = BW_U_STAGES;
    constexpr int PB = (64 * CPR + BW_THREADS - 1) / BW_THREADS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wm = warp % WM, wn = warp / WM;
    pdl_wait();
    int tiles;
    const SegTab tab = load_tab(p, reinterpret_cast<int *>(smem + ST * (SD + SB)), tiles);
    const int per_tile = p.step_end[p.S - 1];
    const int64_t total = int64_t(tiles) * per_tile;
    const int ctas = int(min(int64_t(gridDim.x), total));      // a step each at least
    if (!WHOLE && int(blockIdx.x) >= ctas) return;
    // WHOLE: items in place of steps
    int64_t step = WHOLE ? int64_t(blockIdx.x) : step_begin(total, blockIdx.x, ctas);
    const int64_t end = WHOLE ? int64_t(tiles) * p.S : step_begin(total, blockIdx.x + 1, ctas);
    int tile = 0, s = 0, k = 0;
    if constexpr (!WHOLE) {
        tile = int(step / per_tile);
        k = int(step % per_tile);                              // of the tile, then of the slice
        while (k >= p.step_end[s]) ++s;
        if (s > 0) k -= p.step_end[s - 1];
    }
    while (step < end) {
        if constexpr (WHOLE) {
            tile = int(step / p.S);
            s = int(step % p.S);
        }
        const int seg = find_segment(tab.tile, p.nbins, tile);
        const int id = tab.id[seg];
        const int row0 = tab.start[seg] + (tile - tab.tile[seg]) * BW_TOK;
        const int nrows = min(BW_TOK, tab.start[seg] + tab.count[seg] - row0);
        const int lo = p.off[s], hi = lo + p.n[s];
        const int c0 = p.dy_vec ? lo & ~7 : lo;                // first column of the first step
        const int k_lo = k;
        const int steps = p.step_end[s] - (s > 0 ? p.step_end[s - 1] : 0);
        const int k_hi = WHOLE ? steps : int(min(int64_t(steps), k + (end - step)));
        const uint16_t *bw = p.b[s] + int64_t(id) * p.n[s] * p.r;
        const uint16_t *src[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = (tid + i * BW_THREADS) >> 3;
            const int tok = row < nrows ? checked_token(p.sorted[row0 + row], p.T, p.error_word) : -1;
            src[i] = tok >= 0 ? p.dy + int64_t(tok) * p.dy_ld : nullptr;
        }
        auto issue = [&](int k) {
            if (k < k_hi) {
                uint8_t *at = smem + k % ST * (SD + SB);
                const int col = c0 + k * 64;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = tid + i * BW_THREADS;
                    uint8_t *dst = at + tile_at<8, BW_TOK>(c >> 3, c & 7);
                    if (src[i] != nullptr) copy8(dst, src[i], col + (c & 7) * 8, lo, hi, p.dy_vec);
                    else *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < PB; ++i) {
                    const int c = tid + i * BW_THREADS, row = col + c / CPR - lo, ch = c % CPR;
                    if (c >= 64 * CPR) break;
                    const bool ok = row >= 0 && row < hi - lo && ch * 8 < p.r;
                    cp_async16(smem_addr(at + SD + tile_at<CPR, 64>(c / CPR, ch)),
                               ok ? bw + int64_t(row) * p.r + ch * 8 : bw, ok);
                }
            }
            cp_async_commit();
        };
        float acc[NI][4] = {};
        for (int i = k_lo; i < k_lo + ST - 1; ++i) issue(i);
        float4 u[WHOLE ? RP / 16 : 1];
        if constexpr (WHOLE) {
#pragma unroll
            for (int i = 0; i < RP / 16; ++i) {
                const int at = (tid + i * BW_THREADS) * 4, row = at / RP, col = at % RP;
                u[i] = make_float4(0, 0, 0, 0);
                if (row < nrows && col < p.r) {
                    const int tok = checked_token(p.sorted[row0 + row], p.T, p.error_word);
                    if (tok >= 0)
                        u[i] = *reinterpret_cast<const float4 *>(p.buf + (int64_t(s) * p.T + tok) * p.r + col);
                }
            }
        }
        for (int i = k_lo; i < k_hi; ++i) {
            cp_async_wait<ST - 2>();
            __syncthreads();
            issue(i + ST - 1);
            const uint32_t sd = base + i % ST * (SD + SB), sb = sd + SD;
#pragma unroll
            for (int kk = 0; kk < 64; kk += 16) {
                uint32_t a[4];
                frag_a<8, BW_TOK, true>(sd, wm * 16, kk, a);
                if constexpr (NI == 1) {
                    uint32_t b[2];
                    frag_b1<CPR, 64>(sb, kk, wn * 8, b);
                    mma_bf16_16816(acc[0], a, b[0], b[1]);
                } else {
#pragma unroll
                    for (int j = 0; j < NI; j += 2) {
                        uint32_t b[4];
                        frag_b<CPR, 64, false>(sb, kk, wn * (RP / WN) + 8 * j, b);
                        mma_bf16_16816(acc[j], a, b[0], b[1]);
                        mma_bf16_16816(acc[j + 1], a, b[2], b[3]);
                    }
                }
            }
        }
        const int gq = lane >> 2, t = lane & 3;
        if constexpr (WHOLE) {
            const int64_t out0 = (int64_t(s) * p.rows + int64_t(tile) * BW_TOK) * RP;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                uint16_t *at = p.g + out0 + (wm * 16 + gq) * RP + wn * (RP / WN) + 8 * j + 2 * t;
                const uint2 h = make_uint2(pack_bf16x2(acc[j][0], acc[j][1]), pack_bf16x2(acc[j][2], acc[j][3]));
                *reinterpret_cast<uint32_t *>(at) = h.x;
                *reinterpret_cast<uint32_t *>(at + 8 * RP) = h.y;
                if (p.low != 0) {
                    const uint2 l = rest4(make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]), h);
                    *reinterpret_cast<uint32_t *>(at + p.low) = l.x;
                    *reinterpret_cast<uint32_t *>(at + p.low + 8 * RP) = l.y;
                }
            }
#pragma unroll
            for (int i = 0; i < RP / 16; ++i) {
                uint16_t *at = p.u + out0 + (tid + i * BW_THREADS) * 4;
                const uint2 h = round4(u[i]);
                *reinterpret_cast<uint2 *>(at) = h;
                if (p.low != 0) *reinterpret_cast<uint2 *>(at + p.low) = rest4(u[i], h);
            }
            __syncthreads();                                   // the ring is free
            step += gridDim.x;
            continue;
        }
        float *out = p.part + (int64_t(blockIdx.x) + int64_t(tile) * p.S + s) * BW_TOK * RP;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            float *at = out + (wm * 16 + gq) * RP + wn * (RP / WN) + 8 * j + 2 * t;
            *reinterpret_cast<float2 *>(at) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2 *>(at + 8 * RP) = make_float2(acc[j][2], acc[j][3]);
        }
        __syncthreads();                                       // the ring is free
        step += k_hi - k_lo;
        k = 0;
        if (++s == p.S) {
            s = 0;
            ++tile;
        }
    }
}

// The partial sums of a tile, added in a fixed order and rounded: g; and u
// beside it.  A block takes 16 tokens x 16 columns at a time, a quarter of
// the slots each 64 threads: with few tiles there are many slots of each (a
// block a tile took 53 us at rank 128, 512 tokens, widths 4096, 1024, 1024;
// this 7).
template <int RP>
__global__ void __launch_bounds__(BW_THREADS) join_u_kernel(const __grid_constant__ BackwardArgs p)
{
    constexpr int PARTS = RP / 4, TEAMS = BW_THREADS / 64;
    extern __shared__ __align__(16) int join_tab[];
    __shared__ float4 s_sum[TEAMS - 1][64];
    __shared__ __align__(16) uint16_t s_turned[2][16][16];
    pdl_wait();
    int tiles;
    const SegTab tab = load_tab(p, join_tab, tiles);
    const int per_tile = p.step_end[p.S - 1];
    const int64_t total = int64_t(tiles) * per_tile;
    const int ctas = int(min(int64_t(p.u_ctas), total));
    const int team = threadIdx.x >> 6, t = threadIdx.x & 63;
    for (int unit = blockIdx.x; unit < tiles * p.S * PARTS; unit += gridDim.x) {
        const int item = unit / PARTS, part = unit % PARTS;
        const int tile = item / p.S, s = item % p.S;
        const int row = (part & 3) * 16 + (t >> 2), col = (part >> 2) * 16 + (t & 3) * 4;
        const int64_t first = int64_t(tile) * per_tile + (s > 0 ? p.step_end[s - 1] : 0);
        const int c_lo = step_cta(total, first, ctas);
        const int slots = step_cta(total, int64_t(tile) * per_tile + p.step_end[s] - 1, ctas) + 1 - c_lo;
        const float *from = p.part + (int64_t(c_lo) + item) * BW_TOK * RP + row * RP + col;
        float4 v = make_float4(0, 0, 0, 0);
        const int end = slots * (team + 1) / TEAMS;
#pragma unroll 4
        for (int c = slots * team / TEAMS; c < end; ++c) {
            const float4 x = *reinterpret_cast<const float4 *>(from + int64_t(c) * BW_TOK * RP);
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
        }
        if (team > 0) s_sum[team - 1][t] = v;
        float4 uf = make_float4(0, 0, 0, 0);               // u; then, of team 0, g
        if (team == 1) {
            const int seg = find_segment(tab.tile, p.nbins, tile);
            const int row0 = tab.start[seg] + (tile - tab.tile[seg]) * BW_TOK;
            if (row < tab.start[seg] + tab.count[seg] - row0 && col < p.r) {
                const int tok = checked_token(p.sorted[row0 + row], p.T, p.error_word);
                if (tok >= 0)
                    uf = *reinterpret_cast<const float4 *>(p.buf + (int64_t(s) * p.T + tok) * p.r + col);
            }
        }
        __syncthreads();
        const int64_t out0 = (int64_t(s) * p.rows + int64_t(tile) * BW_TOK) * RP;
        if (team == 0) {
#pragma unroll
            for (int i = 0; i < TEAMS - 1; ++i) {
                const float4 x = s_sum[i][t];
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
            }
            uf = v;
        }
        const uint2 uv = round4(uf);
        if (team == 0 || (team == 1 && p.ut == nullptr)) {
            uint16_t *at = (team == 0 ? p.g : p.u) + out0 + row * RP + col;
            *reinterpret_cast<uint2 *>(at) = uv;
            if (p.low != 0) *reinterpret_cast<uint2 *>(at + p.low) = rest4(uf, uv);
        }
        if (p.ut != nullptr) {
            // transposed: 32 bytes of 16 tokens for each column
            auto turn = [&](const uint2 &v, int64_t low) {
                if (team < 2) {
                    uint16_t(&at)[16][16] = s_turned[team];
                    const int y = t >> 2, x = (t & 3) * 4;
                    at[x][y] = uint16_t(v.x & 0xFFFFu);
                    at[x + 1][y] = uint16_t(v.x >> 16);
                    at[x + 2][y] = uint16_t(v.y & 0xFFFFu);
                    at[x + 3][y] = uint16_t(v.y >> 16);
                }
                __syncthreads();
                if (team == 0) {
                    const int which = t >> 5, x = t >> 1 & 15, half = (t & 1) * 8;
                    *reinterpret_cast<uint4 *>((which == 0 ? p.gt : p.ut) + low + out0 +
                                               ((part >> 2) * 16 + x) * BW_TOK + (part & 3) * 16 + half) =
                        *reinterpret_cast<const uint4 *>(&s_turned[which][x][half]);
                }
            };
            turn(uv, 0);
            if (p.low != 0) {
                __syncthreads();
                turn(rest4(uf, uv), p.low);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- dx

constexpr int BW_X_STAGES = 3;
constexpr int BW_X_LD = BW_COLS + 4;       // floats of a staged row of dx

template <int RP>
constexpr int grad_x_smem()
{
    return BW_X_STAGES * (BW_TOK * RP * 2 + RP * BW_COLS * 2) + BW_TOK * BW_X_LD * 4;
}

// Item: (tile, 128 columns), one step a slice (and term of g); a ring of three
// steps runs across the items.
template <int RP, bool TERMS>
__global__ void __launch_bounds__(BW_THREADS, RP <= 32 ? 3 : 1) grad_x_kernel(const __grid_constant__ BackwardArgs p)
{
    constexpr int CPR = RP / 8, ST = BW_X_STAGES;
    constexpr int SG = BW_TOK * RP * 2, SA = RP * BW_COLS * 2;
    constexpr int PG = (BW_TOK * CPR + BW_THREADS - 1) / BW_THREADS, PA = RP * 16 / BW_THREADS;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *stage = reinterpret_cast<float *>(smem + ST * (SG + SA));
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int m0 = warp % 4 * 16, n0 = warp / 4 * 64;          // 16 tokens x 64 columns a warp
    pdl_wait();
    int tiles;
    const SegTab tab = load_tab(p, reinterpret_cast<int *>(smem + grad_x_smem<RP>()), tiles);
    const int hb = (p.H + BW_COLS - 1) / BW_COLS;
    const int items = tiles * hb;             // T x H fits the memory: below 2^31
    const int steps = TERMS ? 2 * p.S : p.S;

    // the step that is loaded next
    int l_item = blockIdx.x;
    int l_s = 0, l_stage = 0;
    auto issue = [&]() {
        if (l_item < items) {
            const int tile = l_item / hb, h0 = l_item % hb * BW_COLS;
            const int seg = find_segment(tab.tile, p.nbins, tile);
            const bool second = TERMS && l_s >= p.S;
            const int s = second ? l_s - p.S : l_s;
            const uint16_t *gt = p.g + (second ? p.low : 0) + (int64_t(s) * p.rows + int64_t(tile) * BW_TOK) * RP;
            const uint16_t *aw = p.a[s] + int64_t(tab.id[seg]) * p.r * p.H;
            uint8_t *at = smem + l_stage * (SG + SA);
#pragma unroll
            for (int i = 0; i < PG; ++i) {
                const int c = tid + i * BW_THREADS;
                if (c < BW_TOK * CPR)
                    cp_async16(smem_addr(at + tile_at<CPR, BW_TOK>(c / CPR, c % CPR)), gt + c * 8, true);
            }
#pragma unroll
            for (int i = 0; i < PA; ++i) {
                const int c = tid + i * BW_THREADS, row = c >> 4, col = h0 + (c & 15) * 8;
                const bool ok = row < p.r && col < p.H;
                cp_async16(smem_addr(at + SG + tile_at<16, RP>(row, c & 15)),
                           ok ? aw + int64_t(row) * p.H + col : aw, ok);
            }
            if (++l_s == steps) {
                l_s = 0;
                l_item += gridDim.x;
            }
        }
        l_stage = l_stage + 1 == ST ? 0 : l_stage + 1;
        cp_async_commit();
    };
    for (int i = 0; i < ST - 1; ++i) issue();
    int stg = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int tile = item / hb, h0 = item % hb * BW_COLS;
        const int seg = find_segment(tab.tile, p.nbins, tile);
        const int row0 = tab.start[seg] + (tile - tab.tile[seg]) * BW_TOK;
        const int nrows = min(BW_TOK, tab.start[seg] + tab.count[seg] - row0);
        // the rows this thread writes: 16 threads a row, four rows each
        int tok[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (tid >> 4) + 16 * i;
            tok[i] = row < nrows ? checked_token(p.sorted[row0 + row], p.T, p.error_word) : -1;
        }
        float acc[8][4] = {};
        for (int s = 0; s < steps; ++s) {
            cp_async_wait<ST - 2>();
            __syncthreads();
            issue();
            const uint32_t sg = base + stg * (SG + SA), sa = sg + SG;
            stg = stg + 1 == ST ? 0 : stg + 1;
#pragma unroll
            for (int kk = 0; kk < RP; kk += 16) {
                uint32_t a[4];
                frag_a<CPR, BW_TOK, true>(sg, m0, kk, a);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    uint32_t b[4];
                    frag_b<16, RP, false>(sa, kk, n0 + 8 * j, b);
                    mma_bf16_16816(acc[j], a, b[0], b[1]);
                    mma_bf16_16816(acc[j + 1], a, b[2], b[3]);
                }
            }
        }
        const int gq = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float *at = stage + (m0 + gq) * BW_X_LD + n0 + 8 * j + 2 * t;
            *reinterpret_cast<float2 *>(at) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2 *>(at + 8 * BW_X_LD) = make_float2(acc[j][2], acc[j][3]);
        }
        __syncthreads();
        const int col = h0 + (tid & 15) * 8;
        if (col < p.H) {
            uint4 was[4];
            if (p.add) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tok[i] >= 0) was[i] = load8(p.dx + int64_t(tok[i]) * p.dx_ld, col, 0, p.H, p.dx_vec);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (tok[i] < 0) continue;
                const float *v = stage + ((tid >> 4) + 16 * i) * BW_X_LD + (tid & 15) * 8;
                float f[8];
                *reinterpret_cast<float4 *>(f) = *reinterpret_cast<const float4 *>(v);
                *reinterpret_cast<float4 *>(f + 4) = *reinterpret_cast<const float4 *>(v + 4);
                const uint32_t w[4] = {was[i].x, was[i].y, was[i].z, was[i].w};
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = p.scale * f[2 * e], y = p.scale * f[2 * e + 1];
                    if (p.add) {
                        x += bf16_lo(w[e]);
                        y += bf16_hi(w[e]);
                    }
                    o[e] = pack_bf16x2(x, y);
                }
                uint16_t *dst = p.dx + int64_t(tok[i]) * p.dx_ld + col;
                if (p.dx_vec) {
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dst[2 * e] = uint16_t(o[e] & 0xFFFFu);
                        dst[2 * e + 1] = uint16_t(o[e] >> 16);
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
    if (!p.add) clear_rest(p, tab, warp, BW_THREADS / 32);
}

// ---------------------------------------------------------------- dA, dB, dbias

template <int RP> struct WShape { static constexpr int WM = RP >= 64 ? 4 : 8, WN = 8 / WM; };
constexpr int BW_W_STAGES = 3;
constexpr int BW_W_LD = BW_COLS + 8;       // elements of a staged row of dA

template <int RP>
constexpr int grad_w_smem()
{
    return BW_W_STAGES * (BW_TOK * BW_COLS * 2 + BW_TOK * RP * 2) + RP * BW_W_LD * 2;
}

// Item: (adapter, column block): D[128 columns x RP] = sum over the
// adapter's tokens of dy^T u (dB) or x^T g (dA), 64 tokens a step (an
// adapter without tokens has one step of zeros).  Per-token adapters give
// items of a single step, so a ring of three steps runs across the items.
// TERMS: the same steps again for the second terms of g and u.
template <int RP, bool TERMS>
__global__ void __launch_bounds__(BW_THREADS) grad_w_kernel(const __grid_constant__ BackwardArgs p)
{
    constexpr int WM = WShape<RP>::WM, WN = WShape<RP>::WN, ST = BW_W_STAGES;
    constexpr int MI = BW_COLS / WM / 16, NI = RP / WN / 8, CPR = RP / 8;
    constexpr int SZ = BW_TOK * BW_COLS * 2, SV = BW_TOK * RP * 2;
    constexpr int PV = (BW_TOK * CPR + BW_THREADS - 1) / BW_THREADS;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *stage = smem + ST * (SZ + SV);
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wm = warp % WM, wn = warp / WM;
    pdl_wait();
    int tiles;
    int *mem = reinterpret_cast<int *>(smem + grad_w_smem<RP>());
    const SegTab tab = load_tab(p, mem, tiles);
    const int *seg_of = load_seg_of(p, tab, tiles, mem);
    const int blocks = p.block_end[2 * p.S - 1];

    // A block of an adapter's gradients: its product (dB of slice q, or dA of
    // slice q - S) and its first column.  Items are taken gridDim.x apart; the
    // walk adds instead of dividing.
    struct Walk {
        int id, blk, q, c0;
    };
    const int step_id = gridDim.x / blocks, step_blk = gridDim.x % blocks;
    auto place = [&](Walk &w) {
        int q = 0, from = 0;
        while (w.blk >= p.block_end[q]) from = p.block_end[q++];
        w.q = q;
        w.c0 = (w.blk - from) * BW_COLS;
        if (q < p.S) w.c0 += p.dy_vec ? p.off[q] & ~7 : p.off[q];
    };
    auto next = [&](Walk &w) {
        w.id += step_id;
        w.blk += step_blk;
        if (w.blk >= blocks) {
            w.blk -= blocks;
            ++w.id;
        }
        if (w.id < p.L) place(w);
    };
    Walk at;                                    // the item that is multiplied next
    at.id = blockIdx.x / blocks;
    at.blk = blockIdx.x % blocks;
    if (at.id < p.L) place(at);

    // the step that is loaded next, with its tokens
    Walk to = at;
    const uint16_t *z = nullptr, *v = nullptr;
    int64_t z_ld = 0;
    int start = 0, count = 0, l_k = 0, l_half = 1, l_stage = 0, tok[4];
    bool vec = false, whole = false;
    const int z_at = int(tile_at<16, BW_TOK>(tid >> 4, tid & 15));
    auto tokens = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (TERMS && l_k >= l_half ? l_k - l_half : l_k) * BW_TOK + (tid >> 4) + i * 16;
            tok[i] = row < count ? checked_token(p.sorted[start + row], p.T, p.error_word) : -1;
        }
    };
    auto enter = [&]() {
        if (to.id >= p.L) return;
        const bool is_a = to.q >= p.S;
        const int seg = seg_of[to.id], s = is_a ? to.q - p.S : to.q, col = to.c0 + (tid & 15) * 8;
        const int width = is_a ? p.H : p.width;
        start = seg >= 0 ? tab.start[seg] : 0;
        count = seg >= 0 ? tab.count[seg] : 0;
        if constexpr (TERMS) l_half = count > 0 ? (count + BW_TOK - 1) / BW_TOK : 1;
        z = (is_a ? p.x : p.dy) + col;
        z_ld = is_a ? p.x_ld : p.dy_ld;
        vec = is_a ? p.x_vec : p.dy_vec;
        whole = vec && col + 8 <= width;
        v = (is_a ? p.g : p.u) +
            (int64_t(s) * p.rows + (seg >= 0 ? int64_t(tab.tile[seg]) * BW_TOK : 0)) * RP + tid * 8;
        tokens();
    };
    enter();
    auto issue = [&]() {
        if (to.id < p.L) {
            uint8_t *dst = smem + l_stage * (SZ + SV) + z_at;
            if (whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    cp_async16(smem_addr(dst + i * 16 * 128), tok[i] < 0 ? z : z + tok[i] * z_ld, tok[i] >= 0);
            } else {
                const int col = to.c0 + (tid & 15) * 8, width = to.q >= p.S ? p.H : p.width;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(dst + i * 16 * 128) =
                        tok[i] < 0 ? make_uint4(0, 0, 0, 0) : load8(z - col + tok[i] * z_ld, col, 0, width, false);
            }
            const uint32_t sv = base + l_stage * (SZ + SV) + SZ;
            int64_t v_at = int64_t(l_k) * BW_TOK * RP;
            if (TERMS && l_k >= l_half) v_at = p.low + int64_t(l_k - l_half) * BW_TOK * RP;
#pragma unroll
            for (int i = 0; i < PV; ++i) {
                const int c = tid + i * BW_THREADS;
                if (c < BW_TOK * CPR)
                    cp_async16(sv + tile_at<CPR, BW_TOK>(c / CPR, c % CPR),
                               count > 0 ? v + v_at + i * BW_THREADS * 8 : p.g, count > 0);
            }
            if (TERMS ? ++l_k >= (count > 0 ? 2 * l_half : 1) : ++l_k * BW_TOK >= count) {
                l_k = 0;
                next(to);
                enter();
            } else {
                tokens();
            }
        }
        l_stage = l_stage + 1 == ST ? 0 : l_stage + 1;
        cp_async_commit();
    };
    for (int i = 0; i < ST - 1; ++i) issue();
    int stg = 0;
    for (; at.id < p.L; next(at)) {
        const bool is_a = at.q >= p.S;
        const int s = is_a ? at.q - p.S : at.q, seg = seg_of[at.id];
        const int firsts = seg >= 0 ? (tab.count[seg] + BW_TOK - 1) / BW_TOK : 1;
        const int steps = TERMS && seg >= 0 ? 2 * firsts : firsts;
        const int lo = is_a ? 0 : p.off[s], n = is_a ? p.H : p.n[s];
        uint16_t *dbias = is_a ? nullptr : p.dbias[s];
        float acc[MI][NI][4] = {}, ones[MI][4] = {};
        for (int k = 0; k < steps; ++k) {
            cp_async_wait<ST - 2>();
            __syncthreads();
            issue();
            const uint32_t sz = base + stg * (SZ + SV), sv = sz + SZ;
            stg = stg + 1 == ST ? 0 : stg + 1;
#pragma unroll
            for (int kk = 0; kk < BW_TOK; kk += 16) {
                uint32_t a[MI][4];
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    frag_a<16, BW_TOK, false>(sz, wm * (BW_COLS / WM) + i * 16, kk, a[i]);
#pragma unroll
                for (int j = 0; j < NI; j += 2) {
                    uint32_t b[4];
                    frag_b<CPR, BW_TOK, false>(sv, kk, wn * (RP / WN) + 8 * j, b);
#pragma unroll
                    for (int i = 0; i < MI; ++i) {
                        mma_bf16_16816(acc[i][j], a[i], b[0], b[1]);
                        mma_bf16_16816(acc[i][j + 1], a[i], b[2], b[3]);
                    }
                }
                if (dbias != nullptr && wn == 0 && (!TERMS || k < firsts)) {
                    // a product with ones: column 0 of the result
                    const uint32_t one = lane < 4 ? 0x3F803F80u : 0u;
#pragma unroll
                    for (int i = 0; i < MI; ++i) mma_bf16_16816(ones[i], a[i], one, one);
                }
            }
        }
        // out through shared memory, rounded; dA transposed
        const int gq = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int m = wm * (BW_COLS / WM) + i * 16 + gq, c = wn * (RP / WN) + 8 * j + 2 * t;
                if (!is_a) {
                    *reinterpret_cast<uint32_t *>(stage + tile_at<CPR, BW_COLS>(m, c / 8) + c % 8 * 2) =
                        pack_bf16x2(acc[i][j][0], acc[i][j][1]);
                    *reinterpret_cast<uint32_t *>(stage + tile_at<CPR, BW_COLS>(m + 8, c / 8) + c % 8 * 2) =
                        pack_bf16x2(acc[i][j][2], acc[i][j][3]);
                } else {
                    uint16_t *to_m = reinterpret_cast<uint16_t *>(stage) + c * BW_W_LD + m;
                    const uint32_t v0 = pack_bf16x2(p.scale * acc[i][j][0], p.scale * acc[i][j][1]);
                    const uint32_t v1 = pack_bf16x2(p.scale * acc[i][j][2], p.scale * acc[i][j][3]);
                    to_m[0] = uint16_t(v0 & 0xFFFFu);
                    to_m[BW_W_LD] = uint16_t(v0 >> 16);
                    to_m[8] = uint16_t(v1 & 0xFFFFu);
                    to_m[BW_W_LD + 8] = uint16_t(v1 >> 16);
                }
            }
        if (dbias != nullptr && wn == 0 && t == 0) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = at.c0 + wm * (BW_COLS / WM) + i * 16 + gq + 8 * half - lo;
                    if (row >= 0 && row < n)
                        dbias[int64_t(at.id) * n + row] =
                            uint16_t(pack_bf16x2(ones[i][2 * half], 0.0f) & 0xFFFFu);
                }
        }
        __syncthreads();
        if (!is_a) {
            uint16_t *out = p.db[s];
            if (out != nullptr) {
                for (int i = tid; i < BW_COLS * CPR; i += BW_THREADS) {
                    const int m = i / CPR, c = i % CPR, row = at.c0 + m - lo;
                    if (row >= 0 && row < n && c * 8 < p.r)
                        *reinterpret_cast<uint4 *>(out + (int64_t(at.id) * n + row) * p.r + c * 8) =
                            *reinterpret_cast<const uint4 *>(stage + tile_at<CPR, BW_COLS>(m, c));
                }
            }
        } else {
            uint16_t *out = p.da[s] + int64_t(at.id) * p.r * p.H + at.c0;
            for (int i = tid; i < 16 * p.r; i += BW_THREADS) {
                const int c = i >> 4, m = (i & 15) * 8;
                if (at.c0 + m < p.H)
                    *reinterpret_cast<uint4 *>(out + int64_t(c) * p.H + m) =
                        *reinterpret_cast<const uint4 *>(reinterpret_cast<uint16_t *>(stage) + c * BW_W_LD + m);
            }
        }
    }
    cp_async_wait<0>();
}

// ---------------------------------------------------------------- host

static int padded_rank(int r)
{
    int rp = 16;
    while (rp < r) rp *= 2;
    return rp;
}

constexpr int BW_RESIDENT = 4;             // CTAs of a kernel on an SM, at most

// Rows of the laid-out g and u of one slice: every adapter that occurs may
// add a partial tile.
static int64_t backward_rows(int64_t T, int64_t L)
{
    return (T / BW_TOK + (L < T ? L : T)) * BW_TOK;
}

// Copies of the laid-out g or u in the workspace: g, u, and for ranks above
// 32 g transposed; each with its second terms behind it in a small batch.
static int backward_terms(int64_t T) { return T <= BW_TERMS_TOKENS ? 2 : 1; }
static int backward_parts(int64_t T, int rank) { return (rank > 32 ? 3 : 2) * backward_terms(T); }

// g and u, and the slots of partial sums: one an item and one a CTA.
static int64_t backward_bytes(int64_t T, int S, int rank, int64_t L)
{
    const int64_t rows = backward_rows(T, L), one = rows * S * padded_rank(rank) * 2;
    const int64_t slots = rows / BW_TOK * S + BW_RESIDENT * device_sm_count();
    return backward_parts(T, rank) * ((one + 255) / 256 * 256) + slots * BW_TOK * padded_rank(rank) * 4;
}

template <int RP>
static int run_backward(BackwardArgs p, cudaStream_t st)
{
    const bool w_tc = grad_w_tc_fits(p, RP);
    if (!w_tc) p.gt = p.ut = nullptr;
    const int tab = int(seg_tab_bytes(p.nbins));
    const int us = grad_u_smem<RP>() + tab, xs = grad_x_smem<RP>() + tab;
    const int ws = grad_w_smem<RP>() + tab + p.L * 4;
    cudaError_t e;
    static int configured[64] = {0};
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return int(e);
    if (dev >= 64 || !configured[dev]) {
        constexpr int most = int(seg_tab_bytes(LORA_MAX_LORAS + 1)) + LORA_MAX_LORAS * 4;
        if ((e = cudaFuncSetAttribute(grad_u_kernel<RP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      grad_u_smem<RP>() + most)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(grad_u_kernel<RP <= 32 ? RP : 32, true>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      grad_u_smem<RP <= 32 ? RP : 32>() + most)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(grad_x_kernel<RP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      grad_x_smem<RP>() + most)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(grad_x_kernel<RP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      grad_x_smem<RP>() + most)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(grad_w_kernel<RP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      grad_w_smem<RP>() + most)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(grad_w_kernel<RP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      grad_w_smem<RP>() + most)) != cudaSuccess)
            return int(e);
        if (dev < 64) configured[dev] = 1;
    }
    const int sms = device_sm_count();
    // resident CTAs of a kernel by its shared memory
    auto resident = [&](int smem) {
        const int n = 227 * 1024 / (smem + 1024);
        return int64_t(sms) * (n < 1 ? 1 : n > BW_RESIDENT ? BW_RESIDENT : n);
    };
    const int64_t tiles = p.rows / BW_TOK;
    // Ranks above 32 run on tcgen05 where the rows allow TMA.
    int tc = RP >= 64 && p.T > 0 ? launch_grad_u_tc(p, RP, st) : -1;
    if (tc > 0) return tc;
    int longest = 0;                           // steps of a slice
    for (int k = 0; k < p.S; ++k) {
        const int steps = p.step_end[k] - (k > 0 ? p.step_end[k - 1] : 0);
        if (steps > longest) longest = steps;
    }
    if (p.T > 0 && RP <= 32 && longest <= BW_U_WHOLE) {
        const int64_t most = tiles * p.S, grid = most < resident(us) ? most : resident(us);
        e = launch_kernel(grad_u_kernel<RP <= 32 ? RP : 32, true>, dim3(unsigned(grid)), dim3(BW_THREADS), us, st, p);
        if (e != cudaSuccess) return int(e);
    } else if (p.T > 0 && tc < 0) {
        BackwardArgs q = p;
        q.u_ctas = int(resident(us));
        e = launch_kernel(grad_u_kernel<RP, false>, dim3(unsigned(q.u_ctas)), dim3(BW_THREADS), us, st, q);
        if (e != cudaSuccess) return int(e);
        const int64_t most = tiles * p.S * (RP / 4), grid = most < 8 * sms ? most : 8 * sms;
        e = launch_kernel(join_u_kernel<RP>, dim3(unsigned(grid)), dim3(BW_THREADS), tab, st, q);
        if (e != cudaSuccess) return int(e);
    }
    const int64_t items = int64_t(p.L) * p.block_end[2 * p.S - 1];
    if (w_tc) {
        if (int err = launch_grad_w_tc(p, RP, st)) return err;
    } else if (items > 0) {
        const int64_t grid = items < resident(ws) ? items : resident(ws);
        e = launch_kernel(p.low != 0 ? grad_w_kernel<RP, true> : grad_w_kernel<RP, false>, dim3(unsigned(grid)),
                          dim3(BW_THREADS), ws, st, p);
        if (e != cudaSuccess) return int(e);
    }
    // dx last: it may be written over dy or x, which the kernels before read
    if (p.T > 0 && p.dx != nullptr) {
        tc = RP >= 64 ? launch_grad_x_tc(p, RP, st) : -1;
        if (tc > 0) return tc;
        if (tc < 0) {
            const int64_t most = tiles * ((p.H + BW_COLS - 1) / BW_COLS);
            const int64_t grid = most < resident(xs) ? most : resident(xs);
            e = launch_kernel(p.low != 0 ? grad_x_kernel<RP, true> : grad_x_kernel<RP, false>,
                              dim3(unsigned(grid)), dim3(BW_THREADS), xs, st, p);
            if (e != cudaSuccess) return int(e);
        }
    }
    return LORA_OK;
}

}  // namespace lora

LORA_API int64_t lora_linear_backward_workspace(int32_t num_tokens, int32_t hidden,
                                                const int32_t *slice_sizes, int32_t num_slices,
                                                int32_t rank, int32_t max_loras)
{
    if (slice_sizes == nullptr) return LORA_ERR_NULL;
    if (hidden < 8 || hidden % 8 != 0 || num_tokens < 0 || max_loras < 1 || max_loras > LORA_MAX_LORAS)
        return LORA_ERR_SIZE;
    if (num_slices < 1 || num_slices > LORA_MAX_SLICES) return LORA_ERR_SLICES;
    if (rank < 8 || rank > LORA_MAX_RANK || rank % 8 != 0) return LORA_ERR_RANK;
    // a workspace holds every smaller batch too, whose g and u may have more terms
    const int64_t own = lora::backward_bytes(num_tokens, num_slices, rank, max_loras);
    const int64_t small = num_tokens > lora::BW_TERMS_TOKENS
                              ? lora::backward_bytes(lora::BW_TERMS_TOKENS, num_slices, rank, max_loras) : 0;
    return own > small ? own : small;
}

LORA_API int lora_linear_backward(const lora_bf16_t *dy, int64_t dy_ld, int32_t num_tokens,
                                  const lora_bf16_t *x, int32_t hidden, int64_t x_ld,
                                  const float *buf, const lora_bf16_t *const *lora_a,
                                  const lora_bf16_t *const *lora_b, const int32_t *slice_sizes,
                                  int32_t num_slices, int32_t rank, float scale, lora_bf16_t *dx,
                                  int64_t dx_ld, int32_t add_inputs, lora_bf16_t *const *d_lora_a,
                                  lora_bf16_t *const *d_lora_b, lora_bf16_t *const *d_lora_bias,
                                  const lora_meta_t *meta, void *workspace, int64_t workspace_bytes,
                                  void *stream)
{
    using namespace lora;
    NvtxRange nvtx_range("lora_linear_backward");
    if (meta == nullptr || slice_sizes == nullptr || lora_a == nullptr || lora_b == nullptr)
        return LORA_ERR_NULL;
    if (num_slices < 1 || num_slices > LORA_MAX_SLICES) return LORA_ERR_SLICES;
    if (rank < 8 || rank > LORA_MAX_RANK || rank % 8 != 0) return LORA_ERR_RANK;
    if (num_tokens < 0 || hidden < 8 || meta->max_loras < 1 || meta->max_loras > LORA_MAX_LORAS)
        return LORA_ERR_SIZE;
    if (num_tokens > meta->max_num_tokens) return LORA_ERR_TOKENS;
    if (hidden % 8 != 0) return LORA_ERR_ALIGN;
    if (!meta->token_indices_sorted_by_lora_ids || !meta->num_tokens_per_lora ||
        !meta->lora_token_start_loc || !meta->active_lora_ids || !meta->no_lora_flag ||
        !meta->error_word || workspace == nullptr)
        return LORA_ERR_NULL;
    if (num_tokens > 0 && (dy == nullptr || x == nullptr || buf == nullptr)) return LORA_ERR_NULL;
    auto bits = [](const void *ptr) { return reinterpret_cast<uintptr_t>(ptr); };
    BackwardArgs p;
    int64_t width = 0;
    int blocks = 0;
    for (int s = 0; s < LORA_MAX_SLICES; ++s) {
        const bool in = s < num_slices;
        p.a[s] = in ? lora_a[s] : nullptr;
        p.b[s] = in ? lora_b[s] : nullptr;
        p.da[s] = in && d_lora_a != nullptr ? d_lora_a[s] : nullptr;
        p.db[s] = in && d_lora_b != nullptr ? d_lora_b[s] : nullptr;
        p.dbias[s] = in && d_lora_bias != nullptr ? d_lora_bias[s] : nullptr;
        p.n[s] = p.off[s] = 0;
        if (!in) continue;
        if (p.a[s] == nullptr || p.b[s] == nullptr) return LORA_ERR_NULL;
        if (slice_sizes[s] < 1) return LORA_ERR_SIZE;
        if ((bits(p.a[s]) | bits(p.b[s]) | bits(p.da[s]) | bits(p.db[s])) & 15u) return LORA_ERR_ALIGN;
        p.n[s] = slice_sizes[s];
        p.off[s] = int32_t(width);
        width += slice_sizes[s];
        if (width > (int64_t(1) << 30)) return LORA_ERR_SIZE;
    }
    if (dy_ld < width) return LORA_ERR_WIDTH;
    if (x_ld < hidden || (dx != nullptr && dx_ld < hidden)) return LORA_ERR_SIZE;
    if ((bits(buf) & 15u) || (bits(workspace) & 255u)) return LORA_ERR_ALIGN;
    if (workspace_bytes < lora_linear_backward_workspace(num_tokens, hidden, slice_sizes, num_slices, rank,
                                                         meta->max_loras))
        return LORA_ERR_WORKSPACE;
    p.dy = dy;
    p.dy_ld = dy_ld;
    p.x = x;
    p.x_ld = x_ld;
    p.buf = buf;
    p.dx = dx;
    p.dx_ld = dx_ld;
    p.T = num_tokens;
    p.H = hidden;
    p.S = num_slices;
    p.r = rank;
    p.L = meta->max_loras;
    p.width = int32_t(width);
    p.add = add_inputs != 0;
    p.dy_vec = (bits(dy) & 15u) == 0 && dy_ld % 8 == 0;
    p.x_vec = (bits(x) & 15u) == 0 && x_ld % 8 == 0;
    p.dx_vec = (bits(dx) & 15u) == 0 && dx_ld % 8 == 0;
    p.scale = scale;
    for (int s = 0; s < num_slices; ++s) {
        const int lead = p.dy_vec ? p.off[s] & 7 : 0;
        if (p.db[s] != nullptr || p.dbias[s] != nullptr) blocks += (lead + p.n[s] + BW_COLS - 1) / BW_COLS;
        p.block_end[s] = blocks;
    }
    for (int s = 0; s < num_slices; ++s) {
        if (p.da[s] != nullptr) blocks += (hidden + BW_COLS - 1) / BW_COLS;
        p.block_end[num_slices + s] = blocks;
    }
    const int rp = padded_rank(rank);
    p.rows = backward_rows(num_tokens, p.L);
    const int64_t one = (p.rows * num_slices * rp * 2 + 255) / 256 * 256;
    const int64_t part = one * backward_terms(num_tokens);
    p.low = part > one ? one / 2 : 0;
    p.g = reinterpret_cast<uint16_t *>(workspace);
    p.u = reinterpret_cast<uint16_t *>(static_cast<char *>(workspace) + part);
    p.ut = p.u;
    p.gt = reinterpret_cast<uint16_t *>(static_cast<char *>(workspace) + 2 * part);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + backward_parts(num_tokens, rank) * one);
    p.u_ctas = 0;
    int steps = 0;
    for (int s = 0; s < LORA_MAX_SLICES; ++s) {
        if (s < num_slices) steps += ((p.dy_vec ? p.off[s] & 7 : 0) + p.n[s] + 63) / 64;
        p.step_end[s] = steps;
    }
    p.sorted = meta->token_indices_sorted_by_lora_ids;
    p.counts = meta->num_tokens_per_lora;
    p.start_loc = meta->lora_token_start_loc;
    p.active = meta->active_lora_ids;
    p.no_lora = meta->no_lora_flag;
    p.error_word = meta->error_word;
    p.nbins = meta->max_loras + 1;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (rp) {
    case 16: return run_backward<16>(p, st);
    case 32: return run_backward<32>(p, st);
    case 64: return run_backward<64>(p, st);
    default: return run_backward<128>(p, st);
    }
}
