// lora_loss.cuh -- what the kernels of lora_cross_entropy share.
#pragma once

#include <math.h>

#include "lora_common.cuh"

namespace lora {

constexpr float LOSS_LOG2E = 1.4426950408889634f;
constexpr float LOSS_LN2 = 0.6931471805599453f;
constexpr float LOSS_MAX_REF = 3.4028235e38f;     // references stay finite where exponents do not

// What a finished row gives: its loss, the base-2 log of its sum, the factor
// of its accumulated terms (of 2^-ref each) and of the target's row of W
// (1 - p_y).
struct LossRow {
    float loss, lse2, inv, share;
};

// total: the terms of the columns other than the target's, in units of
// 2^ref; logit: the target's exponent.  1 - p_y is total over everything, so
// a sure target costs no digits: where the others weigh less than it, the
// loss is log1p of their ratio, wherever the reference lies.
__device__ __forceinline__ LossRow loss_row(float total, float ref, float logit)
{
    LossRow r;
    const float d = logit - ref;
    if (total == 0.0f) {                          // the target is the only column left
        r.lse2 = logit;
        r.loss = r.inv = r.share = logit - logit; // 0, or NaN where the logit is
    } else if (total <= exp2f(d)) {
        // the others relative to the target; NaN for an infinite one
        const float back = total * exp2f(-d) + (d - d);
        r.loss = log1pf(back);
        r.lse2 = logit + r.loss * LOSS_LOG2E;
        r.share = back / (1.0f + back);
        r.inv = exp2f(-d) / (1.0f + back);
    } else {
        const float all = total + exp2f(d);
        const float lg = log2f(all);
        r.loss = (lg - d) * LOSS_LN2;
        r.lse2 = ref + lg;
        r.share = total / all;
        r.inv = 1.0f / all;
    }
    return r;
}

// One or two tokens (lora_loss_row.cu).
constexpr int LOSS_ROW_TOKENS = 2;
struct LossRowArgs {
    const uint16_t *hidden, *weight;
    int64_t hidden_ld, dh_ld;
    const int32_t *targets;
    const float *token_weight;
    float *loss, *logsumexp;
    uint16_t *dh;
    int32_t T, H, V, nt, slots;
    int32_t *error_word;
    float *logit;          // [T]
    float2 *stat;          // [slots][T]: reference, sum
    float *acc;            // [slots][T][H]; null without a gradient
};
bool loss_row_fits(int32_t T, int32_t H);
int loss_row_slots();
int run_loss_row(LossRowArgs p, cudaStream_t st);

}  // namespace lora
