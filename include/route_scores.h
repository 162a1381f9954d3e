/*
 * route_scores.h -- C ABI of the expert selection from given router logits
 * (libmoe_gb300.so; status codes, element types and stream type from
 * moe_gb300.h).
 *
 * moe_route computes softmax routing from x and W_r in one fused kernel.
 * This entry takes the logits of any router and covers the other routing
 * rules of expert layers: sigmoid scores, a balance bias that moves the
 * choice but not the weights, and a first choice among groups of experts.
 * Its ids and weights go to moe_permute and moe_expert_ffn as moe_route's do.
 *
 * For every token, with L its E logits:
 *   s_e    = 1 / (1 + exp(-L_e))            (MOE_SCORE_SIGMOID)
 *          = exp(L_e - max L) / sum_i exp(L_i - max L)   (MOE_SCORE_SOFTMAX)
 *   c_e    = s_e + bias_e, the value that experts are chosen by
 *   group g holds the E / n_groups consecutive experts from g E / n_groups;
 *   its value is the sum of its group_rank largest c_e (1: its maximum)
 *   chosen: the top_groups groups of largest value, then the top_k experts of
 *   largest c_e inside them; equal values -> lower index first, both times
 *   ids[j] = the chosen experts in descending order of c_e
 *   w[j]   = scale * s_{ids_j} / sum_i s_{ids_i}    (renormalise != 0)
 *          = scale * s_{ids_j}                      (renormalise == 0)
 * Without a bias c_e is taken as L_e itself where only its order counts (the
 * order of the scores without their rounding, which ties values that differ),
 * and a sum of two uses s_e (softmax: exp(L_e - max L), the common factor
 * left out).
 *
 * A logit of -infinity masks its expert: score 0, chosen only when nothing
 * else is left in the chosen groups, lowest index first, with weight 0.  A
 * bias of -infinity leaves the score but takes the expert out of the choice
 * in the same way: if it has to fill a slot its weight is 0.  A token whose
 * chosen experts all have score 0 gets weights 0.  A NaN or +infinity logit
 * (or a bias that is NaN or +infinity) is treated as such a mask and records
 * MOE_ERR_DEVICE_NONFINITE; other tokens are unaffected.
 */
#ifndef ROUTE_SCORES_H
#define ROUTE_SCORES_H

#include "moe_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };

typedef struct {
  int32_t T;             /* tokens, >= 0 (0 is a no-op)                         */
  int32_t n_experts;     /* E: 1..256                                           */
  int32_t top_k;         /* k: 1..min(16, top_groups * E / n_groups)            */
  int32_t n_groups;      /* 1..32, divides E; 1 = no groups                     */
  int32_t top_groups;    /* 1..n_groups                                         */
  int32_t group_rank;    /* 1 or 2: experts whose values rank a group           */
  int32_t score;         /* MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID              */
  int32_t logit_dtype;   /* MOE_F32 or MOE_BF16                                 */
  int32_t renormalise;   /* 0 or 1                                              */
  float scale;           /* finite, > 0                                         */
  int64_t logit_stride;  /* elements from one token's logits to the next's, >= E */
} moe_route_scores_config_t;

/*
 * logits    [T] rows of E elements, logit_stride apart (device, aligned to
 *           its element)
 * bias      [E] float, or NULL
 * topk_ids  [T][k] int32 out
 * topk_w    [T][k] float out
 * Asynchronous on `stream`, no workspace, nothing allocated.  Scores, sums
 * and weights are fp32.
 */
moe_status_t moe_route_scores(const moe_route_scores_config_t* cfg, const void* logits, const float* bias,
                              int32_t* topk_ids, float* topk_w, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ROUTE_SCORES_H */
