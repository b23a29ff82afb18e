/*
 * moe_balance.h - load-balance loss of the router in libnvfp4moe.so.
 *
 * From the router's logits and choices (moe_route), per sequence s:
 *   counts[s][e]  choices of expert e by the sequence's tokens
 *   n_s           its tokens
 *   p_t           score "softmax": softmax of token t's logits; score
 *                 "sigmoid": sigma of the logits divided by their sum
 *   probs[s][e]   mean of p_t[e] over the sequence's tokens
 *   f[s][e]       counts[s][e] E / (k n_s)
 *   loss        = coeff / S' * sum_s sum_e f[s][e] probs[s][e]
 * with S' the number of sequences that have tokens (loss 0 if there is none).
 * The counts carry no gradient:
 *   dloss/dlogit[t][e] = coeff / (S' n_s) p_t[e] (f[s][e] - sum_j f[s][j] p_t[j]) * d
 * with d = 1 for softmax and sigma(-logit) for sigmoid.
 *
 *   - token_mask (uint8 [T], nullable): tokens with 0 are left out: their
 *     logits and choices are read, and dropped whatever they hold (NaN and
 *     infinities too); their gradient is 0.
 *   - seq_offsets (int32 [S+1], nullable, non-decreasing): sequence s is the
 *     tokens [seq_offsets[s], seq_offsets[s+1]).  Tokens in no sequence are
 *     left out.  NULL: one sequence of all T tokens (S = 1).
 *   - choices outside [0, E) (a dropped slot) are not counted.
 *   - the counts are those of the tokens that are not left out.  As the
 *     expert_counts of a product on moe_route's rows, which hold every token,
 *     they serve only without a mask and summed over sequences that together
 *     hold every token.
 *   - an expert masked with a logit of -inf gets p = 0 and gradient 0; a token
 *     whose logits are all -inf has p = 0 throughout.
 * Sums are fp32 in a fixed order (fp64 where the partial sums join): the
 * results are the same from run to run.
 * Conventions are those of nvfp4_moe.h.
 */
#ifndef NVFP4_MOE_BALANCE_H
#define NVFP4_MOE_BALANCE_H

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_BALANCE_SIGMOID = 0, MOE_BALANCE_SOFTMAX = 1 };

/* logits[T][E] of `dtype` (MXFP4_DTYPE_*), rows row_stride elements apart;
 * topk_idx int32 [T][k].  Outputs: loss fp32 [1]; counts int32 [S][E]; tokens
 * int32 [S+1], n_s and behind them S'; probs fp32 [S][E].  Needs
 * 1 <= E <= 1024, 1 <= k <= 32, 1 <= S, T >= 0. */
NVFP4_API size_t moe_balance_loss_workspace_size(int T, int E, int S);
NVFP4_API nvfp4_status moe_balance_loss(const void* logits, int dtype, int T, int E, long long row_stride,
                                        const int32_t* topk_idx, int k, int score, const uint8_t* token_mask,
                                        const int32_t* seq_offsets, int S, float coeff, float* loss, int32_t* counts,
                                        int32_t* tokens, float* probs, void* ws, size_t ws_bytes, void* stream);

/* dlogits[T][E] (the logits' dtype, rows grad_stride elements apart) =
 * grad_loss[0] * dloss/dlogits from the counts and tokens of the forward call
 * with the same arguments.  Every element is written.  dlogits may not share
 * elements with logits: where their memory meets, they are different columns
 * of one buffer, with one stride. */
NVFP4_API nvfp4_status moe_balance_loss_backward(const void* logits, int dtype, int T, int E, long long row_stride,
                                                 int k, int score, const uint8_t* token_mask,
                                                 const int32_t* seq_offsets, int S, float coeff,
                                                 const int32_t* counts, const int32_t* tokens,
                                                 const float* grad_loss, void* dlogits, long long grad_stride,
                                                 void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_MOE_BALANCE_H */
