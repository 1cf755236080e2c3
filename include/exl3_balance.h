/*
 * exl3_balance.h - C ABI of the loss that evens out a router's experts, with their
 * counts, and its gradient (gfx950).  It stands beside the routing of exl3_moe.h,
 * which brings the tokens to the experts that the same ids name.
 *
 * For logits [tokens][experts], p = softmax of a row of them, and ids [tokens][top_k]
 * whose entries outside 0 .. n_experts - 1 are dropped slots (exl3_moe.h):
 *   - a token counts if at least one of its slots is kept (padding has none); V is
 *     their number, c[e] the number of kept slots of expert e;
 *   - loss = coefficient * n_experts * sum_e (c[e] / (V top_k)) * (1 / V) sum_t p[t][e]
 *     over the tokens that count: `coefficient` for an even router, more otherwise;
 *     0 where no token counts;
 *   - gradient (c is a constant of it):
 *       dlogits[t][e] = dloss * coefficient * (n_experts / V) * p[t][e] * (s[e] - sum_j s[j] p[t][j]),
 *       s[e] = c[e] / (V top_k); zeros for a token that does not count.
 * Logits of a token that does not count are not used, whatever they hold.  A logit of
 * -infinity has probability 0, a token with nothing else only zeros; a NaN or +infinity
 * makes its token's probabilities NaN, as a softmax does.  A probability below 2^-126 of
 * its token's largest (a logit 87.4 and more below) counts as 0.
 *
 * Conventions: as in exl3.h and exl3_moe.h.  Sums over tokens are fp32 in an order that
 * depends on the sizes alone, those over experts 64 bits or fp32: results do not depend
 * on timing.  EXL3_EINVAL for null or misaligned pointers (loss, dloss: 4 bytes), bad
 * types, sizes below 1 (no tokens: a loss of 0, counts of 0, no gradient), more than
 * EXL3_MOE_MAX_EXPERTS experts, a coefficient that is not finite; EXL3_EUNSUPPORTED for
 * 2^24 tokens or 2^31 slots.  Results and the workspace share no byte with the
 * arguments or each other (EXL3_EINVAL where they do).  The lanes that hold a token's
 * logits (16 bytes each, 64 lanes at most) read its slots one after the other: meant for
 * a few slots a lane, as many more take time in proportion.
 */
#ifndef EXL3_BALANCE_H
#define EXL3_BALANCE_H

#include "exl3_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * exl3_moe_balance_workspace_bytes: device scratch of exl3_moe_balance_loss (0 for few
 * tokens).  EXL3_EINVAL for n_tokens < 0, n_experts outside 1 .. EXL3_MOE_MAX_EXPERTS.
 * Host-only.
 */
int64_t exl3_moe_balance_workspace_bytes(int32_t n_tokens, int32_t n_experts);

/*
 * exl3_moe_balance_loss: the loss and the counts above.
 *   logits : dtype [n_tokens][n_experts]
 *   ids    : int32 or int64 (id_bytes 4 or 8) [n_tokens][top_k]
 *   loss   : fp32, one value
 *   counts : int32 [n_experts + 1]: c, then V
 *   workspace : device scratch of exl3_moe_balance_workspace_bytes, not initialised
 */
int exl3_moe_balance_loss(const void* logits, int32_t dtype, const void* ids, int32_t id_bytes, int32_t n_tokens,
                          int32_t top_k, int32_t n_experts, double coefficient, float* loss, int32_t* counts,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * exl3_moe_balance_loss_backward: its gradient to the logits.
 *   dloss   : fp32, device, one value: the gradient that reaches the loss
 *   counts  : as exl3_moe_balance_loss wrote them for these ids
 *   dlogits : dtype [n_tokens][n_experts], overwritten
 */
int exl3_moe_balance_loss_backward(const float* dloss, const void* logits, int32_t dtype, const void* ids,
                                   int32_t id_bytes, int32_t n_tokens, int32_t top_k, int32_t n_experts,
                                   const int32_t* counts, double coefficient, void* dlogits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EXL3_BALANCE_H */
