/*
 * exl3_moe.h - C ABI of the mixture-of-experts routing operators for MI355X
 * (gfx950): slots sorted by expert, the tokens' rows brought into that order,
 * and the experts' rows brought back with the router's weights, with the
 * gradients of both.  Between them runs a product per expert: the grouped
 * exl3_mxfp4_linear, or exl3_linear on each expert's rows.
 *
 * A slot is a pair (token t, choice j), flat index t * top_k + j; it asks for
 * expert ids[t][j].  An id outside 0 .. n_experts - 1 marks a dropped slot
 * (padding tokens, overflowing experts).  The sorted order holds the slots of
 * expert 0, of expert 1, ..., and the dropped ones last, each group in the order
 * of the flat index:
 *   order    : int32 [slots], the slot at each place
 *   position : int32 [slots], the place of each slot (order's inverse)
 *   offsets  : int32 [n_experts + 1], first place of each expert;
 *              offsets[n_experts] is the number of slots that are not dropped
 * "rows" below are [slots][n], one per place; those of dropped slots are zero
 * where a call writes them and are not read otherwise.
 *
 * Conventions: as in exl3.h and exl3_mxfp4.h (dtype is exl3_dtype).  position
 * entries outside 0 .. slots - 1 are treated as dropped.  A row that no entry names
 * is left as it was, and one that two entries name holds values of either (as
 * exl3_moe_sort writes position, each row has one entry).  EXL3_EINVAL for null or
 * misaligned pointers (kept: 4 bytes), bad types and sizes below 1 (no tokens or
 * slots are a no-op); EXL3_EUNSUPPORTED for 2^24 tokens, 2^26 - 4 slots (sort: more
 * than 2^30) or n > 2^24.  Results and the workspace share no byte with the
 * arguments or each other (EXL3_EINVAL where they do).  Sums are fp32, in the order
 * of j, rounded once; where position is a permutation results do not depend on
 * timing.
 */
#ifndef EXL3_MOE_H
#define EXL3_MOE_H

#include "exl3_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most experts exl3_moe_sort takes. */
#define EXL3_MOE_MAX_EXPERTS 1024

/*
 * exl3_moe_workspace_bytes: device scratch of exl3_moe_sort (0 for few slots).
 * EXL3_EINVAL for n_slots < 0, n_experts outside 1 .. EXL3_MOE_MAX_EXPERTS.
 * Host-only.
 */
int64_t exl3_moe_workspace_bytes(int32_t n_slots, int32_t n_experts);

/*
 * exl3_moe_sort: the stable sort above.
 *   ids      : int32 or int64 (id_bytes 4 or 8) [n_slots]
 *   order, position, offsets : as above, overwritten
 *   workspace : device scratch of exl3_moe_workspace_bytes, not initialised
 * n_slots == 0 writes offsets only.
 */
int exl3_moe_sort(const void* ids, int32_t id_bytes, int32_t n_slots, int32_t n_experts, int32_t* order,
                  int32_t* position, int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream);

/*
 * exl3_moe_gather: rows[position[t][j]] = x[t], zero for a dropped slot.
 *   x        : dtype [n_tokens][n]
 *   position : int32 [n_tokens][top_k]
 *   kept     : device pointer to offsets[n_experts]
 *   rows     : dtype [n_tokens * top_k][n]; every row that position names is written
 * Its gradient, dx[t] = sum over j of drows[position[t][j]], is
 * exl3_moe_combine without weights.
 */
int exl3_moe_gather(const void* x, int32_t dtype, int32_t n_tokens, int32_t top_k, int32_t n, const int32_t* position,
                    const int32_t* kept, void* rows, void* stream);

/*
 * exl3_moe_combine: y[t] = sum over j of weights[t][j] * rows[position[t][j]],
 * dropped slots left out (whatever their weight).
 *   weights : weights_dtype [n_tokens][top_k], or NULL (all ones)
 *   y       : dtype [n_tokens][n], overwritten
 */
int exl3_moe_combine(const void* rows, int32_t dtype, int32_t n_tokens, int32_t top_k, int32_t n,
                     const int32_t* position, const int32_t* kept, const void* weights, int32_t weights_dtype, void* y,
                     void* stream);

/*
 * exl3_moe_combine_backward: the gradients of exl3_moe_combine,
 *   drows[position[t][j]] = weights[t][j] * dy[t]        (zero for a dropped slot)
 *   dweights[t][j]        = sum over c of rows[position[t][j]][c] * dy[t][c]   (likewise)
 *   drows    : dtype [n_tokens * top_k][n]; every row that position names is written
 *   dweights : weights_dtype [n_tokens][top_k], overwritten
 */
int exl3_moe_combine_backward(const void* dy, const void* rows, int32_t dtype, int32_t n_tokens, int32_t top_k,
                              int32_t n, const int32_t* position, const int32_t* kept, const void* weights,
                              int32_t weights_dtype, void* drows, void* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EXL3_MOE_H */
