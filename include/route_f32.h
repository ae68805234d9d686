/*
 * route_f32.h -- C ABI of libgemm_f32.so, part 4: what stands around products
 * grouped by expert (segment_gemm_f32.h) in a mixture of experts: the router,
 * and the way of the rows (tokens) to the experts and back.
 *
 * The plan. A router gives each of T tokens k slots, each an expert or none (-1).
 * The experts' rows are the slots with an expert, sorted by expert, slots of
 * one expert in ascending order:
 *   offsets  E + 1 int64: expert e has rows offsets[e] .. offsets[e + 1] - 1 (as
 *            gemm_f32_grouped takes them); offsets[0] = 0
 *   order    T k int32: row r is that of slot order[r] = t k + j; -1 from
 *            offsets[E] on
 *   places   T x k int32: the row of slot (t, j), or -1
 * All of it stays in device memory; nothing is read by the host.
 *
 * Matrices are row-major device memory with a pitch in elements, of `type` (a
 * gemm_f32_type); the other arrays are dense. Streams, ownership, errors and
 * thread safety are those of gemm_f32.h; no result depends on timing (but that of
 * places that name a row twice), and none may overlap an operand or another result
 * (GEMM_ERR_ALIAS). Sizes are at most GEMM_F32_MAX_SEGMENT_SIZE, and T k too.
 */
#ifndef ROUTE_F32_H
#define ROUTE_F32_H

#include <stdint.h>

#include "segment_gemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GEMM_F32_SCORE_SOFTMAX = 0,  /* s_e = exp(x_e) / sum of exp(x) over all experts */
    GEMM_F32_SCORE_SIGMOID = 1   /* s_e = 1 / (1 + exp(-x_e)) */
} gemm_f32_score;

#define GEMM_F32_MAX_ROUTE_SLOTS 32  /* k at most */

/*
 * gemm_f32_route -- the k best experts of every token, their weights, and the
 * plan.
 *
 *   logits   x, T x E, of `type`; E from 1 to GEMM_F32_MAX_SEGMENTS
 *   bias     E floats added to the scores where experts are compared, but not
 *            in the weights; NULL: none
 *   mask     T bytes, 0: the token takes no part (a padded batch); NULL: all do
 *   groups, top_groups, group_best
 *            groups > 1: the experts are that many groups of E / groups
 *            neighbours (at most 32); the top_groups groups with the largest sum
 *            of their group_best (1 or 2) best s + bias (or all they have) are
 *            chosen, and experts of theirs alone. groups = 1: all of them.
 *   k        slots of a token, 1 .. min(E, GEMM_F32_MAX_ROUTE_SLOTS)
 *   renormalise  0: weight = scale s_e; 1: scale s_e / (sum of the token's s_e)
 *   experts  T x k int32: the experts with the largest s + bias, largest first,
 *            and, where equal, the lowest index first
 *   weights  T x k float
 *   offsets, order, places  the plan; all three NULL: none
 *
 * Comparisons are those of the real numbers: s + bias is computed in fp32, and
 * again in 64 bits for a token where two of them that matter are closer than the
 * rounding of fp32. Without a bias (and groups of which one best counts) the
 * logits are compared.
 *   x_e or bias_e of -infinity: e is not available. Slots left over have expert
 * -1 and weight 0. The lowest finite value is a number like others.
 *   A NaN (or what becomes one: softmax of +infinity) stays in its token: its
 * experts rank below all others that are available, in ascending order, and
 * weights that have a NaN among their terms are NaN.
 * Weights are to fp32: within (E / 32 + 40) 2^-24 of their value, where their
 * terms' |x - max x| is small; exp's argument is rounded to fp32.
 */
int gemm_f32_route(int type, int score, int64_t T, int64_t E, int64_t k,
                   const void *logits, int64_t ldx,
                   const float *bias, const uint8_t *mask,
                   int64_t groups, int64_t top_groups, int64_t group_best,
                   int renormalise, float scale,
                   int32_t *experts, float *weights,
                   int64_t *offsets, int32_t *order, int32_t *places, void *stream);

/*
 * gemm_f32_route_backward -- the gradient of the logits from that of the weights
 * (the choice of experts is held fixed):
 *
 *   softmax, renormalised   dx_e = w_e (g_e - sum g w / scale)
 *   softmax                 dx_e = w_e g_e - s_e sum g w       (all experts)
 *   sigmoid, renormalised   dx_e = w_e (g_e - sum g w / scale) (1 - s_e)
 *   sigmoid                 dx_e = w_e g_e (1 - s_e)
 *
 *   dweights  g, T x k float
 *   experts, weights  the forward's; slots without an expert (any index outside
 *             [0, E)) take no part; an expert that stands in two slots of a token
 *             gets the sum of both
 *   dlogits   T x E, of `type`, all of it written: zero where it is not above
 * scale must not be 0 where renormalised.
 */
int gemm_f32_route_backward(int type, int score, int64_t T, int64_t E, int64_t k,
                            const float *dweights, const void *logits, int64_t ldx,
                            const int32_t *experts, const float *weights,
                            int renormalise, float scale,
                            void *dlogits, int64_t lddx, void *stream);

/*
 * gemm_f32_route_plan -- the plan of experts that were chosen otherwise: `slots`
 * indices (any value outside [0, E): none).
 */
int gemm_f32_route_plan(int64_t slots, int64_t E, const int32_t *experts,
                        int64_t *offsets, int32_t *order, int32_t *places, void *stream);

/*
 * gemm_f32_dispatch -- each token's row to all of its places: Y[places[t][j]] =
 * X[t]. X is T x D, Y `rows` x D. Rows that no place names are not written; a
 * place outside [0, rows) is none. Each element of a row that is named twice gets
 * the value of one of the two, not always of the same one (a plan names none twice).
 */
int gemm_f32_dispatch(int type, int64_t T, int64_t D, int64_t k, int64_t rows,
                      const void *X, int64_t ldx, const int32_t *places,
                      void *Y, int64_t ldy, void *stream);

/*
 * gemm_f32_combine -- the weighted sum of a token's rows:
 *
 *     O[t] = sum_j w[t][j] Y[places[t][j]],
 *
 * in ascending j, in fp32, rounded once; zero where a token has no place. weights
 * NULL: 1, which is the gradient of gemm_f32_dispatch. Weights of slots without a
 * place are not read into the sum.
 */
int gemm_f32_combine(int type, int64_t T, int64_t D, int64_t k, int64_t rows,
                     const void *Y, int64_t ldy, const int32_t *places, const float *weights,
                     void *O, int64_t ldo, void *stream);

/*
 * gemm_f32_combine_backward -- gradients of gemm_f32_combine:
 *
 *     dY[places[t][j]] = w[t][j] dO[t],   dw[t][j] = sum_d dO[t][d] Y[places[t][j]][d]
 *
 *   dY        rows that no place names are not written; a row named twice as for
 *             gemm_f32_dispatch
 *   dweights  T x k float, 0 for slots without a place
 * One of dY and dweights may be NULL (with weights NULL: 1 there too).
 */
int gemm_f32_combine_backward(int type, int64_t T, int64_t D, int64_t k, int64_t rows,
                              const void *dO, int64_t lddo, const void *Y, int64_t ldy,
                              const int32_t *places, const float *weights,
                              void *dY, int64_t lddy, float *dweights, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ROUTE_F32_H */
