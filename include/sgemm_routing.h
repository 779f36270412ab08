/*
 * sgemm_routing.h -- routing of tokens to experts, and their rows' way there
 * and back (GB300, sm_103a).  Companion of sgemm_experts.h, whose grouped
 * products take the boundaries and the rows that these make: same status
 * codes, types, streams, error behaviour and scratch pool.
 *
 * A token's k choices are a row of `experts` (T x k ints, the best first).  A
 * choice without an expert holds -1.  `slots` (T x k ints) is the row that each
 * choice has among all choices sorted by expert, and -1 where there is none;
 * `offsets` (E + 1 ints) are the boundaries of the experts' rows, offsets[E]
 * the number of choices that have an expert.  Among an expert's rows the
 * tokens keep their order, so results do not depend on timing.
 *
 * Memory.  All pointers are DEVICE pointers owned by the caller, aligned to
 * their element type; leading dimensions are in elements; integer arrays and
 * weights are contiguous.  Outputs must not overlap inputs or one another.
 * Row padding is neither read nor written.  The kernels check every slot and
 * expert that they read: one outside its range is taken as -1.
 * Entry points that may allocate device memory from the library's
 * stream-ordered pool (see sgemm.h), and those that never do:
 *   ROUTING-ALLOCATING: sgemm_route
 *   ROUTING-NON-ALLOCATING: sgemm_route_grad sgemm_spread sgemm_combine sgemm_combine_grad
 */
#ifndef GB300_SGEMM_ROUTING_H
#define GB300_SGEMM_ROUTING_H

#include <stdint.h>

#include "sgemm_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a score is made of a token's logits. */
enum { SGEMM_SCORE_SOFTMAX = 0, SGEMM_SCORE_SIGMOID = 1 };

/* The most experts, choices of a token, and groups of experts. */
enum { SGEMM_ROUTE_MAX_EXPERTS = 1024, SGEMM_ROUTE_MAX_CHOICES = 32, SGEMM_ROUTE_MAX_GROUPS = 32 };

/*
 * sgemm_route -- every token's experts, their weights, and the rows' places
 *
 *     s_e = softmax(logits)_e or sigmoid(logits_e)      scores
 *     c_e = s_e + bias_e                                what experts are chosen by
 *     experts = the k experts with the largest c, largest first
 *     weights = scale * s_e, renormalised: scale * s_e / sum of the chosen s
 *
 *   type, logits, ld   T x E, in HBM as `type`
 *   bias       E floats, or NULL: none.  It has no part in the weights
 *   groups, top_groups, group_best   the experts are `groups` groups of
 *              E / groups neighbours, and only the `top_groups` best are chosen
 *              from.  A group is as good as the sum of its group_best (1 or 2)
 *              largest c, of those there are.  groups = 1: no groups
 *   experts, weights, slots   T x k;  offsets   E + 1
 * An expert whose logit or whose c is -inf is out of service: it is not chosen,
 * and a token that has fewer than k experts left gets -1 with weight 0 in its
 * last places.  So a padding token is a row of -inf.
 * Ties go to the lowest expert and the lowest group.  The choice is that of
 * exact arithmetic: values that lie too near one another for float32 are compared
 * in 64 bits, or by their logits if they all have one bias (64 bits hold many sigmoids equal).  NaN counts as the largest value; it makes its
 * token's weights NaN, as +inf does with a softmax (but only its own weight
 * with sigmoid scores that are not renormalised).
 * Weights are within 2^-18 of the exact ones, relative to the token's
 * largest, and float32's smallest number; renormalised ones do not depend on how small the scores are.
 * Limits: 1 <= k <= 32, k <= E <= 1024, groups <= 32 and a divisor of E, top_groups <= groups.
 */
int sgemm_route(int type, int score, int T, int E, int k,
                const void* logits, int64_t ld,
                const float* bias,
                int groups, int top_groups, int group_best,
                int renormalize, float scale,
                int* experts, float* weights, int* offsets, int* slots,
                void* stream);

/*
 * sgemm_route_grad -- the gradient of the logits (T x E of `type`) from that of
 * the weights (T x k floats), for the experts that sgemm_route chose with the
 * same score, renormalize and scale.  Choices of no expert have no part in it;
 * a token without experts, and experts whose logit is -inf, get zeros.  A token's
 * experts must differ.
 */
int sgemm_route_grad(int type, int score, int T, int E, int k,
                     const void* logits, int64_t ld,
                     const int* experts, const float* dweights,
                     int renormalize, float scale,
                     void* dlogits, int64_t ldd,
                     void* stream);

/*
 * sgemm_spread -- Y[slots[t, j], :] = X[t, :] for slots below offsets[E], and zeros
 * to Y's rows from offsets[E] (taken within [0, R]) on.
 *   X          T x H;   Y   R x H
 *   slots      T x k, different from one another where they are rows of Y
 *   E, offsets as sgemm_route gives them
 * Rows below offsets[E] that no slot names are left as they were.
 * Its gradient is sgemm_combine without weights (of slots below offsets[E]).
 */
int sgemm_spread(int type, int T, int k, int R, int H,
                 const void* X, int64_t ldx,
                 const int* slots, int E, const int* offsets,
                 void* Y, int64_t ldy,
                 void* stream);

/*
 * sgemm_combine -- out[t, :] = sum over j of weights[t, j] * Y[slots[t, j], :]
 * (T x H), summed in float32 in the order of j and rounded once; choices of no
 * row have no part in it, whatever their weight.  weights NULL: ones.
 */
int sgemm_combine(int type, int T, int k, int R, int H,
                  const void* Y, int64_t ldy,
                  const int* slots, const float* weights,
                  void* out, int64_t ldo,
                  void* stream);

/*
 * sgemm_combine_grad -- the gradients of a combination:
 *     dY[slots[t, j], :] = weights[t, j] * dout[t, :] for slots below offsets[E],
 *                          zeros to dY's rows from there on (other rows as
 *                          sgemm_spread), and
 *     dweights[t, j] = sum over h of dout[t, h] * Y[slots[t, j], h], 0 where
 *                      there is no row.
 * dY NULL or dweights NULL: that gradient is not wanted (Y is read for
 * dweights, offsets for dY; either may then be NULL).  weights NULL: ones.
 */
int sgemm_combine_grad(int type, int T, int k, int R, int H,
                       const void* dout, int64_t ldd,
                       const void* Y, int64_t ldy,
                       const int* slots, const float* weights, int E, const int* offsets,
                       void* dY, int64_t lddy, float* dweights,
                       void* stream);

#ifdef __cplusplus
}
#endif
#endif
