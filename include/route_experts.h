/*
 * libroute -- the routed experts' operators, and dropout, C ABI.
 *
 * What a layer runs between the route step's ids and weights (route.h) and the
 * residual stream, forward and backward:
 *
 *   dispatch   the (row, expert) pairs sorted by expert, token rows copied to
 *              their sorted places, and the experts' results brought back as
 *              weighted sums
 *   experts    the gated feed-forward block of every expert on its own run of
 *              the sorted rows
 *   dropout    out = x keep / (1 - p) + residual, from a counter-based generator
 *
 * A plan is a route_layer (route_layer.h): route_layer_destroy, _status,
 * _saved_bytes and _test_stall take these plans too, and route_layer.h's
 * conventions on matrices, types, statuses and streams hold, but:
 *  - dispatch and dropout plans hold no scratch: their calls may run on several
 *    streams at the same time.
 *  - Index arrays are int32 on the device.  The library cannot look at them
 *    before it launches; no value in them makes a kernel read or write outside
 *    the tensors that it was given.
 */
#ifndef ROUTE_EXPERTS_H
#define ROUTE_EXPERTS_H

#include "route_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ROUTE_MAX_EXPERTS 1024
#define ROUTE_MAX_TOPK 32
#define ROUTE_EXPERTS_MAX_ROWS 1048576

/* route_dispatch_prepare: up to `rows` (65536) token rows of `dim` values of
 * `type` (BF16, FP16, FP32), each with `topk` (1..32) expert ids.  The plan's
 * experts are first .. first + experts - 1 (experts 1..1024): pairs with other
 * ids (those of other shards, -1 for padding) belong to nobody here. */
route_status route_dispatch_prepare(int rows, int dim, int type, int experts, int first, int topk,
                                    int device, route_layer **out);

/*
 * route_dispatch_sort: the pairs (r, j) with ids[r, j] among the plan's
 * experts, sorted by expert, pairs of one expert by r and then j.
 *   offsets [experts + 1]  where each expert's run begins; the last: how many
 *                          pairs there are
 *   place [rows][topk]     the place of each pair, -1 if it is none of the plan's
 *   source [rows * topk]   r * topk + j of the pair at each place; what lies
 *                          behind the last pair is left as it was.  May be NULL
 * ids [rows, topk] has row stride ld_ids.  An id may be in a row more than once.
 * With no rows every offset is 0.
 */
route_status route_dispatch_sort(const route_layer *plan, int rows, const int32_t *ids,
                                 int64_t ld_ids, int32_t *offsets, int32_t *place, int32_t *source,
                                 void *stream);

/* route_dispatch_gather: out[place[r, j]] = x[r].  out has `pairs` rows (0 ..
 * the plan's rows * topk, else ROUTE_ERR_ROWS; so in the calls below); a place
 * outside 0 .. pairs - 1 is none, and rows that no place names are left as they
 * were.  Of two pairs with the same place either may win, value by value. */
route_status route_dispatch_gather(const route_layer *plan, int rows, const void *x, int64_t ld_x,
                                   const int32_t *place, int pairs, void *out, int64_t ld_out,
                                   void *stream);

/* route_dispatch_gather_backward: dx[r] = sum over j of dout[place[r, j]], in
 * FP32 and in the order of j. */
route_status route_dispatch_gather_backward(const route_layer *plan, int rows, const void *dout,
                                            int64_t ld_dout, int pairs, const int32_t *place,
                                            void *dx, int64_t ld_dx, void *stream);

/* route_dispatch_combine: out[r] = sum over j of weights[r, j] y[place[r, j]] +
 * residual[r], in FP32 and in the order of j.  weights [rows][topk] FP32 may be
 * NULL (1), residual too (0).  A pair without a place adds nothing, whatever
 * its weight.  out may be the residual. */
route_status route_dispatch_combine(const route_layer *plan, int rows, const void *y, int64_t ld_y,
                                    int pairs, const int32_t *place, const float *weights,
                                    const void *residual, int64_t ld_residual, void *out,
                                    int64_t ld_out, void *stream);

/*
 * route_dispatch_combine_backward:
 *   dy[place[r, j]] = weights[r, j] dout[r],  dweights[r, j] = <dout[r], y[place[r, j]]>
 * dweights [rows][topk] FP32 is 0 where a pair has no place; rows of dy that no
 * place names are left as they were, and of two pairs with the same place either
 * may win, value by value (combine's gradient would be their sum).  Either of dy
 * and dweights may be NULL; y may be NULL without dweights, weights are 1 where
 * NULL.
 */
route_status route_dispatch_combine_backward(const route_layer *plan, int rows, const void *dout,
                                             int64_t ld_dout, const void *y, int64_t ld_y, int pairs,
                                             const int32_t *place, const float *weights, void *dy,
                                             int64_t ld_dy, float *dweights, void *stream);

/*
 * route_experts_prepare: experts (1..1024) gated blocks
 *   h = act(x W_gate[e]) * (x W_up[e]),  out = h W_down[e]
 * with W_gate, W_up [experts][k, f] and W_down [experts][f, n], BF16 or FP16,
 * on up to `rows` (1048576) sorted rows; k, f and n are multiples of 8
 * (ROUTE_ERR_PLAN).  train != 0 prepares for route_experts_backward too.
 *
 * Expert e's rows are offsets[e] .. offsets[e + 1] - 1 (route_dispatch_sort's);
 * offsets outside 0 .. rows are cut to it.  Rows that are nobody's are not
 * written, and what they hold changes no result.  Offsets must not descend:
 * where they do, so that runs overlap, what the call's results hold is
 * unspecified (a row may be any of its experts' or be left as it was).
 *
 * All matrices start on 16 bytes with row strides that are multiples of 8
 * (ROUTE_ERR_ALIGN); es_* are the distances between experts' matrices in
 * values, multiples of 8 and no less than a row.  FP16's range holds for h and
 * the gradients of the pre-activations, as for a gated block.
 */
route_status route_experts_prepare(int rows, int k, int f, int n, int experts, int type, int act,
                                   int train, int device, route_layer **out);

/* route_experts_forward.  saved, if given (plans with train), receives the FP32
 * gate and up sums and h: route_layer_saved_bytes(plan, rows). */
route_status route_experts_forward(const route_layer *plan, int rows, const void *x, int64_t ld_x,
                                   const int32_t *offsets, const void *W_gate, int64_t ld_gate,
                                   int64_t es_gate, const void *W_up, int64_t ld_up, int64_t es_up,
                                   const void *W_down, int64_t ld_down, int64_t es_down, void *out,
                                   int64_t ld_out, void *saved, void *stream);

/*
 * route_experts_backward, for each expert on its rows, with dh = dout W_down^T,
 * dgate = dh * up * act'(gate), dup = dh * act(gate):
 *   dx = dgate W_gate^T + dup W_up^T,  dW_gate = x^T dgate,  dW_up = x^T dup,
 *   dW_down = h^T dout
 * rows, offsets and x are those of the forward call that filled `saved` (whose
 * layout goes by rows).  Any of dx, dW_gate, dW_up and dW_down may be NULL.  The
 * weights' gradients of an expert without rows are 0.  x may be NULL without
 * dW_gate and dW_up.
 */
route_status route_experts_backward(const route_layer *plan, int rows, const void *dout,
                                    int64_t ld_dout, const void *x, int64_t ld_x,
                                    const int32_t *offsets, const void *W_gate, int64_t ld_gate,
                                    int64_t es_gate, const void *W_up, int64_t ld_up, int64_t es_up,
                                    const void *W_down, int64_t ld_down, int64_t es_down,
                                    const void *saved, void *dx, int64_t ld_dx, void *dW_gate,
                                    int64_t ld_dgate, int64_t es_dgate, void *dW_up, int64_t ld_dup,
                                    int64_t es_dup, void *dW_down, int64_t ld_ddown,
                                    int64_t es_ddown, void *stream);

/* route_dropout_prepare: up to `rows` (65536) rows of `dim` values (1..65536);
 * BF16, FP16 or FP32. */
route_status route_dropout_prepare(int rows, int dim, int type, int device, route_layer **out);

/*
 * route_dropout_forward: out = keep * x / (1 - q) + residual, in FP32: 1 / (1 - q),
 * its product with x and the sum are each rounded to it, and a 16-bit result
 * once more.
 *
 * Each value has a lot of 16 bits, and is kept if its lot is at least t =
 * p 65536 rounded to the nearest whole number (0 <= p <= 1): q = t / 65536 is
 * the probability that it is dropped, exactly, and what the kept values are
 * scaled by (p = 0.1 drops 0.100006 of them).  With t = 65536 nothing is kept.
 * A dropped value contributes 0 whatever it is.
 *
 * The lots are those of Philox 4x32 with ten rounds: the key is `seed`, the
 * counter offset + *step + r ceil(dim / 8) + c / 8 (64 bits, which wrap; the
 * upper 64 are 0) for column c of row r, and the lot the (c mod 8)-th 16 bits
 * of its 128, from the lowest.  They depend on nothing else, so no mask is
 * stored and the backward call draws the same; calls whose offsets are at least
 * rows ceil(dim / 8) apart have lots of their own.  `step`, one int64 on the
 * device that is read when the kernel runs, lets a captured call draw new lots
 * at every replay; it may be NULL (0).
 *
 * residual may be NULL; out may be x or the residual.
 */
route_status route_dropout_forward(const route_layer *plan, int rows, const void *x, int64_t ld_x,
                                   double p, uint64_t seed, uint64_t offset, const int64_t *step,
                                   const void *residual, int64_t ld_residual, void *out,
                                   int64_t ld_out, void *stream);

/* route_dropout_backward: dx = keep * dout / (1 - q) with the same lots and the
 * same roundings.  The residual's gradient is dout itself.  dx may be dout. */
route_status route_dropout_backward(const route_layer *plan, int rows, const void *dout,
                                    int64_t ld_dout, double p, uint64_t seed, uint64_t offset,
                                    const int64_t *step, void *dx, int64_t ld_dx, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ROUTE_EXPERTS_H */
