/*
 * libroute -- the layer operators around the route step, C ABI.
 *
 * What a layer runs next to the route step (route.h), forward and backward:
 *
 *   norm    y = (x - mean) / sqrt(var + eps) * gamma + beta   (each token row)
 *   linear  out = act(x W + bias) + residual
 *   gated   out = (act(x W_gate) * (x W_up)) W_down + residual
 *
 * for instance the norm whose rows the route step reads, the shared expert
 * (gated), and the latent's projection back to the hidden width, added to
 * the residual stream (linear).
 *
 * Conventions, besides route.h's on streams, graph capture and errors:
 *  - Matrices are row-major with unit stride between columns; `ld_*` is the
 *    distance between rows in elements, at least the row's length (ignored
 *    where there is one row).  Weights are stored [in, out], like the route
 *    step's.
 *  - Operands and results have the plan's type (route_layer_type); sums,
 *    statistics and kept pre-activations are FP32.  Between an operator's
 *    inputs and its results there is at most one rounding to 16 bits besides
 *    the result's own: h = act(gate) * up before W_down, and the gradients
 *    of pre-activations before the products that read them.  These have the
 *    plan's type and so its range: an FP16 plan's become infinite past 65504,
 *    and lose bits below 6.1e-5, though the result may be far from both.
 *  - Matrices that a product reads (x, dout, the weights) and whose width is
 *    a multiple of 8 start on 16 bytes and have row strides that are
 *    multiples of 8, otherwise ROUTE_ERR_ALIGN.  Where the width is not a
 *    multiple of 8 any alignment and stride will do: rows that TMA cannot
 *    read in place are copied into the plan's scratch first.  All other
 *    tensors need their element's alignment only, and are read and written
 *    in vectors where theirs allows it.
 *  - A plan fixes the widths and the largest row count; a call takes 0 to
 *    that many rows.  With none, forward calls launch nothing and backward
 *    calls write zeros into the parameters' gradients.
 *  - A plan holds scratch memory and must not run on two streams at the same
 *    time.  Calls of several host threads on one plan (and stream) are taken one
 *    after another.  Calls do not allocate.
 *  - Results are reproducible bit for bit: no sum's order depends on timing.
 *  - `out` may be the residual itself (in place); no other output may
 *    overlap an input or another output.
 *  - Statuses: ROUTE_ERR_ROWS (rows outside the plan), ROUTE_ERR_MODE
 *    (unknown type or activation), ROUTE_ERR_PLAN (widths out of range, a
 *    stride below the row's length, a call that the plan was not prepared
 *    for), ROUTE_ERR_NULL, ROUTE_ERR_ALIGN, ROUTE_ERR_DEVICE, ROUTE_ERR_CUDA.
 */
#ifndef ROUTE_LAYER_H
#define ROUTE_LAYER_H

#include "route.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ROUTE_LAYER_MAX_ROWS 65536
#define ROUTE_LAYER_MAX_WIDTH 65536
#define ROUTE_NORM_MAX_WIDTH 16384

typedef enum { ROUTE_BF16 = 0, ROUTE_FP16 = 1, ROUTE_FP32 = 2 } route_layer_type;

typedef enum {
    ROUTE_ACT_NONE = 0,
    ROUTE_ACT_RELU = 1,
    ROUTE_ACT_GELU = 2,      /* z (1 + erf(z / sqrt 2)) / 2 */
    ROUTE_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
    ROUTE_ACT_SILU = 4,      /* z / (1 + exp(-z)) */
    ROUTE_ACT_SIGMOID = 5    /* 1 / (1 + exp(-z)) */
} route_activation;

typedef struct route_layer route_layer; /* opaque: a layer operator's plan */

/* route_norm_prepare: a layer norm of rows of `dim` values (1..16384), type
 * BF16, FP16 or FP32 (x, y, the parameters and all gradients). */
route_status route_norm_prepare(int rows, int dim, int type, int device, route_layer **out);

/* route_linear_prepare: out[rows, n] = act(x[rows, k] W[k, n] + bias[n]) +
 * residual[rows, n].  x, W and bias are BF16 or FP16 (`type`); out and the
 * residual have `out_type`: the same, or FP32 (inference only).  train != 0
 * prepares for route_linear_backward too. */
route_status route_linear_prepare(int rows, int k, int n, int type, int out_type, int act,
                                  int train, int device, route_layer **out);

/* route_gated_prepare: h = act(x[rows, k] W_gate[k, f]) * (x W_up[k, f]),
 * out[rows, n] = h W_down[f, n] + residual[rows, n]; BF16 or FP16.  train != 0
 * prepares for route_gated_backward too. */
route_status route_gated_prepare(int rows, int k, int f, int n, int type, int act, int train,
                                 int device, route_layer **out);

/* route_layer_destroy: free the plan and its scratch memory (synchronises
 * the plan's device).  NULL is accepted and ignored. */
route_status route_layer_destroy(route_layer *plan);

/* route_layer_status: synchronise the plan's device, then report and clear
 * the device-side error word: ROUTE_OK, or ROUTE_ERR_DEVICE_TIMEOUT (a bounded
 * wait expired; the outputs of that launch are invalid). */
route_status route_layer_status(const route_layer *plan);

/* Bytes of the `saved` buffer that a training forward call of `rows` rows
 * fills and its backward call reads (device memory of the caller's, 32-byte
 * aligned; its layout is the library's own): the FP32 pre-activations, and a
 * gated block's h.  0 for plans that save nothing, -1 for a NULL plan. */
int64_t route_layer_saved_bytes(const route_layer *plan, int rows);

/*
 * route_norm_forward: y = (x - mean) rstd gamma + beta for each row, with
 * mean = sum(x) / dim, rstd = 1 / sqrt(sum((x - mean)^2) / dim + eps).
 * gamma, beta [dim]: either may be NULL (1 and 0).  stats [rows][2] FP32, if
 * given, receives (mean, rstd) for the backward pass.  eps >= 0.  y may be x.
 */
route_status route_norm_forward(const route_layer *plan, int rows, const void *x, int64_t ld_x,
                                const void *gamma, const void *beta, float eps, void *y,
                                int64_t ld_y, float *stats, void *stream);

/*
 * route_norm_backward, with g = dy gamma and xh = (x - mean) rstd:
 *   dx = rstd (g - mean(g) - xh mean(g xh))
 *   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
 * Any of dx, dgamma and dbeta may be NULL.  dx may be dy or x.
 */
route_status route_norm_backward(const route_layer *plan, int rows, const void *dy, int64_t ld_dy,
                                 const void *x, int64_t ld_x, const void *gamma,
                                 const float *stats, void *dx, int64_t ld_dx, void *dgamma,
                                 void *dbeta, void *stream);

/*
 * route_linear_forward.  bias and residual may be NULL.  saved, if given
 * (plans with train and an activation), receives z = x W + bias.
 */
route_status route_linear_forward(const route_layer *plan, int rows, const void *x, int64_t ld_x,
                                  const void *W, int64_t ld_W, const void *bias,
                                  const void *residual, int64_t ld_residual, void *out,
                                  int64_t ld_out, void *saved, void *stream);

/*
 * route_linear_backward, with dz = dout * act'(z):
 *   dx = dz W^T,  dW = x^T dz,  dbias = sum over rows of dz (unrounded)
 * The residual's gradient is dout itself.  Any of dx, dW and dbias may be
 * NULL; x may be NULL without dW, W without dx; saved without an activation.
 */
route_status route_linear_backward(const route_layer *plan, int rows, const void *dout,
                                   int64_t ld_dout, const void *x, int64_t ld_x, const void *W,
                                   int64_t ld_W, const void *saved, void *dx, int64_t ld_dx,
                                   void *dW, int64_t ld_dW, void *dbias, void *stream);

/*
 * route_gated_forward.  residual may be NULL.  saved, if given (plans with
 * train), receives the FP32 gate and up sums and h.
 */
route_status route_gated_forward(const route_layer *plan, int rows, const void *x, int64_t ld_x,
                                 const void *W_gate, int64_t ld_gate, const void *W_up,
                                 int64_t ld_up, const void *W_down, int64_t ld_down,
                                 const void *residual, int64_t ld_residual, void *out,
                                 int64_t ld_out, void *saved, void *stream);

/*
 * route_gated_backward, with dh = dout W_down^T, dgate = dh * up * act'(gate),
 * dup = dh * act(gate):
 *   dx = dgate W_gate^T + dup W_up^T,  dW_gate = x^T dgate,  dW_up = x^T dup,
 *   dW_down = h^T dout
 * Any of dx, dW_gate, dW_up and dW_down may be NULL.
 */
route_status route_gated_backward(const route_layer *plan, int rows, const void *dout,
                                  int64_t ld_dout, const void *x, int64_t ld_x, const void *W_gate,
                                  int64_t ld_gate, const void *W_up, int64_t ld_up,
                                  const void *W_down, int64_t ld_down, const void *saved, void *dx,
                                  int64_t ld_dx, void *dW_gate, int64_t ld_dgate, void *dW_up,
                                  int64_t ld_dup, void *dW_down, int64_t ld_ddown, void *stream);

/* route_layer_test_stall: TEST HOOK, as route_test_stall for a linear or
 * gated plan: each product's kernel skips its last copies, so that its waits
 * give up after timeout_ns and route_layer_status reports
 * ROUTE_ERR_DEVICE_TIMEOUT.  enable == 0 restores the default bound (2 s). */
route_status route_layer_test_stall(route_layer *plan, int enable, uint64_t timeout_ns);

#ifdef __cplusplus
}
#endif

#endif /* ROUTE_LAYER_H */
