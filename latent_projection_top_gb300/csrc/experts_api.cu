// C ABI of the routed experts' operators and of dropout: plans, argument
// checks and launches.  Every check of what the host can see happens before
// anything is enqueued.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "experts.cuh"
#include "layer_math.cuh"
#include "layer_plan.h"
#include "route_experts.h"

using namespace route;

namespace {

static_assert(kMaxExperts == ROUTE_MAX_EXPERTS && kMaxTopk == ROUTE_MAX_TOPK, "limits");

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

route_status launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, what);
}

route_status need(const void *p, const char *name, unsigned align) {
    if (!p) return api_fail(ROUTE_ERR_NULL, "%s must be non-NULL", name);
    return check_vec(name, p, (int)align);
}

long long stride_of(int rows, int64_t ld, int cols) { return rows > 1 ? ld : cols; }

// ---- dispatch -------------------------------------------------------------------

route_status check_pairs(const route_layer *p, int pairs) {
    const long long most = (long long)p->rows * p->topk;
    if (pairs < 0 || pairs > most)
        return api_fail(ROUTE_ERR_ROWS, "pairs %d outside the plan's 0-%lld", pairs, most);
    return ROUTE_OK;
}

MoveArgs move_args(const route_layer *p, int rows, int pairs, const int32_t *place, const float *weights) {
    MoveArgs a = {};
    a.rows = rows, a.topk = p->topk, a.dim = p->k, a.type = p->type;
    a.pairs = pairs;
    a.place = place, a.weights = weights;
    return a;
}

// Weighted sums over places: combine, and (without weights and residual) gather's gradient.
route_status combine(const route_layer *p, int rows, const char *y_name, const void *y, int64_t ld_y, int pairs,
                     const int32_t *place, const float *weights, const void *residual, int64_t ld_residual,
                     const char *out_name, void *out, int64_t ld_out, void *stream) {
    route_status st = check_plan(p, kDispatch, rows);
    if (st != ROUTE_OK || (st = check_pairs(p, pairs)) != ROUTE_OK) return st;
    if (rows == 0) return ROUTE_OK;
    const int es = layer_esize(p->type);
    if ((pairs > 0 && (st = check_mat({y_name, y, ld_y, pairs, p->k, es, false})) != ROUTE_OK) ||
        (st = check_mat({out_name, out, ld_out, rows, p->k, es, false})) != ROUTE_OK ||
        (residual && (st = check_mat({"residual", residual, ld_residual, rows, p->k, es, false})) != ROUTE_OK) ||
        (st = need(place, "place", 4)) != ROUTE_OK || (st = check_vec("weights", weights, 4)) != ROUTE_OK)
        return st;
    MoveArgs a = move_args(p, rows, pairs, place, weights);
    a.a = residual, a.ld_a = stride_of(rows, ld_residual, p->k);
    a.b = y, a.ld_b = stride_of(pairs, ld_y, p->k);
    a.out = out, a.ld_out = stride_of(rows, ld_out, p->k);
    DeviceGuard guard(p->device);
    return launched(combine_launch(a, p->sms, static_cast<cudaStream_t>(stream)), "combine kernel launch");
}

// ---- the experts' products --------------------------------------------------------

// The experts' matrices [experts][rows, cols].
struct Stack {
    const char *name;
    const void *p;
    int64_t ld, es;
    int rows, cols;
};

route_status check_stack(const Stack &s, int experts) {
    route_status st = check_mat({s.name, s.p, s.ld, s.rows, s.cols, 2, true});
    if (st != ROUTE_OK || experts == 1) return st;
    if (s.es < s.cols)
        return api_fail(ROUTE_ERR_PLAN, "%s: experts' stride %lld is less than a row of %d", s.name,
                        (long long)s.es, s.cols);
    if (s.es % 8 != 0)
        return api_fail(ROUTE_ERR_ALIGN, "%s: experts' stride must be a multiple of 8", s.name);
    return ROUTE_OK;
}

route_status check_rows(const char *name, const void *p, int64_t ld, int rows, int cols) {
    return check_mat({name, p, ld, rows, cols, 2, true});
}

// Maps of one launch of the rows kernel.
struct Rows {
    const route_layer *p;
    ExpertsMaps maps;
    ExpertsArgs a;
    route_status st = ROUTE_OK;

    Rows(const route_layer *plan, int rows, const int32_t *offsets, int cols, int cols_a_tile, int K, int terms)
        : p(plan) {
        memset(static_cast<void *>(&a), 0, sizeof a);
        a.offsets = offsets;
        a.experts = p->experts, a.rows = rows;
        a.tiles_n = ceil_div(cols, cols_a_tile);
        a.kswitch = ceil_div(K, 64), a.kblocks = terms * a.kswitch;
        a.fp16 = p->type == kFp16;
        a.pairs = p->pairs;
        a.tiles_a_pair = (float)a.tiles_n / (float)a.pairs;
        a.test_stall = p->test_stall;
        a.timeout_ns = p->timeout_ns;
        a.status = p->words;
        a.e.N = cols;
        a.e.out_type = a.e.bias_type = p->type;
        a.e.act = p->act;
        a.e.vec = kVecOut | kVecRes | kVecBias;
    }
    // the rows' operand [rows, K] of a segment
    void tokens(int seg, const void *src, long long ld, int K) {
        for (int i = 0; i < kTokenBoxes && st == ROUTE_OK; ++i)
            st = api_encode_operand(&maps.t[seg][i], src, a.fp16, (uint64_t)K, (uint64_t)a.rows, (uint64_t)ld, 64,
                                    16u * (i + 1), "the sorted rows");
    }
    // a segment's weights: box of 64 columns x 64 rows, or of 64 columns x a CTA's share of the rows
    void weights(int i, const Stack &w, bool n_contiguous) {
        // no higher than the matrix: such a box loads slowly
        const uint32_t box = n_contiguous ? 64u : w.rows < 128 ? (uint32_t)up8(w.rows) : 128u;
        a.w_bytes = n_contiguous ? 2u * 64u * 128u : box * 128u;
        const long long ld = stride_of(w.rows, w.ld, w.cols), es = p->experts > 1 ? w.es : w.rows * ld;
        if (st == ROUTE_OK)
            st = api_encode_operands(&maps.w[i], w.p, a.fp16, (uint64_t)w.cols, (uint64_t)w.rows,
                                     (uint64_t)p->experts, (uint64_t)ld, (uint64_t)es, 64, box, w.name);
    }
    // Where all tiles that there could be are no more than the clusters that the
    // GPU holds at two CTAs an SM, each is split over a cluster (experts_small.cu:
    // 1 row at 2 of 64 experts, 896x448, 10.0 us; by pairs 12.3).
    route_status launch(int epi, bool n_contiguous, bool chained, bool more, cudaStream_t s) {
        if (st != ROUTE_OK) return st;
        a.chained = chained, a.trigger = more;
        const int used = a.rows < a.experts ? a.rows : a.experts;
        const int cols = epi == kEpiGated ? kFewCols / 2 : kFewCols;
        const long long tiles = (long long)used * ceil_div(a.e.N, cols);
        if (n_contiguous && a.rows <= kFewRows && tiles * kFewCtas <= 2ll * p->sms) {
            int ctas = kFewCtas;
            while (ctas > a.kblocks) ctas /= 2;
            a.tiles_n = ceil_div(a.e.N, cols);
            return launched(experts_small_launch(epi, (int)tiles, ctas, maps, a, s), "experts' product kernel launch");
        }
        return launched(experts_launch(epi, n_contiguous, maps, a, s), "experts' product kernel launch");
    }
};

route_status zero_stack(const Stack &w, int experts, cudaStream_t s) {
    if (!w.p) return ROUTE_OK;
    const long long ld = stride_of(w.rows, w.ld, w.cols);
    const bool one = experts == 1 || w.es == w.rows * ld;  // all rows the same distance apart
    const size_t rows = one ? (size_t)experts * w.rows : (size_t)w.rows;
    for (int e = 0; e < (one ? 1 : experts); ++e) {
        const cudaError_t err = cudaMemset2DAsync(const_cast<char *>(static_cast<const char *>(w.p)) + e * w.es * 2,
                                                  (size_t)ld * 2, 0, (size_t)w.cols * 2, rows, s);
        if (err != cudaSuccess) return cuda_fail(err, "cudaMemset2DAsync");
    }
    return ROUTE_OK;
}

// ---- dropout ----------------------------------------------------------------------

route_status dropout(const route_layer *p, int rows, const char *name, const void *x, int64_t ld_x, double prob,
                     uint64_t seed, uint64_t offset, const int64_t *step, const void *residual, int64_t ld_residual,
                     const char *out_name, void *out, int64_t ld_out, void *stream) {
    route_status st = check_plan(p, kDropout, rows);
    if (st != ROUTE_OK) return st;
    if (!(prob >= 0.0 && prob <= 1.0)) return api_fail(ROUTE_ERR_PLAN, "p must be from 0 to 1");
    if (rows == 0) return ROUTE_OK;
    const int es = layer_esize(p->type);
    if ((st = check_mats({{name, x, ld_x, rows, p->k, es, false}, {out_name, out, ld_out, rows, p->k, es, false}})) !=
            ROUTE_OK ||
        (residual && (st = check_mat({"residual", residual, ld_residual, rows, p->k, es, false})) != ROUTE_OK) ||
        (st = check_vec("step", step, 8)) != ROUTE_OK)
        return st;
    DropoutArgs a = {};
    a.rows = rows, a.dim = p->k, a.type = p->type;
    a.threshold = (unsigned)std::floor(prob * 65536.0 + 0.5);
    a.scale = a.threshold < 65536u ? (float)(65536.0 / (65536.0 - a.threshold)) : 0.f;
    a.offset = offset;
    for (int r = 0; r < kPhiloxRounds; ++r) {
        a.keys[2 * r] = (uint32_t)seed + 0x9E3779B9u * (uint32_t)r;
        a.keys[2 * r + 1] = (uint32_t)(seed >> 32) + 0xBB67AE85u * (uint32_t)r;
    }
    a.step = reinterpret_cast<const long long *>(step);
    a.x = x, a.ld_x = stride_of(rows, ld_x, p->k);
    a.residual = residual, a.ld_res = stride_of(rows, ld_residual, p->k);
    a.out = out, a.ld_out = stride_of(rows, ld_out, p->k);
    DeviceGuard guard(p->device);
    return launched(dropout_launch(a, p->sms, static_cast<cudaStream_t>(stream)), "dropout kernel launch");
}

}  // namespace

extern "C" {

route_status route_dispatch_prepare(int rows, int dim, int type, int experts, int first, int topk, int device,
                                    route_layer **out) {
    route_status st =
        layer_check_prepare(rows, ROUTE_LAYER_MAX_ROWS, {dim}, ROUTE_LAYER_MAX_WIDTH, type, true, 0, out);
    if (st != ROUTE_OK) return st;
    if (experts < 1 || experts > ROUTE_MAX_EXPERTS)
        return api_fail(ROUTE_ERR_PLAN, "experts %d outside 1-%d", experts, ROUTE_MAX_EXPERTS);
    if (topk < 1 || topk > ROUTE_MAX_TOPK)
        return api_fail(ROUTE_ERR_PLAN, "topk %d outside 1-%d", topk, ROUTE_MAX_TOPK);
    if (first < 0) return api_fail(ROUTE_ERR_PLAN, "first must not be negative");
    route_layer *p = layer_new_plan(kDispatch, rows, type, 0, 0);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = dim;
    p->experts = experts, p->first = first, p->topk = topk;
    return layer_finish_prepare(p, device, out);
}

route_status route_dispatch_sort(const route_layer *p, int rows, const int32_t *ids, int64_t ld_ids,
                                 int32_t *offsets, int32_t *place, int32_t *source, void *stream) {
    route_status st = check_plan(p, kDispatch, rows);
    if (st != ROUTE_OK || (st = need(offsets, "offsets", 4)) != ROUTE_OK) return st;
    if (rows > 0 && ((st = check_mat({"ids", ids, ld_ids, rows, p->topk, 4, false})) != ROUTE_OK ||
                     (st = need(place, "place", 4)) != ROUTE_OK || (st = check_vec("source", source, 4)) != ROUTE_OK))
        return st;
    SortArgs a = {};
    a.rows = rows, a.topk = p->topk, a.experts = p->experts, a.first = p->first;
    a.ids = ids, a.ld_ids = stride_of(rows, ld_ids, p->topk);
    a.offsets = offsets, a.place = place, a.source = source;
    DeviceGuard guard(p->device);
    return launched(sort_launch(a, p->sort, static_cast<cudaStream_t>(stream)), "sort kernel launch");
}

route_status route_dispatch_gather(const route_layer *p, int rows, const void *x, int64_t ld_x,
                                   const int32_t *place, int pairs, void *out, int64_t ld_out, void *stream) {
    route_status st = check_plan(p, kDispatch, rows);
    if (st != ROUTE_OK || (st = check_pairs(p, pairs)) != ROUTE_OK) return st;
    if (rows == 0 || pairs == 0) return ROUTE_OK;
    const int es = layer_esize(p->type);
    if ((st = check_mats({{"x", x, ld_x, rows, p->k, es, false}, {"out", out, ld_out, pairs, p->k, es, false}})) !=
            ROUTE_OK ||
        (st = need(place, "place", 4)) != ROUTE_OK)
        return st;
    MoveArgs a = move_args(p, rows, pairs, place, nullptr);
    a.a = x, a.ld_a = stride_of(rows, ld_x, p->k);
    a.out = out, a.ld_out = stride_of(pairs, ld_out, p->k);
    DeviceGuard guard(p->device);
    return launched(gather_launch(a, p->sms, static_cast<cudaStream_t>(stream)), "gather kernel launch");
}

route_status route_dispatch_combine(const route_layer *p, int rows, const void *y, int64_t ld_y, int pairs,
                                    const int32_t *place, const float *weights, const void *residual,
                                    int64_t ld_residual, void *out, int64_t ld_out, void *stream) {
    return combine(p, rows, "y", y, ld_y, pairs, place, weights, residual, ld_residual, "out", out, ld_out, stream);
}

route_status route_dispatch_gather_backward(const route_layer *p, int rows, const void *dout, int64_t ld_dout,
                                            int pairs, const int32_t *place, void *dx, int64_t ld_dx,
                                            void *stream) {
    return combine(p, rows, "dout", dout, ld_dout, pairs, place, nullptr, nullptr, 0, "dx", dx, ld_dx, stream);
}

route_status route_dispatch_combine_backward(const route_layer *p, int rows, const void *dout, int64_t ld_dout,
                                             const void *y, int64_t ld_y, int pairs, const int32_t *place,
                                             const float *weights, void *dy, int64_t ld_dy, float *dweights,
                                             void *stream) {
    route_status st = check_plan(p, kDispatch, rows);
    if (st != ROUTE_OK || (st = check_pairs(p, pairs)) != ROUTE_OK) return st;
    if (rows == 0 || (!dy && !dweights)) return ROUTE_OK;
    const int es = layer_esize(p->type);
    if ((st = check_mat({"dout", dout, ld_dout, rows, p->k, es, false})) != ROUTE_OK ||
        (pairs > 0 && dweights && (st = check_mat({"y", y, ld_y, pairs, p->k, es, false})) != ROUTE_OK) ||
        (pairs > 0 && dy && (st = check_mat({"dy", dy, ld_dy, pairs, p->k, es, false})) != ROUTE_OK) ||
        (st = need(place, "place", 4)) != ROUTE_OK || (st = check_vec("weights", weights, 4)) != ROUTE_OK ||
        (st = check_vec("dweights", dweights, 4)) != ROUTE_OK)
        return st;
    MoveArgs a = move_args(p, rows, pairs, place, weights);
    a.a = dout, a.ld_a = stride_of(rows, ld_dout, p->k);
    a.b = dweights ? y : nullptr, a.ld_b = stride_of(pairs, ld_y, p->k);
    a.out = dy, a.ld_out = stride_of(pairs, ld_dy, p->k);
    a.dweights = dweights;
    DeviceGuard guard(p->device);
    return launched(combine_backward_launch(a, p->sms, static_cast<cudaStream_t>(stream)), "combine gradient kernel launch");
}

route_status route_experts_prepare(int rows, int k, int f, int n, int experts, int type, int act, int train,
                                   int device, route_layer **out) {
    route_status st = layer_check_prepare(rows, ROUTE_EXPERTS_MAX_ROWS, {k, f, n}, ROUTE_LAYER_MAX_WIDTH, type,
                                          false, act, out);
    if (st != ROUTE_OK) return st;
    if (experts < 1 || experts > ROUTE_MAX_EXPERTS)
        return api_fail(ROUTE_ERR_PLAN, "experts %d outside 1-%d", experts, ROUTE_MAX_EXPERTS);
    for (int w : {k, f, n})
        if (w % 8 != 0) return api_fail(ROUTE_ERR_PLAN, "width %d is not a multiple of 8", w);
    route_layer *p = layer_new_plan(kExpertBlocks, rows, type, act, train);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = k, p->f = f, p->n = n;
    p->experts = experts;
    return layer_finish_prepare(p, device, out);
}

route_status route_experts_forward(const route_layer *p, int rows, const void *x, int64_t ld_x,
                                   const int32_t *offsets, const void *W_gate, int64_t ld_gate, int64_t es_gate,
                                   const void *W_up, int64_t ld_up, int64_t es_up, const void *W_down,
                                   int64_t ld_down, int64_t es_down, void *out, int64_t ld_out, void *saved,
                                   void *stream) {
    route_status st = check_plan(p, kExpertBlocks, rows);
    if (st != ROUTE_OK) return st;
    std::lock_guard<std::mutex> lock(p->calls);
    if (saved && !p->train) return api_fail(ROUTE_ERR_PLAN, "the plan was prepared without train");
    if (rows == 0) return ROUTE_OK;
    const Stack wg = {"W_gate", W_gate, ld_gate, es_gate, p->k, p->f}, wu = {"W_up", W_up, ld_up, es_up, p->k, p->f},
                wd = {"W_down", W_down, ld_down, es_down, p->f, p->n};
    for (const Stack &w : {wg, wu, wd})
        if ((st = check_stack(w, p->experts)) != ROUTE_OK) return st;
    if ((st = check_rows("x", x, ld_x, rows, p->k)) != ROUTE_OK ||
        (st = check_rows("out", out, ld_out, rows, p->n)) != ROUTE_OK ||
        (st = need(offsets, "offsets", 4)) != ROUTE_OK || (st = check_vec("saved", saved, 32)) != ROUTE_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard guard(p->device);
    const long long ldf = up16(p->f);
    uint8_t *h = saved ? static_cast<uint8_t *>(saved) + saved_h(p, rows) : p->scratch + p->o_h;
    Rows up(p, rows, offsets, p->f, kExpertCols / 2, p->k, 1);
    up.tokens(0, x, stride_of(rows, ld_x, p->k), p->k);
    up.weights(0, wg, true);
    up.weights(1, wu, true);
    up.a.e.out = h, up.a.e.ld_out = ldf;
    up.a.e.saved = static_cast<float *>(saved), up.a.e.ld_saved = ldf;
    up.a.e.saved2 = saved ? up.a.e.saved + (size_t)rows * ldf : nullptr;
    if ((st = up.launch(kEpiGated, true, false, true, s)) != ROUTE_OK) return st;
    Rows down(p, rows, offsets, p->n, kExpertCols, p->f, 1);
    down.tokens(0, h, ldf, p->f);
    down.weights(0, wd, true);
    down.a.e.out = out, down.a.e.ld_out = stride_of(rows, ld_out, p->n);
    return down.launch(kEpiLinear, true, true, false, s);
}

route_status route_experts_backward(const route_layer *p, int rows, const void *dout, int64_t ld_dout, const void *x,
                                    int64_t ld_x, const int32_t *offsets, const void *W_gate, int64_t ld_gate,
                                    int64_t es_gate, const void *W_up, int64_t ld_up, int64_t es_up,
                                    const void *W_down, int64_t ld_down, int64_t es_down, const void *saved,
                                    void *dx, int64_t ld_dx, void *dW_gate, int64_t ld_dgate, int64_t es_dgate,
                                    void *dW_up, int64_t ld_dup, int64_t es_dup, void *dW_down, int64_t ld_ddown,
                                    int64_t es_ddown, void *stream) {
    route_status st = check_plan(p, kExpertBlocks, rows);
    if (st != ROUTE_OK) return st;
    std::lock_guard<std::mutex> lock(p->calls);
    if (!p->train) return api_fail(ROUTE_ERR_PLAN, "the plan was prepared without train");
    const Stack grads[3] = {{"dW_gate", dW_gate, ld_dgate, es_dgate, p->k, p->f},
                            {"dW_up", dW_up, ld_dup, es_dup, p->k, p->f},
                            {"dW_down", dW_down, ld_ddown, es_ddown, p->f, p->n}};
    for (const Stack &g : grads)
        if (g.p && (st = check_stack(g, p->experts)) != ROUTE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard guard(p->device);
    if (rows == 0) {
        for (const Stack &g : grads)
            if ((st = zero_stack(g, p->experts, s)) != ROUTE_OK) return st;
        return ROUTE_OK;
    }
    const bool pre = dx || dW_gate || dW_up;  // the pre-activations' gradients are wanted
    const bool weights = dW_gate || dW_up || dW_down;
    if (!pre && !weights) return ROUTE_OK;
    const Stack wg = {"W_gate", W_gate, ld_gate, es_gate, p->k, p->f}, wu = {"W_up", W_up, ld_up, es_up, p->k, p->f},
                wd = {"W_down", W_down, ld_down, es_down, p->f, p->n};
    if ((st = check_rows("dout", dout, ld_dout, rows, p->n)) != ROUTE_OK ||
        (pre && (st = check_stack(wd, p->experts)) != ROUTE_OK) ||
        ((dW_gate || dW_up) && (st = check_rows("x", x, ld_x, rows, p->k)) != ROUTE_OK) ||
        (dx && ((st = check_stack(wg, p->experts)) != ROUTE_OK || (st = check_stack(wu, p->experts)) != ROUTE_OK ||
                (st = check_rows("dx", dx, ld_dx, rows, p->k)) != ROUTE_OK)) ||
        (st = need(offsets, "offsets", 4)) != ROUTE_OK || (st = need(saved, "saved", 32)) != ROUTE_OK)
        return st;
    const long long ldf = up16(p->f), ldy = stride_of(rows, ld_dout, p->n);
    uint8_t *dg = p->scratch + p->o_dg, *du = p->scratch + p->o_du;
    const uint8_t *h = static_cast<const uint8_t *>(saved) + saved_h(p, rows);
    if (pre) {
        // dh = dout W_down^T, turned into dgate and dup in its epilogue
        Rows g(p, rows, offsets, p->f, kExpertCols, p->n, 1);
        g.tokens(0, dout, ldy, p->n);
        g.weights(0, wd, false);
        g.a.e.out = dg, g.a.e.out2 = du, g.a.e.ld_out = ldf;
        g.a.e.saved = static_cast<float *>(const_cast<void *>(saved)), g.a.e.ld_saved = ldf;
        g.a.e.saved2 = g.a.e.saved + (size_t)rows * ldf;
        if ((st = g.launch(kEpiDGate, false, false, dx || weights, s)) != ROUTE_OK) return st;
    }
    if (dx) {
        Rows g(p, rows, offsets, p->k, kExpertCols, p->f, 2);
        g.tokens(0, dg, ldf, p->f);
        g.tokens(1, du, ldf, p->f);
        g.weights(0, wg, false);
        g.weights(1, wu, false);
        g.a.e.out = dx, g.a.e.ld_out = stride_of(rows, ld_dx, p->k);
        if ((st = g.launch(kEpiLinear, false, true, weights, s)) != ROUTE_OK) return st;
    }
    if (!weights) return ROUTE_OK;
    GradMaps maps;
    GradArgs a;
    memset(static_cast<void *>(&a), 0, sizeof a);
    a.offsets = offsets;
    a.experts = p->experts, a.rows = rows;
    a.fp16 = p->type == kFp16;
    // dx's product has waited for dgate and dup's (without it they are the ones before)
    a.beside = dx != nullptr;
    a.pairs = p->pairs;
    a.test_stall = p->test_stall;
    a.timeout_ns = p->timeout_ns;
    a.status = p->words;
    auto map = [&](CUtensorMap *m, const void *src, long long ld, int cols, const char *what) {
        if (st == ROUTE_OK)
            st = api_encode_operand(m, src, a.fp16, (uint64_t)cols, (uint64_t)rows, (uint64_t)ld, 64, 64, what);
    };
    for (int i = 0; i < 3; ++i) {
        const Stack &g = grads[i];
        if (!g.p) continue;
        auto &q = a.p[a.nprob];
        q.M = g.rows, q.N = g.cols;
        q.tiles_m = ceil_div(q.M, 256), q.tiles_n = ceil_div(q.N, 256);
        q.base = a.per_expert;
        a.per_expert += q.tiles_m * q.tiles_n;
        const long long ld = stride_of(g.rows, g.ld, g.cols), es = p->experts > 1 ? g.es : g.rows * ld;
        if (st == ROUTE_OK)
            st = api_encode_operands(&maps.d[a.nprob], g.p, a.fp16, (uint64_t)g.cols, (uint64_t)g.rows,
                                     (uint64_t)p->experts, (uint64_t)ld, (uint64_t)es, 64, 32, g.name);
        if (i < 2)
            map(&maps.a[a.nprob], x, stride_of(rows, ld_x, p->k), p->k, "x");
        else
            map(&maps.a[a.nprob], h, ldf, p->f, "h");
        if (i < 2)
            map(&maps.b[a.nprob], i == 0 ? dg : du, ldf, p->f, "the pre-activations' gradient");
        else
            map(&maps.b[a.nprob], dout, ldy, p->n, "dout");
        ++a.nprob;
    }
    if (st != ROUTE_OK) return st;
    return launched(experts_grad_launch(maps, a, s), "weights' gradient kernel launch");
}

route_status route_dropout_prepare(int rows, int dim, int type, int device, route_layer **out) {
    route_status st =
        layer_check_prepare(rows, ROUTE_LAYER_MAX_ROWS, {dim}, ROUTE_LAYER_MAX_WIDTH, type, true, 0, out);
    if (st != ROUTE_OK) return st;
    route_layer *p = layer_new_plan(kDropout, rows, type, 0, 0);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = dim;
    return layer_finish_prepare(p, device, out);
}

route_status route_dropout_forward(const route_layer *p, int rows, const void *x, int64_t ld_x, double prob,
                                   uint64_t seed, uint64_t offset, const int64_t *step, const void *residual,
                                   int64_t ld_residual, void *out, int64_t ld_out, void *stream) {
    return dropout(p, rows, "x", x, ld_x, prob, seed, offset, step, residual, ld_residual, "out", out, ld_out, stream);
}

route_status route_dropout_backward(const route_layer *p, int rows, const void *dout, int64_t ld_dout, double prob,
                                    uint64_t seed, uint64_t offset, const int64_t *step, void *dx, int64_t ld_dx,
                                    void *stream) {
    return dropout(p, rows, "dout", dout, ld_dout, prob, seed, offset, step, nullptr, 0, "dx", dx, ld_dx, stream);
}

}  // extern "C"
