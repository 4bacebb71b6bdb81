// C ABI of the layer operators: plans, argument checks, the choice of tile
// and split for every product, and the launches.  Every check happens on the
// host before anything is enqueued.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "experts.cuh"
#include "layer_math.cuh"
#include "layer_plan.h"

using namespace route;

namespace {

// A launch's split products have at most two items a CTA pair: FP32 partials
// of a 256 x 256 tile each.
constexpr size_t kTilePartBytes = 256 * 256 * 4;

int vec_bits(const void *out, long long ld_out, const void *out2, const void *res, long long ld_res,
             int out_type, const void *bias) {
    // four values at a time
    const int bytes = 4 * layer_esize(out_type);
    auto rows_on = [&](const void *p, long long ld) {
        return p == nullptr || (aligned(p, (unsigned)bytes) && ld % 4 == 0);
    };
    int v = 0;
    if (rows_on(out, ld_out) && rows_on(out2, ld_out)) v |= kVecOut;
    if (rows_on(res, ld_res)) v |= kVecRes;
    if (aligned(bias, 8)) v |= kVecBias;
    if (out_type != kFp32 && aligned(bias, 16)) v |= kVecAny;
    if (out_type != kFp32 && aligned(out, 16) && ld_out % 8 == 0 && aligned(bias, 16) && aligned(res, 16) &&
        (res == nullptr || ld_res % 8 == 0))
        v |= kVecPacked;
    return v;
}

// ---- products -------------------------------------------------------------------

struct Operand {
    const void *p;
    long long ld;
};

// Operands as TMA can read them: in place, or copied into scratch by one
// launch for all of a call's.
struct Copies {
    const route_layer *p;
    RepackArgs args;
    explicit Copies(const route_layer *plan) : p(plan) { args.count = 0; }
    Operand operand(const void *src, long long ld, int rows, int cols, size_t scratch) {
        if (cols % 8 == 0) return {src, rows > 1 ? ld : cols};
        if (aligned(src, 16) && ld % 8 == 0 && rows > 1) return {src, ld};
        auto &c = args.c[args.count++];
        c.src = src, c.ld_src = rows > 1 ? ld : cols;
        c.dst = p->scratch + scratch, c.ld_dst = up8(cols);
        c.rows = rows, c.cols = cols;
        return {c.dst, c.ld_dst};
    }
    route_status launch(cudaStream_t stream) {
        if (args.count == 0) return ROUTE_OK;
        const cudaError_t e = repack_launch(args, stream);
        return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "operand copy");
    }
};

// A product of a launch: its form, the rows and columns of its result (gated:
// hidden columns), its contraction's terms and each one's length.
struct Prod {
    int id;  // its place among the products that the choice of tiles goes by
    int form, M, N, terms, K;
    Operand a[2], b[2];  // of each term (gated: b of gate and of up)
    Epilogue e;
    int kblocks() const { return terms * ((K + 63) / 64); }
};

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// The choice with the smallest estimated time, from what the kernels measure:
// a launch of pair tiles has 5.0 us (4.5 with 128 columns) besides its
// k-blocks, of 0.34 us in a 256 x 256 tile and 0.29 us in a 256 x 128 tile,
// and 1.8 us more where the epilogue does more than store; the small tiles
// have 2.6 us and are bound by what an SM reads, about 70 bytes a nanosecond.
Choice choose(const route_layer *p, int epi, const Prod *w, int count) {
    Choice best = {false, 256, {1, 1, 1, 1}, 1e30};
    double &t_best = best.us;
    int rows = 0, kmost = 0;
    bool tt = false;
    for (int i = 0; i < count; ++i) {
        rows = rows < w[i].M ? w[i].M : rows;
        kmost = kmost < w[i].kblocks() ? w[i].kblocks() : kmost;
        tt = tt || w[i].form == kFormTT;
    }
    for (int bn : {256, 128}) {
        const int cols = epi == kEpiGated ? bn / 2 : bn;
        const double kb_us = bn == 256 ? 0.34 : 0.29;
        const double drain_us = (bn == 256 ? 1.0 : 0.55) * (epi == kEpiLinear ? 2.5 : 4.0);
        const double start_us = (bn == 256 ? 5.0 : 4.5) + (epi == kEpiLinear ? 0.0 : 1.8);
        long long tiles[kGemmMaxProblems];
        double work = 0;
        for (int i = 0; i < count; ++i) {
            tiles[i] = (long long)ceil_div(w[i].M, kGemmBM) * ceil_div(w[i].N, cols);
            work += (double)tiles[i] * w[i].kblocks();
        }
        // No contraction is left longer than `part` of an equal share: without
        // splits, and with several sizes of them.
        for (double part : {0.0, 2.0, 1.0, 0.7, 0.5, 0.34, 0.25}) {
            Choice c = {false, bn, {1, 1, 1, 1}, 0};
            long long items = 0, split_items = 0;
            double longest = 0, level = 0, t = start_us;
            for (int i = 0; i < count; ++i) {
                int s = part > 0 ? (int)(w[i].kblocks() * p->pairs / (work * part) + 0.99) : 1;
                s = s > kGemmMaxSplits ? kGemmMaxSplits : s;
                s = s > w[i].kblocks() / 2 ? w[i].kblocks() / 2 : s;
                s = s < 1 ? 1 : s;
                c.splits[i] = s;
                items += tiles[i] * s;
                double one = ceil_div(w[i].kblocks(), s) * kb_us;
                longest = longest < one ? one : longest;
                // a tile's epilogue hides behind the next one's k-blocks
                one = one < drain_us ? drain_us : one;
                level += (double)tiles[i] * s * one / p->pairs;
                if (s > 1) {
                    split_items += tiles[i] * s;
                    t += 3.5 + (double)w[i].M * w[i].N * (epi == kEpiGated ? 2 : 1) * 4.0 * (s + 1) / 4e6;
                }
            }
            if (split_items > 2 * p->pairs) continue;
            if (count == 1) {  // equal items
                t += longest + (ceil_div(items, p->pairs) - 1) * (longest < drain_us ? drain_us : longest);
            } else {
                // items do not end together (16x3584x7168's backward pass 27.6 us, 32.4
                // without this; with 0.7 512x2048x512 7.6, so 6.7)
                level += 0.35 * longest;
                t += level > longest ? level : longest;
            }
            c.us = t;
            if (t < t_best) best = c;
        }
    }
    {
        int need = tt ? 64 : 16;
        while (need < 128 && need < rows) need *= 2;
        const int cols = epi == kEpiGated ? kSmallTile / 2 : kSmallTile;
        // fewer rows a tile than there are: more CTAs for short contractions
        for (int bn = tt ? 64 : 16; bn <= need; bn *= 2) {
            long long tiles = 0;
            for (int i = 0; i < count; ++i)
                tiles += (long long)ceil_div(w[i].M, bn) * ceil_div(w[i].N, cols);
            for (int s = 1; s <= kSmallMaxSplits && s <= kmost; s *= 2) {
                if (tiles * s > 8192) break;
                double longest = 0, level = 0;
                for (int i = 0; i < count; ++i) {
                    const int box = w[i].form != kFormTT && w[i].M < bn ? w[i].M : bn;
                    const double kb = ceil_div(w[i].kblocks(), s) * (16384 + box * 128) / 70e3;
                    const double drain = (epi == kEpiLinear ? 0.025 : 0.045) * box / s;
                    double one = kb + 0.8 + drain;
                    longest = longest < one ? one : longest;
                    // two CTAs of an SM hide each other's start and end, not more
                    const double half = 0.5 * (4.0 + kb + drain);
                    one = one < half ? half : one;
                    const long long ctas = (long long)ceil_div(w[i].M, bn) * ceil_div(w[i].N, cols) * s;
                    level += (double)ctas * one / p->sms;
                }
                // one round of CTAs is as long as the longest of them; of several, not all
                // end together (3000x256x2048's backward pass 16.1 us, 17.1 without)
                if (tiles * s <= p->sms) level = 0;
                double t = count > 1 && level > 0 ? level + 0.3 * longest : longest;
                t = t < longest ? longest : t < level ? level : t;
                // CTAs past two an SM start when others have left
                t += 2.6 + (s > 1 ? 0.3 : 0.0) + 3.0 * (ceil_div(tiles * s, 2 * p->sms) - 1);
                if (t < t_best) best = {true, bn, {s, s, s, s}, t};
            }
        }
    }
    return best;
}

const Choice &choice_of(const route_layer *p, ChoiceSlot slot, int rows, int epi, const Prod *w, int count) {
    ChoiceMemo &m = p->memo[slot];
    if (m.rows != rows) m.c = choose(p, epi, w, count), m.rows = rows;
    return m.c;
}

void set_tiles(GemmProblem &q, int tile_rows, int tile_cols, int pairs) {
    q.tiles_m = ceil_div(q.e.M, tile_rows);
    q.tiles_n = ceil_div(q.e.N, tile_cols);
    // Column tiles of a band: with up to 16 tiles either way the whole of that
    // way stays in L2 while the other streams past it (all 14 columns of
    // 8192x3584x3584: 130.8 us, 8 of them 133.6; 2 columns with all 16 rows of
    // 4096x3584x7168: 129.0, 8 columns 131.9), else about a square of tiles at
    // work (8192x3584x7168: 8 columns 264.7, 28 270.8, 2 269.3).
    int band = q.tiles_n <= 16 ? q.tiles_n : q.tiles_m <= 16 ? 2 : 8;
    // With few rows, as many tiles as pairs in a band (512x3584x16384 42.4 us, by
    // the line above 43.1; with 8 rows of tiles, 2048x7168x7168, 113.8 and 109.3).
    const int least = ceil_div(pairs, q.tiles_m);
    band = q.tiles_m < 8 && band < least ? least : band;
    q.band = band < q.tiles_n ? band : q.tiles_n;
}

// Who takes which items when there are few of them and their products'
// contractions differ: the longest first, each to the pair with the least so
// far.  (Items in turn leave some pairs with two long ones: dx and dW of
// 2050x896x3584 then take 89 k-blocks where this takes 66.)  No item is shorter
// than a tile's epilogue, `drain` k-blocks.
void deal_items(GemmArgs &a, int pairs, int drain) {
    // a heap of the pairs, the least loaded (then the lowest) on top
    int heap[kGemmMaxPairs];
    for (int j = 0; j < pairs; ++j) heap[j] = j;
    auto add_to_top = [&](int cost) {
        const int key = heap[0] + cost * kGemmMaxPairs;
        int i = 0;
        for (;;) {
            int c = 2 * i + 1;
            if (c >= pairs) break;
            if (c + 1 < pairs && heap[c + 1] < heap[c]) ++c;
            if (heap[c] >= key) break;
            heap[i] = heap[c];
            i = c;
        }
        heap[i] = key;
    };
    a.listed = 1;
    for (int c = 0; c < a.nprob; ++c) {
        const int items = (c + 1 < a.nprob ? a.p[c + 1].item_base : a.items) - a.p[c].item_base;
        const int blocks = ceil_div(a.p[c].kblocks, a.p[c].splits), cost = blocks < drain ? drain : blocks;
        for (int j = 0; j < pairs; ++j) a.count[c][j] = 0;
        for (int i = 0; i < items; ++i) {
            ++a.count[c][heap[0] % kGemmMaxPairs];
            add_to_top(cost);
        }
        int at = 0;
        for (int j = 0; j < pairs; ++j) a.first[c][j] = (uint16_t)at, at += a.count[c][j];
    }
}

// Launch `count` products with one epilogue and, when pair tiles are split,
// the kernels that finish them.  `more`: another kernel of the call follows;
// `chained`: the one before is a product that does not write the B of this
// launch's NT and NN products.
route_status run(const route_layer *p, int epi, Prod *w, int count, const Choice &ch, bool chained,
                 bool more, cudaStream_t stream) {
    GemmMaps maps;
    GemmArgs a;
    memset(&a, 0, offsetof(GemmArgs, first));
    a.nprob = count;
    a.splits = ch.splits[0];
    a.fp16 = p->type == kFp16;
    a.timeout_ns = p->timeout_ns;
    a.status = p->words;
    a.test_stall = p->test_stall;

    struct {
        const void *ptr;
        long long ld, inner, outer;
        uint32_t box;
    } made[kGemmMaxMaps];
    int nmaps = 0;
    route_status st = ROUTE_OK;
    // The map of `o` [outer, inner] in boxes of 64 x box_outer; operands that
    // two products share have one.
    auto map = [&](const Operand &o, long long inner, long long outer, uint32_t box, const char *what) {
        for (int i = 0; i < nmaps; ++i)
            if (made[i].ptr == o.p && made[i].ld == o.ld && made[i].inner == inner &&
                made[i].outer == outer && made[i].box == box)
                return (uint8_t)i;
        if (st == ROUTE_OK)
            st = api_encode_operand(&maps.m[nmaps], o.p, a.fp16, (uint64_t)inner, (uint64_t)outer,
                                    (uint64_t)(outer > 1 ? o.ld : up8(inner)), 64, box, what);
        made[nmaps] = {o.p, o.ld, inner, outer, box};
        return (uint8_t)nmaps++;
    };

    const int width = ch.small ? kSmallTile : ch.bn;
    const int tile_rows = ch.small ? ch.bn : kGemmBM, tile_cols = epi == kEpiGated ? width / 2 : width;
    const uint32_t cta_rows = ch.small ? (uint32_t)ch.bn : 128u;  // A rows a CTA loads
    const uint32_t cta_cols = ch.small ? (uint32_t)kSmallTile : (uint32_t)ch.bn / 2;
    // the longest items first
    auto item_blocks = [&](const Prod &x) { return ceil_div(x.kblocks(), ch.splits[x.id]); };
    for (int i = 1; i < count; ++i)
        for (int j = i; j > 0 && item_blocks(w[j]) > item_blocks(w[j - 1]); --j) {
            const Prod t = w[j];
            w[j] = w[j - 1], w[j - 1] = t;
        }
    float *part = reinterpret_cast<float *>(p->scratch + p->o_part);
    int unfinished = 0;
    for (int i = 0; i < count; ++i) {
        GemmProblem &q = a.p[i];
        const Prod &x = w[i];
        q.e = x.e;
        q.e.M = x.M, q.e.N = x.N;
        q.form = x.form;
        q.kblocks = x.kblocks(), q.kswitch = x.kblocks() / x.terms;
        // A box is no higher than its tensor (one that is loads slowly, 98
        // against 25 us at 8x3584x7168).
        const uint32_t box = (uint32_t)x.M >= cta_rows ? cta_rows : (uint32_t)up8(x.M);
        q.a_bytes = (x.form == kFormTT ? cta_rows : box) * 64 * 2;
        for (int t = 0; t < x.terms; ++t) {
            if (x.form == kFormTT)
                q.a[t] = map(x.a[t], x.M, x.K, 64, "x");
            else
                q.a[t] = map(x.a[t], x.K, x.M, box, "rows' operand");
            if (x.form == kFormNN)
                q.b[t][0] = map(x.b[t], x.K, x.N, cta_cols, "W");
            else
                q.b[t][0] = map(x.b[t], x.N, x.K, 64, "columns' operand");
            q.b[t][1] = epi == kEpiGated ? map(x.b[1], x.N, x.K, 64, "W_up") : q.b[t][0];
        }
        set_tiles(q, tile_rows, tile_cols, p->pairs);
        q.item_base = a.items;
        q.splits = ch.splits[x.id];
        a.items += q.tiles_m * q.tiles_n * (ch.small ? 1 : q.splits);
        if (!ch.small && q.splits > 1) {
            q.e.part = part;
            q.e.ld_part = up16(x.N) * (epi == kEpiGated ? 2 : 1);
            part += (size_t)q.splits * x.M * q.e.ld_part;
            ++unfinished;
        }
    }
    if (st != ROUTE_OK) return st;
    if (ch.small) {
        a.trigger = more;
        const cudaError_t e = small_launch(epi, ch.bn, maps, a, chained, stream);
        return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "product kernel launch");
    }
    a.pairs = a.items < p->pairs ? a.items : p->pairs;
    if (count > 1 && a.items <= 4 * p->pairs && p->pairs <= kGemmMaxPairs) deal_items(a, a.pairs, ch.bn == 256 ? 7 : 5);
    a.trigger = more || unfinished > 0;
    const int form = w[0].form == kFormNT ? kFormNT : epi == kEpiDGate ? kFormNN : kFormMixed;
    cudaError_t e = gemm_launch(form, epi, ch.bn, maps, a, stream);
    if (e != cudaSuccess) return cuda_fail(e, "product kernel launch");
    for (int i = 0; i < count; ++i)
        if (a.p[i].splits > 1) {
            FinishArgs f;
            f.splits = a.p[i].splits;
            f.trigger = more || --unfinished > 0;
            f.e = a.p[i].e;
            e = gemm_finish_launch(epi, f, stream);
            if (e != cudaSuccess) return cuda_fail(e, "product finish kernel launch");
        }
    return ROUTE_OK;
}

// A product whose result goes to out[M, N].
Prod product(const route_layer *p, int form, int M, int N, int K, const Operand &a, const Operand &b,
             void *out, long long ld_out, int out_type) {
    Prod w;
    memset(static_cast<void *>(&w), 0, sizeof w);
    w.form = form, w.M = M, w.N = N, w.terms = 1, w.K = K;
    w.a[0] = a, w.b[0] = b;
    w.e.out = out;
    w.e.ld_out = M > 1 ? ld_out : up16(N);
    w.e.out_type = out_type;
    w.e.bias_type = p->type;
    w.e.vec = vec_bits(out, w.e.ld_out, nullptr, nullptr, 0, out_type, nullptr);
    return w;
}

// out[M, N] = act(A[M, K] W[K, N] + bias) + residual.
route_status forward_product(const route_layer *p, ChoiceSlot slot, const Operand &A, const Operand &W, int M, int K,
                             int N, int act, const void *bias, const void *residual, int64_t ld_res,
                             void *out, int64_t ld_out, int out_type, float *saved, bool chained,
                             cudaStream_t stream) {
    Prod w = product(p, kFormNT, M, N, K, A, W, out, ld_out, out_type);
    w.e.bias = bias;
    w.e.residual = residual;
    w.e.ld_res = M > 1 ? ld_res : up16(N);
    w.e.act = act;
    w.e.saved = saved, w.e.ld_saved = up16(N);
    w.e.vec = vec_bits(out, w.e.ld_out, nullptr, residual, w.e.ld_res, out_type, bias);
    const int epi = act == kActNone ? kEpiLinear : kEpiAct;
    return run(p, epi, &w, 1, choice_of(p, slot, M, epi, &w, 1), chained, false, stream);
}

// A backward pass's products: dx (all[0]) and the weights' gradients, those
// whose result is wanted.  One launch, unless the contractions (over the
// widths for dx, over the rows for the others) differ so much that no one
// way to cut them suits both.  What is chosen goes by all of them, so that a
// gradient's bits do not depend on which others are asked for.  `more`:
// another kernel of the call follows.
route_status backward_products(const route_layer *p, int rows, Prod *all, int count, bool chained,
                               bool more, cudaStream_t stream) {
    for (int i = 0; i < count; ++i) all[i].id = i;
    const Choice &one = choice_of(p, kSlotBackward, rows, kEpiLinear, all, count);
    const Choice &input = choice_of(p, kSlotInput, rows, kEpiLinear, all, 1);
    const Choice &weights = choice_of(p, kSlotWeights, rows, kEpiLinear, all + 1, count - 1);
    Prod w[kGemmMaxProblems];
    int n = 0;
    // (the second launch's start hides behind the first, but for 1.4 us: 16x3584x7168
    // 27.6 us in two launches, 32.8 in one; 2050x896x3584 25.5 in one, 33.2 in two)
    if (input.us + weights.us + 1.4 < one.us) {
        Prod *dx = all[0].e.out ? all : nullptr;
        for (int i = 1; i < count; ++i)
            if (all[i].e.out) w[n] = all[i], w[n++].id = i - 1;
        route_status st;
        if (dx && (st = run(p, kEpiLinear, dx, 1, input, chained, more || n > 0, stream)) != ROUTE_OK) return st;
        return n ? run(p, kEpiLinear, w, n, weights, false, more, stream) : ROUTE_OK;
    }
    for (int i = 0; i < count; ++i)
        if (all[i].e.out) w[n++] = all[i];
    return n ? run(p, kEpiLinear, w, n, one, chained, more, stream) : ROUTE_OK;
}

route_status zero_matrix(void *p, int64_t ld, int rows, int cols, int esize, cudaStream_t stream) {
    if (!p) return ROUTE_OK;
    const cudaError_t e = cudaMemset2DAsync(p, (size_t)(rows > 1 ? ld : cols) * esize, 0,
                                            (size_t)cols * esize, (size_t)rows, stream);
    return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "cudaMemset2DAsync");
}

}  // namespace

namespace route {

// ---- plans ------------------------------------------------------------------------

route_status layer_finish_prepare(route_layer *p, int device, route_layer **out) {
    DeviceGuard guard(device);
    if (guard.err != cudaSuccess) {
        delete p;
        return cuda_fail(guard.err, "cudaSetDevice");
    }
    cudaDeviceProp prop;
    cudaError_t e = cudaGetDeviceProperties(&prop, device);
    route_status st = ROUTE_OK;
    const bool products = p->kind == kLinear || p->kind == kGated;
    if (e != cudaSuccess) {
        st = cuda_fail(e, "cudaGetDeviceProperties");
    } else if (prop.major != 10 || prop.minor != 3) {
        st = api_fail(ROUTE_ERR_DEVICE, "device %d is sm_%d%d; this library is built for sm_103a only",
                      device, prop.major, prop.minor);
    } else if (products && ((size_t)gemm_smem_bytes() > prop.sharedMemPerBlockOptin ||
                            (size_t)small_smem_bytes() > prop.sharedMemPerBlockOptin ||
                            prop.multiProcessorCount < 2)) {
        st = api_fail(ROUTE_ERR_DEVICE, "the product kernels need %d B of shared memory per block",
                      gemm_smem_bytes());
    } else if (p->kind == kExpertBlocks && ((size_t)experts_smem_bytes() > prop.sharedMemPerBlockOptin ||
                                            prop.multiProcessorCount < 2)) {
        st = api_fail(ROUTE_ERR_DEVICE, "the experts' kernels need %d B of shared memory per block",
                      experts_smem_bytes());
    } else if ((e = p->kind == kNorm           ? norm_configure()
                    : p->kind == kDispatch     ? sort_configure()
                    : p->kind == kExpertBlocks ? experts_configure()
                                               : cudaSuccess) != cudaSuccess ||
               (p->kind == kExpertBlocks && (e = experts_small_configure()) != cudaSuccess) ||
               (products && ((e = gemm_configure()) != cudaSuccess || (e = small_configure()) != cudaSuccess))) {
        st = cuda_fail(e, "cudaFuncSetAttribute");
    }
    if (st != ROUTE_OK) {
        delete p;
        return st;
    }
    p->device = device;
    p->sms = prop.multiProcessorCount;
    p->pairs = p->sms / 2;
    p->timeout_ns = kTimeoutNs;
    if (p->kind == kDispatch) p->sort = sort_shape();

    size_t at = 0;
    auto area = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) & ~size_t(255);
        return o;
    };
    const size_t R = (size_t)p->rows;
    auto copy = [&](size_t rows, int cols) { return area(cols % 8 ? rows * up8(cols) * 2 : 0); };
    if (p->kind == kNorm) {
        p->o_part = area(norm_part_floats(p->k, p->sms) * 4);
    } else if (p->kind == kExpertBlocks) {
        p->o_h = area(R * up16(p->f) * 2);
        if (p->train) {
            p->o_dg = area(R * up16(p->f) * 2);
            p->o_du = area(R * up16(p->f) * 2);
        }
    } else if (products) {
        p->o_part = area(2 * (size_t)p->pairs * kTilePartBytes);
        p->o_x = copy(R, p->k);
        if (p->kind == kLinear) {
            p->o_w[0] = copy(p->k, p->n);
            p->o_dg = area(p->train && (p->act != kActNone || p->n % 8) ? R * up16(p->n) * 2 : 0);
            p->o_sum = area(p->train ? dz_part_floats(p->n) * 4 : 0);
        } else {
            p->o_w[0] = copy(p->k, p->f);
            p->o_w[1] = copy(p->k, p->f);
            p->o_w[2] = copy(p->f, p->n);
            p->o_h = area(R * up16(p->f) * 2);
            if (p->train) {
                p->o_dout = copy(R, p->n);
                p->o_dg = area(R * up16(p->f) * 2);
                p->o_du = area(R * up16(p->f) * 2);
            }
        }
    }
    p->scratch_bytes = at;
    if ((e = cudaMalloc(&p->words, kWords * sizeof(unsigned))) != cudaSuccess ||
        (e = cudaMemset(p->words, 0, kWords * sizeof(unsigned))) != cudaSuccess ||
        (e = cudaMalloc(&p->scratch, at ? at : 256)) != cudaSuccess) {
        if (p->words) cudaFree(p->words);
        delete p;
        return cuda_fail(e, "plan memory");
    }
    *out = p;
    return ROUTE_OK;
}

route_status layer_check_prepare(int rows, int max_rows, std::initializer_list<int> widths, int max_width,
                                 int type, bool fp32, int act, route_layer **out) {
    if (!out) return api_fail(ROUTE_ERR_NULL, "out must be non-NULL");
    *out = nullptr;
    if (rows < 1 || rows > max_rows)
        return api_fail(ROUTE_ERR_ROWS, "rows %d outside 1-%d", rows, max_rows);
    for (int w : widths)
        if (w < 1 || w > max_width)
            return api_fail(ROUTE_ERR_PLAN, "width %d outside 1-%d", w, max_width);
    if (type != kBf16 && type != kFp16 && !(fp32 && type == kFp32))
        return api_fail(ROUTE_ERR_MODE, "type %d is not one of this operator's", type);
    if (act < 0 || act >= kActCount) return api_fail(ROUTE_ERR_MODE, "unknown activation %d", act);
    return ROUTE_OK;
}

route_layer *layer_new_plan(LayerKind kind, int rows, int type, int act, int train) {
    route_layer *p = new (std::nothrow) route_layer();  // all zero
    if (!p) return nullptr;
    p->kind = kind;
    p->rows = rows;
    p->type = p->out_type = type;
    p->act = act;
    p->train = train != 0;
    return p;
}

}  // namespace route

extern "C" {

route_status route_norm_prepare(int rows, int dim, int type, int device, route_layer **out) {
    route_status st = layer_check_prepare(rows, ROUTE_LAYER_MAX_ROWS, {dim}, ROUTE_NORM_MAX_WIDTH, type, true, 0, out);
    if (st != ROUTE_OK) return st;
    route_layer *p = layer_new_plan(kNorm, rows, type, 0, 0);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = dim;
    return layer_finish_prepare(p, device, out);
}

route_status route_linear_prepare(int rows, int k, int n, int type, int out_type, int act,
                                  int train, int device, route_layer **out) {
    route_status st = layer_check_prepare(rows, ROUTE_LAYER_MAX_ROWS, {k, n}, ROUTE_LAYER_MAX_WIDTH, type, false, act, out);
    if (st != ROUTE_OK) return st;
    if (out_type != type && out_type != kFp32)
        return api_fail(ROUTE_ERR_MODE, "out_type %d is neither the plan's type nor FP32", out_type);
    if (train && out_type != type)
        return api_fail(ROUTE_ERR_PLAN, "a training plan's results have the plan's type");
    route_layer *p = layer_new_plan(kLinear, rows, type, act, train);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = k, p->n = n;
    p->out_type = out_type;
    return layer_finish_prepare(p, device, out);
}

route_status route_gated_prepare(int rows, int k, int f, int n, int type, int act, int train,
                                 int device, route_layer **out) {
    route_status st = layer_check_prepare(rows, ROUTE_LAYER_MAX_ROWS, {k, f, n}, ROUTE_LAYER_MAX_WIDTH, type, false, act, out);
    if (st != ROUTE_OK) return st;
    route_layer *p = layer_new_plan(kGated, rows, type, act, train);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = k, p->f = f, p->n = n;
    return layer_finish_prepare(p, device, out);
}

route_status route_layer_destroy(route_layer *p) {
    if (!p) return ROUTE_OK;
    DeviceGuard guard(p->device);
    const cudaError_t e = cudaDeviceSynchronize();
    cudaFree(p->words);
    cudaFree(p->scratch);
    delete p;
    return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "cudaDeviceSynchronize");
}

route_status route_layer_status(const route_layer *p) {
    if (!p) return api_fail(ROUTE_ERR_NULL, "plan is NULL");
    DeviceGuard guard(p->device);
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
    unsigned w = 0;
    if ((e = cudaMemcpy(&w, p->words, sizeof w, cudaMemcpyDeviceToHost)) != cudaSuccess ||
        (e = cudaMemset(p->words, 0, sizeof w)) != cudaSuccess)
        return cuda_fail(e, "status word");
    if (w & kStatusTimeout)
        return api_fail(ROUTE_ERR_DEVICE_TIMEOUT, "a kernel gave up waiting; its outputs are invalid");
    return ROUTE_OK;
}

int64_t route_layer_saved_bytes(const route_layer *p, int rows) {
    if (!p) return -1;
    if (rows <= 0 || !p->train) return 0;
    if (p->kind == kLinear) return p->act == kActNone ? 0 : (int64_t)rows * up16(p->n) * 4;
    if (p->kind == kGated || p->kind == kExpertBlocks)
        return (int64_t)saved_h(p, rows) + (int64_t)rows * up16(p->f) * 2;
    return 0;
}

route_status route_layer_test_stall(route_layer *p, int enable, uint64_t timeout_ns) {
    if (!p) return api_fail(ROUTE_ERR_NULL, "plan is NULL");
    p->test_stall = enable != 0;
    p->timeout_ns = enable ? timeout_ns : kTimeoutNs;
    return ROUTE_OK;
}

route_status route_norm_forward(const route_layer *p, int rows, const void *x, int64_t ld_x,
                                const void *gamma, const void *beta, float eps, void *y,
                                int64_t ld_y, float *stats, void *stream) {
    route_status st = check_plan(p, kNorm, rows);
    if (st != ROUTE_OK) return st;
    std::lock_guard<std::mutex> lock(p->calls);
    if (!(eps >= 0.f) || std::isinf(eps))
        return api_fail(ROUTE_ERR_PLAN, "eps must be finite and not negative");
    if (rows == 0) return ROUTE_OK;
    const int es = layer_esize(p->type);
    if ((st = check_mats({{"x", x, ld_x, rows, p->k, es, false},
                          {"y", y, ld_y, rows, p->k, es, false}})) != ROUTE_OK ||
        (st = check_vec("gamma", gamma, es)) != ROUTE_OK ||
        (st = check_vec("beta", beta, es)) != ROUTE_OK ||
        (st = check_vec("stats", stats, 8)) != ROUTE_OK)
        return st;
    NormArgs a = {};
    a.rows = rows, a.dim = p->k, a.type = p->type;
    a.eps = eps;
    a.x = x, a.ld_x = rows > 1 ? ld_x : p->k;
    a.gamma = gamma, a.beta = beta;
    a.y = y, a.ld_y = rows > 1 ? ld_y : p->k;
    a.stats = stats;
    a.sms = p->sms;
    DeviceGuard guard(p->device);
    const cudaError_t e = norm_forward_launch(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "norm kernel launch");
}

route_status route_norm_backward(const route_layer *p, int rows, const void *dy, int64_t ld_dy,
                                 const void *x, int64_t ld_x, const void *gamma,
                                 const float *stats, void *dx, int64_t ld_dx, void *dgamma,
                                 void *dbeta, void *stream) {
    route_status st = check_plan(p, kNorm, rows);
    if (st != ROUTE_OK) return st;
    std::lock_guard<std::mutex> lock(p->calls);
    const int es = layer_esize(p->type);
    if ((st = check_vec("gamma", gamma, es)) != ROUTE_OK ||
        (st = check_vec("dgamma", dgamma, es)) != ROUTE_OK ||
        (st = check_vec("dbeta", dbeta, es)) != ROUTE_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard guard(p->device);
    if (rows == 0) {
        if ((st = zero_matrix(dgamma, p->k, 1, p->k, es, s)) != ROUTE_OK) return st;
        return zero_matrix(dbeta, p->k, 1, p->k, es, s);
    }
    if ((st = check_mats({{"dy", dy, ld_dy, rows, p->k, es, false},
                          {"x", x, ld_x, rows, p->k, es, false}})) != ROUTE_OK ||
        (dx && (st = check_mat({"dx", dx, ld_dx, rows, p->k, es, false})) != ROUTE_OK))
        return st;
    if (!stats) return api_fail(ROUTE_ERR_NULL, "stats must be non-NULL");
    if ((st = check_vec("stats", stats, 8)) != ROUTE_OK) return st;
    if (!dx && !dgamma && !dbeta) return ROUTE_OK;
    NormArgs a = {};
    a.rows = rows, a.dim = p->k, a.type = p->type;
    a.x = x, a.ld_x = rows > 1 ? ld_x : p->k;
    a.gamma = gamma;
    a.stats = const_cast<float *>(stats);
    a.dy = dy, a.ld_dy = rows > 1 ? ld_dy : p->k;
    a.dx = dx, a.ld_dx = rows > 1 ? ld_dx : p->k;
    a.dgamma = dgamma, a.dbeta = dbeta;
    a.part = reinterpret_cast<float *>(p->scratch + p->o_part);
    a.sms = p->sms;
    const cudaError_t e = norm_backward_launch(a, s);
    return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "norm gradient kernel launch");
}

route_status route_linear_forward(const route_layer *p, int rows, const void *x, int64_t ld_x,
                                  const void *W, int64_t ld_W, const void *bias,
                                  const void *residual, int64_t ld_residual, void *out,
                                  int64_t ld_out, void *saved, void *stream) {
    route_status st = check_plan(p, kLinear, rows);
    if (st != ROUTE_OK) return st;
    std::lock_guard<std::mutex> lock(p->calls);
    if (saved && (!p->train || p->act == kActNone))
        return api_fail(ROUTE_ERR_PLAN, "the plan saves nothing (no training, or no activation)");
    if (rows == 0) return ROUTE_OK;
    const int es = layer_esize(p->out_type);
    if ((st = check_mats({{"x", x, ld_x, rows, p->k, 2, true},
                          {"W", W, ld_W, p->k, p->n, 2, true},
                          {"out", out, ld_out, rows, p->n, es, false}})) != ROUTE_OK ||
        (residual &&
         (st = check_mat({"residual", residual, ld_residual, rows, p->n, es, false})) != ROUTE_OK) ||
        (st = check_vec("bias", bias, 2)) != ROUTE_OK ||
        (st = check_vec("saved", saved, 32)) != ROUTE_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard guard(p->device);
    Copies copies(p);
    const Operand ox = copies.operand(x, ld_x, rows, p->k, p->o_x);
    const Operand ow = copies.operand(W, ld_W, p->k, p->n, p->o_w[0]);
    if ((st = copies.launch(s)) != ROUTE_OK) return st;
    return forward_product(p, kSlotForward, ox, ow, rows, p->k, p->n, p->act, bias, residual, ld_residual, out,
                           ld_out, p->out_type, static_cast<float *>(saved), false, s);
}

route_status route_linear_backward(const route_layer *p, int rows, const void *dout,
                                   int64_t ld_dout, const void *x, int64_t ld_x, const void *W,
                                   int64_t ld_W, const void *saved, void *dx, int64_t ld_dx,
                                   void *dW, int64_t ld_dW, void *dbias, void *stream) {
    route_status st = check_plan(p, kLinear, rows);
    if (st != ROUTE_OK) return st;
    std::lock_guard<std::mutex> lock(p->calls);
    if (!p->train) return api_fail(ROUTE_ERR_PLAN, "the plan was prepared without train");
    if (dW && (st = check_mat({"dW", dW, ld_dW, p->k, p->n, 2, false})) != ROUTE_OK) return st;
    if ((st = check_vec("dbias", dbias, 2)) != ROUTE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard guard(p->device);
    if (rows == 0) {
        if ((st = zero_matrix(dW, ld_dW, p->k, p->n, 2, s)) != ROUTE_OK) return st;
        return zero_matrix(dbias, p->n, 1, p->n, 2, s);
    }
    if ((st = check_mat({"dout", dout, ld_dout, rows, p->n, 2, true})) != ROUTE_OK ||
        (dW && (st = check_mat({"x", x, ld_x, rows, p->k, 2, true})) != ROUTE_OK) ||
        (dx && ((st = check_mat({"W", W, ld_W, p->k, p->n, 2, true})) != ROUTE_OK ||
                (st = check_mat({"dx", dx, ld_dx, rows, p->k, 2, false})) != ROUTE_OK)))
        return st;
    if (p->act != kActNone && !saved) return api_fail(ROUTE_ERR_NULL, "saved must be non-NULL");
    if ((st = check_vec("saved", saved, 32)) != ROUTE_OK) return st;
    if (!dx && !dW && !dbias) return ROUTE_OK;

    // dz: dout itself where there is no activation and TMA can read it
    Operand dz = {dout, rows > 1 ? ld_dout : p->n};
    const bool in_place = p->act == kActNone && aligned(dout, 16) &&
                          (rows > 1 ? ld_dout % 8 == 0 : p->n % 8 == 0);
    const bool make_dz = !in_place && (dx || dW);
    DzArgs a = {};
    if (make_dz || dbias) {
        a.rows = rows, a.n = p->n, a.type = p->type, a.act = p->act;
        a.dout = dout, a.ld_dout = dz.ld;
        if (p->act != kActNone) a.z = static_cast<const float *>(saved), a.ld_z = up16(p->n);
        if (make_dz) {
            a.dz = p->scratch + p->o_dg, a.ld_dz = up16(p->n);
            dz = {a.dz, a.ld_dz};
        }
        a.sums_only = in_place;
        a.dbias = dbias;
        a.part = reinterpret_cast<float *>(p->scratch + p->o_sum);
        const cudaError_t e = dz_launch(a, s);
        if (e != cudaSuccess) return cuda_fail(e, "pre-activation gradient kernel launch");
    }
    auto sums = [&](bool after) {
        const cudaError_t e = dbias ? bias_launch(a, after, s) : cudaSuccess;
        return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "bias gradient kernel launch");
    };
    if (!dx && !dW) return sums(false);
    // dx = dz W^T and dW = x^T dz
    Copies copies(p);
    const Operand ox = dW ? copies.operand(x, ld_x, rows, p->k, p->o_x) : Operand{nullptr, 0};
    const Operand ow = dx ? copies.operand(W, ld_W, p->k, p->n, p->o_w[0]) : Operand{nullptr, 0};
    if ((st = copies.launch(s)) != ROUTE_OK) return st;
    Prod all[2] = {product(p, kFormNN, rows, p->k, p->n, dz, ow, dx, ld_dx, p->type),
                   product(p, kFormTT, p->k, p->n, rows, ox, dz, dW, ld_dW, p->type)};
    // dz's kernel, if it was the last one, waited and does not write W
    st = backward_products(p, rows, all, 2, make_dz && copies.args.count == 0, dbias != nullptr, s);
    return st != ROUTE_OK ? st : sums(true);
}

route_status route_gated_forward(const route_layer *p, int rows, const void *x, int64_t ld_x,
                                 const void *W_gate, int64_t ld_gate, const void *W_up,
                                 int64_t ld_up, const void *W_down, int64_t ld_down,
                                 const void *residual, int64_t ld_residual, void *out,
                                 int64_t ld_out, void *saved, void *stream) {
    route_status st = check_plan(p, kGated, rows);
    if (st != ROUTE_OK) return st;
    std::lock_guard<std::mutex> lock(p->calls);
    if (saved && !p->train) return api_fail(ROUTE_ERR_PLAN, "the plan was prepared without train");
    if (rows == 0) return ROUTE_OK;
    if ((st = check_mats({{"x", x, ld_x, rows, p->k, 2, true},
                          {"W_gate", W_gate, ld_gate, p->k, p->f, 2, true},
                          {"W_up", W_up, ld_up, p->k, p->f, 2, true},
                          {"W_down", W_down, ld_down, p->f, p->n, 2, true},
                          {"out", out, ld_out, rows, p->n, 2, false}})) != ROUTE_OK ||
        (residual &&
         (st = check_mat({"residual", residual, ld_residual, rows, p->n, 2, false})) != ROUTE_OK) ||
        (st = check_vec("saved", saved, 32)) != ROUTE_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard guard(p->device);
    Copies copies(p);
    const Operand ox = copies.operand(x, ld_x, rows, p->k, p->o_x);
    const Operand og = copies.operand(W_gate, ld_gate, p->k, p->f, p->o_w[0]);
    const Operand ou = copies.operand(W_up, ld_up, p->k, p->f, p->o_w[1]);
    const Operand od = copies.operand(W_down, ld_down, p->f, p->n, p->o_w[2]);
    if ((st = copies.launch(s)) != ROUTE_OK) return st;
    // h = act(x W_gate) * (x W_up): one kernel for both projections
    const long long ldf = up16(p->f);
    uint8_t *h = saved ? static_cast<uint8_t *>(saved) + saved_h(p, rows) : p->scratch + p->o_h;
    Prod w = product(p, kFormNT, rows, p->f, p->k, ox, og, h, ldf, p->type);
    w.b[1] = ou;
    w.e.act = p->act;
    w.e.saved = static_cast<float *>(saved), w.e.ld_saved = ldf;
    w.e.saved2 = saved ? w.e.saved + (size_t)rows * ldf : nullptr;
    if ((st = run(p, kEpiGated, &w, 1, choice_of(p, kSlotForward, rows, kEpiGated, &w, 1), false, true, s)) != ROUTE_OK) return st;
    return forward_product(p, kSlotDown, {h, ldf}, od, rows, p->f, p->n, kActNone, nullptr, residual,
                           ld_residual, out, ld_out, p->type, nullptr, true, s);
}

route_status route_gated_backward(const route_layer *p, int rows, const void *dout,
                                  int64_t ld_dout, const void *x, int64_t ld_x, const void *W_gate,
                                  int64_t ld_gate, const void *W_up, int64_t ld_up,
                                  const void *W_down, int64_t ld_down, const void *saved, void *dx,
                                  int64_t ld_dx, void *dW_gate, int64_t ld_dgate, void *dW_up,
                                  int64_t ld_dup, void *dW_down, int64_t ld_ddown, void *stream) {
    route_status st = check_plan(p, kGated, rows);
    if (st != ROUTE_OK) return st;
    std::lock_guard<std::mutex> lock(p->calls);
    if (!p->train) return api_fail(ROUTE_ERR_PLAN, "the plan was prepared without train");
    const Mat grads[3] = {{"dW_gate", dW_gate, ld_dgate, p->k, p->f, 2, false},
                          {"dW_up", dW_up, ld_dup, p->k, p->f, 2, false},
                          {"dW_down", dW_down, ld_ddown, p->f, p->n, 2, false}};
    for (const Mat &m : grads)
        if (m.p && (st = check_mat(m)) != ROUTE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard guard(p->device);
    if (rows == 0) {
        for (const Mat &m : grads)
            if ((st = zero_matrix(const_cast<void *>(m.p), m.ld, m.rows, m.cols, 2, s)) != ROUTE_OK)
                return st;
        return ROUTE_OK;
    }
    const bool pre = dx || dW_gate || dW_up;  // the pre-activations' gradients are wanted
    if (!pre && !dW_down) return ROUTE_OK;
    if ((st = check_mat({"dout", dout, ld_dout, rows, p->n, 2, true})) != ROUTE_OK ||
        (pre && (st = check_mat({"W_down", W_down, ld_down, p->f, p->n, 2, true})) != ROUTE_OK) ||
        ((dW_gate || dW_up) && (st = check_mat({"x", x, ld_x, rows, p->k, 2, true})) != ROUTE_OK) ||
        (dx && ((st = check_mat({"W_gate", W_gate, ld_gate, p->k, p->f, 2, true})) != ROUTE_OK ||
                (st = check_mat({"W_up", W_up, ld_up, p->k, p->f, 2, true})) != ROUTE_OK ||
                (st = check_mat({"dx", dx, ld_dx, rows, p->k, 2, false})) != ROUTE_OK)))
        return st;
    if (!saved) return api_fail(ROUTE_ERR_NULL, "saved must be non-NULL");
    if ((st = check_vec("saved", saved, 32)) != ROUTE_OK) return st;

    const long long ldf = up16(p->f);
    const bool weights = dW_gate || dW_up || dW_down;
    const Operand none = {nullptr, 0};
    Copies copies(p);
    const Operand dy = copies.operand(dout, ld_dout, rows, p->n, p->o_dout);
    const Operand od = pre ? copies.operand(W_down, ld_down, p->f, p->n, p->o_w[2]) : none;
    const Operand og = dx ? copies.operand(W_gate, ld_gate, p->k, p->f, p->o_w[0]) : none;
    const Operand ou = dx ? copies.operand(W_up, ld_up, p->k, p->f, p->o_w[1]) : none;
    const Operand ox = dW_gate || dW_up ? copies.operand(x, ld_x, rows, p->k, p->o_x) : none;
    if ((st = copies.launch(s)) != ROUTE_OK) return st;
    const Operand dg = {p->scratch + p->o_dg, ldf}, du = {p->scratch + p->o_du, ldf};
    if (pre) {
        // dh = dout W_down^T, turned into dgate and dup in its epilogue
        Prod w = product(p, kFormNN, rows, p->f, p->n, dy, od, const_cast<void *>(dg.p), ldf, p->type);
        w.e.ld_out = ldf;
        w.e.out2 = const_cast<void *>(du.p);
        w.e.act = p->act;
        w.e.saved = static_cast<float *>(const_cast<void *>(saved)), w.e.ld_saved = ldf;
        w.e.saved2 = w.e.saved + (size_t)rows * ldf;
        if ((st = run(p, kEpiDGate, &w, 1, choice_of(p, kSlotDGate, rows, kEpiDGate, &w, 1), false, dx || weights, s)) != ROUTE_OK) return st;
    }
    // dx = dgate W_gate^T + dup W_up^T and the weights' gradients
    const Operand h = {static_cast<const uint8_t *>(saved) + saved_h(p, rows), ldf};
    Prod all[4] = {product(p, kFormNN, rows, p->k, p->f, dg, og, dx, ld_dx, p->type),
                   product(p, kFormTT, p->k, p->f, rows, ox, dg, dW_gate, ld_dgate, p->type),
                   product(p, kFormTT, p->k, p->f, rows, ox, du, dW_up, ld_dup, p->type),
                   product(p, kFormTT, p->f, p->n, rows, h, dy, dW_down, ld_ddown, p->type)};
    all[0].terms = 2, all[0].a[1] = du, all[0].b[1] = ou;
    return backward_products(p, rows, all, 4, pre, false, s);
}

}  // extern "C"
