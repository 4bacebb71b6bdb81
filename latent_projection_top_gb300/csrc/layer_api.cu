// C ABI of the layer operators: plans, argument checks, the choice of tile
// and split for every product, and the launches.  Every check happens on the
// host before anything is enqueued.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <initializer_list>
#include <new>

#include "api_util.h"
#include "layer.cuh"
#include "layer_math.cuh"
#include "route_layer.h"

using namespace route;

namespace {
enum LayerKind { kNorm, kLinear, kGated };
}

struct route_layer {
    LayerKind kind;
    int rows, k, f, n;
    int type, out_type, act, train;
    int device, sms, pairs;
    int test_stall;
    unsigned long long timeout_ns;
    unsigned *words;   // device status word
    uint8_t *scratch;
    size_t scratch_bytes;
    // offsets into scratch (0 size where the plan needs none)
    size_t o_part;     // split partials, or column-sum partials
    size_t o_x, o_w[3], o_dout, o_h, o_dg, o_du;
};

namespace {

constexpr unsigned long long kTimeoutNs = 2000000000ull;
// Split products have at most one item a CTA pair: FP32 partials of a
// 256 x 256 tile each.
constexpr size_t kTilePartBytes = 256 * 256 * 4;

route_status cuda_fail(cudaError_t e, const char *what) {
    return api_fail(ROUTE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    cudaError_t err;
    explicit DeviceGuard(int dev) {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != dev) {
            err = cudaSetDevice(dev);
            changed = err == cudaSuccess;
        }
    }
    ~DeviceGuard() {
        if (changed) cudaSetDevice(prev);
    }
};

long long up8(long long v) { return (v + 7) & ~7ll; }
long long up16(long long v) { return (v + 15) & ~15ll; }
bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---- argument checks ----------------------------------------------------------

// A matrix argument: its name, width and whether a product reads it by TMA.
struct Mat {
    const char *name;
    const void *p;
    int64_t ld;
    int rows, cols, esize;
    bool operand;
};

route_status check_mat(const Mat &m) {
    if (!m.p) return api_fail(ROUTE_ERR_NULL, "%s must be non-NULL", m.name);
    if (!aligned(m.p, (unsigned)m.esize))
        return api_fail(ROUTE_ERR_ALIGN, "%s is not aligned to its element", m.name);
    if (m.rows > 1 && m.ld < m.cols)
        return api_fail(ROUTE_ERR_PLAN, "%s: row stride %lld is less than its %d columns", m.name,
                        (long long)m.ld, m.cols);
    if (m.operand && m.cols % 8 == 0 && (!aligned(m.p, 16) || (m.rows > 1 && m.ld % 8 != 0)))
        return api_fail(ROUTE_ERR_ALIGN,
                        "%s must start on 16 bytes with a row stride that is a multiple of 8", m.name);
    return ROUTE_OK;
}

route_status check_mats(std::initializer_list<Mat> ms) {
    for (const Mat &m : ms)
        if (m.p || m.cols > 0) {
            const route_status st = check_mat(m);
            if (st != ROUTE_OK) return st;
        }
    return ROUTE_OK;
}

route_status check_vec(const char *name, const void *p, int esize) {
    if (p && !aligned(p, (unsigned)esize))
        return api_fail(ROUTE_ERR_ALIGN, "%s is not aligned to its element", name);
    return ROUTE_OK;
}

route_status check_plan(const route_layer *p, LayerKind kind, int rows) {
    if (!p) return api_fail(ROUTE_ERR_NULL, "plan is NULL");
    if (p->kind != kind) return api_fail(ROUTE_ERR_PLAN, "the plan is another operator's");
    if (rows < 0 || rows > p->rows)
        return api_fail(ROUTE_ERR_ROWS, "rows %d outside the plan's 0-%d", rows, p->rows);
    return ROUTE_OK;
}

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
    return v;
}

// ---- products -------------------------------------------------------------------

struct Operand {
    const void *p;
    long long ld;
};

// An operand as TMA can read it: in place, or copied into scratch.
route_status operand(const route_layer *p, const void *src, long long ld, int rows, int cols,
                     size_t scratch, cudaStream_t stream, Operand *out) {
    if (cols % 8 == 0) {
        *out = {src, rows > 1 ? ld : cols};
        return ROUTE_OK;
    }
    const long long ldp = up8(cols);
    if (aligned(src, 16) && ld % 8 == 0 && rows > 1) {
        *out = {src, ld};
        return ROUTE_OK;
    }
    void *dst = p->scratch + scratch;
    const cudaError_t e = repack_launch(src, rows > 1 ? ld : cols, dst, ldp, rows, cols, stream);
    if (e != cudaSuccess) return cuda_fail(e, "operand copy");
    *out = {dst, ldp};
    return ROUTE_OK;
}

// How a launch covers its products: CTA-pair tiles of 256 x bn
// (layer_gemm.cu), or 128-column tiles of bn rows (layer_small.cu), and the
// splits of the contraction.
struct Choice {
    bool small;
    int bn, splits;
};

struct Shape {
    int M, N;  // N: columns of D (gated: hidden columns)
};

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// The choice with the smallest estimated time, from what the kernels measure:
// a k-block of a pair's 256 x 256 tile takes 0.34 us and of a 256 x 128 tile
// 0.30 us; the small tiles are bound by what an SM reads, about 70 bytes a
// nanosecond, or by memory.
Choice choose(const route_layer *p, int form, int epi, const Shape *shape, int count, int kblocks) {
    Choice best = {false, 256, 1};
    double t_best = 1e30, elems = 0;
    int rows = 0;
    for (int i = 0; i < count; ++i) {
        elems += (double)shape[i].M * shape[i].N * (epi == kEpiGated ? 2 : 1);
        rows = rows < shape[i].M ? shape[i].M : rows;
    }
    for (int bn : {256, 128}) {
        long long tiles = 0;
        const int cols = epi == kEpiGated ? bn / 2 : bn;
        for (int i = 0; i < count; ++i)
            tiles += (long long)ceil_div(shape[i].M, kGemmBM) * ceil_div(shape[i].N, cols);
        const int most = tiles >= p->pairs ? 1 : (int)(p->pairs / tiles);
        for (int s = 1; s <= most && (s == 1 || kblocks / s >= 2); ++s) {
            const int waves = ceil_div(tiles * s, p->pairs);
            double t = 7.0 + waves * (ceil_div(kblocks, s) * (bn == 256 ? 0.34 : 0.30));
            if (s > 1) t += 2.5 + elems * 4.0 * (s + 1) / 4e6;
            if (t < t_best) t_best = t, best = {false, bn, s};
        }
    }
    {
        int bn = form == kFormTT ? 64 : 16;
        while (bn < 128 && bn < rows) bn *= 2;
        long long tiles = 0;
        const int cols = epi == kEpiGated ? kSmallTile / 2 : kSmallTile;
        for (int i = 0; i < count; ++i)
            tiles += (long long)ceil_div(shape[i].M, bn) * ceil_div(shape[i].N, cols);
        int s = 1;
        while (s < kSmallMaxSplits && tiles * s * 2 <= 2 * p->sms && s * 2 <= kblocks) s *= 2;
        const double kb_us = (16384 + bn * 128) / 70e3;
        const double t = 5.0 + ceil_div(tiles * s, p->sms) * (ceil_div(kblocks, s) * kb_us + 0.5);
        if (t < t_best) best = {true, bn, s};
    }
    return best;
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
    const int least = ceil_div(pairs, q.tiles_m);  // as many tiles as pairs in a band
    band = q.tiles_m < 8 && band < least ? least : band;
    q.band = band < q.tiles_n ? band : q.tiles_n;
}

struct Product {
    GemmMaps maps;
    GemmArgs args;
    int nmaps = 0;
    bool fp16;
    Product(const route_layer *p) : fp16(p->type == kFp16) {
        memset(&args, 0, sizeof args);
        args.fp16 = fp16;
        args.a_bytes = 128 * 64 * 2;
        args.timeout_ns = p->timeout_ns;
        args.status = p->words;
        args.test_stall = p->test_stall;
    }
    // Rows of the boxes of a K-contiguous A (a tile's rows for one CTA, or
    // what there is of M: a box higher than its tensor loads slowly, 98
    // against 25 us at 8x3584x7168) and of a K-contiguous B.
    uint32_t a_rows(int M, const Choice &ch) {
        const uint32_t most = ch.small ? (uint32_t)ch.bn : 128u;
        const uint32_t r = (uint32_t)M >= most ? most : (uint32_t)up8(M);
        args.a_bytes = r * 64 * 2;
        return r;
    }
    static uint32_t b_rows(const Choice &ch) {
        return ch.small ? (uint32_t)kSmallTile : (uint32_t)ch.bn / 2;
    }
    // A map of `o` [outer, inner] in boxes of box_inner x box_outer.
    route_status map(const Operand &o, long long inner, long long outer, uint32_t box_outer,
                     const char *what, uint8_t *index) {
        *index = (uint8_t)nmaps;
        return api_encode_operand(&maps.m[nmaps++], o.p, fp16, (uint64_t)inner, (uint64_t)outer,
                                  (uint64_t)(outer > 1 ? o.ld : up8(inner)), 64, box_outer, what);
    }
};

// Launch the product(s) and, when pair tiles are split, the kernel(s) that
// finish them.  `more`: another kernel of the call follows; `chained`: the
// one before is a product that does not write this one's B.
route_status run(const route_layer *p, Product &pr, int form, int epi, const Choice &ch,
                 bool chained, bool more, cudaStream_t stream) {
    GemmArgs &a = pr.args;
    const int width = ch.small ? kSmallTile : ch.bn;
    a.splits = ch.splits;
    int items = 0;
    float *part = reinterpret_cast<float *>(p->scratch + p->o_part);
    for (int i = 0; i < a.nprob; ++i) {
        GemmProblem &q = a.p[i];
        set_tiles(q, ch.small ? ch.bn : kGemmBM, epi == kEpiGated ? width / 2 : width, p->pairs);
        q.item_base = items;
        items += q.tiles_m * q.tiles_n * (ch.small ? 1 : ch.splits);
        if (!ch.small && ch.splits > 1) {
            q.e.part = part;
            q.e.ld_part = up16(q.e.N) * (epi == kEpiGated ? 2 : 1);
            part += (size_t)ch.splits * q.e.M * q.e.ld_part;
        }
    }
    a.items = items;
    if (ch.small) {
        if (form == kFormTT) a.a_bytes = (unsigned)ch.bn * 64 * 2;
        a.trigger = more;
        const cudaError_t e = small_launch(form, epi, ch.bn, pr.maps, a, chained, stream);
        return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "product kernel launch");
    }
    a.pairs = items < p->pairs ? items : p->pairs;
    a.trigger = more || ch.splits > 1;
    cudaError_t e = gemm_launch(form, epi, ch.bn, pr.maps, a, stream);
    if (e != cudaSuccess) return cuda_fail(e, "product kernel launch");
    if (ch.splits > 1)
        for (int i = 0; i < a.nprob; ++i) {
            FinishArgs f;
            f.splits = ch.splits;
            f.trigger = more || i + 1 < a.nprob;
            f.e = a.p[i].e;
            e = gemm_finish_launch(epi, f, stream);
            if (e != cudaSuccess) return cuda_fail(e, "product finish kernel launch");
        }
    return ROUTE_OK;
}

Choice choose_one(const route_layer *p, int form, int epi, int M, int N, int kblocks) {
    const Shape s = {M, N};
    return choose(p, form, epi, &s, 1, kblocks);
}

int kblocks_of(int k) { return (k + 63) / 64; }

void set_out(GemmProblem &q, void *out, long long ld_out, int out_type) {
    q.e.out = out;
    q.e.ld_out = q.e.M > 1 ? ld_out : up16(q.e.N);
    q.e.out_type = out_type;
    q.e.vec = vec_bits(q.e.out, q.e.ld_out, nullptr, nullptr, 0, out_type, nullptr);
}

// out[M, N] = epilogue(A[M, K] W[K, N]): A K-contiguous, W N-contiguous.
route_status forward_product(const route_layer *p, const Operand &A, const Operand &W, int M, int K,
                             int N, int act, const void *bias, const void *residual, int64_t ld_res,
                             void *out, int64_t ld_out, int out_type, float *saved, bool chained,
                             cudaStream_t stream) {
    Product pr(p);
    GemmProblem &q = pr.args.p[0];
    pr.args.nprob = 1;
    q.e.M = M, q.e.N = N;
    q.kblocks = q.kswitch = kblocks_of(K);
    set_out(q, out, ld_out, out_type);
    q.e.bias = bias, q.e.bias_type = p->type;
    q.e.residual = residual;
    q.e.ld_res = M > 1 ? ld_res : up16(N);
    q.e.act = act;
    q.e.saved = saved, q.e.ld_saved = up16(N);
    q.e.vec = vec_bits(out, q.e.ld_out, nullptr, residual, q.e.ld_res, out_type, bias);
    const int epi = act == kActNone ? kEpiLinear : kEpiAct;
    const Choice ch = choose_one(p, kFormNT, epi, M, N, q.kblocks);
    route_status st;
    if ((st = pr.map(A, K, M, pr.a_rows(M, ch), "x", &q.a[0])) != ROUTE_OK ||
        (st = pr.map(W, N, K, 64, "W", &q.b[0][0])) != ROUTE_OK)
        return st;
    q.b[0][1] = q.b[0][0];
    return run(p, pr, kFormNT, epi, ch, chained, false, stream);
}

// out[M, K] = sum over i of dz_i[M, N] W_i[K, N]^T, one or two terms.
route_status input_grad(const route_layer *p, int terms, const Operand *dz, const Operand *W, int M,
                        int N, int K, void *out, int64_t ld_out, bool chained, bool more,
                        cudaStream_t stream) {
    Product pr(p);
    GemmProblem &q = pr.args.p[0];
    pr.args.nprob = 1;
    q.e.M = M, q.e.N = K;
    q.kswitch = kblocks_of(N);
    q.kblocks = terms * q.kswitch;
    set_out(q, out, ld_out, p->type);
    const Choice ch = choose_one(p, kFormNN, kEpiLinear, M, K, q.kblocks);
    for (int i = 0; i < terms; ++i) {
        route_status st;
        if ((st = pr.map(dz[i], N, M, pr.a_rows(M, ch), "dz", &q.a[i])) != ROUTE_OK ||
            (st = pr.map(W[i], N, K, pr.b_rows(ch), "W", &q.b[i][0])) != ROUTE_OK)
            return st;
        q.b[i][1] = q.b[i][0];
    }
    return run(p, pr, kFormNN, kEpiLinear, ch, chained, more, stream);
}

// dW_i[K_i, N_i] = x_i[rows, K_i]^T dz_i[rows, N_i] for up to three weights.
struct WeightGrad {
    Operand x, dz;
    int K, N;
    void *dW;
    int64_t ld;
};
// `shapes`: of all the weights the operator has, so that a gradient's bits do
// not depend on which others are asked for.
route_status weight_grads(const route_layer *p, const WeightGrad *w, int count, int rows,
                          const Shape *shapes, int all, cudaStream_t stream) {
    Product pr(p);
    pr.args.nprob = count;
    for (int i = 0; i < count; ++i) {
        GemmProblem &q = pr.args.p[i];
        q.e.M = w[i].K, q.e.N = w[i].N;
        q.kblocks = q.kswitch = kblocks_of(rows);
        set_out(q, w[i].dW, w[i].ld, p->type);
        route_status st;
        if ((st = pr.map(w[i].x, q.e.M, rows, 64, "x", &q.a[0])) != ROUTE_OK ||
            (st = pr.map(w[i].dz, q.e.N, rows, 64, "dz", &q.b[0][0])) != ROUTE_OK)
            return st;
        q.b[0][1] = q.b[0][0];
    }
    const Choice ch = choose(p, kFormTT, kEpiLinear, shapes, all, kblocks_of(rows));
    return run(p, pr, kFormTT, kEpiLinear, ch, false, false, stream);
}

route_status zero_matrix(void *p, int64_t ld, int rows, int cols, int esize, cudaStream_t stream) {
    if (!p) return ROUTE_OK;
    const cudaError_t e = cudaMemset2DAsync(p, (size_t)(rows > 1 ? ld : cols) * esize, 0,
                                            (size_t)cols * esize, (size_t)rows, stream);
    return e == cudaSuccess ? ROUTE_OK : cuda_fail(e, "cudaMemset2DAsync");
}

// ---- plans ------------------------------------------------------------------------

route_status finish_prepare(route_layer *p, int device, route_layer **out) {
    DeviceGuard guard(device);
    if (guard.err != cudaSuccess) {
        delete p;
        return cuda_fail(guard.err, "cudaSetDevice");
    }
    cudaDeviceProp prop;
    cudaError_t e = cudaGetDeviceProperties(&prop, device);
    route_status st = ROUTE_OK;
    if (e != cudaSuccess) {
        st = cuda_fail(e, "cudaGetDeviceProperties");
    } else if (prop.major != 10 || prop.minor != 3) {
        st = api_fail(ROUTE_ERR_DEVICE, "device %d is sm_%d%d; this library is built for sm_103a only",
                      device, prop.major, prop.minor);
    } else if (p->kind != kNorm && ((size_t)gemm_smem_bytes() > prop.sharedMemPerBlockOptin ||
                                    (size_t)small_smem_bytes() > prop.sharedMemPerBlockOptin ||
                                    prop.multiProcessorCount < 2)) {
        st = api_fail(ROUTE_ERR_DEVICE, "the product kernels need %d B of shared memory per block",
                      gemm_smem_bytes());
    } else if (p->kind == kNorm && (e = norm_configure()) != cudaSuccess) {
        st = cuda_fail(e, "cudaFuncSetAttribute");
    } else if (p->kind != kNorm && ((e = gemm_configure()) != cudaSuccess ||
                                    (e = small_configure()) != cudaSuccess)) {
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
    } else {
        size_t part = (size_t)p->pairs * kTilePartBytes;
        if (p->kind == kLinear && p->train && part < dz_part_floats(p->n) * 4)
            part = dz_part_floats(p->n) * 4;
        p->o_part = area(part);
        p->o_x = copy(R, p->k);
        if (p->kind == kLinear) {
            p->o_w[0] = copy(p->k, p->n);
            p->o_dg = area(p->train && (p->act != kActNone || p->n % 8) ? R * up16(p->n) * 2 : 0);
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

route_status check_prepare(int rows, std::initializer_list<int> widths, int max_width, int type,
                           bool fp32, int act, route_layer **out) {
    if (!out) return api_fail(ROUTE_ERR_NULL, "out must be non-NULL");
    *out = nullptr;
    if (rows < 1 || rows > ROUTE_LAYER_MAX_ROWS)
        return api_fail(ROUTE_ERR_ROWS, "rows %d outside 1-%d", rows, ROUTE_LAYER_MAX_ROWS);
    for (int w : widths)
        if (w < 1 || w > max_width)
            return api_fail(ROUTE_ERR_PLAN, "width %d outside 1-%d", w, max_width);
    if (type != kBf16 && type != kFp16 && !(fp32 && type == kFp32))
        return api_fail(ROUTE_ERR_MODE, "type %d is not one of this operator's", type);
    if (act < 0 || act >= kActCount) return api_fail(ROUTE_ERR_MODE, "unknown activation %d", act);
    return ROUTE_OK;
}

route_layer *new_plan(LayerKind kind, int rows, int type, int act, int train) {
    route_layer *p = new (std::nothrow) route_layer;
    if (!p) return nullptr;
    memset(static_cast<void *>(p), 0, sizeof *p);
    p->kind = kind;
    p->rows = rows;
    p->type = p->out_type = type;
    p->act = act;
    p->train = train != 0;
    return p;
}

// Offsets of the parts of `saved`.
size_t saved_h(const route_layer *p, int rows) { return (size_t)rows * 2 * up16(p->f) * 4; }

}  // namespace

extern "C" {

route_status route_norm_prepare(int rows, int dim, int type, int device, route_layer **out) {
    route_status st = check_prepare(rows, {dim}, ROUTE_NORM_MAX_WIDTH, type, true, 0, out);
    if (st != ROUTE_OK) return st;
    route_layer *p = new_plan(kNorm, rows, type, 0, 0);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = dim;
    return finish_prepare(p, device, out);
}

route_status route_linear_prepare(int rows, int k, int n, int type, int out_type, int act,
                                  int train, int device, route_layer **out) {
    route_status st = check_prepare(rows, {k, n}, ROUTE_LAYER_MAX_WIDTH, type, false, act, out);
    if (st != ROUTE_OK) return st;
    if (out_type != type && out_type != kFp32)
        return api_fail(ROUTE_ERR_MODE, "out_type %d is neither the plan's type nor FP32", out_type);
    if (train && out_type != type)
        return api_fail(ROUTE_ERR_PLAN, "a training plan's results have the plan's type");
    route_layer *p = new_plan(kLinear, rows, type, act, train);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = k, p->n = n;
    p->out_type = out_type;
    return finish_prepare(p, device, out);
}

route_status route_gated_prepare(int rows, int k, int f, int n, int type, int act, int train,
                                 int device, route_layer **out) {
    route_status st = check_prepare(rows, {k, f, n}, ROUTE_LAYER_MAX_WIDTH, type, false, act, out);
    if (st != ROUTE_OK) return st;
    route_layer *p = new_plan(kGated, rows, type, act, train);
    if (!p) return api_fail(ROUTE_ERR_CUDA, "out of host memory");
    p->k = k, p->f = f, p->n = n;
    return finish_prepare(p, device, out);
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
    if (w & kStatusBounds)
        return api_fail(ROUTE_ERR_DEVICE_BOUNDS, "a kernel skipped an index out of range");
    if (w & kStatusTimeout)
        return api_fail(ROUTE_ERR_DEVICE_TIMEOUT, "a kernel gave up waiting; its outputs are invalid");
    return ROUTE_OK;
}

int64_t route_layer_saved_bytes(const route_layer *p, int rows) {
    if (!p) return -1;
    if (rows <= 0 || !p->train) return 0;
    if (p->kind == kLinear) return p->act == kActNone ? 0 : (int64_t)rows * up16(p->n) * 4;
    if (p->kind == kGated) return (int64_t)saved_h(p, rows) + (int64_t)rows * up16(p->f) * 2;
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
    Operand ox, ow;
    if ((st = operand(p, x, ld_x, rows, p->k, p->o_x, s, &ox)) != ROUTE_OK ||
        (st = operand(p, W, ld_W, p->k, p->n, p->o_w[0], s, &ow)) != ROUTE_OK)
        return st;
    return forward_product(p, ox, ow, rows, p->k, p->n, p->act, bias, residual, ld_residual, out,
                           ld_out, p->out_type, static_cast<float *>(saved), false, s);
}

route_status route_linear_backward(const route_layer *p, int rows, const void *dout,
                                   int64_t ld_dout, const void *x, int64_t ld_x, const void *W,
                                   int64_t ld_W, const void *saved, void *dx, int64_t ld_dx,
                                   void *dW, int64_t ld_dW, void *dbias, void *stream) {
    route_status st = check_plan(p, kLinear, rows);
    if (st != ROUTE_OK) return st;
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
    if (make_dz || dbias) {
        DzArgs a = {};
        a.rows = rows, a.n = p->n, a.type = p->type, a.act = p->act;
        a.dout = dout, a.ld_dout = dz.ld;
        if (p->act != kActNone) a.z = static_cast<const float *>(saved), a.ld_z = up16(p->n);
        if (make_dz) {
            a.dz = p->scratch + p->o_dg, a.ld_dz = up16(p->n);
            dz = {a.dz, a.ld_dz};
        }
        a.dbias = dbias;
        a.part = reinterpret_cast<float *>(p->scratch + p->o_part);
        a.trigger = dx || dW;
        const cudaError_t e = dz_launch(a, s);
        if (e != cudaSuccess) return cuda_fail(e, "pre-activation gradient kernel launch");
    }
    if (dx) {
        Operand ow;
        if ((st = operand(p, W, ld_W, p->k, p->n, p->o_w[0], s, &ow)) != ROUTE_OK ||
            (st = input_grad(p, 1, &dz, &ow, rows, p->n, p->k, dx, ld_dx, false, dW != nullptr, s)) != ROUTE_OK)
            return st;
    }
    if (dW) {
        WeightGrad g = {{}, dz, p->k, p->n, dW, ld_dW};
        if ((st = operand(p, x, ld_x, rows, p->k, p->o_x, s, &g.x)) != ROUTE_OK) return st;
        const Shape shape = {p->k, p->n};
        return weight_grads(p, &g, 1, rows, &shape, 1, s);
    }
    return ROUTE_OK;
}

route_status route_gated_forward(const route_layer *p, int rows, const void *x, int64_t ld_x,
                                 const void *W_gate, int64_t ld_gate, const void *W_up,
                                 int64_t ld_up, const void *W_down, int64_t ld_down,
                                 const void *residual, int64_t ld_residual, void *out,
                                 int64_t ld_out, void *saved, void *stream) {
    route_status st = check_plan(p, kGated, rows);
    if (st != ROUTE_OK) return st;
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
    Operand ox, og, ou, od;
    if ((st = operand(p, x, ld_x, rows, p->k, p->o_x, s, &ox)) != ROUTE_OK ||
        (st = operand(p, W_gate, ld_gate, p->k, p->f, p->o_w[0], s, &og)) != ROUTE_OK ||
        (st = operand(p, W_up, ld_up, p->k, p->f, p->o_w[1], s, &ou)) != ROUTE_OK ||
        (st = operand(p, W_down, ld_down, p->f, p->n, p->o_w[2], s, &od)) != ROUTE_OK)
        return st;
    // h = act(x W_gate) * (x W_up): one kernel for both projections
    const long long ldf = up16(p->f);
    uint8_t *h = saved ? static_cast<uint8_t *>(saved) + saved_h(p, rows) : p->scratch + p->o_h;
    {
        Product pr(p);
        GemmProblem &q = pr.args.p[0];
        pr.args.nprob = 1;
        q.e.M = rows, q.e.N = p->f;
        q.kblocks = q.kswitch = kblocks_of(p->k);
        set_out(q, h, ldf, p->type);
        q.e.act = p->act;
        q.e.saved = static_cast<float *>(saved), q.e.ld_saved = ldf;
        q.e.saved2 = saved ? q.e.saved + (size_t)rows * ldf : nullptr;
        const Choice ch = choose_one(p, kFormNT, kEpiGated, rows, p->f, q.kblocks);
        if ((st = pr.map(ox, p->k, rows, pr.a_rows(rows, ch), "x", &q.a[0])) != ROUTE_OK ||
            (st = pr.map(og, p->f, p->k, 64, "W_gate", &q.b[0][0])) != ROUTE_OK ||
            (st = pr.map(ou, p->f, p->k, 64, "W_up", &q.b[0][1])) != ROUTE_OK ||
            (st = run(p, pr, kFormNT, kEpiGated, ch, false, true, s)) != ROUTE_OK)
            return st;
    }
    return forward_product(p, {h, ldf}, od, rows, p->f, p->n, kActNone, nullptr, residual,
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
    Operand dy;
    if ((st = operand(p, dout, ld_dout, rows, p->n, p->o_dout, s, &dy)) != ROUTE_OK) return st;
    Operand dz[2] = {{p->scratch + p->o_dg, ldf}, {p->scratch + p->o_du, ldf}};
    if (pre) {
        // dh = dout W_down^T, turned into dgate and dup in its epilogue
        Operand od;
        if ((st = operand(p, W_down, ld_down, p->f, p->n, p->o_w[2], s, &od)) != ROUTE_OK) return st;
        Product pr(p);
        GemmProblem &q = pr.args.p[0];
        pr.args.nprob = 1;
        q.e.M = rows, q.e.N = p->f;
        q.kblocks = q.kswitch = kblocks_of(p->n);
        set_out(q, const_cast<void *>(dz[0].p), ldf, p->type);
        q.e.ld_out = ldf;
        q.e.out2 = const_cast<void *>(dz[1].p);
        q.e.act = p->act;
        q.e.saved = static_cast<float *>(const_cast<void *>(saved)), q.e.ld_saved = ldf;
        q.e.saved2 = q.e.saved + (size_t)rows * ldf;
        const Choice ch = choose_one(p, kFormNN, kEpiDGate, rows, p->f, q.kblocks);
        if ((st = pr.map(dy, p->n, rows, pr.a_rows(rows, ch), "dout", &q.a[0])) != ROUTE_OK ||
            (st = pr.map(od, p->n, p->f, pr.b_rows(ch), "W_down", &q.b[0][0])) != ROUTE_OK)
            return st;
        q.b[0][1] = q.b[0][0];
        if ((st = run(p, pr, kFormNN, kEpiDGate, ch, false, true, s)) != ROUTE_OK) return st;
    }
    const bool weights = dW_gate || dW_up || dW_down;
    if (dx) {
        Operand w[2];
        const bool chained = p->f % 8 == 0;  // no copy of the weights between the two products
        if ((st = operand(p, W_gate, ld_gate, p->k, p->f, p->o_w[0], s, &w[0])) != ROUTE_OK ||
            (st = operand(p, W_up, ld_up, p->k, p->f, p->o_w[1], s, &w[1])) != ROUTE_OK ||
            (st = input_grad(p, 2, dz, w, rows, p->f, p->k, dx, ld_dx, chained, weights, s)) != ROUTE_OK)
            return st;
    }
    if (!weights) return ROUTE_OK;
    WeightGrad g[3];
    int count = 0;
    if (dW_gate || dW_up) {
        Operand ox;
        if ((st = operand(p, x, ld_x, rows, p->k, p->o_x, s, &ox)) != ROUTE_OK) return st;
        if (dW_gate) g[count++] = {ox, dz[0], p->k, p->f, dW_gate, ld_dgate};
        if (dW_up) g[count++] = {ox, dz[1], p->k, p->f, dW_up, ld_dup};
    }
    if (dW_down) {
        const Operand h = {static_cast<const uint8_t *>(saved) + saved_h(p, rows), ldf};
        g[count++] = {h, dy, p->f, p->n, dW_down, ld_ddown};
    }
    const Shape shapes[3] = {{p->k, p->f}, {p->k, p->f}, {p->f, p->n}};
    return weight_grads(p, g, count, rows, shapes, 3, s);
}

}  // extern "C"
