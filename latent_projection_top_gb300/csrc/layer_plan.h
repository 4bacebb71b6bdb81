// A layer operator's plan and what its C entry points share (layer_api.cu,
// experts_api.cu): argument checks and the device's memory.  Host code.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <new>

#include "api_util.h"
#include "layer.cuh"
#include "route_layer.h"

namespace route {

enum LayerKind { kNorm, kLinear, kGated, kDropout, kDispatch, kExpertBlocks };

// How a launch covers its products: CTA-pair tiles of 256 x bn
// (layer_gemm.cu), or 128-column tiles of bn rows (layer_small.cu), and the
// splits of the contraction.
struct Choice {
    bool small;
    int bn;
    int splits[kGemmMaxProblems];  // of each product (small tiles: the same for all)
    double us;                     // the estimate that it was chosen by
};

// What the last call of a kind chose, for its number of rows.
enum ChoiceSlot { kSlotForward, kSlotDown, kSlotDGate, kSlotBackward, kSlotInput, kSlotWeights, kSlots };
struct ChoiceMemo {
    int rows;
    Choice c;
};

}  // namespace route

struct route_layer {
    route::LayerKind kind;
    int rows, k, f, n;
    int type, out_type, act, train;
    int experts, first, topk;  // routed experts' plans: experts here, the first one's id, ids a row
    route::SortShape sort;  // a dispatch plan's: what a sort may have of the device
    int device, sms, pairs;
    int test_stall;
    unsigned long long timeout_ns;
    unsigned *words;   // device status word
    uint8_t *scratch;
    size_t scratch_bytes;
    // offsets into scratch (0 size where the plan needs none)
    size_t o_part;     // split partials (norm: column-sum partials)
    size_t o_sum;      // the bias gradient's partials
    size_t o_x, o_w[3], o_dout, o_h, o_dg, o_du;
    // Held for the whole of a call: its kernels share the scratch, and follow one
    // another in the stream without another call's between them.
    mutable std::mutex calls;
    mutable route::ChoiceMemo memo[route::kSlots];
};

namespace route {

constexpr unsigned long long kTimeoutNs = 2000000000ull;

inline route_status cuda_fail(cudaError_t e, const char *what) {
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

inline long long up8(long long v) { return (v + 7) & ~7ll; }
inline long long up16(long long v) { return (v + 15) & ~15ll; }
inline bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---- argument checks ----------------------------------------------------------

// A matrix argument: its name, width and whether a product reads it by TMA.
struct Mat {
    const char *name;
    const void *p;
    int64_t ld;
    int rows, cols, esize;
    bool operand;
};

inline route_status check_mat(const Mat &m) {
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

inline route_status check_mats(std::initializer_list<Mat> ms) {
    for (const Mat &m : ms)
        if (const route_status st = check_mat(m)) return st;
    return ROUTE_OK;
}

inline route_status check_vec(const char *name, const void *p, int esize) {
    if (p && !aligned(p, (unsigned)esize))
        return api_fail(ROUTE_ERR_ALIGN, "%s is not aligned to its element", name);
    return ROUTE_OK;
}

inline route_status check_plan(const route_layer *p, LayerKind kind, int rows) {
    if (!p) return api_fail(ROUTE_ERR_NULL, "plan is NULL");
    if (p->kind != kind) return api_fail(ROUTE_ERR_PLAN, "the plan is another operator's");
    if (rows < 0 || rows > p->rows)
        return api_fail(ROUTE_ERR_ROWS, "rows %d outside the plan's 0-%d", rows, p->rows);
    return ROUTE_OK;
}

// Where a block's h is in `saved`, behind the FP32 sums of gate and up.
inline size_t saved_h(const route_layer *p, int rows) { return (size_t)rows * 2 * up16(p->f) * 4; }

route_status layer_check_prepare(int rows, int max_rows, std::initializer_list<int> widths, int max_width,
                                 int type, bool fp32, int act, route_layer **out);
route_layer *layer_new_plan(LayerKind kind, int rows, int type, int act, int train);
// Binds the plan to its device and allocates its scratch; frees it on an error.
route_status layer_finish_prepare(route_layer *p, int device, route_layer **out);

}  // namespace route
