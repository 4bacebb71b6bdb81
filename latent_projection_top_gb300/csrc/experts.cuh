// Launch arguments and internal launch entry points of the routed experts'
// operators (dispatch_kernel.cu, experts_kernel.cu) and of dropout
// (dropout_kernel.cu); their C ABI is in experts_api.cu.
#pragma once

#include "layer.cuh"

namespace route {

// ---- tokens sorted by expert and back ---------------------------------------------

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 32;

struct SortArgs {
    int rows, topk, experts, first;
    const int *ids;             // [rows, topk], row stride ld_ids
    long long ld_ids;
    int *offsets;               // [experts + 1]
    int *place;                 // [rows][topk]
    int *source;                // [rows * topk] or null
};
cudaError_t sort_configure();
// The CTAs that a cluster may have and the clusters that run side by side on the
// current device.
SortShape sort_shape();
cudaError_t sort_launch(const SortArgs &args, SortShape most_of, cudaStream_t stream);

// What gather and combine, and their gradients, read and write: rows of `dim`
// values in the tokens' order (a) and in the experts' order (b).
struct MoveArgs {
    int rows, topk, dim, type;
    int pairs;                  // rows of b: a place outside 0 .. pairs - 1 is none
    const int *place;           // [rows][topk]
    const float *weights;       // [rows][topk]; null: 1
    const void *a;              // gather: x; combine: the residual or null; gradient: dout
    long long ld_a;
    const void *b;              // the experts' rows that are read
    long long ld_b;
    void *out;                  // gather, gradient: experts' rows (or null); combine: tokens' rows
    long long ld_out;
    float *dweights;            // [rows][topk] or null
};
cudaError_t gather_launch(const MoveArgs &args, int sms, cudaStream_t stream);
cudaError_t combine_launch(const MoveArgs &args, int sms, cudaStream_t stream);
cudaError_t combine_backward_launch(const MoveArgs &args, int sms, cudaStream_t stream);

// ---- the experts' products ----------------------------------------------------------

// Maps of the rows, one for each height of a box: 16 (i + 1) rows.
constexpr int kTokenBoxes = 8;
struct ExpertsMaps {
    CUtensorMap w[2];                // the weights [experts][..][..] (gated: of gate and of up)
    CUtensorMap t[2][kTokenBoxes];   // the rows of each segment of the contraction
};

// D[r, c] = sum_k A[r, k] B_e[k, c] for the rows r of every expert e
// (offsets[e] .. offsets[e + 1]) and what the epilogue makes of it.
struct ExpertsArgs {
    const int *offsets;
    int experts, rows;          // rows of A: offsets past them are cut
    int tiles_n;                // column tiles: 256 columns (gated: 128 hidden ones) of a CTA pair
    int kblocks, kswitch;       // blocks of 64 from kswitch on come from the second segment
    unsigned w_bytes;           // bytes of a CTA's weight boxes of a k-block
    int fp16;
    int trigger;                // another kernel of the call follows
    // The call's kernel before this one waited for its own predecessors before it
    // let this one launch, and writes neither the offsets nor the weights: both
    // are read at once.
    int chained;
    int pairs;                  // CTA pairs launched
    float tiles_a_pair;         // tiles_n / pairs
    int test_stall;
    unsigned long long timeout_ns;
    unsigned *status;
    Epilogue e;                 // M is set for each run of rows
};

// dW_e[m, n] = sum over the rows r of expert e of A[r, m] B[r, n], 16-bit results.
constexpr int kMaxGrads = 3;
struct GradMaps {
    CUtensorMap a[kMaxGrads], b[kMaxGrads];
    CUtensorMap d[kMaxGrads];   // the results [experts][M][N], in boxes of 32 rows x 64 columns
};
struct GradArgs {
    const int *offsets;
    int experts, rows;
    int nprob;
    int fp16;
    // The call's kernel before this one waited for what made A and B before it let
    // this one launch, and writes neither: the two run side by side, and this one
    // waits for it before it ends.
    int beside;
    int pairs;
    int per_expert;             // tiles of one expert, of all problems
    int test_stall;
    unsigned long long timeout_ns;
    unsigned *status;
    struct {
        int M, N, tiles_m, tiles_n, base;
    } p[kMaxGrads];
};

constexpr int kExpertCols = 256;   // weight columns of a tile
constexpr int kExpertRows = 256;   // token rows of a tile, at most
cudaError_t experts_configure();
int experts_smem_bytes();
cudaError_t experts_launch(int epi, bool n_contiguous, const ExpertsMaps &maps, const ExpertsArgs &args,
                           cudaStream_t stream);

// Products of few rows (at most kFewRows) and few tiles, of weights whose columns
// are contiguous: `tiles` tiles of 128 columns (gated: 64 hidden ones), one for
// each column tile of every expert that could have rows, over `ctas` CTAs each.
constexpr int kFewRows = 32;
constexpr int kFewCols = 128;
constexpr int kFewCtas = 8;
cudaError_t experts_small_configure();
cudaError_t experts_small_launch(int epi, int tiles, int ctas, const ExpertsMaps &maps, const ExpertsArgs &args,
                                 cudaStream_t stream);

cudaError_t experts_grad_launch(const GradMaps &maps, const GradArgs &args, cudaStream_t stream);

// ---- dropout ----------------------------------------------------------------------------

constexpr int kPhiloxRounds = 10;
struct DropoutArgs {
    int rows, dim, type;
    unsigned threshold;         // of 65536: lots below it are dropped
    float scale;                // 65536 / (65536 - threshold)
    uint32_t keys[2 * kPhiloxRounds];  // each round's
    unsigned long long offset;
    const long long *step;      // added to the offset; may be null
    const void *x;
    long long ld_x;
    const void *residual;       // may be null
    long long ld_res;
    void *out;
    long long ld_out;
};
cudaError_t dropout_launch(const DropoutArgs &args, int sms, cudaStream_t stream);

}  // namespace route
