// Launch arguments and internal launch entry points of the layer operators
// (layer norm, linear, gated block): the kernels' side is in layer_gemm.cu,
// layer_small.cu, layer_elem.cu and layer_norm.cu, the C ABI's in layer_api.cu
// (layer_call.cpp, the Python module, sees the C ABI only).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace route {

enum LayerType : int { kBf16 = 0, kFp16 = 1, kFp32 = 2 };
enum LayerAct : int {
    kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActSigmoid = 5,
    kActCount = 6
};
__host__ __device__ constexpr int layer_esize(int type) { return type == kFp32 ? 4 : 2; }

// What the epilogue makes of a tile's FP32 sums.
enum LayerEpi : int {
    kEpiLinear = 0,  // out = v + bias + residual
    kEpiGated = 1,   // v = (gate, up): out = act(gate) * up, both kept when `saved` is set
    kEpiDGate = 2,   // v = dh: out = dh * up * act'(gate), out2 = dh * act(gate), from `saved`
    kEpiAct = 3,     // out = act(v + bias) + residual, z = v + bias kept when `saved` is set
    kEpiCount = 4
};
__host__ __device__ constexpr bool epi_linear(int epi) { return epi == kEpiLinear || epi == kEpiAct; }

// What becomes of a product's sums D[M, N].  A kernel copies this into
// registers: read from the launch's arguments with an index that is known
// only at run time, a step of the epilogue waited for each field (a tile's
// epilogue took 20 us).
struct Epilogue {
    int M, N;                   // rows and columns of the result (gated: N hidden columns)
    int out_type;               // type of out, out2 and residual
    int bias_type;
    int act;
    int vec;                    // what may be read and written as vectors (kVec*)
    const void *bias;           // [N]
    const void *residual;       // [M, N], row stride ld_res
    void *out;                  // [M, N], row stride ld_out
    void *out2;                 // kEpiDGate: d up, same layout
    float *saved, *saved2;      // FP32 pre-activations (gated: of gate and of up), row stride ld_saved
    float *part;                // splits > 1: FP32 partials [split][M][ld_part]
    long long ld_res, ld_out, ld_saved, ld_part;
};

enum GemmForm : int {
    kFormNT = 0,  // A rows K-contiguous, B [K, N] N-contiguous (forward)
    kFormNN = 1,  // A rows K-contiguous, B [N, K] K-contiguous (input gradients)
    kFormTT = 2,  // A [K, M] M-contiguous, B [K, N] N-contiguous (weight gradients)
    kFormMixed = 3  // (a kernel's) NN and TT, as each problem says
};

// One matrix product D[M, N] = A B with a contraction of `kblocks` blocks of
// 64 (blocks from `kswitch` on come from the second pair of operands).  Map
// indexes name entries of GemmMaps.
struct GemmProblem {
    Epilogue e;
    int form;
    int tiles_m, tiles_n, band; // row tiles, column tiles, column tiles of a band
    int item_base;              // first work item of this problem
    int splits;                 // K splits of a tile
    int kblocks, kswitch;
    unsigned a_bytes;           // bytes of an A box: fewer rows than a tile's when M is less
    uint8_t a[2], b[2][2];      // A map of each segment, B map of each segment and CTA of the pair
};

constexpr int kGemmMaxProblems = 4;
constexpr int kGemmMaxMaps = 12;
constexpr int kGemmMaxPairs = 80;  // pairs that `count` can describe
constexpr int kGemmMaxSplits = 32;

struct GemmMaps {
    CUtensorMap m[kGemmMaxMaps];
};

struct GemmArgs {
    int nprob;                  // problems, the longest contraction first
    int items;                  // work items: tiles x splits over all problems
    int splits;                 // (small tiles) K splits of every tile: the CTAs of a cluster
    int pairs;                  // CTA pairs launched
    int listed;                 // pair j takes items first[c][j] .. of problem c, count[c][j] of them
                                // (else items j, j + pairs, .. of all)
    int fp16;                   // operands are FP16 (else BF16)
    int trigger;                // a kernel of the same call follows: let it launch early
    int test_stall;
    unsigned long long timeout_ns;
    unsigned *status;
    GemmProblem p[kGemmMaxProblems];
    uint16_t first[kGemmMaxProblems][kGemmMaxPairs], count[kGemmMaxProblems][kGemmMaxPairs];
};

// Partials of a split product summed in split order, then the epilogue.
struct FinishArgs {
    int splits;
    int trigger;
    Epilogue e;
};

constexpr int kGemmBM = 256;
cudaError_t gemm_configure();
int gemm_smem_bytes();
// bn: 256 or 128 accumulator columns a tile.
cudaError_t gemm_launch(int form, int epi, int bn, const GemmMaps &maps, const GemmArgs &args,
                        cudaStream_t stream);
cudaError_t gemm_finish_launch(int epi, const FinishArgs &args, cudaStream_t stream);

// Products of few rows or few tiles: 128 columns x up to 128 rows a tile, the
// contraction split over the CTAs of a cluster (args.splits: 1, 2, 4 or 8).
// Takes the same arguments as gemm_launch; `rows`: MMA rows a tile (16, 32,
// 64 or 128).  With `chained` the call's kernel before this one waited for
// its own predecessors before it let this one launch, and does not write the
// columns' operand of the NT and NN products, which is then read at once.
constexpr int kSmallTile = 128;
constexpr int kSmallMaxSplits = 8;
cudaError_t small_configure();
int small_smem_bytes();
cudaError_t small_launch(int epi, int rows, const GemmMaps &maps, const GemmArgs &args,
                         bool chained, cudaStream_t stream);

// dst[r, 0..cols) = src[r, 0..cols) of 16-bit values, for operands whose rows
// TMA cannot read where they are; all of a call's in one launch.
constexpr int kMaxRepacks = 5;
struct RepackArgs {
    int count;
    struct {
        const void *src;
        void *dst;
        long long ld_src, ld_dst;
        int rows, cols;
    } c[kMaxRepacks];
};
cudaError_t repack_launch(const RepackArgs &args, cudaStream_t stream);

// dz = dout * act'(z) (z: FP32, row stride ld_z; null: dz = dout), written
// with row stride ld_dz unless dz is null.  dbias (type `type`): column sums
// of the unrounded dz, in two steps with FP32 partials in `part`
// (dz_part_floats(n) floats): dz_launch makes them with dz, or bias_launch
// from dout (`sums_only`: no activation, and the products read dout itself);
// bias_launch adds them.
struct DzArgs {
    int rows, n, type, act;
    const void *dout;
    long long ld_dout;
    const float *z;
    long long ld_z;
    void *dz;
    long long ld_dz;
    int sums_only;
    void *dbias;
    float *part;
};
size_t dz_part_floats(int n);
// The kernel of a call that always has one after it.
cudaError_t dz_launch(const DzArgs &args, cudaStream_t stream);
// `after`: the call's kernel before this one has waited for all that came
// before it, dz_launch's kernel among it, and writes nothing that is read
// here: the sums then run beside it.
cudaError_t bias_launch(const DzArgs &args, bool after, cudaStream_t stream);

// What a sort may have of the device (experts.cuh).
struct SortShape {
    int ctas, slices;
};

struct NormArgs {
    int rows, dim, type;
    float eps;
    const void *x;
    long long ld_x;
    const void *gamma, *beta;
    void *y;
    long long ld_y;
    float *stats;               // [rows][2]: mean, 1 / sqrt(var + eps); may be null (forward)
    // backward
    const void *dy;
    long long ld_dy;
    void *dx;
    long long ld_dx;
    void *dgamma, *dbeta;
    float *part;                // norm_part_floats(dim, sms) floats
    int sms;
};
cudaError_t norm_configure();
size_t norm_part_floats(int dim, int sms);
cudaError_t norm_forward_launch(const NormArgs &args, cudaStream_t stream);
cudaError_t norm_backward_launch(const NormArgs &args, cudaStream_t stream);

}  // namespace route
