// The layer operators' elementwise kernels: copies of operands that TMA
// cannot read in place, and a linear layer's d pre-activation with the
// column sums that are its bias's gradient.
#include "layer.cuh"
#include "layer_math.cuh"

namespace route {
namespace {

constexpr int kDzCols = 256;       // columns of a block: 32 threads of 8
constexpr int kDzRows = 2;
constexpr int kDzMaxBlocks = 128;  // row blocks: partial sums a column

// Bound by HBM: 2405x4151 BF16 6.5 us (40 MB in and out, 6.1 TB/s).
//
// Eight values a thread; columns past `cols` become zeros up to the next
// multiple of 8 (ld_dst is one).
__global__ void __launch_bounds__(256) repack_kernel(const __grid_constant__ RepackArgs args) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // a product of the same call follows
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const auto &a = args.c[blockIdx.y];
    const uint16_t *src = static_cast<const uint16_t *>(a.src);
    uint16_t *dst = static_cast<uint16_t *>(a.dst);
    const long long ld_src = a.ld_src, ld_dst = a.ld_dst;
    const int cols = a.cols, groups = (cols + 7) >> 3;
    const long long total = (long long)a.rows * groups;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const int r = (int)(i / groups), c = (int)(i % groups) * 8;
        const uint16_t *s = src + (long long)r * ld_src + c;
        uint32_t w[4];
        if (c + 8 <= cols) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = s[2 * e] | ((uint32_t)s[2 * e + 1] << 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = c + 2 * e < cols ? s[2 * e] : 0u;
                const uint32_t hi = c + 2 * e + 1 < cols ? s[2 * e + 1] : 0u;
                w[e] = lo | (hi << 16);
            }
        }
        *reinterpret_cast<uint4 *>(dst + (long long)r * ld_dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Bound by what it reads and writes, 8 bytes a value: 2050x3584 gelu 10 us (59
// MB, 5.9 TB/s, some of it from L2).
//
// dz = dout * act'(z) for a block of rows and 256 columns: a warp walks rows,
// a thread holds 8 columns and the FP32 sums of the dz it made, before they
// are rounded to 16 bits for the products.
__global__ void __launch_bounds__(256, 4) dz_kernel(const __grid_constant__ DzArgs a, int rows_per_block,
                                                 int vec) {
    __shared__ float s_sum[8][kDzCols];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // products or the sums follow
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * kDzCols + lane * 8;
    const int r1 = min(a.rows, (int)(blockIdx.y + 1) * rows_per_block);
    float sum[8] = {};
    if (c < a.n) {
        const int n = a.n - c;
        const uint16_t *dout = static_cast<const uint16_t *>(a.dout);
        uint16_t *dz = static_cast<uint16_t *>(a.dz);
        // two rows at a time, so that their loads are on the way together (four, with
        // half as many blocks an SM, took 2 us longer: backward 2050x896x3584, gelu)
        for (int r = blockIdx.y * rows_per_block + warp; r < r1; r += 8 * kDzRows) {
            uint4 t[kDzRows];
            float4 z0[kDzRows], z1[kDzRows];
#pragma unroll
            for (int k = 0; k < kDzRows; ++k) {
                const int row = r + 8 * k;
                if (row >= r1) break;
                const uint16_t *s = dout + (long long)row * a.ld_dout + c;
                if (vec && n >= 8) {
                    t[k] = *reinterpret_cast<const uint4 *>(s);
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = 2 * e < n ? s[2 * e] : 0u, hi = 2 * e + 1 < n ? s[2 * e + 1] : 0u;
                        w[e] = lo | (hi << 16);
                    }
                    t[k] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (a.z != nullptr) {
                    const float4 *q = reinterpret_cast<const float4 *>(a.z + (long long)row * a.ld_z + c);
                    z0[k] = q[0], z1[k] = q[1];
                }
            }
#pragma unroll
            for (int k = 0; k < kDzRows; ++k) {
                const int row = r + 8 * k;
                if (row >= r1) break;
                float v[8];
                const uint32_t w[4] = {t[k].x, t[k].y, t[k].z, t[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack16(w[e], a.type);
                    v[2 * e] = f.x, v[2 * e + 1] = f.y;
                }
                if (a.z != nullptr) {
                    float z[8] = {z0[k].x, z0[k].y, z0[k].z, z0[k].w, z1[k].x, z1[k].y, z1[k].z, z1[k].w}, d[8];
                    act_slopes<8>(a.act, z, z, d);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = e < n ? v[e] * d[e] : 0.f;
                }
                // 16 bits: an operand of the products (the sums below take it unrounded)
                if (dz != nullptr)  // ld_dz is a multiple of 8
                    *reinterpret_cast<uint4 *>(dz + (long long)row * a.ld_dz + c) =
                        make_uint4(pack16(v[0], v[1], a.type), pack16(v[2], v[3], a.type),
                                   pack16(v[4], v[5], a.type), pack16(v[6], v[7], a.type));
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += v[e];
            }
        }
    }
    if (a.dbias == nullptr) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) s_sum[warp][lane * 8 + e] = sum[e];
    __syncthreads();
    const int col = blockIdx.x * kDzCols + threadIdx.x;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += s_sum[w][threadIdx.x];
    if (col < a.n) a.part[(long long)blockIdx.y * a.n + col] = t;
}

// The column sums of dout itself, a row of partials a warp: as dz_kernel, of
// 16-bit values and with nothing to write.  This kernel and the next read what
// was there before these were launched: with `after` they wait only before
// they leave, so that they start as blocks of the products leave (backward
// 2050x896x3584 without activation 32.2 us, with the sums ahead of the
// products 36.4, without dbias 27.2; with gelu 42.5, 44.3 and 40.7).  Few rows
// make one block of rows, which adds its own partials.
constexpr int kBiasRows = 4;  // rows whose loads are on the way together
constexpr int kBiasWarps = 4;
constexpr int kBiasMaxBlocks = kDzMaxBlocks / kBiasWarps;
// dbias alone, 3584 columns: 128 rows 4.2 us, in row blocks 5.4; 256 rows 4.4, in one 6.8.
constexpr int kBiasOneBlock = 128;  // rows
__global__ void __launch_bounds__(32 * kBiasWarps)
    bias_part_kernel(const __grid_constant__ DzArgs a, int rows_per_warp, int vec, int after) {
    const bool all = gridDim.y == 1;
    if (!after) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0 && !all) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, part = blockIdx.y * kBiasWarps + (threadIdx.x >> 5);
    const int c = blockIdx.x * kDzCols + lane * 8, n = a.n - c;
    const int r1 = min(a.rows, (part + 1) * rows_per_warp);
    if (n > 0) {
        float sum[8] = {};
        const uint16_t *s = static_cast<const uint16_t *>(a.dout) + c;
        for (int r = part * rows_per_warp; r < r1; r += kBiasRows) {
            uint32_t w[kBiasRows][4] = {};
#pragma unroll
            for (int k = 0; k < kBiasRows; ++k) {
                if (r + k >= r1) break;
                const uint16_t *q = s + (long long)(r + k) * a.ld_dout;
                if (vec && n >= 8) {
                    const uint4 t = *reinterpret_cast<const uint4 *>(q);
                    w[k][0] = t.x, w[k][1] = t.y, w[k][2] = t.z, w[k][3] = t.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = 2 * e < n ? q[2 * e] : 0u, hi = 2 * e + 1 < n ? q[2 * e + 1] : 0u;
                        w[k][e] = lo | (hi << 16);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBiasRows; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack16(w[k][e], a.type);
                    sum[2 * e] += f.x, sum[2 * e + 1] += f.y;
                }
        }
        float *out = a.part + (long long)part * a.n + c;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) out[e] = sum[e];
    }
    if (all) {
        __syncthreads();
        for (int t = threadIdx.x; t < kDzCols && t < a.n - (int)blockIdx.x * kDzCols; t += 32 * kBiasWarps) {
            const float *p = a.part + blockIdx.x * kDzCols + t;
            float v = p[0];
#pragma unroll
            for (int w = 1; w < kBiasWarps; ++w) v += p[(long long)w * a.n];
            store_elem(a.dbias, a.type, blockIdx.x * kDzCols + t, v);
        }
    }
    if (after) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Column sums of `blocks` rows of partials: each of four warps adds every
// fourth, and the sums meet in order.
__global__ void __launch_bounds__(32 * kBiasWarps)
    bias_sum_kernel(const float *part, int blocks, int n, void *out, int type, int after) {
    __shared__ float s_sum[kBiasWarps][32];
    if (!after) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < n) {
#pragma unroll 16
        for (int b = warp; b < blocks; b += kBiasWarps) t += __ldcg(part + (long long)b * n + c);
    }
    s_sum[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < n) {
#pragma unroll
        for (int w = 1; w < kBiasWarps; ++w) t += s_sum[w][lane];
        store_elem(out, type, c, t);
    }
    if (after) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_pdl(void (*fn)(P...), dim3 grid, dim3 block, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[1];
    c.gridDim = grid;
    c.blockDim = block;
    c.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, fn, static_cast<P>(args)...);
}

}  // namespace

cudaError_t repack_launch(const RepackArgs &args, cudaStream_t stream) {
    long long most = 0;
    for (int i = 0; i < args.count; ++i) {
        const long long n = (long long)args.c[i].rows * ((args.c[i].cols + 7) / 8);
        most = most < n ? n : most;
    }
    const unsigned blocks = (unsigned)(most / 256 < 1216 ? (most + 255) / 256 : 1216);
    return launch_pdl(repack_kernel, dim3(blocks, args.count), dim3(256), stream, args);
}

size_t dz_part_floats(int n) { return (size_t)kDzMaxBlocks * n; }

namespace {

// Row blocks of dz_kernel and the rows of each: about eight blocks an SM,
// eight rows at least to a block.
int dz_blocks(int rows, int n, int &per) {
    int rb = 608 / ((n + kDzCols - 1) / kDzCols);
    rb = rb < 1 ? 1 : rb > kDzMaxBlocks ? kDzMaxBlocks : rb;
    rb = rb > (rows + 7) / 8 ? (rows + 7) / 8 : rb;
    per = (rows + rb - 1) / rb;
    return (rows + per - 1) / per;
}

int dout_vec(const DzArgs &a) {
    return (reinterpret_cast<uintptr_t>(a.dout) & 15u) == 0 && (a.ld_dout % 8 == 0 || a.rows == 1);
}

}  // namespace

cudaError_t dz_launch(const DzArgs &args, cudaStream_t stream) {
    if (args.sums_only) return cudaSuccess;
    int per;
    const int rb = dz_blocks(args.rows, args.n, per);
    return launch_pdl(dz_kernel, dim3((args.n + kDzCols - 1) / kDzCols, rb), dim3(256), stream, args, per,
                      dout_vec(args));
}

cudaError_t bias_launch(const DzArgs &args, bool after, cudaStream_t stream) {
    int per, parts = 0;
    if (args.sums_only) {
        // four rows at least to a warp
        int blocks = (args.rows + kBiasRows * kBiasWarps - 1) / (kBiasRows * kBiasWarps);
        blocks = args.rows <= kBiasOneBlock ? 1 : blocks;
        blocks = blocks > kBiasMaxBlocks ? kBiasMaxBlocks : blocks;
        parts = blocks * kBiasWarps;
        per = (args.rows + parts - 1) / parts;
        const cudaError_t e =
            launch_pdl(bias_part_kernel, dim3((args.n + kDzCols - 1) / kDzCols, blocks), dim3(32 * kBiasWarps),
                       stream, args, per, dout_vec(args), (int)after);
        if (e != cudaSuccess || blocks == 1) return e;
        after = false;  // these sums are of the kernel just launched
    } else {
        parts = dz_blocks(args.rows, args.n, per);
    }
    return launch_pdl(bias_sum_kernel, dim3((args.n + 31) / 32), dim3(32 * kBiasWarps), stream,
                      static_cast<const float *>(args.part), parts, args.n, args.dbias, args.type, (int)after);
}

}  // namespace route
