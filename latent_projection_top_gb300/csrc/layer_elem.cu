// The layer operators' elementwise kernels: copies of operands that TMA
// cannot read in place, and a linear layer's d pre-activation with the
// column sums that are its bias's gradient.
#include "layer.cuh"
#include "layer_math.cuh"

namespace route {
namespace {

constexpr int kDzCols = 256;       // columns of a block: 32 threads of 8
constexpr int kDzMaxBlocks = 128;  // row blocks: partial sums a column

// Eight values a thread; columns past `cols` become zeros up to the next
// multiple of 8 (ld_dst is one).
__global__ void __launch_bounds__(256)
    repack_kernel(const uint16_t *src, long long ld_src, uint16_t *dst, long long ld_dst, int rows,
                  int cols) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int groups = (cols + 7) >> 3;
    const long long total = (long long)rows * groups;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const int r = (int)(i / groups), c = (int)(i % groups) * 8;
        const uint16_t *s = src + (long long)r * ld_src + c;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = c + 2 * e < cols ? s[2 * e] : 0u;
            const uint32_t hi = c + 2 * e + 1 < cols ? s[2 * e + 1] : 0u;
            w[e] = lo | (hi << 16);
        }
        *reinterpret_cast<uint4 *>(dst + (long long)r * ld_dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// dz = dout * act'(z) for a block of rows and 256 columns: a warp walks rows,
// a thread holds 8 columns and the FP32 sums of the dz it made, before they
// are rounded to 16 bits for the products.
__global__ void __launch_bounds__(256) dz_kernel(const __grid_constant__ DzArgs a, int rows_per_block,
                                                 int vec) {
    __shared__ float s_sum[8][kDzCols];
    if (threadIdx.x == 0 && a.trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * kDzCols + lane * 8;
    const int r1 = min(a.rows, (int)(blockIdx.y + 1) * rows_per_block);
    float sum[8] = {};
    if (c < a.n) {
        const int n = a.n - c;
        const uint16_t *dout = static_cast<const uint16_t *>(a.dout);
        uint16_t *dz = static_cast<uint16_t *>(a.dz);
        for (int r = blockIdx.y * rows_per_block + warp; r < r1; r += 8) {
            float v[8];
            const uint16_t *s = dout + (long long)r * a.ld_dout + c;
            if (vec && n >= 8) {
                const uint4 t = *reinterpret_cast<const uint4 *>(s);
                const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack16(w[e], a.type);
                    v[2 * e] = f.x, v[2 * e + 1] = f.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = e < n ? load_elem(s, a.type, e) : 0.f;
            }
            if (a.z != nullptr) {
                const float4 *q = reinterpret_cast<const float4 *>(a.z + (long long)r * a.ld_z + c);
                const float4 z0 = q[0], z1 = q[1];
                float z[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w}, d[8];
                act_slopes<8>(a.act, z, z, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = e < n ? v[e] * d[e] : 0.f;
            }
            if (dz != nullptr)  // ld_dz is a multiple of 8
                *reinterpret_cast<uint4 *>(dz + (long long)r * a.ld_dz + c) =
                    make_uint4(pack16(v[0], v[1], a.type), pack16(v[2], v[3], a.type),
                               pack16(v[4], v[5], a.type), pack16(v[6], v[7], a.type));
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += v[e];
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

// Column sums of `blocks` rows of partials, in order within each of eight
// runs and then run by run.
__global__ void __launch_bounds__(256) colsum_kernel(const float *part, int blocks, int n, void *out,
                                                     int type, int trigger) {
    __shared__ float s_sum[8][33];
    if (threadIdx.x == 0 && trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < n)
        for (int b = warp; b < blocks; b += 8) t += part[(long long)b * n + c];
    s_sum[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < n) {
#pragma unroll
        for (int w = 1; w < 8; ++w) t += s_sum[w][lane];
        store_elem(out, type, c, t);
    }
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

cudaError_t repack_launch(const void *src, long long ld_src, void *dst, long long ld_dst, int rows,
                          int cols, cudaStream_t stream) {
    const long long total = (long long)rows * ((cols + 7) / 8);
    const unsigned blocks = (unsigned)(total / 256 < 2432 ? (total + 255) / 256 : 2432);
    return launch_pdl(repack_kernel, dim3(blocks), dim3(256), stream,
                      static_cast<const uint16_t *>(src), ld_src, static_cast<uint16_t *>(dst),
                      ld_dst, rows, cols);
}

size_t dz_part_floats(int n) { return (size_t)kDzMaxBlocks * n; }

cudaError_t dz_launch(const DzArgs &args, cudaStream_t stream) {
    const int cb = (args.n + kDzCols - 1) / kDzCols;
    // about eight blocks an SM, eight rows at least to a block
    int rb = 1216 / cb;
    rb = rb < 1 ? 1 : rb > kDzMaxBlocks ? kDzMaxBlocks : rb;
    rb = rb > (args.rows + 7) / 8 ? (args.rows + 7) / 8 : rb;
    const int per = (args.rows + rb - 1) / rb;
    rb = (args.rows + per - 1) / per;
    const int vec = (reinterpret_cast<uintptr_t>(args.dout) & 15u) == 0 && args.ld_dout % 8 == 0;
    DzArgs first = args;
    first.trigger = args.trigger || args.dbias != nullptr;
    cudaError_t e = launch_pdl(dz_kernel, dim3(cb, rb), dim3(256), stream, first, per, vec);
    if (e != cudaSuccess || args.dbias == nullptr) return e;
    return launch_pdl(colsum_kernel, dim3((args.n + 31) / 32), dim3(256), stream,
                      static_cast<const float *>(args.part), rb, args.n, args.dbias, args.type,
                      args.trigger);
}

}  // namespace route
