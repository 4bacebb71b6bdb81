// Layer norm of token rows, forward and backward.
//
//   y  = (x - mean) r gamma + beta,  r = 1 / sqrt(var + eps)
//   dx = r (g - mean(g) - xh mean(g xh)),  g = dy gamma,  xh = (x - mean) r
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// A row is held in the registers of T threads (up to 32 values each), so x
// and dy are read once and the variance is the sum of squared deviations
// from the mean, not a difference of large sums.  Sums are FP32.
#include "layer.cuh"
#include "layer_math.cuh"

namespace route {
namespace {

constexpr int kV = 4;  // runs of eight values a thread
constexpr int kMaxPart = 304;

// Where value e of run v of thread t sits in the row: whole 16-byte vectors
// when rows are aligned for it, else one element a thread at a time.
template <int T, bool VEC>
__device__ __forceinline__ int col_of(int v, int e, int t) {
    return VEC ? (v * T + t) * 8 + e : (v * 8 + e) * T + t;
}

template <int T, bool VEC>
__device__ __forceinline__ void load_run(const void *p, int type, long long row, int v, int t,
                                         int dim, float (&x)[8]) {
    if constexpr (VEC) {
        const int c = (v * T + t) * 8;
        if (c < dim) {  // dim is a multiple of 8
            if (type == kFp32) {
                const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + row + c);
                const float4 a = q[0], b = q[1];
                x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
                x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
            } else {
                const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + row + c);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack16(w[e], type);
                    x[2 * e] = f.x, x[2 * e + 1] = f.y;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = col_of<T, false>(v, e, t);
            x[e] = c < dim ? load_elem(p, type, row + c) : 0.f;
        }
    }
}

template <int T, bool VEC>
__device__ __forceinline__ void store_run(void *p, int type, long long row, int v, int t, int dim,
                                          const float (&x)[8]) {
    if constexpr (VEC) {
        const int c = (v * T + t) * 8;
        if (c >= dim) return;
        if (type == kFp32) {
            float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + row + c);
            q[0] = make_float4(x[0], x[1], x[2], x[3]);
            q[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + row + c) =
                make_uint4(pack16(x[0], x[1], type), pack16(x[2], x[3], type),
                           pack16(x[4], x[5], type), pack16(x[6], x[7], type));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = col_of<T, false>(v, e, t);
            if (c < dim) store_elem(p, type, row + c, x[e]);
        }
    }
}

// Sum over the T threads of a row, the same in every thread and every run.
template <int T>
__device__ __forceinline__ float row_sum(float v, float *scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (T > 32) {
        const int w = threadIdx.x >> 5;
        __syncthreads();  // the last sum has been read
        if ((threadIdx.x & 31) == 0) scratch[w] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < T / 32; ++i) v += scratch[i];
    }
    return v;
}

template <int T, bool VEC>
__global__ void __launch_bounds__(T > 32 ? T : 128)
    norm_forward_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float scratch[T / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kRows = T > 32 ? 1 : 4;
    const int t = threadIdx.x % T;
    const int r = blockIdx.x * kRows + threadIdx.x / T;
    if (r >= a.rows) return;  // whole rows: every thread of a row
    const long long row = (long long)r * a.ld_x;
    float x[kV][8];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        load_run<T, VEC>(a.x, a.type, row, v, t, a.dim, x[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[v][e];
    }
    const float inv = 1.f / (float)a.dim;
    const float mean = row_sum<T>(s, scratch) * inv;
    s = 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[v][e] -= mean;
            if (col_of<T, VEC>(v, e, t) < a.dim) s += x[v][e] * x[v][e];
        }
    const float rstd = 1.f / sqrtf(row_sum<T>(s, scratch) * inv + a.eps);
    if (t == 0 && a.stats != nullptr) {
        a.stats[2 * (long long)r] = mean;
        a.stats[2 * (long long)r + 1] = rstd;
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        float g[8], b[8];
        if (a.gamma != nullptr) {
            load_run<T, VEC>(a.gamma, a.type, 0, v, t, a.dim, g);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = 1.f;
        }
        if (a.beta != nullptr) {
            load_run<T, VEC>(a.beta, a.type, 0, v, t, a.dim, b);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] = x[v][e] * rstd * g[e] + b[e];
        store_run<T, VEC>(a.y, a.type, (long long)r * a.ld_y, v, t, a.dim, x[v]);
    }
}

// Rows are dealt to `gridDim.x` blocks; a thread keeps the gain's and
// offset's gradient sums of its own columns over its rows in registers and
// writes them once, as one row of partials a block.
template <int T, bool VEC>
__global__ void __launch_bounds__(T > 32 ? T : 128)
    norm_backward_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kRows = T > 32 ? 1 : 4;
    __shared__ float scratch[T / 32];
    __shared__ float s_acc[T > 32 ? 1 : kRows * 1024];
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    const float inv = 1.f / (float)a.dim;
    float dg[kV][8] = {}, db[kV][8] = {};
    for (int r = blockIdx.x * kRows + sub; r < a.rows; r += gridDim.x * kRows) {
        const float mean = a.stats[2 * (long long)r], rstd = a.stats[2 * (long long)r + 1];
        float xh[kV][8], g[kV][8];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            float gm[8];
            load_run<T, VEC>(a.x, a.type, (long long)r * a.ld_x, v, t, a.dim, xh[v]);
            load_run<T, VEC>(a.dy, a.type, (long long)r * a.ld_dy, v, t, a.dim, g[v]);
            if (a.gamma != nullptr) {
                load_run<T, VEC>(a.gamma, a.type, 0, v, t, a.dim, gm);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) gm[e] = 1.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[v][e] = (xh[v][e] - mean) * rstd;
                dg[v][e] += g[v][e] * xh[v][e];
                db[v][e] += g[v][e];
                g[v][e] *= gm[e];  // zero past the row's end: dy is
                s1 += g[v][e];
                s2 += g[v][e] * xh[v][e];
            }
        }
        if (a.dx == nullptr) continue;
        s1 = row_sum<T>(s1, scratch) * inv;
        s2 = row_sum<T>(s2, scratch) * inv;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[v][e] = rstd * (g[v][e] - s1 - xh[v][e] * s2);
            store_run<T, VEC>(a.dx, a.type, (long long)r * a.ld_dx, v, t, a.dim, g[v]);
        }
    }
    if (a.part == nullptr) return;
    float *part = a.part + (long long)blockIdx.x * 2 * a.dim;
    if constexpr (T > 32) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = col_of<T, VEC>(v, e, t);
                if (c < a.dim) part[c] = dg[v][e], part[a.dim + c] = db[v][e];
            }
    } else {
        // the block's rows meet in shared memory, gradient by gradient
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < kV; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s_acc[sub * 1024 + col_of<T, VEC>(v, e, t)] = k ? db[v][e] : dg[v][e];
            __syncthreads();
            for (int c = threadIdx.x; c < a.dim; c += 32 * kRows) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kRows; ++i) sum += s_acc[i * 1024 + c];
                part[k * a.dim + c] = sum;
            }
        }
    }
}

// Column sums of the blocks' partials: dgamma in the first dim columns,
// dbeta in the rest.
__global__ void __launch_bounds__(256) norm_sum_kernel(const float *part, int blocks, int dim,
                                                       void *dgamma, void *dbeta, int type) {
    __shared__ float s_sum[8][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < 2 * dim)
        for (int b = warp; b < blocks; b += 8) t += part[(long long)b * 2 * dim + c];
    s_sum[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < 2 * dim) {
#pragma unroll
        for (int w = 1; w < 8; ++w) t += s_sum[w][lane];
        if (c < dim) {
            if (dgamma != nullptr) store_elem(dgamma, type, c, t);
        } else if (dbeta != nullptr) {
            store_elem(dbeta, type, c - dim, t);
        }
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

bool rows_aligned(const void *p, long long ld, int esize) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * esize % 16 == 0);
}

// Threads of a row: 32 values a thread at most.
int threads_of(int dim) { return dim <= 1024 ? 32 : dim <= 4096 ? 128 : dim <= 8192 ? 256 : 512; }

template <bool VEC>
cudaError_t forward(const NormArgs &a, cudaStream_t stream) {
    switch (threads_of(a.dim)) {
        case 32: return launch_pdl(norm_forward_kernel<32, VEC>, dim3((a.rows + 3) / 4), dim3(128), stream, a);
        case 128: return launch_pdl(norm_forward_kernel<128, VEC>, dim3(a.rows), dim3(128), stream, a);
        case 256: return launch_pdl(norm_forward_kernel<256, VEC>, dim3(a.rows), dim3(256), stream, a);
        default: return launch_pdl(norm_forward_kernel<512, VEC>, dim3(a.rows), dim3(512), stream, a);
    }
}

template <bool VEC>
cudaError_t backward(const NormArgs &a, int grid, cudaStream_t stream) {
    switch (threads_of(a.dim)) {
        case 32: return launch_pdl(norm_backward_kernel<32, VEC>, dim3(grid), dim3(128), stream, a);
        case 128: return launch_pdl(norm_backward_kernel<128, VEC>, dim3(grid), dim3(128), stream, a);
        case 256: return launch_pdl(norm_backward_kernel<256, VEC>, dim3(grid), dim3(256), stream, a);
        default: return launch_pdl(norm_backward_kernel<512, VEC>, dim3(grid), dim3(512), stream, a);
    }
}

}  // namespace

size_t norm_part_floats(int dim, int sms) {
    (void)sms;
    return (size_t)kMaxPart * 2 * dim;
}

cudaError_t norm_forward_launch(const NormArgs &a, cudaStream_t stream) {
    const int es = layer_esize(a.type);
    const bool vec = a.dim % 8 == 0 && rows_aligned(a.x, a.ld_x, es) && rows_aligned(a.y, a.ld_y, es) &&
                     rows_aligned(a.gamma, 0, es) && rows_aligned(a.beta, 0, es);
    return vec ? forward<true>(a, stream) : forward<false>(a, stream);
}

cudaError_t norm_backward_launch(const NormArgs &args, cudaStream_t stream) {
    NormArgs a = args;
    const int es = layer_esize(a.type);
    const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
    if (!sums) a.part = nullptr;
    const bool vec = a.dim % 8 == 0 && rows_aligned(a.x, a.ld_x, es) && rows_aligned(a.dy, a.ld_dy, es) &&
                     rows_aligned(a.dx, a.ld_dx, es) && rows_aligned(a.gamma, 0, es);
    const int per = threads_of(a.dim) == 32 ? 4 : 1;
    int grid = (a.rows + per - 1) / per;
    grid = grid < kMaxPart ? grid : kMaxPart;
    const cudaError_t e = vec ? backward<true>(a, grid, stream) : backward<false>(a, grid, stream);
    if (e != cudaSuccess || !sums) return e;
    return launch_pdl(norm_sum_kernel, dim3((2 * a.dim + 31) / 32), dim3(256), stream,
                      static_cast<const float *>(a.part), grid, a.dim, a.dgamma, a.dbeta, a.type);
}

}  // namespace route
