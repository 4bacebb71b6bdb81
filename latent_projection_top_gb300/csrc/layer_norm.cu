// Layer norm of token rows, forward and backward.
//
//   y  = (x - mean) r gamma + beta,  r = 1 / sqrt(var + eps)
//   dx = r (g - mean(g) - xh mean(g xh)),  g = dy gamma,  xh = (x - mean) r
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Bound by HBM: forward 16384x7168 BF16 85 us (5.5 TB/s), backward 8192x7168
// 65.5 us (5.4 TB/s; 58 without the parameters' sums).
//
// x and dy are read once, and the variance is the sum of squared deviations
// from the mean, not a difference of large sums; nor is xh one of large
// products.  Sums are FP32.
#include <initializer_list>

#include "layer.cuh"
#include "layer_math.cuh"
#include "layer_ptx.cuh"

namespace route {
namespace {

constexpr int kMaxBlocks = 3;  // backward blocks an SM, at most

// Threads of a block and rows it holds, with up to t threads a row.
__host__ __device__ constexpr int block_of(int t) { return t > 32 ? t : 128; }
__host__ __device__ constexpr int rows_of(int t) { return block_of(t) / t; }

// ---- rows aligned for 16-byte access: a ring of rows in shared memory --------
//
// Memory-bound: 3 (forward: 2) times the row's bytes and little else, so what
// counts is that enough bytes are always on their way (about 45 KB an SM at
// this memory's rate and latency).  Blocks are persistent; a thread copies
// the 16-byte vectors that it will itself use of the next rows into its own
// places of a ring (cp.async: no registers held, no barrier to hand a row
// over), and per row the block meets only to add the row's sums.

// A 16-byte vector as it lies in memory, and as FP32 pairs: the arithmetic
// runs on pairs (fma.rn.f32x2), half the instructions, which at two or three
// blocks an SM bound the backward pass before memory does.
template <int TY>
constexpr int kVec = 16 / layer_esize(TY);  // values of a vector
template <int TY>
constexpr int kPairs = kVec<TY> / 2;
struct Run {
    uint32_t w[4];
};
template <int TY>
__device__ __forceinline__ void unpack_run(const Run &q, uint64_t (&x)[kPairs<TY>]) {
#pragma unroll
    for (int e = 0; e < kPairs<TY>; ++e) {
        if constexpr (TY == kFp32) {
            x[e] = ptx::f32x2_pack(__uint_as_float(q.w[2 * e]), __uint_as_float(q.w[2 * e + 1]));
        } else {
            const float2 f = unpack16(q.w[e], TY);
            x[e] = ptx::f32x2_pack(f.x, f.y);
        }
    }
}
// The same of a parameter's vector inside the loop over rows.  Unpacking does
// not change from row to row, and hoisted out of the loop it would hold twice
// the registers and spill (forward 16384x7168: 171 us); the empty statement
// keeps it in.
template <int TY>
__device__ __forceinline__ void unpack_param(Run &q, uint64_t (&x)[kPairs<TY>]) {
    if constexpr (TY != kFp32)
#pragma unroll
        for (int e = 0; e < 4; ++e) asm volatile("" : "+r"(q.w[e]));
    unpack_run<TY>(q, x);
}
__device__ __forceinline__ uint64_t pair(float v) { return ptx::f32x2_pack(v, v); }
__device__ __forceinline__ float pair_sum(uint64_t v) {
    float a, b;
    ptx::f32x2_unpack(v, a, b);
    return a + b;
}

// A row's T threads (a block, or a warp) hold V vectors each: vector v of
// thread t starts at column (v T + t) kVec.
template <int V, int TY>
struct Ring {
    // bytes of a row's place
    static __host__ __device__ constexpr uint32_t row_bytes(int T) { return (uint32_t)V * T * 16; }
    // Neighbours in t are neighbours in shared memory.
    static __device__ __forceinline__ uint32_t at(uint32_t base, int v, int T, int t) {
        return base + (uint32_t)(v * T + t) * 16u;
    }
    static __device__ __forceinline__ void copy(uint32_t base, const void *p, long long row, int dim,
                                                int T, int t) {
        const char *src = static_cast<const char *>(p) + row * layer_esize(TY) + t * 16;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if ((v * T + t) * kVec<TY> < dim)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(base, v, T, t)),
                             "l"(src + v * T * 16)
                             : "memory");
    }
    static __device__ __forceinline__ void load(uint32_t base, int v, int T, int t, Run &q) {
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(q.w[0]), "=r"(q.w[1]), "=r"(q.w[2]), "=r"(q.w[3])
                     : "r"(at(base, v, T, t))
                     : "memory");
    }
    static __device__ __forceinline__ void load(uint32_t base, int v, int T, int t,
                                                uint64_t (&x)[kPairs<TY>]) {
        Run q;
        load(base, v, T, t, q);
        unpack_run<TY>(q, x);
    }
};

// Store a vector at column i.
template <int TY>
__device__ __forceinline__ void store_pairs(void *p, long long i, const uint64_t (&x)[kPairs<TY>]) {
    float f[kVec<TY>];
#pragma unroll
    for (int e = 0; e < kPairs<TY>; ++e) ptx::f32x2_unpack(x[e], f[2 * e], f[2 * e + 1]);
    if constexpr (TY == kFp32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
    else
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
            make_uint4(pack16(f[0], f[1], TY), pack16(f[2], f[3], TY), pack16(f[4], f[5], TY),
                       pack16(f[6], f[7], TY));
}
// FP32 values of a vector's columns.
template <int TY>
__device__ __forceinline__ void store_sums(float *p, const uint64_t (&x)[kPairs<TY>]) {
#pragma unroll
    for (int e = 0; e < kPairs<TY>; e += 2) {
        float4 f;
        ptx::f32x2_unpack(x[e], f.x, f.y);
        ptx::f32x2_unpack(x[e + 1], f.z, f.w);
        *reinterpret_cast<float4 *>(p + 2 * e) = f;
    }
}

// A parameter's values of this thread, kept packed in registers.
template <int V, int TY>
__device__ __forceinline__ void load_param(const void *p, int T, int t, int dim, float none, Run (&q)[V]) {
    const uint32_t fill = TY == kFp32 ? __float_as_uint(none) : pack16(none, none, TY);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (p != nullptr && (v * T + t) * kVec<TY> < dim) {
            const uint4 x = static_cast<const uint4 *>(p)[v * T + t];
            q[v].w[0] = x.x, q[v].w[1] = x.y, q[v].w[2] = x.z, q[v].w[3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) q[v].w[e] = fill;
        }
    }
}

// Sums over a row's threads, the same in every thread and every run.  One
// barrier: consecutive sums use alternate scratch.
template <int MAXT>
__device__ __forceinline__ float row_sum(float a, float2 (*scratch)[MAXT / 32], int &turn, int T) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    if constexpr (MAXT > 32) {
        if ((threadIdx.x & 31) == 0) scratch[turn][threadIdx.x >> 5].x = a;
        __syncthreads();
        a = 0.f;
#pragma unroll
        for (int i = 0; i < MAXT / 32; ++i)
            if (32 * i < T) a += scratch[turn][i].x;
        turn ^= 1;
    }
    return a;
}
template <int MAXT>
__device__ __forceinline__ void row_sums(float &a, float &b, float2 (*scratch)[MAXT / 32], int &turn, int T) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if constexpr (MAXT > 32) {
        if ((threadIdx.x & 31) == 0) scratch[turn][threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < MAXT / 32; ++i)
            if (32 * i < T) {
                const float2 s = scratch[turn][i];
                a += s.x, b += s.y;
            }
        turn ^= 1;
    }
}

template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }


// Blocks an SM and rows of a ring: up to ~190 KB of rows an SM.  `t`: the
// most threads of a row that a kernel is made for.
__host__ __device__ constexpr int fwd_blocks(int t, int ty) {
    return t <= 128 ? 4 : t == 256 ? 2 : 1;
}
__host__ __device__ constexpr int bwd_blocks(int t, int ty) {
    return t == 32 ? 3 : t == 128 ? 3 : t == 256 ? (ty != kFp32 ? 2 : 1) : 1;
}
__host__ __device__ constexpr int depth_of(uint32_t block_bytes, uint32_t row_bytes) {
    const uint32_t d = block_bytes / row_bytes;
    return d > 6 ? 6 : d < 2 ? 2 : (int)d;
}
template <int T, int V, int TY>
__host__ __device__ constexpr int fwd_depth() {
    return depth_of(190u * 1024u / fwd_blocks(T, TY), Ring<V, TY>::row_bytes(T) * rows_of(T));
}
template <int T, int V, int TY>
__host__ __device__ constexpr int bwd_depth() {
    return depth_of(190u * 1024u / bwd_blocks(T, TY), 2 * Ring<V, TY>::row_bytes(T) * rows_of(T));
}

// MAXT: 32 (a warp a row, four rows a block), else the most threads of a
// block, which holds one row.
template <int MAXT, int V, int TY>
__global__ void __launch_bounds__(block_of(MAXT), fwd_blocks(MAXT, TY))
    norm_forward_ring_kernel(const __grid_constant__ NormArgs a) {
    using R = Ring<V, TY>;
    constexpr int kP = kPairs<TY>;
    constexpr int P = fwd_depth<MAXT, V, TY>(), kRows = rows_of(MAXT);
    extern __shared__ uint4 ring[];
    __shared__ float2 scratch[2][MAXT / 32];
    const int T = MAXT == 32 ? 32 : blockDim.x;
    const int t = threadIdx.x % T;
    const uint32_t place = R::row_bytes(T);
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + (threadIdx.x / T) * P * place;
    const int stride = gridDim.x * kRows;
    const int r0 = blockIdx.x * kRows + threadIdx.x / T;
    int turn = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
    for (int i = 0; i < P - 1; ++i) {
        if (r0 + i * stride < a.rows)
            R::copy(mine + i * place, a.x, (long long)(r0 + i * stride) * a.ld_x, a.dim, T, t);
        copy_commit();
    }
    Run gamma[V], beta[V];
    load_param<V, TY>(a.gamma, T, t, a.dim, 1.f, gamma);
    load_param<V, TY>(a.beta, T, t, a.dim, 0.f, beta);
    const float inv = 1.f / (float)a.dim;
    int slot = 0;
    for (int r = r0; r < a.rows; r += stride) {
        const int slot_in = slot == 0 ? P - 1 : slot - 1;
        if (r + (P - 1) * stride < a.rows)
            R::copy(mine + slot_in * place, a.x, (long long)(r + (P - 1) * stride) * a.ld_x, a.dim, T, t);
        copy_commit();
        copy_wait<P - 1>();
        const uint32_t base = mine + slot * place;
        slot = slot + 1 == P ? 0 : slot + 1;
        uint64_t x[V][kP], acc = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if ((v * T + t) * kVec<TY> >= a.dim) break;
            R::load(base, v, T, t, x[v]);
#pragma unroll
            for (int e = 0; e < kP; ++e) acc = ptx::f32x2_add(acc, x[v][e]);
        }
        const float mean = row_sum<MAXT>(pair_sum(acc), scratch, turn, T) * inv;
        const uint64_t mean2 = pair(-mean);
        acc = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if ((v * T + t) * kVec<TY> >= a.dim) break;
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                x[v][e] = ptx::f32x2_add(x[v][e], mean2);
                acc = ptx::f32x2_fma(x[v][e], x[v][e], acc);
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<MAXT>(pair_sum(acc), scratch, turn, T) * inv + a.eps);
        const uint64_t rstd2 = pair(rstd);
        if (t == 0 && a.stats != nullptr)
            *reinterpret_cast<float2 *>(a.stats + 2 * (long long)r) = make_float2(mean, rstd);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * kVec<TY>;
            if (c >= a.dim) break;
            uint64_t g[kP], b[kP];
            unpack_run<TY>(gamma[v], g);
            unpack_run<TY>(beta[v], b);
#pragma unroll
            for (int e = 0; e < kP; ++e)
                x[v][e] = ptx::f32x2_fma(ptx::f32x2_mul(x[v][e], rstd2), g[e], b[e]);
            store_pairs<TY>(a.y, (long long)r * a.ld_y + c, x[v]);
        }
    }
}

// A thread keeps the gain's and offset's gradient sums of its own columns
// over its rows in registers and writes them once, as a row of partials a
// block; x and dy are read from the ring twice rather than kept.
template <int MAXT, int V, int TY>
__global__ void __launch_bounds__(block_of(MAXT), bwd_blocks(MAXT, TY))
    norm_backward_ring_kernel(const __grid_constant__ NormArgs a) {
    using R = Ring<V, TY>;
    constexpr int kP = kPairs<TY>;
    constexpr int P = bwd_depth<MAXT, V, TY>(), kRows = rows_of(MAXT);
    extern __shared__ uint4 ring[];
    __shared__ float2 scratch[2][MAXT / 32];
    const int T = MAXT == 32 ? 32 : blockDim.x;
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    const uint32_t place = R::row_bytes(T);
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + sub * P * 2 * place;
    const int stride = gridDim.x * kRows;
    const int r0 = blockIdx.x * kRows + sub;
    int turn = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the sums follow; the last kernel of a call lets nothing launch early
    if (threadIdx.x == 0 && a.part != nullptr) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto copy_row = [&](int r, int slot) {
        R::copy(mine + slot * 2 * place, a.x, (long long)r * a.ld_x, a.dim, T, t);
        R::copy(mine + slot * 2 * place + place, a.dy, (long long)r * a.ld_dy, a.dim, T, t);
    };
    const float2 *stats = reinterpret_cast<const float2 *>(a.stats);
#pragma unroll
    for (int i = 0; i < P - 1; ++i) {
        if (r0 + i * stride < a.rows) copy_row(r0 + i * stride, i);
        copy_commit();
    }
    Run gamma[V];
    load_param<V, TY>(a.gamma, T, t, a.dim, 1.f, gamma);
    const float inv = 1.f / (float)a.dim;
    uint64_t dg[V][kP] = {}, db[V][kP] = {};
    float2 ms = r0 < a.rows ? stats[r0] : make_float2(0.f, 0.f);
    int slot = 0;
    for (int r = r0; r < a.rows; r += stride) {
        const int slot_in = slot == 0 ? P - 1 : slot - 1;
        if (r + (P - 1) * stride < a.rows) copy_row(r + (P - 1) * stride, slot_in);
        copy_commit();
        const float rstd = ms.y;
        // xh = (x - mean) rstd: x rstd - mean rstd, an instruction less (8192x7168
        // BF16 63.9 against 65.5 us), is a difference of large products in rows that
        // are far from zero (dgamma wrong by 1e-4 at 4096 deviations)
        const uint64_t rstd2 = pair(rstd), mean2 = pair(-ms.x);
        if (r + stride < a.rows) ms = stats[r + stride];
        copy_wait<P - 1>();
        const uint32_t base = mine + slot * 2 * place;
        slot = slot + 1 == P ? 0 : slot + 1;
        uint64_t a1 = 0u, a2 = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if ((v * T + t) * kVec<TY> >= a.dim) break;
            uint64_t x[kP], dy[kP], g[kP];
            R::load(base, v, T, t, x);
            R::load(base + place, v, T, t, dy);
            unpack_param<TY>(gamma[v], g);
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                const uint64_t xh = ptx::f32x2_mul(ptx::f32x2_add(x[e], mean2), rstd2);
                const uint64_t gy = ptx::f32x2_mul(dy[e], g[e]);
                dg[v][e] = ptx::f32x2_fma(dy[e], xh, dg[v][e]);
                db[v][e] = ptx::f32x2_add(dy[e], db[v][e]);
                a1 = ptx::f32x2_add(a1, gy);
                a2 = ptx::f32x2_fma(gy, xh, a2);
            }
        }
        if (a.dx == nullptr) continue;
        float s1 = pair_sum(a1), s2 = pair_sum(a2);
        row_sums<MAXT>(s1, s2, scratch, turn, T);
        // dx = rstd g dy - (rstd s1 + rstd s2 xh)
        const uint64_t k1 = pair(-rstd * s1 * inv), k2 = pair(-rstd * s2 * inv);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * kVec<TY>;
            if (c >= a.dim) break;
            uint64_t x[kP], dy[kP], g[kP];
            R::load(base, v, T, t, x);
            R::load(base + place, v, T, t, dy);
            unpack_param<TY>(gamma[v], g);
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                const uint64_t xh = ptx::f32x2_mul(ptx::f32x2_add(x[e], mean2), rstd2);
                dy[e] = ptx::f32x2_fma(ptx::f32x2_mul(dy[e], g[e]), rstd2, ptx::f32x2_fma(xh, k2, k1));
            }
            store_pairs<TY>(a.dx, (long long)r * a.ld_dx + c, dy);
        }
    }
    if (a.part == nullptr) return;
    float *part = a.part + (long long)blockIdx.x * 2 * a.dim;
    if constexpr (MAXT > 32) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * kVec<TY>;
            if (c < a.dim) {
                store_sums<TY>(part + c, dg[v]);
                store_sums<TY>(part + a.dim + c, db[v]);
            }
        }
    } else {
        // the block's rows meet in the ring's memory, gradient by gradient
        copy_wait<0>();
        float *acc = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
                store_sums<TY>(acc + (sub * V * 32 + v * 32 + t) * kVec<TY>, k ? db[v] : dg[v]);
            __syncthreads();
            for (int c = threadIdx.x; c < a.dim; c += block_of(MAXT)) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kRows; ++i) sum += acc[i * V * 32 * kVec<TY> + c];
                part[k * a.dim + c] = sum;
            }
        }
    }
}

// ---- any alignment: one element a thread at a time ------------------------------
//
// A row is held in the registers of T threads (up to 32 values each), thread
// t's value i at column i T + t.  The backward pass's rows come through a
// ring as above, but as the 4-byte words that they lie in (rows of 16-bit
// values may start in the middle of one), each copied by any thread of the
// row (8192x1001 BF16: 29 us, loaded directly 45).  The forward pass has
// registers for enough blocks to load directly (20 us, through a ring 49).

template <int TY>
__host__ __device__ constexpr uint32_t loose_bytes(int t) {  // a row's place
    return (uint32_t)(32 * t * layer_esize(TY) + 16);
}
// Two places of FP32 rows past 8192 do not fit: those are loaded directly.
template <int T, int TY>
constexpr bool kLooseRing = !(T == 512 && TY == kFp32);
__host__ __device__ constexpr int loose_blocks(int t) { return t == 512 ? 1 : t == 256 ? 2 : 3; }
template <int T, int TY>
__host__ __device__ constexpr int loose_depth() {
    return depth_of(186u * 1024u / loose_blocks(T), 2 * loose_bytes<TY>(T) * rows_of(T));
}

// Eight values at a time that no thread has are passed over, of 16-bit types
// (backward 8689x107 12.0 us, 17.6 with all 32; 1989x5149 42.6 and 55.4; where
// nothing can be passed over 8192x1001 29.3 and 27.8.  FP32, whose values need
// no unpacking, loses: 1989x5149 79.5 and 67.8).
template <int TY>
constexpr bool kSkip = TY != kFp32;

template <int T, int TY>
__device__ __forceinline__ void copy_words(uint32_t base, const void *p, long long row, int dim, int t) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) + (uintptr_t)(row * layer_esize(TY));
    const uintptr_t from = at & ~(uintptr_t)3;
    const int words = (int)((at - from + (uintptr_t)dim * layer_esize(TY) + 3) / 4);
    for (int i = t; i < words; i += T)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(base + 4u * i), "l"(from + 4u * i) : "memory");
}
// Values of the row that copy_words brought.
template <int T, int TY>
__device__ __forceinline__ void take_values(uint32_t base, const void *p, long long row, int t, int dim,
                                            float (&x)[32]) {
    if constexpr (TY == kFp32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            x[i] = 0.f;
            if (i * T + t < dim)
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[i]) : "r"(base + 4u * (i * T + t)) : "memory");
        }
    } else {
        base += (uint32_t)(reinterpret_cast<uintptr_t>(p) + (uintptr_t)(row * 2)) & 2u;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (kSkip<TY> && i % 8 == 0 && i * T >= dim) break;
            uint16_t w = 0;
            if (i * T + t < dim)
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(base + 2u * (i * T + t)) : "memory");
            x[i] = unpack16(w, TY).x;
        }
    }
}
template <int T, int TY>
__device__ __forceinline__ void load_values(const void *p, long long row, int t, int dim, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i * T + t < dim ? load_elem(p, TY, row + i * T + t) : 0.f;
}
template <int T>
__device__ __forceinline__ void row_sync() {
    if (T > 32)
        __syncthreads();
    else
        __syncwarp();
}

// Sum over the T threads of a row, the same in every thread and every run.
template <int T>
__device__ __forceinline__ float sum_of_row(float v, float *scratch) {
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

template <int T, int TY>
__global__ void __launch_bounds__(block_of(T)) norm_forward_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float scratch[T / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = threadIdx.x % T;
    const int r = blockIdx.x * rows_of(T) + threadIdx.x / T;
    if (r >= a.rows) return;  // whole rows: every thread of a row
    float x[32], s = 0.f;
    load_values<T, TY>(a.x, (long long)r * a.ld_x, t, a.dim, x);
#pragma unroll
    for (int i = 0; i < 32; ++i) s += x[i];
    const float inv = 1.f / (float)a.dim;
    const float mean = sum_of_row<T>(s, scratch) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (i % 8 == 0 && i * T >= a.dim) break;
        x[i] -= mean;
        if (i * T + t < a.dim) s += x[i] * x[i];
    }
    const float rstd = 1.f / sqrtf(sum_of_row<T>(s, scratch) * inv + a.eps);
    if (t == 0 && a.stats != nullptr)
        *reinterpret_cast<float2 *>(a.stats + 2 * (long long)r) = make_float2(mean, rstd);
    // FP32: eight columns' parameters before the first of their stores, ahead
    // of which a load does not move (8192x1001: 13.0 us, one by one 22.6; two-
    // byte loads, whose unpacking fills the time, 24.3 and 20.2)
    constexpr int kTogether = TY == kFp32 ? 8 : 1;
#pragma unroll
    for (int k = 0; k < 32; k += kTogether) {
        // no thread has any of these (8192x129 BF16 5.5 us, all 32 worked on 7.9)
        if (k % 8 == 0 && k * T >= a.dim) break;
        float g[kTogether], b[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            const int c = (k + i) * T + t;
            g[i] = a.gamma != nullptr && c < a.dim ? load_elem(a.gamma, TY, c) : 1.f;
            b[i] = a.beta != nullptr && c < a.dim ? load_elem(a.beta, TY, c) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            const int c = (k + i) * T + t;
            if (c < a.dim) store_elem(a.y, TY, (long long)r * a.ld_y + c, x[k + i] * rstd * g[i] + b[i]);
        }
    }
}

template <int T, int TY>
__global__ void __launch_bounds__(block_of(T), loose_blocks(T)) norm_backward_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kRows = rows_of(T);
    constexpr bool RING = kLooseRing<T, TY>;
    constexpr int P = RING ? loose_depth<T, TY>() : 1;
    constexpr uint32_t kPlace = loose_bytes<TY>(T);
    extern __shared__ uint4 ring[];
    __shared__ float scratch[T / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the sums follow; the last kernel of a call lets nothing launch early
    if (threadIdx.x == 0 && a.part != nullptr) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + sub * P * 2 * kPlace;
    const int stride = gridDim.x * kRows, r0 = blockIdx.x * kRows + sub;
    auto copy_row = [&](int r, int place) {
        copy_words<T, TY>(mine + place * 2 * kPlace, a.x, (long long)r * a.ld_x, a.dim, t);
        copy_words<T, TY>(mine + place * 2 * kPlace + kPlace, a.dy, (long long)r * a.ld_dy, a.dim, t);
    };
    if constexpr (RING)
        for (int i = 0; i < P - 1; ++i) {
            if (r0 + i * stride < a.rows) copy_row(r0 + i * stride, i);
            copy_commit();
        }
    const float inv = 1.f / (float)a.dim;
    float dg[32] = {}, db[32] = {};
    int slot = 0;
    for (int r = r0; r < a.rows; r += stride) {
        const float2 ms = *reinterpret_cast<const float2 *>(a.stats + 2 * (long long)r);
        const float mean = ms.x, rstd = ms.y;
        float xh[32], g[32], s1 = 0.f, s2 = 0.f;
        if constexpr (RING) {
            row_sync<T>();  // every thread has taken the last row's values
            if (r + (P - 1) * stride < a.rows) copy_row(r + (P - 1) * stride, slot == 0 ? P - 1 : slot - 1);
            copy_commit();
            copy_wait<P - 1>();
            row_sync<T>();
            const uint32_t base = mine + slot * 2 * kPlace;
            take_values<T, TY>(base, a.x, (long long)r * a.ld_x, t, a.dim, xh);
            take_values<T, TY>(base + kPlace, a.dy, (long long)r * a.ld_dy, t, a.dim, g);
            slot = slot + 1 == P ? 0 : slot + 1;
        } else {
            load_values<T, TY>(a.x, (long long)r * a.ld_x, t, a.dim, xh);
            load_values<T, TY>(a.dy, (long long)r * a.ld_dy, t, a.dim, g);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (kSkip<TY> && i % 8 == 0 && i * T >= a.dim) break;
            const float gm = a.gamma != nullptr && i * T + t < a.dim ? load_elem(a.gamma, TY, i * T + t) : 1.f;
            xh[i] = (xh[i] - mean) * rstd;
            dg[i] += g[i] * xh[i];
            db[i] += g[i];
            g[i] *= gm;  // zero past the row's end: dy is
            s1 += g[i];
            s2 += g[i] * xh[i];
        }
        if (a.dx == nullptr) continue;
        s1 = sum_of_row<T>(s1, scratch) * inv;
        s2 = sum_of_row<T>(s2, scratch) * inv;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (kSkip<TY> && i % 8 == 0 && i * T >= a.dim) break;
            if (i * T + t < a.dim)
                store_elem(a.dx, TY, (long long)r * a.ld_dx + i * T + t, rstd * (g[i] - s1 - xh[i] * s2));
        }
    }
    if (a.part == nullptr) return;
    float *part = a.part + (long long)blockIdx.x * 2 * a.dim;
    if constexpr (T > 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int c = i * T + t;
            if (c < a.dim) part[c] = dg[i], part[a.dim + c] = db[i];
        }
    } else {
        // the block's rows meet in the ring's memory, gradient by gradient
        copy_wait<0>();
        float *s_acc = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 32; ++i) s_acc[sub * 1024 + i * T + t] = k ? db[i] : dg[i];
            __syncthreads();
            for (int c = threadIdx.x; c < a.dim; c += block_of(T)) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kRows; ++i) sum += s_acc[i * 1024 + c];
                part[k * a.dim + c] = sum;
            }
        }
    }
}

// Column sums of the blocks' partials (read from L2, where they were just
// written): dgamma in the first dim columns, dbeta in the rest.  A block
// takes 32 columns; each of its 16 warps adds every sixteenth row, and the
// sums meet in order (8192x7168: 304 rows, 17 MB, about 3 us).
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps)
    norm_sum_kernel(const float *part, int blocks, int dim, void *dgamma, void *dbeta, int type) {
    __shared__ float s_sum[kSumWarps][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < 2 * dim) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += kSumWarps) t += __ldcg(part + (long long)b * 2 * dim + c);
    }
    s_sum[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < 2 * dim) {
#pragma unroll
        for (int w = 1; w < kSumWarps; ++w) t += s_sum[w][lane];
        if (c < dim) {
            if (dgamma != nullptr) store_elem(dgamma, type, c, t);
        } else if (dbeta != nullptr) {
            store_elem(dbeta, type, c - dim, t);
        }
    }
}

template <class... P, class... A>
cudaError_t launch_pdl(void (*fn)(P...), int grid, int block, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[1];
    c.gridDim = dim3(grid);
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
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

// Threads of a ring kernel's block: as few whole warps as hold the row in
// four runs a thread.
int threads_for(int t, int dim) { return t == 32 ? block_of(t) : ((dim + 31) / 32 + 31) / 32 * 32; }

int blocks_for(int rows, int t, int most) {
    const int need = (rows + rows_of(t) - 1) / rows_of(t);
    return need < most ? need : most;
}

template <int T, int V, int TY>
constexpr size_t fwd_smem() {
    return (size_t)fwd_depth<T, V, TY>() * rows_of(T) * Ring<V, TY>::row_bytes(T);
}
template <int T, int V, int TY>
constexpr size_t bwd_smem() {
    return (size_t)bwd_depth<T, V, TY>() * rows_of(T) * 2 * Ring<V, TY>::row_bytes(T);
}

// FP32 rows past 8192: two places of x and dy would not fit.
template <int T, int TY>
constexpr bool kHasBackwardRing = !(T == 512 && TY == kFp32);

template <int T, int V, int TY>
cudaError_t configure_one() {
    static_assert(fwd_smem<T, V, TY>() <= 224 * 1024, "shared memory");
    static_assert(!kHasBackwardRing<T, TY> || bwd_smem<T, V, TY>() <= 224 * 1024, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(norm_forward_ring_kernel<T, V, TY>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)fwd_smem<T, V, TY>());
    if constexpr (kHasBackwardRing<T, TY>)
        if (e == cudaSuccess) e = cudaFuncSetAttribute(norm_backward_ring_kernel<T, V, TY>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)bwd_smem<T, V, TY>());
    return e;
}
// Vectors a thread that hold n times eight values.
template <int TY>
constexpr int runs(int n) {
    return n * 8 / kVec<TY>;
}
template <int TY>
cudaError_t configure_type() {
    cudaError_t e = configure_one<32, runs<TY>(1), TY>();
    if (e == cudaSuccess) e = configure_one<32, runs<TY>(4), TY>();
    if (e == cudaSuccess) e = configure_one<128, runs<TY>(4), TY>();
    if (e == cudaSuccess) e = configure_one<256, runs<TY>(4), TY>();
    if (e == cudaSuccess) e = configure_one<512, runs<TY>(4), TY>();
    return e;
}

template <int T, int V, int TY>
cudaError_t forward_ring(const NormArgs &a, cudaStream_t stream) {
    return launch_pdl(norm_forward_ring_kernel<T, V, TY>,
                      blocks_for(a.rows, T, a.sms * fwd_blocks(T, TY)), threads_for(T, a.dim),
                      fwd_smem<T, V, TY>(), stream, a);
}
template <int TY>
cudaError_t forward_aligned(const NormArgs &a, cudaStream_t stream) {
    if (a.dim <= 256) return forward_ring<32, runs<TY>(1), TY>(a, stream);
    switch (threads_of(a.dim)) {
        case 32: return forward_ring<32, runs<TY>(4), TY>(a, stream);
        case 128: return forward_ring<128, runs<TY>(4), TY>(a, stream);
        case 256: return forward_ring<256, runs<TY>(4), TY>(a, stream);
        default: return forward_ring<512, runs<TY>(4), TY>(a, stream);
    }
}


template <int T, int TY>
constexpr size_t loose_smem() {
    return kLooseRing<T, TY> ? (size_t)loose_depth<T, TY>() * 2 * loose_bytes<TY>(T) * rows_of(T) : 0;
}
template <int T, int TY>
cudaError_t configure_loose() {
    static_assert(loose_smem<T, TY>() <= 224 * 1024, "shared memory");
    static_assert(T > 32 || loose_smem<T, TY>() >= 4 * 1024 * 4, "the gradients' sums");
    return cudaFuncSetAttribute(norm_backward_kernel<T, TY>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)loose_smem<T, TY>());
}
template <int T, int TY>
cudaError_t backward_loose(const NormArgs &a, int *grid, cudaStream_t stream) {
    *grid = blocks_for(a.rows, T, loose_blocks(T) * a.sms);
    return launch_pdl(norm_backward_kernel<T, TY>, *grid, block_of(T), loose_smem<T, TY>(), stream, a);
}
template <int TY>
cudaError_t forward_any(const NormArgs &a, cudaStream_t stream) {
    const int t = threads_of(a.dim), grid = (a.rows + rows_of(t) - 1) / rows_of(t);
    return launch_pdl(t == 32    ? norm_forward_kernel<32, TY>
                      : t == 128 ? norm_forward_kernel<128, TY>
                      : t == 256 ? norm_forward_kernel<256, TY>
                                 : norm_forward_kernel<512, TY>,
                      grid, block_of(t), 0, stream, a);
}
template <int TY>
cudaError_t backward_any(const NormArgs &a, int *grid, cudaStream_t stream) {
    const int t = threads_of(a.dim);
    return t == 32    ? backward_loose<32, TY>(a, grid, stream)
           : t == 128 ? backward_loose<128, TY>(a, grid, stream)
           : t == 256 ? backward_loose<256, TY>(a, grid, stream)
                      : backward_loose<512, TY>(a, grid, stream);
}

template <int T, int V, int TY>
cudaError_t backward_ring(const NormArgs &a, int *grid, cudaStream_t stream) {
    // A block writes its gradients' sums whatever rows it had: with three rows at
    // least to a block, the same number of blocks on every SM (300x7168 8.6 us,
    // a block a row 11.4; 4096x1024 10.9 and 12.0; with six rows 1024x2048 takes
    // 9.6, so 8.5).
    const int groups = (a.rows + rows_of(T) - 1) / rows_of(T);
    int each = bwd_blocks(T, TY);
    if (a.part != nullptr && each > groups / (3 * a.sms)) each = groups / (3 * a.sms);
    *grid = blocks_for(a.rows, T, a.sms * (each < 1 ? 1 : each));
    return launch_pdl(norm_backward_ring_kernel<T, V, TY>, *grid, threads_for(T, a.dim),
                      bwd_smem<T, V, TY>(), stream, a);
}
template <int TY>
cudaError_t backward_aligned(const NormArgs &a, int *grid, cudaStream_t stream) {
    if (a.dim <= 256) return backward_ring<32, runs<TY>(1), TY>(a, grid, stream);
    switch (threads_of(a.dim)) {
        case 32: return backward_ring<32, runs<TY>(4), TY>(a, grid, stream);
        case 128: return backward_ring<128, runs<TY>(4), TY>(a, grid, stream);
        case 256: return backward_ring<256, runs<TY>(4), TY>(a, grid, stream);
        default:
            if constexpr (kHasBackwardRing<512, TY>) return backward_ring<512, runs<TY>(4), TY>(a, grid, stream);
            return backward_any<TY>(a, grid, stream);
    }
}

}  // namespace

namespace {
template <int TY>
cudaError_t configure_loose_type() {
    cudaError_t e = configure_loose<32, TY>();
    if (e == cudaSuccess) e = configure_loose<128, TY>();
    if (e == cudaSuccess) e = configure_loose<256, TY>();
    return e == cudaSuccess ? configure_loose<512, TY>() : e;
}
}  // namespace

cudaError_t norm_configure() {
    for (cudaError_t e : {configure_type<kBf16>(), configure_type<kFp16>(), configure_type<kFp32>(),
                          configure_loose_type<kBf16>(), configure_loose_type<kFp16>(),
                          configure_loose_type<kFp32>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

size_t norm_part_floats(int dim, int sms) { return (size_t)kMaxBlocks * sms * 2 * dim; }

template <int TY>
static cudaError_t forward_typed(const NormArgs &a, cudaStream_t stream) {
    const int es = layer_esize(TY);
    const bool vec = a.dim % 8 == 0 && rows_aligned(a.x, a.ld_x, es) && rows_aligned(a.y, a.ld_y, es) &&
                     rows_aligned(a.gamma, 0, es) && rows_aligned(a.beta, 0, es);
    return vec ? forward_aligned<TY>(a, stream) : forward_any<TY>(a, stream);
}

template <int TY>
static cudaError_t backward_typed(const NormArgs &a, int *grid, cudaStream_t stream) {
    const int es = layer_esize(TY);
    const bool vec = a.dim % 8 == 0 && rows_aligned(a.x, a.ld_x, es) && rows_aligned(a.dy, a.ld_dy, es) &&
                     rows_aligned(a.dx, a.ld_dx, es) && rows_aligned(a.gamma, 0, es);
    return vec ? backward_aligned<TY>(a, grid, stream) : backward_any<TY>(a, grid, stream);
}

cudaError_t norm_forward_launch(const NormArgs &a, cudaStream_t stream) {
    return a.type == kBf16   ? forward_typed<kBf16>(a, stream)
           : a.type == kFp16 ? forward_typed<kFp16>(a, stream)
                             : forward_typed<kFp32>(a, stream);
}

cudaError_t norm_backward_launch(const NormArgs &args, cudaStream_t stream) {
    NormArgs a = args;
    const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
    if (!sums) a.part = nullptr;
    int grid = 0;
    const cudaError_t e = a.type == kBf16   ? backward_typed<kBf16>(a, &grid, stream)
                          : a.type == kFp16 ? backward_typed<kFp16>(a, &grid, stream)
                                            : backward_typed<kFp32>(a, &grid, stream);
    if (e != cudaSuccess || !sums) return e;
    return launch_pdl(norm_sum_kernel, (2 * a.dim + 31) / 32, 32 * kSumWarps, 0, stream,
                      static_cast<const float *>(a.part), grid, a.dim, a.dgamma, a.dbeta, a.type);
}

}  // namespace route
