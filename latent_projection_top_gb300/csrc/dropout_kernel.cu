// Dropout from a counter-based generator, added to a residual.
//
// Every eight values of a row share one counter, and the 128 bits that Philox
// 4x32 of ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011) makes of it: 16 bits, a lot, for each.  A value
// is dropped if its lot is below the threshold.  Nothing but the seed and the
// offset is kept: the backward pass draws the same lots.
#include "experts.cuh"
#include "layer_math.cuh"

namespace route {
namespace {

// The 128 bits of one counter: 64 bits of it are used, the others are 0.
__device__ __forceinline__ uint4 philox(unsigned long long counter, unsigned long long key) {
    uint4 c = make_uint4((uint32_t)counter, (uint32_t)(counter >> 32), 0u, 0u);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const unsigned long long p0 = 0xD2511F53ull * c.x, p1 = 0xCD9E8D57ull * c.z;
        c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ k0, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k1, (uint32_t)p0);
        k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
    }
    return c;
}

// Eight values from element i on, `n` of them there; `vec`: as vectors.
template <int TY>
__device__ __forceinline__ void load8(const void *p, long long i, int n, bool vec, float (&v)[8]) {
    if constexpr (TY == kFp32) {
        const float *q = static_cast<const float *>(p) + i;
        if (vec) {
            const float4 a = reinterpret_cast<const float4 *>(q)[0], b = reinterpret_cast<const float4 *>(q)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? q[e] : 0.f;
        }
    } else {
        const uint16_t *q = static_cast<const uint16_t *>(p) + i;
        uint32_t w[4];
        if (vec) {
            const uint4 t = *reinterpret_cast<const uint4 *>(q);
            w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = 2 * e < n ? q[2 * e] : 0u, hi = 2 * e + 1 < n ? q[2 * e + 1] : 0u;
                w[e] = lo | (hi << 16);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack16(w[e], TY);
            v[2 * e] = f.x, v[2 * e + 1] = f.y;
        }
    }
}

template <int TY>
__device__ __forceinline__ void store8(void *p, long long i, int n, bool vec, const float (&v)[8]) {
    if constexpr (TY == kFp32) {
        float *q = static_cast<float *>(p) + i;
        if (vec) {
            reinterpret_cast<float4 *>(q)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(q)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) q[e] = v[e];
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack16(v[2 * e], v[2 * e + 1], TY);
        uint16_t *q = static_cast<uint16_t *>(p) + i;
        if (vec) {
            *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (2 * e < n) q[2 * e] = (uint16_t)w[e];
                if (2 * e + 1 < n) q[2 * e + 1] = (uint16_t)(w[e] >> 16);
            }
        }
    }
}

// Eight values a thread.  A dropped value is not multiplied: an infinity or a
// NaN there is gone.
template <int TY>
__global__ void __launch_bounds__(256) dropout_kernel(const __grid_constant__ DropoutArgs a, int vec) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int groups = (a.dim + 7) >> 3;
    const long long all = (long long)a.rows * groups;
    unsigned long long offset = a.offset;
    if (a.step != nullptr) offset += (unsigned long long)*a.step;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < all;
         i += (long long)gridDim.x * blockDim.x) {
        const int r = (int)(i / groups), c = (int)(i - (long long)r * groups) * 8, n = a.dim - c;
        const bool whole = vec && n >= 8;
        float v[8], res[8];
        load8<TY>(a.x, r * a.ld_x + c, n, whole, v);
        if (a.residual != nullptr) load8<TY>(a.residual, r * a.ld_res + c, n, whole, res);
        const uint4 bits = philox(offset + (unsigned long long)i, a.seed);
        const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t lot = (w[e / 2] >> (16 * (e % 2))) & 0xFFFFu;
            v[e] = lot >= a.threshold ? v[e] * a.scale : 0.f;
            if (a.residual != nullptr) v[e] += res[e];
        }
        store8<TY>(a.out, r * a.ld_out + c, n, whole, v);
    }
}

}  // namespace

cudaError_t dropout_launch(const DropoutArgs &args, int sms, cudaStream_t stream) {
    const int bytes = 16, per = bytes / layer_esize(args.type);
    auto rows_on = [&](const void *p, long long ld) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld % per == 0);
    };
    int vec = rows_on(args.x, args.ld_x) && rows_on(args.residual, args.ld_res) && rows_on(args.out, args.ld_out);
    const long long all = (long long)args.rows * ((args.dim + 7) / 8);
    const long long blocks = (all + 255) / 256, most = 8ll * sms;
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[1];
    c.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    c.blockDim = dim3(256);
    c.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    void *params[] = {const_cast<DropoutArgs *>(&args), &vec};
    const void *k = args.type == kBf16   ? reinterpret_cast<const void *>(dropout_kernel<kBf16>)
                    : args.type == kFp16 ? reinterpret_cast<const void *>(dropout_kernel<kFp16>)
                                         : reinterpret_cast<const void *>(dropout_kernel<kFp32>);
    return cudaLaunchKernelExC(&c, k, params);
}

}  // namespace route
