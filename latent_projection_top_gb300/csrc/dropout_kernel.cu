// Dropout from a counter-based generator, added to a residual.
//
// Every eight values of a row share one counter, and the 128 bits that Philox
// 4x32 of ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011) makes of it: 16 bits, a lot, for each.  A value
// is dropped if its lot is below the threshold.  Nothing but the seed and the
// offset is kept: the backward pass draws the same lots.
#include <type_traits>

#include "experts.cuh"
#include "layer_math.cuh"

namespace route {
namespace {

// The 128 bits of one counter: 64 bits of it are used, the others are 0.
__device__ __forceinline__ uint4 philox(unsigned long long counter, const DropoutArgs &a) {
    uint4 c = make_uint4((uint32_t)counter, (uint32_t)(counter >> 32), 0u, 0u);
#pragma unroll
    for (int r = 0; r < kPhiloxRounds; ++r) {
        const unsigned long long p0 = 0xD2511F53ull * c.x, p1 = 0xCD9E8D57ull * c.z;
        c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ a.keys[2 * r], (uint32_t)p1,
                       (uint32_t)(p0 >> 32) ^ c.w ^ a.keys[2 * r + 1], (uint32_t)p0);
    }
    return c;
}

// The comparison of the e-th of a counter's lots with the threshold: both in
// the upper half of a word, so that an odd one needs no shift.
struct Lots {
    uint32_t least;
    bool none;  // a threshold that no lot reaches
    __device__ __forceinline__ explicit Lots(const DropoutArgs &a)
        : least(a.threshold << 16), none(a.threshold > 0xFFFFu) {}
    __device__ __forceinline__ bool keep(const uint4 &bits, int e) const {
        const uint32_t w = e < 2 ? bits.x : e < 4 ? bits.y : e < 6 ? bits.z : bits.w;
        return (e % 2 ? w : w << 16) >= least && !none;
    }
};

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

__device__ __forceinline__ unsigned long long first_counter(const DropoutArgs &a) {
    return a.offset + (a.step != nullptr ? (unsigned long long)*a.step : 0ull);
}

// Rows that take 16 bytes at a time: eight values, a counter's, a thread.  FLAT:
// the rows follow one another in every matrix.  A dropped value is not
// multiplied: an infinity or a NaN there is gone.
//
// Bound by HBM where a residual is added (8192x7168 BF16 51 us, 352 MB, 6.9 TB/s),
// else by the instructions issued, of which ten rounds are 40 for eight values and
// half of those at half the rate (41 us, 235 MB, 5.7 TB/s).
template <int TY, bool FLAT>
__global__ void __launch_bounds__(256) dropout_kernel(const __grid_constant__ DropoutArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const unsigned groups = (unsigned)(a.dim + 7) >> 3, all = (unsigned)a.rows * groups;
    const unsigned step = gridDim.x * blockDim.x;
    const unsigned long long offset = first_counter(a);
    const Lots lots(a);
    for (unsigned i = blockIdx.x * blockDim.x + threadIdx.x; i < all; i += step) {
        long long x = 8ll * i, res = x, out = x;
        int n = 8;
        if (!FLAT) {
            const unsigned r = i / groups;
            const int c = (int)(i - r * groups) * 8;
            n = a.dim - c;
            x = r * a.ld_x + c, res = r * a.ld_res + c, out = r * a.ld_out + c;
        }
        const bool whole = FLAT || n >= 8;
        float v[8], add[8];
        load8<TY>(a.x, x, n, whole, v);
        if (a.residual != nullptr) load8<TY>(a.residual, res, n, whole, add);
        const uint4 bits = philox(offset + i, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = lots.keep(bits, e) ? v[e] * a.scale : 0.f;
        if (a.residual != nullptr)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += add[e];
        store8<TY>(a.out, out, n, whole, v);
    }
}

// Rows at any alignment: a warp takes 256 values of a row, each lane draws the
// lots of eight neighbours, and then has every 32nd value, so that its accesses
// are whole stretches of the row (8192x3583 BF16 with a residual 46 us; eight
// neighbours a lane, 68).
template <int TY>
__global__ void __launch_bounds__(256) dropout_any_kernel(const __grid_constant__ DropoutArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int groups = (a.dim + 7) >> 3, pieces = (a.dim + 255) >> 8, lane = threadIdx.x & 31;
    const unsigned long long offset = first_counter(a);
    const Lots lots(a);
    const unsigned all = (unsigned)a.rows * (unsigned)pieces, step = gridDim.x * (blockDim.x >> 5);
    for (unsigned i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < all; i += step) {
        const int r = (int)(i / (unsigned)pieces), c = (int)(i - (unsigned)r * pieces) * 256;
        const uint4 bits = philox(offset + (unsigned long long)((long long)r * groups + c / 8 + lane), a);
        uint32_t keep = 0u;  // bit e: the lane's eight neighbours' e-th
#pragma unroll
        for (int e = 0; e < 8; ++e) keep |= (lots.keep(bits, e) ? 1u : 0u) << e;
        const long long at = c + lane, ix = r * a.ld_x + at, ir = r * a.ld_res + at, io = r * a.ld_out + at;
        auto take = [&](auto all_there) {
            constexpr bool whole = decltype(all_there)::value;
            float v[8], res[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool there = whole || at + 32 * j < a.dim;
                v[j] = there ? load_elem(a.x, TY, ix + 32 * j) : 0.f;
                res[j] = there && a.residual != nullptr ? load_elem(a.residual, TY, ir + 32 * j) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t of = __shfl_sync(0xFFFFFFFFu, keep, 4 * j + (lane >> 3));
                v[j] = (of >> (lane & 7)) & 1u ? v[j] * a.scale : 0.f;
                if (a.residual != nullptr) v[j] += res[j];
                if (whole || at + 32 * j < a.dim) store_elem(a.out, TY, io + 32 * j, v[j]);
            }
        };
        if (c + 256 <= a.dim)
            take(std::true_type{});
        else
            take(std::false_type{});
    }
}

}  // namespace

cudaError_t dropout_launch(const DropoutArgs &args, int sms, cudaStream_t stream) {
    const int bytes = 16, per = bytes / layer_esize(args.type);
    auto rows_on = [&](const void *p, long long ld) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld % per == 0);
    };
    const bool vec = rows_on(args.x, args.ld_x) && rows_on(args.residual, args.ld_res) && rows_on(args.out, args.ld_out);
    // threads, a group or a lane each
    const long long all = (long long)args.rows * (vec ? (args.dim + 7) / 8 : (args.dim + 255) / 256 * 32);
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
    void *params[] = {const_cast<DropoutArgs *>(&args)};
    const bool flat = args.dim % 8 == 0 && args.ld_x == args.dim && args.ld_out == args.dim &&
                      (args.residual == nullptr || args.ld_res == args.dim);
#define ROUTE_DROPOUT(T)                                                  \
    (!vec   ? reinterpret_cast<const void *>(dropout_any_kernel<T>)       \
     : flat ? reinterpret_cast<const void *>(dropout_kernel<T, true>)     \
            : reinterpret_cast<const void *>(dropout_kernel<T, false>))
    const void *k = args.type == kBf16   ? ROUTE_DROPOUT(kBf16)
                    : args.type == kFp16 ? ROUTE_DROPOUT(kFp16)
                                         : ROUTE_DROPOUT(kFp32);
#undef ROUTE_DROPOUT
    return cudaLaunchKernelExC(&c, k, params);
}

}  // namespace route
