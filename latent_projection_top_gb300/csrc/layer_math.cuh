// Activations, 16-bit conversions and guarded vector access shared by the
// layer operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "layer.cuh"

namespace route {

// 1 / (1 + exp(-z)), the fast exponential and division: a few units in the
// last place, and 0 and 1 at the ends.
__device__ __forceinline__ float sigmoid_(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// The normal distribution's cumulative function and exp(-z^2 / 2), which the
// derivative of gelu needs as well.  With x = |z| / sqrt 2 and
// t = 1 / (1 + p x), erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2) within 1.5e-7
// (Abramowitz and Stegun, formula 7.1.26); no branches, so that a thread's
// values are computed side by side.
__device__ __forceinline__ float normal_cdf(float z, float &bell) {
    const float t = __fdividef(1.f, 1.f + 0.3275911f * 0.70710678f * fabsf(z));
    bell = __expf(-0.5f * z * z);
    const float q = t * (0.254829592f +
                         t * (-0.284496736f +
                              t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    const float tail = 0.5f * q * bell;
    return z < 0.f ? tail : 1.f - tail;
}

// The inner argument of gelu's tanh form, doubled: (1 + tanh u) / 2 is
// sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3).
__device__ __forceinline__ float tanh_arg(float z) {
    return 1.5957691f * z * (1.f + 0.044715f * z * z);
}

// v = act(v).  The activation is chosen once for all values: every form is
// free of branches, and W of them are in flight together (chosen per value,
// a tile's epilogue took nine times the tile's products).  NaN stays NaN.
template <int W>
__device__ __forceinline__ void act_values(int act, float (&v)[W]) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];
            break;
        case kActGelu:
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float bell;
                v[j] *= normal_cdf(v[j], bell);
            }
            break;
        case kActGeluTanh:
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] *= sigmoid_(tanh_arg(v[j]));
            break;
        case kActSilu:
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] *= sigmoid_(v[j]);
            break;
        case kActSigmoid:
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] = sigmoid_(v[j]);
            break;
        default: break;
    }
}

// a = act(z), d = act'(z); a may be z.
template <int W>
__device__ __forceinline__ void act_slopes(int act, const float (&z)[W], float (&a)[W], float (&d)[W]) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int j = 0; j < W; ++j) {
                d[j] = z[j] > 0.f ? 1.f : 0.f;
                a[j] = z[j] < 0.f ? 0.f : z[j];
            }
            break;
        case kActGelu:
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float bell;
                const float c = normal_cdf(z[j], bell), x = z[j];
                d[j] = c + x * 0.39894228f * bell;
                a[j] = x * c;
            }
            break;
        case kActGeluTanh:
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float x = z[j], s = sigmoid_(tanh_arg(x));
                d[j] = s + x * s * (1.f - s) * 1.5957691f * (1.f + 0.134145f * x * x);
                a[j] = x * s;
            }
            break;
        case kActSilu:
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float x = z[j], s = sigmoid_(x);
                d[j] = s * (1.f + x * (1.f - s));
                a[j] = x * s;
            }
            break;
        case kActSigmoid:
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float s = sigmoid_(z[j]);
                d[j] = s * (1.f - s);
                a[j] = s;
            }
            break;
        default:
#pragma unroll
            for (int j = 0; j < W; ++j) d[j] = 1.f, a[j] = z[j];
            break;
    }
}

__device__ __forceinline__ float load_elem(const void *p, int type, long long i) {
    if (type == kFp32) return static_cast<const float *>(p)[i];
    if (type == kFp16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ void store_elem(void *p, int type, long long i, float v) {
    if (type == kFp32)
        static_cast<float *>(p)[i] = v;
    else if (type == kFp16)
        static_cast<__half *>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// Two values of a 16-bit type from / to one word.
__device__ __forceinline__ float2 unpack16(uint32_t w, int type) {
    if (type == kFp16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack16(float a, float b, int type) {
    if (type == kFp16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void st_global_v8(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void ld_global_v8(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}

// W consecutive values at element i; `n` of them exist; `vec`: the address is
// aligned for whole-vector access (32 bytes for W = 16, 8 for W = 4).
template <int W>
__device__ __forceinline__ void load_vec(const void *p, int type, long long i, int n, bool vec,
                                         float (&v)[W]) {
    if (vec && n >= W) {
        if (type == kFp32) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
#pragma unroll
            for (int j = 0; j < W / 4; ++j) {
                const float4 t = q[j];
                v[4 * j] = t.x, v[4 * j + 1] = t.y, v[4 * j + 2] = t.z, v[4 * j + 3] = t.w;
            }
        } else if constexpr (W == 16) {
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 t = q[j];
                const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack16(w[e], type);
                    v[8 * j + 2 * e] = f.x, v[8 * j + 2 * e + 1] = f.y;
                }
            }
        } else {
            static_assert(W == 4, "vector width");
            const uint2 t = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
            const float2 f0 = unpack16(t.x, type), f1 = unpack16(t.y, type);
            v[0] = f0.x, v[1] = f0.y, v[2] = f1.x, v[3] = f1.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = j < n ? load_elem(p, type, i + j) : 0.f;
    }
}

// `vec`: 0 element by element, 1 the address is 16-byte aligned (8 for
// W = 4), 2 it is 32-byte aligned.
template <int W>
__device__ __forceinline__ void store_vec(void *p, int type, long long i, int n, int vec,
                                          const float (&v)[W]) {
    if (vec != 0 && n >= W) {
        if (type == kFp32) {
            float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
#pragma unroll
            for (int j = 0; j < W / 4; ++j)
                q[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else if constexpr (W == 16) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack16(v[2 * e], v[2 * e + 1], type);
            if (vec == 2) {
                st_global_v8(static_cast<uint16_t *>(p) + i, w);
            } else {
                uint4 *q = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i);
                q[0] = make_uint4(w[0], w[1], w[2], w[3]);
                q[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        } else {
            static_assert(W == 4, "vector width");
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) =
                make_uint2(pack16(v[0], v[1], type), pack16(v[2], v[3], type));
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j < n) store_elem(p, type, i + j, v[j]);
    }
}

// GemmProblem::vec
constexpr int kVecOut = 3, kVecRes = 4, kVecBias = 8;  // kVecOut: store_vec's `vec`

// Offsets of column c's pair in a gated block's saved row: 16 gate values,
// then the 16 up values of the same columns, so that one thread's 16-column
// chunk is one 128-byte line.
__host__ __device__ constexpr int saved_gate(int c) { return (c >> 4) * 32 + (c & 15); }

// What the epilogue of W columns of a row reads from memory besides bias,
// as it lies there: loaded ahead of its use (before the tile's sums are
// complete, and a chunk ahead of the one in work), because a load's latency
// in each of a tile's chunks costs more than the tile's products.
template <int EPI, int W>
struct EpiIn {
    static constexpr int kWords = EPI == kEpiDGate ? 2 * W : EPI == kEpiLinear ? W : 1;
    uint32_t w[kWords];
};

template <int EPI, int W>
__device__ __forceinline__ void epi_load(const GemmProblem &p, int r, int c, EpiIn<EPI, W> &in) {
    if (r >= p.M || c >= p.N) return;
    if constexpr (EPI == kEpiLinear) {
        if (p.residual == nullptr) return;
        const long long i = (long long)r * p.ld_res + c;
        const int n = p.N - c;
        if ((p.vec & kVecRes) && n >= W) {
            if (p.out_type == kFp32) {
                const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p.residual) + i);
#pragma unroll
                for (int j = 0; j < W / 4; ++j) {
                    const uint4 t = q[j];
                    in.w[4 * j] = t.x, in.w[4 * j + 1] = t.y, in.w[4 * j + 2] = t.z, in.w[4 * j + 3] = t.w;
                }
            } else if constexpr (W >= 8) {
                const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.residual) + i);
#pragma unroll
                for (int j = 0; j < W / 8; ++j) {
                    const uint4 t = q[j];
                    in.w[4 * j] = t.x, in.w[4 * j + 1] = t.y, in.w[4 * j + 2] = t.z, in.w[4 * j + 3] = t.w;
                }
            } else {
                const uint2 t = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.residual) + i);
                in.w[0] = t.x, in.w[1] = t.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j)
                in.w[j] = j >= n ? 0u
                          : p.out_type == kFp32 ? static_cast<const uint32_t *>(p.residual)[i + j]
                                                : static_cast<const uint16_t *>(p.residual)[i + j];
        }
    } else if constexpr (EPI == kEpiDGate) {
        const float *s = p.saved + (long long)r * p.ld_saved + saved_gate(c);
        if constexpr (W == 16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t t[8];
                ld_global_v8(s + 8 * k, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) in.w[8 * k + e] = t[e];
            }
        } else {
            const uint4 g = *reinterpret_cast<const uint4 *>(s);
            const uint4 u = *reinterpret_cast<const uint4 *>(s + 16);
            in.w[0] = g.x, in.w[1] = g.y, in.w[2] = g.z, in.w[3] = g.w;
            in.w[4] = u.x, in.w[5] = u.y, in.w[6] = u.z, in.w[7] = u.w;
        }
    }
}

// FP32 values to the plan's own memory, rows padded to whole chunks.
template <int W>
__device__ __forceinline__ void store_saved(float *p, const float (&v)[W]) {
    if constexpr (W == 16) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = __float_as_uint(v[8 * k + e]);
            st_global_v8(p + 8 * k, t);
        }
    } else {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

// The epilogue of W columns from column c of row r: v holds the FP32 sums
// (gated: u the up sums), `in` what epi_load read for them.
template <int EPI, int W>
__device__ __forceinline__ void epilogue(const GemmProblem &p, int r, int c, float (&v)[W],
                                         const float (&u)[W], const EpiIn<EPI, W> &in) {
    const int n = p.N - c;  // columns that exist
    if (r >= p.M || n <= 0) return;
    const long long o = (long long)r * p.ld_out + c;
    if constexpr (EPI == kEpiLinear) {
        if (p.bias != nullptr) {
            float b[W];
            load_vec<W>(p.bias, p.bias_type, c, n, (p.vec & kVecBias) != 0, b);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] += b[j];
        }
        if (p.saved != nullptr) store_saved<W>(p.saved + (long long)r * p.ld_saved + c, v);
        act_values<W>(p.act, v);
        if (p.residual != nullptr) {
            if (p.out_type == kFp32) {
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] += __uint_as_float(in.w[j]);
            } else if ((p.vec & kVecRes) && n >= W) {
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    const float2 f = unpack16(in.w[j], p.out_type);
                    v[2 * j] += f.x, v[2 * j + 1] += f.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] += unpack16(in.w[j], p.out_type).x;
            }
        }
        store_vec<W>(p.out, p.out_type, o, n, p.vec & kVecOut, v);
    } else if constexpr (EPI == kEpiGated) {
        if (p.saved != nullptr) {
            float *s = p.saved + (long long)r * p.ld_saved + saved_gate(c);
            store_saved<W>(s, v);
            store_saved<W>(s + 16, u);
        }
        act_values<W>(p.act, v);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] *= u[j];
        store_vec<W>(p.out, p.out_type, o, n, p.vec & kVecOut, v);
    } else {
        float a[W], d[W];
#pragma unroll
        for (int j = 0; j < W; ++j) a[j] = __uint_as_float(in.w[j]);
        act_slopes<W>(p.act, a, a, d);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            a[j] *= v[j];
            d[j] *= v[j] * __uint_as_float(in.w[W + j]);
        }
        store_vec<W>(p.out, p.out_type, o, n, p.vec & kVecOut, d);
        store_vec<W>(p.out2, p.out_type, o, n, p.vec & kVecOut, a);
    }
}

}  // namespace route
