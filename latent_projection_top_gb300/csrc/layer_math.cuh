// Activations, 16-bit conversions and guarded vector access shared by the
// layer operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "layer.cuh"

namespace route {

__device__ __forceinline__ float sigmoidf_(float z) { return 1.f / (1.f + expf(-z)); }

// act(z).  NaN stays NaN in every form.
__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case kActRelu: return z < 0.f ? 0.f : z;
        case kActGelu: return 0.5f * z * erfcf(-0.70710678f * z);
        case kActGeluTanh:  // z (1 + tanh u) / 2 = z sigmoid(2 u)
            return z * sigmoidf_(1.5957691f * (z + 0.044715f * z * z * z));
        case kActSilu: return z * sigmoidf_(z);
        case kActSigmoid: return sigmoidf_(z);
        default: return z;
    }
}

// act(z) and act'(z).
__device__ __forceinline__ void act_both(int act, float z, float &a, float &d) {
    switch (act) {
        case kActRelu:
            a = z < 0.f ? 0.f : z;
            d = z > 0.f ? 1.f : 0.f;
            break;
        case kActGelu: {
            const float c = 0.5f * erfcf(-0.70710678f * z);
            a = z * c;
            d = c + z * 0.39894228f * expf(-0.5f * z * z);
            break;
        }
        case kActGeluTanh: {
            const float s = sigmoidf_(1.5957691f * (z + 0.044715f * z * z * z));
            a = z * s;
            d = s + z * s * (1.f - s) * 1.5957691f * (1.f + 0.134145f * z * z);
            break;
        }
        case kActSilu: {
            const float s = sigmoidf_(z);
            a = z * s;
            d = s * (1.f + z * (1.f - s));
            break;
        }
        case kActSigmoid:
            a = sigmoidf_(z);
            d = a * (1.f - a);
            break;
        default:
            a = z;
            d = 1.f;
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

// The epilogue of W columns from column c of row r (r < M): v holds the FP32
// sums (gated: u the up sums).
template <int EPI, int W>
__device__ __forceinline__ void epilogue(const GemmProblem &p, int r, int c, float (&v)[W],
                                         const float (&u)[W]) {
    const int n = p.N - c;  // columns that exist
    if (n <= 0) return;
    const long long o = (long long)r * p.ld_out + c;
    if constexpr (EPI == kEpiLinear) {
        if (p.bias != nullptr) {
            float b[W];
            load_vec<W>(p.bias, p.bias_type, c, n, (p.vec & kVecBias) != 0, b);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] += b[j];
        }
        if (p.saved != nullptr)  // rows padded to whole chunks: no guard
            store_vec<W>(p.saved, kFp32, (long long)r * p.ld_saved + c, W, 1, v);
        if (p.act != kActNone) {
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] = act_value(p.act, v[j]);
        }
        if (p.residual != nullptr) {
            float b[W];
            load_vec<W>(p.residual, p.out_type, (long long)r * p.ld_res + c, n, (p.vec & kVecRes) != 0, b);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] += b[j];
        }
        store_vec<W>(p.out, p.out_type, o, n, p.vec & kVecOut, v);
    } else if constexpr (EPI == kEpiGated) {
        if (p.saved != nullptr) {
            const long long s = (long long)r * p.ld_saved + saved_gate(c);
            store_vec<W>(p.saved, kFp32, s, W, 1, v);
            store_vec<W>(p.saved, kFp32, s + 16, W, 1, u);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = act_value(p.act, v[j]) * u[j];
        store_vec<W>(p.out, p.out_type, o, n, p.vec & kVecOut, v);
    } else {
        const long long s = (long long)r * p.ld_saved + saved_gate(c);
        float g[W], up[W];
        load_vec<W>(p.saved, kFp32, s, W, true, g);
        load_vec<W>(p.saved, kFp32, s + 16, W, true, up);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float a, d;
            act_both(p.act, g[j], a, d);
            g[j] = v[j] * up[j] * d;
            up[j] = v[j] * a;
        }
        store_vec<W>(p.out, p.out_type, o, n, p.vec & kVecOut, g);
        store_vec<W>(p.out2, p.out_type, o, n, p.vec & kVecOut, up);
    }
}

}  // namespace route
