// Activations, 16-bit conversions and guarded vector access shared by the
// layer operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "layer.cuh"
#include "layer_ptx.cuh"

namespace route {

__device__ __forceinline__ float ex2_(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 1 / (1 + exp(-z)), the fast exponential and reciprocal: a few units in the
// last place, and 0 and 1 at the ends.
__device__ __forceinline__ float sigmoid_(float z) { return rcp_(1.f + ex2_(-1.44269504f * z)); }

// The normal distribution's tail for two values at a time, a = min(|z|, 30):
// half of erfc(a / sqrt 2), as bell = exp(-a^2 / 2) times t P(t), t = 1 / (1 +
// 0.2735 a).  P is the polynomial of degree 8 whose largest relative error for
// a from 0 to 30 is least: fitted for this file (reweighted least squares in
// FP64), 4e-8.  With FP32's roundings the tail is within 4e-7 of itself for a
// up to 1, 1.5e-6 up to 5 (the exponent's rounding).  A polynomial of degree 4
// (Abramowitz and Stegun, formula 7.1.26) is right to 1.5e-7 of 1, which at
// z = -3.5 is 2e-4 of gelu; it saves 2-5% of a product with little else to do
// (2048x64x3584 10.8 us, so 11.3; 4096x3584x7168 120.5 and 121.5).  No branches,
// and FP32 pairs, because an epilogue's activations are bound by the
// instructions issued.  Past 30 all are 0.
__device__ __forceinline__ void normal_tail(float z0, float z1, uint64_t &a, uint64_t &tail, uint64_t &bell) {
    a = ptx::f32x2_pack(fminf(fabsf(z0), 30.f), fminf(fabsf(z1), 30.f));
    auto both = [](float c) { return ptx::f32x2_pack(c, c); };
    float e0, e1, d0, d1;
    ptx::f32x2_unpack(ptx::f32x2_mul(ptx::f32x2_mul(a, a), both(-0.5f * 1.44269504f)), e0, e1);
    ptx::f32x2_unpack(ptx::f32x2_fma(a, both(0.273499995f), both(1.f)), d0, d1);
    bell = ptx::f32x2_pack(ex2_(e0), ex2_(e1));
    const uint64_t t = ptx::f32x2_pack(rcp_(d0), rcp_(d1));
    uint64_t q = ptx::f32x2_fma(t, both(0.0278880764f), both(-0.11606431f));
    q = ptx::f32x2_fma(q, t, both(0.142815575f));
    q = ptx::f32x2_fma(q, t, both(-0.0457833074f));
    q = ptx::f32x2_fma(q, t, both(0.0940481573f));
    q = ptx::f32x2_fma(q, t, both(0.0768939033f));
    q = ptx::f32x2_fma(q, t, both(0.102065168f));
    q = ptx::f32x2_fma(q, t, both(0.109023206f));
    q = ptx::f32x2_fma(q, t, both(0.109113552f));
    tail = ptx::f32x2_mul(ptx::f32x2_mul(q, t), bell);
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
            for (int j = 0; j < W; j += 2) {  // z Phi(z) = max(z, 0) - |z| tail(|z|)
                uint64_t a, tail, bell;
                normal_tail(v[j], v[j + 1], a, tail, bell);
                float b0, b1;
                ptx::f32x2_unpack(ptx::f32x2_mul(a, tail), b0, b1);
                v[j] = max_nan(v[j], 0.f) - b0;
                v[j + 1] = max_nan(v[j + 1], 0.f) - b1;
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
            for (int j = 0; j < W; j += 2) {  // the slope is Phi(z) + z bell / sqrt(2 pi)
                uint64_t m, tail, bell;
                normal_tail(z[j], z[j + 1], m, tail, bell);
                float t[2], b[2], p[2];
                ptx::f32x2_unpack(tail, t[0], t[1]);
                ptx::f32x2_unpack(ptx::f32x2_mul(m, tail), b[0], b[1]);
                ptx::f32x2_unpack(
                    ptx::f32x2_mul(ptx::f32x2_mul(m, bell), ptx::f32x2_pack(0.39894228f, 0.39894228f)),
                    p[0], p[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = z[j + e];
                    d[j + e] = x < 0.f ? t[e] - p[e] : 1.f - t[e] + p[e];
                    if (x != x) d[j + e] = x;
                    a[j + e] = max_nan(x, 0.f) - b[e];
                }
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

// Four values of a type as they lie in memory (16-bit types: packed in the
// first two words), at element i; `n` of them exist; `vec`: the address is
// aligned for them all.
__device__ __forceinline__ void load4_raw(const void *p, int type, long long i, int n, bool vec,
                                          uint32_t (&w)[4]) {
    if (type == kFp32) {
        const uint32_t *q = static_cast<const uint32_t *>(p) + i;
        if (vec && n >= 4) {
            const uint4 t = *reinterpret_cast<const uint4 *>(q);
            w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = j < n ? q[j] : 0u;
        }
    } else {
        const uint16_t *q = static_cast<const uint16_t *>(p) + i;
        if (vec && n >= 4) {
            const uint2 t = *reinterpret_cast<const uint2 *>(q);
            w[0] = t.x, w[1] = t.y;
        } else {
            uint32_t e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = j < n ? q[j] : 0u;
            w[0] = e[0] | (e[1] << 16), w[1] = e[2] | (e[3] << 16);
        }
    }
}
__device__ __forceinline__ float4 values4(const uint32_t (&w)[4], int type) {
    if (type == kFp32)
        return make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]),
                           __uint_as_float(w[3]));
    const float2 a = unpack16(w[0], type), b = unpack16(w[1], type);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(void *p, int type, long long i, int n, bool vec, const float (&v)[4]) {
    if (!vec || n < 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) store_elem(p, type, i + j, v[j]);
    } else if (type == kFp32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) =
            make_uint2(pack16(v[0], v[1], type), pack16(v[2], v[3], type));
    }
}

// Epilogue::vec: rows that may be read and written four values at a time.
constexpr int kVecOut = 1, kVecRes = 2, kVecBias = 4;
// 16-bit rows of the result and the residual, and the bias, that may be
// accessed eight values at a time; of these the bias only.
constexpr int kVecPacked = 8, kVecAny = 16;

// The epilogues work on four columns of a row a thread, neighbouring threads
// on neighbouring columns, so that what they read and write of a row is whole
// lines.  (A row a thread, as the sums leave TMEM, wrote 32 bytes of 32 lines
// an instruction: 34 us for the 59 MB result of 4096x64x7168.)

// What they read from memory besides the bias, as it lies there: loaded
// ahead of its use, because a load's latency in each of a tile's steps costs
// more than the tile's products.
template <int EPI>
struct EpiIn {
    static constexpr int kWords = EPI == kEpiDGate ? 8 : epi_linear(EPI) ? 4 : 1;
    uint32_t w[kWords];
};

template <int EPI>
__device__ __forceinline__ void epi_load(const Epilogue &p, int r, int c, EpiIn<EPI> &in) {
    if (r >= p.M || c >= p.N) return;
    if constexpr (epi_linear(EPI)) {
        if (p.residual != nullptr)
            load4_raw(p.residual, p.out_type, (long long)r * p.ld_res + c, p.N - c,
                      (p.vec & kVecRes) != 0, in.w);
    } else if constexpr (EPI == kEpiDGate) {
        const long long i = (long long)r * p.ld_saved + c;
        const uint4 g = *reinterpret_cast<const uint4 *>(p.saved + i);
        const uint4 u = *reinterpret_cast<const uint4 *>(p.saved2 + i);
        in.w[0] = g.x, in.w[1] = g.y, in.w[2] = g.z, in.w[3] = g.w;
        in.w[4] = u.x, in.w[5] = u.y, in.w[6] = u.z, in.w[7] = u.w;
    }
}

// The epilogue of four columns from column c (a multiple of 4) of row r: v
// holds the FP32 sums (gated: u the up sums), `in` what epi_load read.
//
// A gated block's h, d gate and d up are rounded to the operands' 16 bits here,
// as dz is in layer_elem.cu: the next product reads them as tensor-core
// operands, which have no more (in FP32 they would take two or three products
// of 16-bit parts each).  With the result's own rounding the error against 64
// bits is 1.4 times that of one rounding; in FP16 they are infinite past 65504.
template <int EPI>
__device__ __forceinline__ void epilogue(const Epilogue &p, int r, int c, float (&v)[4],
                                         const float (&u)[4], const EpiIn<EPI> &in) {
    const int n = p.N - c;  // columns that exist
    if (r >= p.M || n <= 0) return;
    const long long o = (long long)r * p.ld_out + c;
    const bool vec = (p.vec & kVecOut) != 0;
    // rows of what is kept are padded to whole groups: no guard
    auto keep = [&](float *q, const float (&x)[4]) {
        *reinterpret_cast<float4 *>(q + (long long)r * p.ld_saved + c) = make_float4(x[0], x[1], x[2], x[3]);
    };
    if constexpr (epi_linear(EPI)) {
        if (p.bias != nullptr) {
            uint32_t w[4];
            load4_raw(p.bias, p.bias_type, c, n, (p.vec & kVecBias) != 0, w);
            const float4 b = values4(w, p.bias_type);
            v[0] += b.x, v[1] += b.y, v[2] += b.z, v[3] += b.w;
        }
        if constexpr (EPI == kEpiAct) {
            if (p.saved != nullptr) keep(p.saved, v);
            act_values<4>(p.act, v);
        }
        if (p.residual != nullptr) {
            const float4 b = values4(in.w, p.out_type);
            v[0] += b.x, v[1] += b.y, v[2] += b.z, v[3] += b.w;
        }
        store4(p.out, p.out_type, o, n, vec, v);
    } else if constexpr (EPI == kEpiGated) {
        if (p.saved != nullptr) {
            keep(p.saved, v);
            keep(p.saved2, u);
        }
        act_values<4>(p.act, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= u[j];
        store4(p.out, p.out_type, o, n, vec, v);
    } else {
        float a[4], d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = __uint_as_float(in.w[j]);
        act_slopes<4>(p.act, a, a, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] *= v[j];
            d[j] *= v[j] * __uint_as_float(in.w[4 + j]);
        }
        store4(p.out, p.out_type, o, n, vec, d);
        store4(p.out2, p.out_type, o, n, vec, a);
    }
}

// The same for R steps at once: a thread's four columns c of the rows r,
// r + step, ..  Each question that is the same for the whole tile (which
// type, is there a bias, ..) is asked once for 4 R values: asked for every
// four, the questions and not the memory set the time (plain 4096x64x7168:
// 77 us).  What is asked for a step is whether its row exists.
template <int EPI, int R>
struct GroupIn {
    static constexpr int kWords = EPI == kEpiDGate ? 8 : epi_linear(EPI) ? 2 : 1;
    uint32_t w[R][kWords];
};

template <int EPI, int R>
__device__ __forceinline__ void group_load(const Epilogue &p, int r, int c, int step, GroupIn<EPI, R> &in) {
    if (c >= p.N) return;
    if constexpr (epi_linear(EPI)) {
        if (p.residual == nullptr || p.out_type == kFp32) return;
        const uint16_t *q = static_cast<const uint16_t *>(p.residual) + (long long)r * p.ld_res + c;
        const long long move = step * p.ld_res;
        if ((p.vec & kVecRes) && c + 4 <= p.N) {
#pragma unroll
            for (int j = 0; j < R; ++j, q += move)
                if (r + j * step < p.M) {
                    const uint2 t = *reinterpret_cast<const uint2 *>(q);
                    in.w[j][0] = t.x, in.w[j][1] = t.y;
                }
        } else {
#pragma unroll
            for (int j = 0; j < R; ++j, q += move)
                if (r + j * step < p.M) {
                    const uint32_t e1 = c + 1 < p.N ? q[1] : 0, e2 = c + 2 < p.N ? q[2] : 0,
                                   e3 = c + 3 < p.N ? q[3] : 0;
                    in.w[j][0] = q[0] | (e1 << 16), in.w[j][1] = e2 | (e3 << 16);
                }
        }
    } else if constexpr (EPI == kEpiDGate) {
        const float *g = p.saved + (long long)r * p.ld_saved + c, *u = p.saved2 + (long long)r * p.ld_saved + c;
        const long long move = step * p.ld_saved;
#pragma unroll
        for (int j = 0; j < R; ++j, g += move, u += move)
            if (r + j * step < p.M) {
                const uint4 x = *reinterpret_cast<const uint4 *>(g), y = *reinterpret_cast<const uint4 *>(u);
                in.w[j][0] = x.x, in.w[j][1] = x.y, in.w[j][2] = x.z, in.w[j][3] = x.w;
                in.w[j][4] = y.x, in.w[j][5] = y.y, in.w[j][6] = y.z, in.w[j][7] = y.w;
            }
    }
}

// `vec`: rows take four values at a time; `n`: columns that exist.
template <int TY, int R>
__device__ __forceinline__ void group_store(void *out, long long ld, int r, int M, int c, int n, int step,
                                            bool vec, const float (&v)[4 * R]) {
    const long long move = step * ld;
    if constexpr (TY == kFp32) {
        float *q = static_cast<float *>(out) + (long long)r * ld + c;
#pragma unroll
        for (int j = 0; j < R; ++j, q += move)
            if (r + j * step < M) {
                if (vec && n >= 4) {
                    *reinterpret_cast<float4 *>(q) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < n) q[e] = v[4 * j + e];
                }
            }
    } else {
        uint16_t *q = static_cast<uint16_t *>(out) + (long long)r * ld + c;
        if (vec && n >= 4) {
#pragma unroll
            for (int j = 0; j < R; ++j, q += move)
                if (r + j * step < M)
                    *reinterpret_cast<uint2 *>(q) =
                        make_uint2(pack16(v[4 * j], v[4 * j + 1], TY), pack16(v[4 * j + 2], v[4 * j + 3], TY));
        } else {
#pragma unroll
            for (int j = 0; j < R; ++j, q += move)
                if (r + j * step < M) {
                    const uint32_t a = pack16(v[4 * j], v[4 * j + 1], TY), b = pack16(v[4 * j + 2], v[4 * j + 3], TY);
                    if (n > 0) q[0] = (uint16_t)a;
                    if (n > 1) q[1] = (uint16_t)(a >> 16);
                    if (n > 2) q[2] = (uint16_t)b;
                    if (n > 3) q[3] = (uint16_t)(b >> 16);
                }
        }
    }
}
template <int R>
__device__ __forceinline__ void group_store(void *out, const Epilogue &p, int r, int c, int step,
                                            const float (&v)[4 * R]) {
    const bool vec = (p.vec & kVecOut) != 0;
    if (p.out_type == kBf16)
        group_store<kBf16, R>(out, p.ld_out, r, p.M, c, p.N - c, step, vec, v);
    else if (p.out_type == kFp16)
        group_store<kFp16, R>(out, p.ld_out, r, p.M, c, p.N - c, step, vec, v);
    else
        group_store<kFp32, R>(out, p.ld_out, r, p.M, c, p.N - c, step, vec, v);
}
// FP32 values to memory of the plan's own, whose rows are padded.
template <int R>
__device__ __forceinline__ void group_keep(float *out, long long ld, int r, int M, int c, int step,
                                           const float (&v)[4 * R]) {
    group_store<kFp32, R>(out, ld, r, M, c, 4, step, true, v);
}

template <int EPI, int R>
__device__ __forceinline__ void group_epilogue(const Epilogue &p, int r, int c, int step, float (&v)[4 * R],
                                               float (&u)[EPI == kEpiGated ? 4 * R : 1],
                                               const GroupIn<EPI, R> &in) {
    if (c >= p.N) return;
    if constexpr (epi_linear(EPI)) {
        if (p.bias != nullptr) {
            uint32_t w[4];
            load4_raw(p.bias, p.bias_type, c, p.N - c, (p.vec & kVecBias) != 0, w);
            const float4 b = values4(w, p.bias_type);
#pragma unroll
            for (int j = 0; j < R; ++j) v[4 * j] += b.x, v[4 * j + 1] += b.y, v[4 * j + 2] += b.z, v[4 * j + 3] += b.w;
        }
        if constexpr (EPI == kEpiAct) {
            if (p.saved != nullptr) group_keep<R>(p.saved, p.ld_saved, r, p.M, c, step, v);
            act_values<4 * R>(p.act, v);
        }
        if (p.residual != nullptr) {
            if (p.out_type == kFp32) {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (r + j * step < p.M) {
                        uint32_t w[4];
                        load4_raw(p.residual, kFp32, (long long)(r + j * step) * p.ld_res + c, p.N - c,
                                  (p.vec & kVecRes) != 0, w);
                        const float4 b = values4(w, kFp32);
                        v[4 * j] += b.x, v[4 * j + 1] += b.y, v[4 * j + 2] += b.z, v[4 * j + 3] += b.w;
                    }
            } else if (p.out_type == kBf16) {
#pragma unroll
                for (int e = 0; e < 2 * R; ++e) {
                    const float2 f = unpack16(in.w[e / 2][e % 2], kBf16);
                    v[2 * e] += f.x, v[2 * e + 1] += f.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2 * R; ++e) {
                    const float2 f = unpack16(in.w[e / 2][e % 2], kFp16);
                    v[2 * e] += f.x, v[2 * e + 1] += f.y;
                }
            }
        }
        group_store<R>(p.out, p, r, c, step, v);
    } else if constexpr (EPI == kEpiGated) {
        if (p.saved != nullptr) {
            group_keep<R>(p.saved, p.ld_saved, r, p.M, c, step, v);
            group_keep<R>(p.saved2, p.ld_saved, r, p.M, c, step, u);
        }
        act_values<4 * R>(p.act, v);
#pragma unroll
        for (int j = 0; j < 4 * R; ++j) v[j] *= u[j];
        group_store<R>(p.out, p, r, c, step, v);
    } else {
        float a[4 * R], d[4 * R];
#pragma unroll
        for (int j = 0; j < 4 * R; ++j) a[j] = __uint_as_float(in.w[j / 4][j % 4]);
        act_slopes<4 * R>(p.act, a, a, d);
#pragma unroll
        for (int j = 0; j < 4 * R; ++j) {
            a[j] *= v[j];
            d[j] *= v[j] * __uint_as_float(in.w[j / 4][4 + j % 4]);
        }
        group_store<R>(p.out, p, r, c, step, d);
        group_store<R>(p.out2, p, r, c, step, a);
    }
}

// ---- a row's columns a thread, to be stored as 16-bit values ------------------

__device__ __forceinline__ void add_values(bool half, const uint32_t (&w)[4], float *v) {
    if (half) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack16(w[e], kFp16);
            v[2 * e] += f.x, v[2 * e + 1] += f.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack16(w[e], kBf16);
            v[2 * e] += f.x, v[2 * e + 1] += f.y;
        }
    }
}
template <int W>
__device__ __forceinline__ void packed_bias(const Epilogue &p, int c, bool half, float (&v)[W]) {
    const uint16_t *b = static_cast<const uint16_t *>(p.bias) + c;
#pragma unroll
    for (int h = 0; h < W; h += 8) {
        if (c + h >= p.N) break;
        if (c + h + 8 <= p.N) {
            const uint4 t = *reinterpret_cast<const uint4 *>(b + h);
            const uint32_t w[4] = {t.x, t.y, t.z, t.w};
            add_values(half, w, v + h);
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (c + h + e < p.N) v[h + e] += load_elem(b, half ? kFp16 : kBf16, h + e);
        }
    }
}
template <int W>
__device__ __forceinline__ void pack_values(bool half, const float (&v)[W], uint32_t (&w)[W / 2]) {
    if (half) {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) w[e] = pack16(v[2 * e], v[2 * e + 1], kFp16);
    } else {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) w[e] = pack16(v[2 * e], v[2 * e + 1], kBf16);
    }
}

// ---- the same, one column a thread --------------------------------------------
//
// For rows that cannot be accessed four values at a time (odd widths):
// neighbouring threads still take neighbouring columns, so that an
// instruction's accesses are one stretch of a row (four scattered values a
// thread write every 32-byte sector four times).  Of linear results only: what
// a gated block's products write (h, d gate, d up) has padded rows.

// Column c of rows r, r + step, .. of the residual: R of them.
template <int R>
__device__ __forceinline__ void column_load(const Epilogue &p, int r, int c, int step, uint32_t (&in)[R]) {
    if (c >= p.N || p.residual == nullptr) return;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int row = r + j * step;
        if (row >= p.M) break;
        const long long i = (long long)row * p.ld_res + c;
        in[j] = p.out_type == kFp32 ? static_cast<const uint32_t *>(p.residual)[i]
                                    : static_cast<const uint16_t *>(p.residual)[i];
    }
}

template <int R>
__device__ __forceinline__ void column_store(void *out, int type, long long ld, int r, int M, int c, int step,
                                             const float (&v)[R]) {
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (r + j * step < M) store_elem(out, type, (long long)(r + j * step) * ld + c, v[j]);
}

template <int EPI, int R>
__device__ __forceinline__ void column_epilogue(const Epilogue &p, int r, int c, int step, float (&v)[R],
                                                const uint32_t (&in)[R]) {
    static_assert(epi_linear(EPI), "rows of a gated block's products are padded");
    if (c >= p.N) return;
    if (p.bias != nullptr) {
        const float b = load_elem(p.bias, p.bias_type, c);
#pragma unroll
        for (int j = 0; j < R; ++j) v[j] += b;
    }
    if constexpr (EPI == kEpiAct) {
        if (p.saved != nullptr) column_store<R>(p.saved, kFp32, p.ld_saved, r, p.M, c, step, v);
        act_values<R>(p.act, v);
    }
    if (p.residual != nullptr) {
#pragma unroll
        for (int j = 0; j < R; ++j)
            v[j] += p.out_type == kFp32 ? __uint_as_float(in[j]) : unpack16(in[j], p.out_type).x;
    }
    column_store<R>(p.out, p.out_type, p.ld_out, r, p.M, c, step, v);
}

}  // namespace route
