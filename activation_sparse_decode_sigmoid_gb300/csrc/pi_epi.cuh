// Device side of the products' epilogues: activations, their derivatives, and
// 8 consecutive outputs of a row at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pi_block.h"

namespace pi {
namespace {

template <typename T> struct C16;
template <> struct C16<__half> {
    static __device__ __forceinline__ float one(uint16_t u) { return __half2float(__ushort_as_half(u)); }
    static __device__ __forceinline__ uint16_t round(float f) { return __half_as_ushort(__float2half_rn(f)); }
    static __device__ __forceinline__ uint32_t round2(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <> struct C16<__nv_bfloat16> {
    static __device__ __forceinline__ float one(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }
    static __device__ __forceinline__ uint16_t round(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
    static __device__ __forceinline__ uint32_t round2(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// Clamp that keeps NaN (fminf and fmaxf would drop it): beyond +-lim the
// smooth functions below are within 2e-33 of their limits, and inf * 0 is avoided.
__device__ __forceinline__ float clampn(float z, float lim) { return z < -lim ? -lim : (z > lim ? lim : z); }

// 1 - Phi(x) for x >= 0 as exp(-x^2 / 2) t P(t), t = 1 / (1 + 0.35 x), with ex =
// exp(-x^2 / 2), which the derivative needs too.  t P(t) is the polynomial of
// seven terms nearest to erfcx(x / sqrt 2) / 2 over x <= 13.5 (beyond, ex is 0 or
// subnormal) in the sense of the largest relative error over 1 + 0.6 x^2, by
// linear programming: 1.3e-7, below what x^2 and the exponential lose.  So the
// tail keeps its relative precision, (8 + 4 x^2) steps of 2^-23 in all: GELU's
// values there are small, not 0.  (An approximation that was exact in absolute
// terms, two terms shorter, was off by 0.36 % at 6 and 1.5 % at 9.)
__device__ __forceinline__ float upper_tail(float x, float &ex)
{
    ex = __expf(-0.5f * x * x);
    const float t = __fdividef(1.f, fmaf(0.35f, x, 1.f));
    float q = fmaf(t, 0.045681693f, -0.18852648f);
    q = fmaf(t, q, 0.21733934f);
    q = fmaf(t, q, 0.0041316487f);
    q = fmaf(t, q, 0.14506322f);
    q = fmaf(t, q, 0.13650973f);
    q = fmaf(t, q, 0.13980091f);
    return t * q * ex;
}

// fn(z), and with both also fn'(z), which shares its exponential.  __expf(a) is
// off by up to 2 + 1.173 |a| steps of 2^-23, __fdividef by 2: below 2^-13 of the
// value where it is smallest, below 2^-16 where f16 has normal numbers, so far
// below the half step of a 16-bit output (2^-8, 2^-11).  fp32 outputs
// (pi_linear's out_dtype) have these errors as they are.  (Where a derivative
// crosses 0 they are relative to its terms, not to their sum.)
template <int FN> __device__ __forceinline__ float act_one(float z)
{
    if (FN == PI_FN_RELU) return z < 0.f ? 0.f : z;
    if (FN == PI_FN_SQRELU) return z < 0.f ? 0.f : z * z;
    if (FN == PI_FN_SIGMOID) return __fdividef(1.f, 1.f + __expf(-z)); // (0 below -87)
    if (FN == PI_FN_SILU) return z < -80.f ? -0.f : __fdividef(z, 1.f + __expf(-z));
    if (FN == PI_FN_GELU) {
        float ex;
        const float q = upper_tail(fabsf(clampn(z, 30.f)), ex);
        return z < -30.f ? -0.f : z * (z < 0.f ? q : 1.f - q);
    }
    if (FN == PI_FN_GELU_TANH) { // z (1 + tanh t) / 2 = z / (1 + exp(-2 t))
        const float c = clampn(z, 30.f);
        const float t = 0.79788456f * (c + 0.044715f * c * c * c);
        return z < -30.f ? -0.f : __fdividef(z, 1.f + __expf(-2.f * clampn(t, 40.f)));
    }
    return z;
}

template <int FN> __device__ __forceinline__ void act_both(float z, float &f, float &df)
{
    if (FN == PI_FN_RELU) f = z < 0.f ? 0.f : z, df = z > 0.f ? 1.f : 0.f;
    else if (FN == PI_FN_SQRELU) f = z < 0.f ? 0.f : z * z, df = z < 0.f ? 0.f : 2.f * z;
    else if (FN == PI_FN_SIGMOID) { // p (1 - p) = e q^2, the same on both sides: 1 - p has nothing left of it above 17
        const float e = __expf(-fabsf(z)), q = __fdividef(1.f, 1.f + e);
        f = z < 0.f ? e * q : q, df = e * q * q;
    } else if (FN == PI_FN_SILU) {
        const float c = clampn(z, 80.f);
        const float p = __fdividef(1.f, 1.f + __expf(-c));
        f = z < -80.f ? -0.f : z * p, df = p * (1.f + c * (1.f - p));
    } else if (FN == PI_FN_GELU) {
        const float c = clampn(z, 30.f);
        float ex;
        const float q = upper_tail(fabsf(c), ex), p = z < 0.f ? q : 1.f - q;
        f = z < -30.f ? -0.f : z * p;
        df = fmaf(0.39894228f * c, ex, p);
    } else if (FN == PI_FN_GELU_TANH) {
        const float c = clampn(z, 10.f);
        const float t = 0.79788456f * (c + 0.044715f * c * c * c);
        const float p = __fdividef(1.f, 1.f + __expf(-2.f * clampn(t, 40.f))); // (1 + tanh t) / 2
        f = z < -10.f ? -0.f : z * p;
        df = p + 2.f * c * p * (1.f - p) * 0.79788456f * (1.f + 0.134145f * c * c);
    } else
        f = z, df = 1.f;
}

template <int FN, int W> __device__ __forceinline__ void act_of(float (&v)[W])
{
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = act_one<FN>(v[i]);
}

template <int FN> __device__ __forceinline__ void both8_of(const float (&z)[8], float (&f)[8], float (&df)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) act_both<FN>(z[i], f[i], df[i]);
}

// (The choice of function stays outside the elements: inside an unrolled
// loop it filled the instruction cache, and a 2048 x 28672 x 8192 product
// with EPI_DACT took 1055 us.)
template <int W> __device__ __forceinline__ void acts(int fn, float (&v)[W])
{
    switch (fn) {
    case PI_FN_RELU: act_of<PI_FN_RELU>(v); break;
    case PI_FN_SQRELU: act_of<PI_FN_SQRELU>(v); break;
    case PI_FN_SIGMOID: act_of<PI_FN_SIGMOID>(v); break;
    case PI_FN_SILU: act_of<PI_FN_SILU>(v); break;
    case PI_FN_GELU: act_of<PI_FN_GELU>(v); break;
    case PI_FN_GELU_TANH: act_of<PI_FN_GELU_TANH>(v); break;
    default: break;
    }
}

__device__ __forceinline__ void both8(int fn, const float (&z)[8], float (&f)[8], float (&df)[8])
{
    switch (fn) {
    case PI_FN_RELU: both8_of<PI_FN_RELU>(z, f, df); break;
    case PI_FN_SQRELU: both8_of<PI_FN_SQRELU>(z, f, df); break;
    case PI_FN_SIGMOID: both8_of<PI_FN_SIGMOID>(z, f, df); break;
    case PI_FN_SILU: both8_of<PI_FN_SILU>(z, f, df); break;
    case PI_FN_GELU: both8_of<PI_FN_GELU>(z, f, df); break;
    case PI_FN_GELU_TANH: both8_of<PI_FN_GELU_TANH>(z, f, df); break;
    default: both8_of<PI_FN_NONE>(z, f, df); break;
    }
}

__device__ __forceinline__ float act1(int fn, float z)
{
    switch (fn) {
    case PI_FN_RELU: return act_one<PI_FN_RELU>(z);
    case PI_FN_SQRELU: return act_one<PI_FN_SQRELU>(z);
    case PI_FN_SIGMOID: return act_one<PI_FN_SIGMOID>(z);
    case PI_FN_SILU: return act_one<PI_FN_SILU>(z);
    case PI_FN_GELU: return act_one<PI_FN_GELU>(z);
    case PI_FN_GELU_TANH: return act_one<PI_FN_GELU_TANH>(z);
    default: return z;
    }
}

// ---------------------------------------------------------------- 8 elements
template <typename T> __device__ __forceinline__ void unpack8(const uint4 &q, float (&v)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = C16<T>::one((uint16_t)(w[i] & 0xffffu));
        v[2 * i + 1] = C16<T>::one((uint16_t)(w[i] >> 16));
    }
}

template <typename T> __device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(C16<T>::round2(v[0], v[1]), C16<T>::round2(v[2], v[3]), C16<T>::round2(v[4], v[5]),
                      C16<T>::round2(v[6], v[7]));
}

// 8 16-bit elements at p (n of them exist; the rest read as 0)
template <typename T> __device__ __forceinline__ void load8(const uint16_t *p, int n, bool vec, float (&v)[8])
{
    if (vec && n >= 8) {
        unpack8<T>(*reinterpret_cast<const uint4 *>(p), v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? C16<T>::one(p[i]) : 0.f;
}

template <typename T> __device__ __forceinline__ void store8(uint16_t *p, int n, bool vec, const float (&v)[8])
{
    if (vec && n >= 8) {
        *reinterpret_cast<uint4 *>(p) = pack8<T>(v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = C16<T>::round(v[i]);
}

__device__ __forceinline__ void load8f(const float *p, int n, bool vec, float (&v)[8])
{
    if (vec && n >= 8) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
}

__device__ __forceinline__ void store8f(float *p, int n, bool vec, const float (&v)[8])
{
    if (vec && n >= 8) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
}

// The epilogue of row `row`, columns [col, col + 8) (col a multiple of 8;
// the caller checks row < M and col < N): v the accumulators, v2 the second
// product's (EPI_GATED).
template <typename T, int MODE>
__device__ __forceinline__ void epilogue8(const Epi &e, int N, int64_t row, int col, float (&v)[8], float (&v2)[8])
{
    const int n = N - col;
    if (MODE == EPI_LINEAR) {
        if (e.bias) {
            float b[8];
            load8<T>(e.bias + col, n, e.vec & V_BIAS, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += b[i];
        }
        if (e.out2) store8<T>(e.out2 + row * e.ld2 + col, n, e.vec & V_OUT2, v);
        acts(e.fn, v);
        if (e.scale != 1.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= e.scale;
        }
        if (e.res) {
            float r[8];
            if (e.out32) load8f(static_cast<const float *>(e.res) + row * e.ldr + col, n, e.vec & V_RES, r);
            else load8<T>(static_cast<const uint16_t *>(e.res) + row * e.ldr + col, n, e.vec & V_RES, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
        }
        if (e.out32) store8f(static_cast<float *>(e.out) + row * e.ldo + col, n, e.vec & V_OUT, v);
        else store8<T>(static_cast<uint16_t *>(e.out) + row * e.ldo + col, n, e.vec & V_OUT, v);
    } else if (MODE == EPI_GATED) {
        if (e.bias) {
            float b[8];
            load8<T>(e.bias + col, n, e.vec & V_BIAS, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += b[i];
        }
        if (e.bias2) {
            float b[8];
            load8<T>(e.bias2 + col, n, e.vec & V_BIAS2, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v2[i] += b[i];
        }
        if (e.out2) store8<T>(e.out2 + row * e.ld2 + col, n, e.vec & V_OUT2, v);
        if (e.out3) store8<T>(e.out3 + row * e.ld3 + col, n, e.vec & V_OUT3, v2);
        acts(e.fn, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= v2[i];
        store8<T>(static_cast<uint16_t *>(e.out) + row * e.ldo + col, n, e.vec & V_OUT, v);
    } else {
        float g[8], f[8], df[8];
        load8<T>(e.in1 + row * e.ldi1 + col, n, e.vec & V_IN1, g);
        both8(e.fn, g, f, df);
        if (e.in2) {
            float u[8];
            load8<T>(e.in2 + row * e.ldi2 + col, n, e.vec & V_IN2, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                u[i] *= v[i] * df[i];
                v[i] *= f[i];
            }
            store8<T>(static_cast<uint16_t *>(e.out) + row * e.ldo + col, n, e.vec & V_OUT, u);
            store8<T>(e.out2 + row * e.ld2 + col, n, e.vec & V_OUT2, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= e.scale * df[i];
            store8<T>(static_cast<uint16_t *>(e.out) + row * e.ldo + col, n, e.vec & V_OUT, v);
        }
    }
}

// The epilogue of one element (EPI_LINEAR, EPI_GATED).
template <typename T, int MODE>
__device__ __forceinline__ void epilogue1(const Epi &e, int64_t row, int col, float v, float v2)
{
    if (e.bias) v += C16<T>::one(e.bias[col]);
    if (MODE == EPI_GATED && e.bias2) v2 += C16<T>::one(e.bias2[col]);
    if (e.out2) e.out2[row * e.ld2 + col] = C16<T>::round(v);
    if (MODE == EPI_GATED && e.out3) e.out3[row * e.ld3 + col] = C16<T>::round(v2);
    v = act1(e.fn, v);
    if (MODE == EPI_GATED) v *= v2;
    else {
        v *= e.scale;
        if (e.res)
            v += e.out32 ? static_cast<const float *>(e.res)[row * e.ldr + col]
                         : C16<T>::one(static_cast<const uint16_t *>(e.res)[row * e.ldr + col]);
        if (e.out32) {
            static_cast<float *>(e.out)[row * e.ldo + col] = v;
            return;
        }
    }
    static_cast<uint16_t *>(e.out)[row * e.ldo + col] = C16<T>::round(v);
}

} // namespace
} // namespace pi
