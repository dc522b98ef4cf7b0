// Microscaled matrices (PI_MX8, PI_MX4), device side: a block's scale, its
// elements' rounding, and where they lie.
//
// A block's scale is the least power of two s with amax / s <= the type's
// largest value (448 = 1.75 2^8, 6 = 1.5 2^2): taken from the bits of amax, so
// it is exact.  x / s is a product with a power of two, exact as long as it is
// normal (what is not lies far below half of the least element), and the
// conversion rounds it once, to nearest, ties to even.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pi.h"
#include "pi_kernels.h"

namespace pi {

// rows and columns are padded to tiles of 128 in the scales, columns in the codes
inline __host__ __device__ int mx_tiles(int n) { return (n + 127) / 128; }
inline __host__ __device__ int64_t mx_row_bytes(int kind, int cols) { return (int64_t)mx_tiles(cols) * (kind == PI_MX8 ? 128 : 64); }
inline __host__ __device__ int64_t mx_scale_bytes(int rows, int cols) { return (int64_t)mx_tiles(rows) * mx_tiles(cols) * 512; }

// the scales of row r, blocks 4 t to 4 t + 3: four bytes in a row
inline __host__ __device__ int64_t mx_scale_at(int64_t r, int t, int tiles)
{
    return ((r >> 7) * tiles + t) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

#ifdef __CUDACC__
namespace {

template <int KIND> struct Mx; // KIND: PI_MX8, PI_MX4
template <> struct Mx<PI_MX8> {
    static constexpr uint32_t emax = 8, mant = 0x600000u; // 448's exponent and mantissa bits
};
template <> struct Mx<PI_MX4> {
    static constexpr uint32_t emax = 2, mant = 0x400000u; // 6's
};

// largest magnitude so far, as the bits of a non-negative float: NaN and
// infinity come out above everything
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// the scale's byte
template <int KIND> __device__ __forceinline__ uint32_t mx_scale(uint32_t amax)
{
    if (amax >= 0x7f800000u) return 255u;
    const uint32_t e = (amax >> 23) + ((amax & 0x7fffffu) > Mx<KIND>::mant ? 1u : 0u);
    return e > Mx<KIND>::emax ? e - Mx<KIND>::emax : 0u;
}
// what elements are multiplied with (a byte of 255: with NaN)
__device__ __forceinline__ float mx_inverse(uint32_t code)
{
    return code == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - code) << 23); // (code <= 253: a normal power)
}
__device__ __forceinline__ float mx_power(uint32_t code)
{
    return code == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(code ? code << 23 : 0x400000u);
}

// eight elements: 8 or 4 bytes
template <int KIND> __device__ __forceinline__ uint2 mx_pack8(const float (&v)[8])
{
    uint2 q = make_uint2(0, 0);
    if (KIND == PI_MX8) { // (NaN: 0x7f)
        asm("{ .reg .b16 a, b, c, d; cvt.rn.satfinite.e4m3x2.f32 a, %3, %2; cvt.rn.satfinite.e4m3x2.f32 b, %5, %4;"
            " cvt.rn.satfinite.e4m3x2.f32 c, %7, %6; cvt.rn.satfinite.e4m3x2.f32 d, %9, %8; mov.b32 %0, {a, b}; mov.b32 %1, {c, d}; }"
            : "=r"(q.x), "=r"(q.y)
            : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    } else {
        asm("{ .reg .b8 a, b, c, d; cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;"
            " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7; mov.b32 %0, {a, b, c, d}; }"
            : "=r"(q.x)
            : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    }
    return q;
}

// eight values times a power of two
template <int KIND> __device__ __forceinline__ uint2 mx_pack8(const float (&v)[8], uint32_t code)
{
    const float m = mx_inverse(code);
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i] * m;
    uint2 q = mx_pack8<KIND>(t);
    if (KIND == PI_MX4 && code == 255u) q.x = 0; // (4 bits have no NaN: the scale says it)
    return q;
}

// eight elements' values, without the scale
template <int KIND> __device__ __forceinline__ void mx_unpack8(const uint2 &q, float (&v)[8])
{
    uint32_t h[4];
    if (KIND == PI_MX8) {
        asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
            : "=r"(h[0]), "=r"(h[1]) : "r"(q.x));
        asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
            : "=r"(h[2]), "=r"(h[3]) : "r"(q.y));
    } else {
        asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b;"
            " cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(q.x));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __half2float(__ushort_as_half((uint16_t)h[i]));
        v[2 * i + 1] = __half2float(__ushort_as_half((uint16_t)(h[i] >> 16)));
    }
}

// Eight columns [c, c + 8) of row r, held by one of four neighbouring lanes
// (XOR: their distance's lowest step, 1 or 8) that hold a block; all of a
// warp's lanes call it.  on: the row exists and c lies inside the padded row;
// what lies past the row's end is 0 in v.
template <int XOR> __device__ __forceinline__ uint32_t mx_amax4(uint32_t a)
{
    a = max(a, __shfl_xor_sync(0xffffffffu, a, XOR));
    return max(a, __shfl_xor_sync(0xffffffffu, a, 2 * XOR));
}
template <int XOR>
__device__ __forceinline__ void mx_store8(int kind, uint8_t *codes, int64_t ld, uint8_t *scales, int tiles, int64_t r, int c, bool on,
                                          const float (&v)[8])
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, mag(v[i]));
    a = mx_amax4<XOR>(on ? a : 0u);
    if (!on) return;
    const uint32_t code = kind == PI_MX8 ? mx_scale<PI_MX8>(a) : mx_scale<PI_MX4>(a);
    if (kind == PI_MX8) *reinterpret_cast<uint2 *>(codes + r * ld + c) = mx_pack8<PI_MX8>(v, code);
    else *reinterpret_cast<uint32_t *>(codes + r * ld + (c >> 1)) = mx_pack8<PI_MX4>(v, code).x;
    if ((c & 31) == 0) scales[mx_scale_at(r, c >> 7, tiles) + ((c >> 5) & 3)] = (uint8_t)code;
}

// Zeros for the scales of rows [T, T rounded up to 128): thread i of n.
__device__ __forceinline__ void mx_pad_scales(uint8_t *scales, int T, int tiles, int64_t i, int64_t n)
{
    const int64_t words = (int64_t)((128 - (T & 127)) & 127) * tiles;
    for (; i < words; i += n) *reinterpret_cast<uint32_t *>(scales + mx_scale_at(T + i / tiles, (int)(i % tiles), tiles)) = 0u;
}

} // namespace
#endif
} // namespace pi
