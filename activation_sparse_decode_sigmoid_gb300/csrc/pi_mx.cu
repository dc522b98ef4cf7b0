// Microscaled matrices: quantisation, the values back, and the C entry points
// of the products of such matrices (a linear layer, a gated FFN).
//
// Both conversions move T K (e + b) bytes, for e bytes an element and b = 33 / 32
// or 17 / 32 a code with its share of the scale.  28672 x 8192, there and back: rows
// of 16 bits that start on 16-byte boundaries are bound by HBM (from and to bf16 84
// and 87 us in 4 bits, 101 and 102 in 8: 6.8 to 7.1 TB/s), rows of 32 bits come to
// 5.2 to 5.5 TB/s (205 to 217 us).  Rows on other boundaries are read and written
// element by element, neighbouring threads 32 elements apart (writing: 8), and take 3 to 7 times as
// long: bf16 395 to 412 us there, 493 to 600 back, fp32 767 to 778 and 601 to 738.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pi.h"
#include "pi_block.h"
#include "pi_epi.cuh"
#include "pi_kernels.h"
#include "pi_mx.cuh"

namespace pi {
namespace {

constexpr int kMaxT = 1 << 22, kMaxDim = 1 << 20;

struct MxP {
    const void *x;   // or the output of the way back
    int64_t ldx;
    int vec;         // 16-byte accesses to x
    int T, K, tiles;
    uint8_t *codes, *scales;
    int64_t ld;
};

// T: __half, __nv_bfloat16 or float
template <typename T> __device__ __forceinline__ void store_any(void *p, int64_t at, int n, bool vec, const float (&v)[8])
{
    store8<T>(static_cast<uint16_t *>(p) + at, n, vec, v);
}
template <> __device__ __forceinline__ void store_any<float>(void *p, int64_t at, int n, bool vec, const float (&v)[8])
{
    store8f(static_cast<float *>(p) + at, n, vec, v);
}

// A block as a thread loads it: 32 elements of 16 or 32 bits.
template <typename T> struct Raw {
    uint32_t w[16];
    __device__ __forceinline__ void load(const void *p, int64_t at, int n, bool vec)
    {
        const uint16_t *s = static_cast<const uint16_t *>(p) + at;
        if (vec && n >= 32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(s) + i);
                w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            w[i] = 2 * i < n ? s[2 * i] : 0u;
            if (2 * i + 1 < n) w[i] |= (uint32_t)s[2 * i + 1] << 16;
        }
    }
    // the largest magnitude, as a float's bits (two halves at a time: as integers they order alike, NaN above all)
    __device__ __forceinline__ uint32_t amax() const
    {
        uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
        for (int i = 1; i < 16; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        return mag(C16<T>::one((uint16_t)max(m & 0xffffu, m >> 16)));
    }
    // elements 8 j to 8 j + 7 times a power of two
    __device__ __forceinline__ void scaled(int j, float m, float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) scale2(w[4 * j + i], m, v[2 * i], v[2 * i + 1]);
    }
    static __device__ __forceinline__ void scale2(uint32_t w, float m, float &a, float &b);
};
template <> __device__ __forceinline__ void Raw<__half>::scale2(uint32_t w, float m, float &a, float &b)
{
    a = C16<__half>::one((uint16_t)w) * m, b = C16<__half>::one((uint16_t)(w >> 16)) * m;
}
// (bf16 holds every power of two that a scale can be: one instruction an element; -0 added keeps the zeros' signs)
template <> __device__ __forceinline__ void Raw<__nv_bfloat16>::scale2(uint32_t w, float m, float &a, float &b)
{
    asm("{ .reg .b16 l, h, x; .reg .b32 z; mov.b32 {l, h}, %2; mov.b32 {x, _}, %3; fma.rn.f32.bf16 %0, l, x, %4; fma.rn.f32.bf16 %1, h, x, %4; }"
        : "=f"(a), "=f"(b)
        : "r"(w), "r"(__float_as_uint(m) >> 16), "f"(-0.f));
}
template <> struct Raw<float> {
    float f[32];
    __device__ __forceinline__ void load(const void *p, int64_t at, int n, bool vec)
    {
        const float *s = static_cast<const float *>(p) + at;
        if (vec && n >= 32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 q = __ldg(reinterpret_cast<const float4 *>(s) + i);
                f[4 * i] = q.x, f[4 * i + 1] = q.y, f[4 * i + 2] = q.z, f[4 * i + 3] = q.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = i < n ? s[i] : 0.f;
    }
    __device__ __forceinline__ uint32_t amax() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max(m, mag(f[i]));
        return m;
    }
    __device__ __forceinline__ void scaled(int j, float m, float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[8 * j + i] * m;
    }
};

// A thread has a block: neither its largest magnitude nor its scale is shared.
// (8 elements a thread and the rest by shuffles took 166 us for 28672 x 8192 from bf16 to
// 4 bits, twice what memory needs.)
constexpr int kQThreads = 128;
__host__ __device__ inline int quantize_rows(int nb) { return nb < kQThreads ? kQThreads / nb : 1; }

template <typename T, int KIND> __global__ void __launch_bounds__(kQThreads) mx_quantize_rows(const __grid_constant__ MxP p)
{
    pdl_enter();
    // blocks of a row; CTAs to a row, or rows to a CTA
    const int nb = p.tiles * 4, per = (nb + kQThreads - 1) / kQThreads, rows = quantize_rows(nb);
    const int64_t r = (int64_t)(blockIdx.x / per) * rows + (rows > 1 ? threadIdx.x / nb : 0);
    const int b = rows > 1 ? threadIdx.x % nb : (int)(blockIdx.x % per) * kQThreads + threadIdx.x;
    if (b >= nb || (rows > 1 && threadIdx.x >= rows * nb) || r >= (int64_t)mx_tiles(p.T) * 128) return;
    uint8_t *scale = p.scales + mx_scale_at(r, b >> 2, p.tiles) + (b & 3);
    if (r >= p.T) { // (rows behind the last: zeros up to the tile's end)
        *scale = 0;
        return;
    }
    Raw<T> x;
    x.load(p.x, r * p.ldx + b * 32, p.K - b * 32, p.vec);
    const uint32_t code = mx_scale<KIND>(x.amax());
    const float m = mx_inverse(code);
    uint2 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[8];
        x.scaled(j, m, v);
        q[j] = mx_pack8<KIND>(v);
    }
    *scale = (uint8_t)code;
    uint4 *o = reinterpret_cast<uint4 *>(p.codes + r * p.ld + b * (KIND == PI_MX8 ? 32 : 16));
    if (KIND == PI_MX8) {
        o[0] = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
        o[1] = make_uint4(q[2].x, q[2].y, q[3].x, q[3].y);
    } else // (4 bits have no NaN: the scale says it)
        o[0] = code == 255u ? make_uint4(0, 0, 0, 0) : make_uint4(q[0].x, q[1].x, q[2].x, q[3].x);
}

// The way back: a warp takes 256 columns of kRows rows, its loads in flight together.
constexpr int kRows = 4, kWarps = 8;
template <typename T, int KIND> __global__ void __launch_bounds__(32 * kWarps) mx_dequantize_rows(const __grid_constant__ MxP p)
{
    pdl_enter();
    const int ncb = (p.tiles + 1) / 2, lane = threadIdx.x & 31;
    const int c = (int)(blockIdx.x % ncb) * 256 + lane * 8, n = p.K - c;
    const int64_t r0 = ((int64_t)(blockIdx.x / ncb) * kWarps + (threadIdx.x >> 5)) * kRows;
    if (n <= 0) return;
    uint2 q[kRows];
    uint32_t s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i;
        if (r >= p.T) continue;
        if (KIND == PI_MX8) q[i] = *reinterpret_cast<const uint2 *>(p.codes + r * p.ld + c);
        else q[i] = make_uint2(*reinterpret_cast<const uint32_t *>(p.codes + r * p.ld + (c >> 1)), 0);
        s[i] = p.scales[mx_scale_at(r, c >> 7, p.tiles) + ((c >> 5) & 3)];
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (r0 + i >= p.T) continue;
        float v[8];
        mx_unpack8<KIND>(q[i], v);
        const float m = mx_power(s[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= m;
        store_any<T>(const_cast<void *>(p.x), (r0 + i) * p.ldx + c, n, p.vec, v);
    }
}

// ------------------------------------------------------------------ checks
bool is16(int dt) { return dt == PI_F16 || dt == PI_BF16; }
bool is_float(int dt) { return is16(dt) || dt == PI_F32; }
bool is_mx(int k) { return k == PI_MX8 || k == PI_MX4; }
bool aligned16(const void *p, int64_t ld, int elem) { return ((uintptr_t)p & 15) == 0 && (ld * elem) % 16 == 0; }

#define CUX(call)                                                                                          \
    do {                                                                                                   \
        cudaError_t e_ = (call);                                                                           \
        if (e_ != cudaSuccess) return ctx_fail(c, PI_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_));   \
    } while (0)

pi_status check_sizes(pi_ctx *c, int rows, int cols, int kind)
{
    if (!is_mx(kind)) return ctx_fail(c, PI_ERR_ARG, "kind %d is not PI_MX8 or PI_MX4", kind);
    if (rows < 0 || rows > kMaxT) return ctx_fail(c, PI_ERR_SHAPE, "%d rows, outside [0, %d]", rows, kMaxT);
    if (cols < 1 || cols > kMaxDim) return ctx_fail(c, PI_ERR_SHAPE, "%d columns, outside [1, %d]", cols, kMaxDim);
    return PI_OK;
}

// A microscaled matrix's buffers and row stride (0: packed).
pi_status check_mx(pi_ctx *c, const char *what, const pi_mx *m, int rows, int cols, int kind, int64_t &ld)
{
    const int64_t row = mx_row_bytes(kind, cols);
    if (!ld) ld = row;
    if (ld < row) return ctx_fail(c, PI_ERR_SHAPE, "%s: row stride %lld below the row's %lld bytes", what, (long long)ld, (long long)row);
    if (ld % 32) return ctx_fail(c, PI_ERR_ARG, "%s: row stride %lld is not a multiple of 32 bytes", what, (long long)ld);
    if (!rows) return PI_OK;
    if (!m || !m->codes || !m->scales) return ctx_fail(c, PI_ERR_ARG, "%s: codes or scales are NULL", what);
    if ((uintptr_t)m->codes % 32 || (uintptr_t)m->scales % 16)
        return ctx_fail(c, PI_ERR_ARG, "%s: codes have to start at a multiple of 32 bytes, scales at one of 16", what);
    return PI_OK;
}

template <int KIND> cudaError_t run_quantize(const MxP &p, int dt, cudaStream_t s, unsigned grid)
{
    return dt == PI_F32   ? launch_pdl(mx_quantize_rows<float, KIND>, dim3(grid), dim3(kQThreads), 0, s, p)
           : dt == PI_F16 ? launch_pdl(mx_quantize_rows<__half, KIND>, dim3(grid), dim3(kQThreads), 0, s, p)
                          : launch_pdl(mx_quantize_rows<__nv_bfloat16, KIND>, dim3(grid), dim3(kQThreads), 0, s, p);
}
template <int KIND> cudaError_t run_dequantize(const MxP &p, int dt, cudaStream_t s, unsigned grid)
{
    return dt == PI_F32   ? launch_pdl(mx_dequantize_rows<float, KIND>, dim3(grid), dim3(32 * kWarps), 0, s, p)
           : dt == PI_F16 ? launch_pdl(mx_dequantize_rows<__half, KIND>, dim3(grid), dim3(32 * kWarps), 0, s, p)
                          : launch_pdl(mx_dequantize_rows<__nv_bfloat16, KIND>, dim3(grid), dim3(32 * kWarps), 0, s, p);
}

pi_status convert(pi_ctx *c, const pi_mx_desc *desc, const void *x, const pi_mx *q, bool back)
{
    if (!desc) return ctx_fail(c, PI_ERR_ARG, "desc is NULL");
    const pi_mx_desc d = *desc;
    if (pi_status st = check_sizes(c, d.rows, d.cols, d.kind)) return st;
    if (!is_float(d.dtype)) return ctx_fail(c, PI_ERR_ARG, "dtype %d is not PI_F16, PI_BF16 or PI_F32", d.dtype);
    const int elem = d.dtype == PI_F32 ? 4 : 2;
    MxP p = {};
    p.ldx = d.ldx ? d.ldx : d.cols;
    if (p.ldx < d.cols) return ctx_fail(c, PI_ERR_SHAPE, "row stride %lld below the row's %d elements", (long long)d.ldx, d.cols);
    p.ld = d.ldq;
    if (pi_status st = check_mx(c, "q", q, d.rows, d.cols, d.kind, p.ld)) return st;
    if (!d.rows) return PI_OK;
    if (!x) return ctx_fail(c, PI_ERR_ARG, "%s is NULL", back ? "y" : "x");
    if (pi_status st = check_elements(c, elem, {x})) return st;
    p.x = x, p.T = d.rows, p.K = d.cols, p.tiles = mx_tiles(d.cols);
    p.vec = ((uintptr_t)x & 15) == 0 && (d.rows == 1 || p.ldx * elem % 16 == 0);
    p.codes = static_cast<uint8_t *>(q->codes), p.scales = static_cast<uint8_t *>(q->scales);
    const CtxView v = ctx_view(c);
    DeviceGuard g(v.device);
    const unsigned grid = back ? (unsigned)((d.rows + kRows * kWarps - 1) / (kRows * kWarps) * ((p.tiles + 1) / 2))
                               : (unsigned)(((int64_t)mx_tiles(d.rows) * 128 + quantize_rows(p.tiles * 4) - 1) / quantize_rows(p.tiles * 4) *
                                            ((p.tiles * 4 + kQThreads - 1) / kQThreads));
    if (back) CUX(d.kind == PI_MX8 ? run_dequantize<PI_MX8>(p, d.dtype, v.stream, grid) : run_dequantize<PI_MX4>(p, d.dtype, v.stream, grid));
    else CUX(d.kind == PI_MX8 ? run_quantize<PI_MX8>(p, d.dtype, v.stream, grid) : run_quantize<PI_MX4>(p, d.dtype, v.stream, grid));
    return PI_OK;
}

pi_status check_kinds(pi_ctx *c, int xk, int wk, int &ops)
{
    if (!is_mx(xk) || !is_mx(wk)) return ctx_fail(c, PI_ERR_ARG, "x_kind %d or w_kind %d is not PI_MX8 or PI_MX4", xk, wk);
    if (xk == PI_MX4 && wk == PI_MX8) return ctx_fail(c, PI_ERR_UNSUPPORTED, "4-bit x with 8-bit weights");
    ops = wk == PI_MX8 ? OPS_MX88 : xk == PI_MX8 ? OPS_MX84 : OPS_MX44;
    return PI_OK;
}

pi_status check_ws(pi_ctx *c, const void *ws, size_t have, size_t need)
{
    if (need && (!ws || have < need))
        return ctx_fail(c, PI_ERR_ARG, "workspace of %zu bytes needed, %zu given", need, ws ? have : (size_t)0);
    if (((uintptr_t)ws & 15) != 0) return ctx_fail(c, PI_ERR_ARG, "workspace not 16-byte aligned");
    return PI_OK;
}

// The product x W^T of a linear layer, without its buffers.
pi_status check_linear(pi_ctx *c, const pi_mx_linear_desc *desc, pi_mx_linear_desc &d, Gemm &g)
{
    if (!desc) return ctx_fail(c, PI_ERR_ARG, "desc is NULL");
    d = *desc;
    g = Gemm{};
    if (!is16(d.dtype)) return ctx_fail(c, PI_ERR_ARG, "dtype %d is not PI_F16 or PI_BF16", d.dtype);
    if (d.out_dtype != d.dtype && d.out_dtype != PI_F32)
        return ctx_fail(c, PI_ERR_ARG, "out_dtype %d is neither dtype nor PI_F32", d.out_dtype);
    if (d.fn < PI_FN_NONE || d.fn > PI_FN_GELU_TANH) return ctx_fail(c, PI_ERR_ARG, "fn %d invalid", d.fn);
    if (!std::isfinite(d.scale)) return ctx_fail(c, PI_ERR_ARG, "scale is not finite");
    if (pi_status st = check_kinds(c, d.x_kind, d.w_kind, g.ops)) return st;
    if (pi_status st = check_sizes(c, d.T, d.K, d.x_kind)) return st;
    if (d.N < 1 || d.N > kMaxDim) return ctx_fail(c, PI_ERR_SHAPE, "N %d outside [1, %d]", d.N, kMaxDim);
    for (int64_t *l : {&d.ldr, &d.ldy}) {
        if (!*l) *l = d.N;
        if (*l < d.N) return ctx_fail(c, PI_ERR_SHAPE, "row stride %lld below the row's %d elements", (long long)*l, d.N);
    }
    g.mode = EPI_LINEAR, g.segs = 1;
    g.M = d.T, g.N = d.N, g.K[0] = d.K;
    g.e.fn = d.fn, g.e.scale = d.scale, g.e.out32 = d.out_dtype == PI_F32;
    g.e.ldr = d.ldr, g.e.ldo = d.ldy;
    return PI_OK;
}

void set_mx(Mat &m, const uint8_t *&scales, const pi_mx &q, int64_t ld)
{
    m = {q.codes, ld, 0};
    scales = static_cast<const uint8_t *>(q.scales);
}

// The two products of an FFN, without the caller's buffers; a lies in the workspace.
struct Ffn {
    pi_mx_gated_ffn_desc d;
    Gemm up, down;
    size_t codes, scales, gemm; // bytes of the workspace's parts
    size_t bytes() const { return codes ? 32 + codes + scales + gemm : 0; } // (32: a starts on such a boundary)
};

pi_status check_ffn(pi_ctx *c, const pi_mx_gated_ffn_desc *desc, const CtxView &v, Ffn &f)
{
    if (!desc) return ctx_fail(c, PI_ERR_ARG, "desc is NULL");
    f = Ffn{};
    f.d = *desc;
    pi_mx_gated_ffn_desc &d = f.d;
    if (!is16(d.dtype)) return ctx_fail(c, PI_ERR_ARG, "dtype %d is not PI_F16 or PI_BF16", d.dtype);
    if (d.fn < PI_FN_NONE || d.fn > PI_FN_GELU_TANH) return ctx_fail(c, PI_ERR_ARG, "fn %d invalid", d.fn);
    if (d.gated != 0 && d.gated != 1) return ctx_fail(c, PI_ERR_ARG, "gated %d is not 0 or 1", d.gated);
    int ops = 0;
    if (pi_status st = check_kinds(c, d.x_kind, d.w_kind, ops)) return st;
    if (pi_status st = check_sizes(c, d.T, d.d, d.x_kind)) return st;
    if (d.n < 1 || d.n > kMaxDim) return ctx_fail(c, PI_ERR_SHAPE, "n %d outside [1, %d]", d.n, kMaxDim);
    if (!d.ldy) d.ldy = d.d;
    if (d.ldy < d.d) return ctx_fail(c, PI_ERR_SHAPE, "row stride %lld below the row's %d elements", (long long)d.ldy, d.d);
    const int64_t lda = mx_row_bytes(d.x_kind, d.n);
    Gemm &u = f.up, &w = f.down;
    u.mode = d.gated ? EPI_GATED : EPI_LINEAR, w.mode = EPI_LINEAR;
    u.segs = w.segs = 1, u.ops = w.ops = ops, u.M = w.M = d.T, u.N = d.n, u.K[0] = d.d, w.N = d.d, w.K[0] = d.n;
    u.e.fn = d.fn, u.e.scale = w.e.scale = 1.f;
    u.e.mx = d.x_kind, u.e.mx_tiles = mx_tiles(d.n), u.e.ldo = lda;
    w.a[0].ld = lda, w.e.ldo = d.ldy;
    w.early = 1; // the weights are older than the product before
    if (!d.T) return PI_OK;
    f.codes = ((size_t)d.T * lda + 255) / 256 * 256;
    f.scales = (size_t)mx_scale_bytes(d.T, d.n);
    f.gemm = std::max(gemm_workspace(u, v), gemm_workspace(w, v));
    return PI_OK;
}

} // namespace
} // namespace pi

using namespace pi;

extern "C" {

pi_status pi_mx_bytes(int32_t rows, int32_t cols, int32_t kind, size_t *codes, size_t *scales)
{
    if (!codes || !scales || !is_mx(kind)) return PI_ERR_ARG;
    if (rows < 0 || rows > kMaxT || cols < 1 || cols > kMaxDim) return PI_ERR_SHAPE;
    *codes = (size_t)rows * mx_row_bytes(kind, cols);
    *scales = (size_t)mx_scale_bytes(rows, cols);
    return PI_OK;
}

pi_status pi_mx_quantize(pi_ctx *c, const pi_mx_desc *desc, const void *x, const pi_mx *q)
{
    return c ? convert(c, desc, x, q, false) : PI_ERR_ARG;
}

pi_status pi_mx_dequantize(pi_ctx *c, const pi_mx_desc *desc, const pi_mx *q, void *y)
{
    return c ? convert(c, desc, y, q, true) : PI_ERR_ARG;
}

pi_status pi_mx_linear_workspace(pi_ctx *c, const pi_mx_linear_desc *desc, size_t *bytes)
{
    if (!c) return PI_ERR_ARG;
    if (!bytes) return ctx_fail(c, PI_ERR_ARG, "bytes is NULL");
    pi_mx_linear_desc d;
    Gemm g;
    if (pi_status st = check_linear(c, desc, d, g)) return st;
    *bytes = d.T ? gemm_workspace(g, ctx_view(c)) : 0;
    return PI_OK;
}

pi_status pi_mx_linear(pi_ctx *c, const pi_mx_linear_desc *desc, const pi_mx *x, const pi_mx *w, const void *b,
                       const void *residual, void *y, void *ws, size_t ws_bytes)
{
    if (!c) return PI_ERR_ARG;
    pi_mx_linear_desc d;
    Gemm g;
    if (pi_status st = check_linear(c, desc, d, g)) return st;
    if (pi_status st = check_mx(c, "x", x, d.T, d.K, d.x_kind, d.ldx)) return st;
    if (!d.T) return PI_OK;
    if (pi_status st = check_mx(c, "w", w, d.N, d.K, d.w_kind, d.ldw)) return st;
    if (!y) return ctx_fail(c, PI_ERR_ARG, "y is NULL");
    const int oe = g.e.out32 ? 4 : 2;
    if (pi_status st = check_elements(c, 2, {b})) return st;
    if (pi_status st = check_elements(c, oe, {residual, y})) return st;
    const CtxView v = ctx_view(c);
    if (pi_status st = check_ws(c, ws, ws_bytes, gemm_workspace(g, v))) return st;
    set_mx(g.a[0], g.sa, *x, d.ldx);
    set_mx(g.b[0], g.sb[0], *w, d.ldw);
    Epi &e = g.e;
    e.bias = static_cast<const uint16_t *>(b), e.res = residual, e.out = y;
    e.vec = (residual && aligned16(residual, d.ldr, oe) ? V_RES : 0u) | (aligned16(y, d.ldy, oe) ? V_OUT : 0u) |
            (b && aligned16(b, 0, 2) ? V_BIAS : 0u);
    DeviceGuard guard(v.device);
    CUX(launch_gemm(g, d.dtype == PI_BF16, v, ws));
    return PI_OK;
}

pi_status pi_mx_gated_ffn_workspace(pi_ctx *c, const pi_mx_gated_ffn_desc *desc, size_t *bytes)
{
    if (!c) return PI_ERR_ARG;
    if (!bytes) return ctx_fail(c, PI_ERR_ARG, "bytes is NULL");
    Ffn f;
    if (pi_status st = check_ffn(c, desc, ctx_view(c), f)) return st;
    *bytes = f.bytes();
    return PI_OK;
}

pi_status pi_mx_gated_ffn(pi_ctx *c, const pi_mx_gated_ffn_desc *desc, const pi_mx_gated_ffn_weights *w, const pi_mx *x,
                          void *y, void *ws, size_t ws_bytes)
{
    if (!c) return PI_ERR_ARG;
    const CtxView v = ctx_view(c);
    Ffn f;
    if (pi_status st = check_ffn(c, desc, v, f)) return st;
    pi_mx_gated_ffn_desc &d = f.d;
    if (!w) return ctx_fail(c, PI_ERR_ARG, "weights are NULL");
    if (!d.gated && (w->gate.codes || w->gate.scales || w->b_gate))
        return ctx_fail(c, PI_ERR_ARG, "gate weights given, but gated is 0");
    if (pi_status st = check_mx(c, "x", x, d.T, d.d, d.x_kind, d.ldx)) return st;
    if (!d.T) return PI_OK;
    if (d.gated)
        if (pi_status st = check_mx(c, "w_gate", &w->gate, d.n, d.d, d.w_kind, d.ld_gate)) return st;
    if (pi_status st = check_mx(c, "w_up", &w->up, d.n, d.d, d.w_kind, d.ld_up)) return st;
    if (pi_status st = check_mx(c, "w_down", &w->down, d.d, d.n, d.w_kind, d.ld_down)) return st;
    if (!y) return ctx_fail(c, PI_ERR_ARG, "y is NULL");
    if (pi_status st = check_elements(c, 2, {w->b_gate, w->b_up, w->b_down, y})) return st;
    if (pi_status st = check_ws(c, ws, ws_bytes, f.bytes())) return st;
    uint8_t *const base = reinterpret_cast<uint8_t *>(((uintptr_t)ws + 31) / 32 * 32);
    const pi_mx a = {base, base + f.codes};
    Gemm &u = f.up, &o = f.down;
    set_mx(u.a[0], u.sa, *x, d.ldx);
    const void *first = w->b_up, *second = nullptr;
    if (d.gated) {
        set_mx(u.b[0], u.sb[0], w->gate, d.ld_gate);
        set_mx(u.b[1], u.sb[1], w->up, d.ld_up);
        first = w->b_gate, second = w->b_up;
    } else
        set_mx(u.b[0], u.sb[0], w->up, d.ld_up);
    u.e.bias = static_cast<const uint16_t *>(first), u.e.bias2 = static_cast<const uint16_t *>(second);
    u.e.out = a.codes, u.e.mx_scales = static_cast<uint8_t *>(a.scales);
    u.e.vec = (first && aligned16(first, 0, 2) ? V_BIAS : 0u) | (second && aligned16(second, 0, 2) ? V_BIAS2 : 0u);
    set_mx(o.a[0], o.sa, a, o.a[0].ld);
    set_mx(o.b[0], o.sb[0], w->down, d.ld_down);
    o.e.bias = static_cast<const uint16_t *>(w->b_down), o.e.out = y;
    o.e.vec = (aligned16(y, d.ldy, 2) ? V_OUT : 0u) | (w->b_down && aligned16(w->b_down, 0, 2) ? V_BIAS : 0u);
    void *gws = base + f.codes + f.scales;
    DeviceGuard guard(v.device);
    CUX(launch_gemm(u, d.dtype == PI_BF16, v, gws));
    CUX(launch_gemm(o, d.dtype == PI_BF16, v, gws));
    return PI_OK;
}

} // extern "C"
