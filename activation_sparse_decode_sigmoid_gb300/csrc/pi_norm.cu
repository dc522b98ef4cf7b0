// The norms before and after a block, with its gate and residual scale
// (pi_norm_residual and its backward pass):
//
//     v  = y or norm_post(y),  x' = rs x + bs gate v,  h = norm_pre(x')
//
// Backward, with xh, yh the normalised rows, r their 1 / sqrt(... + eps):
//     dxh = dh w_pre,  D = dx' + r_x (dxh - [mean dxh] - xh mean(dxh xh))
//     dx = rs D,  dv = bs gate D
//     dyh = dv w_post,  dy = r_y (dyh - [mean dyh] - yh mean(dyh yh))   ([]: layer norm only)
//     P1 = sum dh xh, P0 = sum dh  over tokens: dw_pre, db_pre
//     S1 = sum D yh, S0 = sum D    over the tokens of one gate row:
//         dgate = bs (w_post S1 + b_post S0),  dw_post += bs gate S1,  db_post += bs gate S0
// The forward pass is bound by HBM (a few operations per element).  The backward
// pass, about 50 instructions per element of six arrays, fills neither: HBM is
// half busy and 0.58 instructions issue per cycle, because all warps of an SM
// work on one row and stand at its barriers and results together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "pi.h"
#include "pi_block.h"
#include "pi_epi.cuh"
#include "pi_kernels.h"
#include "pi_mx.cuh"
#include "pi_tc.cuh"

namespace pi {
namespace {

constexpr int kMaxT = 1 << 22, kMaxNormD = 16384;

// Tokens whose column sums one unit of norm_bwd_cols adds up: enough units for
// eight CTAs of 1024 columns on every SM, 4 to 64 tokens each.
int unit_rows(int T, int d, int sms)
{
    const int64_t want = (int64_t)T * ((d + 1023) / 1024) / (8 * sms);
    return (int)std::min<int64_t>(64, std::max<int64_t>(4, want));
}

struct NormP {
    int Tn, d, pre, post, x32;
    int gate_rows; // tokens per gate row (>= 1)
    float rs, bs, eps;
    const void *x;              // forward: x; backward: x'
    const uint16_t *y, *gate;   // or NULL
    const uint16_t *w_pre, *b_pre, *w_post, *b_post;
    void *xo;                   // forward: x' (or NULL)
    uint16_t *h;                // or NULL
    int64_t ldx, ldxo, ldy, ldh, ldgate, lddx; // (ldx: of `x`, ldxo: of xo or dxo)
    unsigned vec;               // 16-byte accesses: 1 x, 2 xo, 4 y, 8 h, 16 gate, 32.. parameters, 64 dx, 128 dy, 256 dxo
    // backward
    const void *dxo;
    const uint16_t *dh;
    void *dx;
    uint16_t *dy;
    float *stats;               // [T][8]: mean_x, r_x, c1, c2, mean_y, r_y
    float *part;                // [units][4][d]: P1, P0, S1, S0
    int units, per_group;       // units in all, and per gate row
    int unit;                   // tokens of a unit
    int per_token;              // a gate row per token: S1, S0 carry the gate, dgate is written by the row kernel
    void *dgate, *dw_pre, *db_pre, *dw_post, *db_post;
    int g32, acc;
    // h microscaled: its kind (0: 16 bits), ldh its bytes a row
    int mx, mx_tiles;
    uint8_t *mx_scales;
};

enum : unsigned { NV_X = 1, NV_XO = 2, NV_Y = 4, NV_H = 8, NV_GATE = 16, NV_PAR = 32, NV_DX = 64, NV_DY = 128, NV_DXO = 256, NV_DGATE = 512 };

template <typename T> __device__ __forceinline__ void loadx8(const void *p, int x32, int64_t at, int n, bool vec, float (&v)[8])
{
    if (x32) load8f(static_cast<const float *>(p) + at, n, vec, v);
    else load8<T>(static_cast<const uint16_t *>(p) + at, n, vec, v);
}

template <typename T> __device__ __forceinline__ void storex8(void *p, int x32, int64_t at, int n, bool vec, const float (&v)[8])
{
    if (x32) store8f(static_cast<float *>(p) + at, n, vec, v);
    else store8<T>(static_cast<uint16_t *>(p) + at, n, vec, v);
}

// Sums of two values over the CTA, in a fixed order; every thread gets them.
// buf: 128 floats of shared memory, one half of 64 on every other call.
__device__ __forceinline__ float2 cta_sum2(float a, float b, float *buf, int &flip)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    const int nw = blockDim.x >> 5;
    if (nw == 1) return make_float2(a, b);
    float *s = buf + (flip ? 64 : 0);
    flip ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = a, s[32 + (threadIdx.x >> 5)] = b;
    __syncthreads();
    const int l = threadIdx.x & 31;
    a = l < nw ? s[l] : 0.f;
    b = l < nw ? s[32 + l] : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
}

// mean and 1 / sqrt(variance or mean square + eps) of a row held in V chunks
// of 8 per thread (two passes over the registers for a layer norm).  Elements
// behind the row count nowhere: a norm without weight and gate leaves -mean r there.
template <int V>
__device__ __forceinline__ void row_stats(int kind, const float (&v)[V][8], int d, float eps, float *buf, int &flip,
                                          float &mean, float &r)
{
    mean = 0.f;
    if (kind == PI_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) s += c + j < d ? v[i][j] : 0.f;
        }
        mean = cta_sum2(s, 0.f, buf, flip).x / (float)d;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = c + j < d ? v[i][j] - mean : 0.f;
            q = fmaf(t, t, q);
        }
    }
    r = 1.f / sqrtf(cta_sum2(q, 0.f, buf, flip).x / (float)d + eps);
}

// v = (v - mean) r w + b
template <typename T, int V>
__device__ __forceinline__ void apply_norm(const NormP &p, float (&v)[V][8], const uint16_t *w, const uint16_t *b,
                                           float mean, float r)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8, n = p.d - c;
        if (n <= 0) continue;
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = (v[i][j] - mean) * r;
        if (w) {
            load8<T>(w + c, n, p.vec & NV_PAR, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= t[j];
        }
        if (b) {
            load8<T>(b + c, n, p.vec & NV_PAR, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += t[j];
        }
    }
}

// 8 columns of a microscaled h: four neighbouring lanes hold a block.
__device__ __forceinline__ void norm_store_mx(const NormP &p, int64_t t, int c, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j >= p.d) v[j] = 0.f;
    mx_store8<1>(p.mx, reinterpret_cast<uint8_t *>(p.h), p.ldh, p.mx_scales, p.mx_tiles, t, c, c < p.mx_tiles * 128, v);
}

// Forward: one CTA per token, the row in registers.
// MX: h is microscaled.
template <typename T, int V, bool MX> __global__ void __launch_bounds__(1024) norm_fwd(const __grid_constant__ NormP p)
{
    __shared__ float buf[128];
    int flip = 0;
    pdl_enter();
    const int64_t t = blockIdx.x;
    if (MX && t >= p.Tn) { // CTAs behind the rows
        mx_pad_scales(p.mx_scales, p.Tn, p.mx_tiles, (t - p.Tn) * blockDim.x + threadIdx.x, (int64_t)(gridDim.x - p.Tn) * blockDim.x);
        return;
    }
    float x[V][8], y[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8, n = p.d - c;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = y[i][j] = 0.f;
        if (n <= 0) continue;
        loadx8<T>(p.x, p.x32, t * p.ldx + c, n, p.vec & NV_X, x[i]);
        if (p.y) load8<T>(p.y + t * p.ldy + c, n, p.vec & NV_Y, y[i]);
    }
    float mean, r;
    if (p.y && p.post != PI_NORM_NONE) {
        row_stats<V>(p.post, y, p.d, p.eps, buf, flip, mean, r);
        apply_norm<T, V>(p, y, p.w_post, p.b_post, mean, r);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8, n = p.d - c;
        if (n <= 0) continue;
        float g[8];
        if (p.y) {
            if (p.gate) load8<T>(p.gate + t / p.gate_rows * p.ldgate + c, n, p.vec & NV_GATE, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = fmaf(p.bs * (p.gate ? g[j] : 1.f), y[i][j], p.rs * x[i][j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= p.rs;
        }
        if (p.xo) storex8<T>(p.xo, p.x32, t * p.ldxo + c, n, p.vec & NV_XO, x[i]);
    }
    if (!p.h) return;
    row_stats<V>(p.pre, x, p.d, p.eps, buf, flip, mean, r);
    apply_norm<T, V>(p, x, p.w_pre, p.b_pre, mean, r);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8, n = p.d - c;
        if (MX) norm_store_mx(p, t, c, x[i]);
        else if (n > 0) store8<T>(p.h + t * p.ldh + c, n, p.vec & NV_H, x[i]);
    }
}

// Statistics of a row read from memory (two passes for a layer norm).
template <typename T>
__device__ __forceinline__ void mem_stats(int kind, const void *x, int x32, int64_t at, bool vec, int d, float eps,
                                          float *buf, int &flip, float &mean, float &r)
{
    mean = 0.f;
    if (kind == PI_NORM_LAYER) {
        float s = 0.f;
        for (int c = threadIdx.x * 8; c < d; c += blockDim.x * 8) {
            float v[8];
            loadx8<T>(x, x32, at + c, d - c, vec, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[j];
        }
        mean = cta_sum2(s, 0.f, buf, flip).x / (float)d;
    }
    float q = 0.f;
    for (int c = threadIdx.x * 8; c < d; c += blockDim.x * 8) {
        float v[8];
        loadx8<T>(x, x32, at + c, d - c, vec, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u = c + j < d ? v[j] - mean : 0.f;
            q = fmaf(u, u, q);
        }
    }
    r = 1.f / sqrtf(cta_sum2(q, 0.f, buf, flip).x / (float)d + eps);
}

// One column chunk of a token in the backward pass: D, and the normalised
// x' and y (y itself without a post norm).
template <typename T>
__device__ __forceinline__ void bwd_chunk(const NormP &p, int64_t t, int c, const float (&st)[6], float (&D)[8],
                                          float (&xh)[8], float (&dh)[8], float (&yh)[8])
{
    const int n = p.d - c;
    if (p.dxo) loadx8<T>(p.dxo, p.x32, t * p.ldxo + c, n, p.vec & NV_DXO, D);
    else {
#pragma unroll
        for (int j = 0; j < 8; ++j) D[j] = 0.f;
    }
    if (p.pre != PI_NORM_NONE && p.dh) {
        float w[8];
        loadx8<T>(p.x, p.x32, t * p.ldx + c, n, p.vec & NV_X, xh);
        load8<T>(p.dh + t * p.ldh + c, n, p.vec & NV_H, dh);
        if (p.w_pre) load8<T>(p.w_pre + c, n, p.vec & NV_PAR, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            xh[j] = (xh[j] - st[0]) * st[1];
            D[j] += st[1] * (dh[j] * (p.w_pre ? w[j] : 1.f) - st[2] - xh[j] * st[3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) xh[j] = dh[j] = 0.f;
    }
    if (p.y) {
        load8<T>(p.y + t * p.ldy + c, n, p.vec & NV_Y, yh);
#pragma unroll
        for (int j = 0; j < 8; ++j) yh[j] = (yh[j] - st[4]) * st[5];
    }
}

// Backward, rows: dx, dy, the rows' statistics, and dgate with a gate row per token.
template <typename T> __global__ void __launch_bounds__(512) norm_bwd_rows(const __grid_constant__ NormP p)
{
    __shared__ float buf[128];
    int flip = 0;
    pdl_enter();
    const int64_t t = blockIdx.x;
    const int d = p.d, step = blockDim.x * 8;
    float st[6] = {0.f, 1.f, 0.f, 0.f, 0.f, 1.f};
    float D[8], xh[8], dh[8], yh[8], g[8], w[8];
    if (p.pre != PI_NORM_NONE && p.dh) {
        mem_stats<T>(p.pre, p.x, p.x32, t * p.ldx, p.vec & NV_X, d, p.eps, buf, flip, st[0], st[1]);
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x * 8; c < d; c += step) {
            loadx8<T>(p.x, p.x32, t * p.ldx + c, d - c, p.vec & NV_X, xh);
            load8<T>(p.dh + t * p.ldh + c, d - c, p.vec & NV_H, dh);
            if (p.w_pre) load8<T>(p.w_pre + c, d - c, p.vec & NV_PAR, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = dh[j] * (p.w_pre ? w[j] : 1.f); // (0 past the row)
                s1 += q;
                s2 = fmaf(q, (xh[j] - st[0]) * st[1], s2);
            }
        }
        const float2 s = cta_sum2(s1, s2, buf, flip);
        st[2] = p.pre == PI_NORM_LAYER ? s.x / (float)d : 0.f;
        st[3] = s.y / (float)d;
    }
    float c1 = 0.f, c2 = 0.f;
    if (p.y && p.post != PI_NORM_NONE) {
        mem_stats<T>(p.post, p.y, 0, t * p.ldy, p.vec & NV_Y, d, p.eps, buf, flip, st[4], st[5]);
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x * 8; c < d; c += step) {
            bwd_chunk<T>(p, t, c, st, D, xh, dh, yh);
            if (p.gate) load8<T>(p.gate + t / p.gate_rows * p.ldgate + c, d - c, p.vec & NV_GATE, g);
            if (p.w_post) load8<T>(p.w_post + c, d - c, p.vec & NV_PAR, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q =
                    c + j < d ? p.bs * (p.gate ? g[j] : 1.f) * D[j] * (p.w_post ? w[j] : 1.f) : 0.f;
                s1 += q;
                s2 = fmaf(q, yh[j], s2);
            }
        }
        const float2 s = cta_sum2(s1, s2, buf, flip);
        c1 = p.post == PI_NORM_LAYER ? s.x / (float)d : 0.f;
        c2 = s.y / (float)d;
    }
    for (int c = threadIdx.x * 8; c < d; c += step) {
        const int n = d - c;
        bwd_chunk<T>(p, t, c, st, D, xh, dh, yh);
        if (p.y && (p.dy || (p.per_token && p.dgate))) {
            if (p.gate) load8<T>(p.gate + t / p.gate_rows * p.ldgate + c, n, p.vec & NV_GATE, g);
            if (p.w_post) load8<T>(p.w_post + c, n, p.vec & NV_PAR, w);
            if (p.per_token && p.dgate) {
                float b[8], o[8];
                if (p.b_post) load8<T>(p.b_post + c, n, p.vec & NV_PAR, b);
                const int64_t at = t * d + c;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = p.bs * D[j] * fmaf(yh[j], p.w_post ? w[j] : 1.f, p.b_post ? b[j] : 0.f);
                if (p.acc) {
                    float old[8];
                    loadx8<T>(p.dgate, p.g32, at, n, p.vec & NV_DGATE, old);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] += old[j];
                }
                storex8<T>(p.dgate, p.g32, at, n, p.vec & NV_DGATE, o);
            }
            if (p.dy) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float dv = p.bs * (p.gate ? g[j] : 1.f) * D[j];
                    o[j] = p.post == PI_NORM_NONE ? dv : st[5] * (dv * (p.w_post ? w[j] : 1.f) - c1 - yh[j] * c2);
                }
                store8<T>(p.dy + t * p.ldy + c, n, p.vec & NV_DY, o);
            }
        }
        if (p.dx) {
#pragma unroll
            for (int j = 0; j < 8; ++j) D[j] *= p.rs;
            storex8<T>(p.dx, p.x32, t * p.lddx + c, n, p.vec & NV_DX, D);
        }
    }
    if (p.stats && threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < 6; ++i) p.stats[t * 8 + i] = st[i];
    }
}

// Tokens of unit u: [t0, t1) (all of one gate row unless per_token).
__device__ __forceinline__ void unit_tokens(const NormP &p, int u, int &t0, int &t1)
{
    const int g = u / p.per_group, k = u % p.per_group;
    const int end = p.per_token ? p.Tn : (int)min((int64_t)p.Tn, (int64_t)(g + 1) * p.gate_rows);
    t0 = (p.per_token ? 0 : g * p.gate_rows) + k * p.unit;
    t1 = min(end, t0 + p.unit);
}

// Backward, columns: one CTA adds up one unit's tokens over 1024 columns.
template <typename T> __global__ void __launch_bounds__(128) norm_bwd_cols(const __grid_constant__ NormP p)
{
    pdl_enter();
    const int ncb = (p.d + 1023) / 1024;
    const int u = blockIdx.x / ncb, c = (blockIdx.x % ncb) * 1024 + threadIdx.x * 8;
    if (c >= p.d) return;
    int t0, t1;
    unit_tokens(p, u, t0, t1);
    float P1[8] = {}, P0[8] = {}, S1[8] = {}, S0[8] = {};
    for (int64_t t = t0; t < t1; ++t) {
        float st[6], D[8], xh[8], dh[8], yh[8], g[8];
#pragma unroll
        for (int i = 0; i < 6; ++i) st[i] = p.stats[t * 8 + i];
#pragma unroll
        for (int j = 0; j < 8; ++j) yh[j] = 0.f;
        bwd_chunk<T>(p, t, c, st, D, xh, dh, yh);
        if (p.per_token) load8<T>(p.gate + t * p.ldgate + c, p.d - c, p.vec & NV_GATE, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (p.per_token) D[j] *= g[j];
            P1[j] = fmaf(dh[j], xh[j], P1[j]);
            P0[j] += dh[j];
            S1[j] = fmaf(D[j], yh[j], S1[j]);
            S0[j] += D[j];
        }
    }
    float *o = p.part + (int64_t)u * 4 * p.d + c;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j < p.d) {
            o[j] = P1[j];
            o[p.d + j] = P0[j];
            o[2 * (int64_t)p.d + j] = S1[j];
            o[3 * (int64_t)p.d + j] = S0[j];
        }
}

template <typename T> __device__ __forceinline__ void put(const NormP &p, void *out, int64_t at, float v)
{
    if (!out) return;
    if (p.g32) {
        float *o = static_cast<float *>(out) + at;
        *o = p.acc ? *o + v : v;
    } else {
        uint16_t *o = static_cast<uint16_t *>(out) + at;
        *o = C16<T>::round(p.acc ? C16<T>::one(*o) + v : v);
    }
}

// Backward, the units' partials in a fixed order: 32 columns a CTA, 16 lanes
// that share them.  blockIdx.y 0: the parameters' gradients; y > 0: the gate
// rows y - 1, y - 1 + (gridDim.y - 1), ...
constexpr int kSumLanes = 16;

template <typename T> __global__ void __launch_bounds__(32 * kSumLanes) norm_bwd_sum(const __grid_constant__ NormP p, int groups)
{
    __shared__ float red[kSumLanes][4][32];
    pdl_enter();
    const int l = threadIdx.x & 31, k = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
    const bool in = c < p.d;
    const int64_t d = p.d;
    if (blockIdx.y > 0) {
        const float w = in && p.w_post ? C16<T>::one(p.w_post[c]) : 1.f, b = in && p.b_post ? C16<T>::one(p.b_post[c]) : 0.f;
        for (int g = (int)blockIdx.y - 1; g < groups; g += (int)gridDim.y - 1) {
            float s1 = 0.f, s0 = 0.f;
            if (in) {
#pragma unroll 4
                for (int i = k; i < p.per_group; i += kSumLanes) {
                    const float *o = p.part + ((int64_t)g * p.per_group + i) * 4 * d + c;
                    s1 += o[2 * d];
                    s0 += o[3 * d];
                }
            }
            red[k][0][l] = s1, red[k][1][l] = s0;
            __syncthreads();
            if (in && k == 0) {
                for (int j = 1; j < kSumLanes; ++j) s1 += red[j][0][l], s0 += red[j][1][l];
                put<T>(p, p.dgate, g * d + c, p.bs * fmaf(w, s1, b * s0));
            }
            __syncthreads();
        }
        return;
    }
    float v[4] = {}; // P1, P0, gate S1, gate S0
    if (in) {
#pragma unroll 4
        for (int i = k; i < p.units; i += kSumLanes) {
            const float *o = p.part + (int64_t)i * 4 * d + c;
            const float gate = p.gate && !p.per_token ? C16<T>::one(p.gate[(int64_t)(i / p.per_group) * p.ldgate + c]) : 1.f;
            v[0] += o[0];
            v[1] += o[d];
            v[2] = fmaf(gate, o[2 * d], v[2]);
            v[3] = fmaf(gate, o[3 * d], v[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[k][i][l] = v[i];
    __syncthreads();
    if (!in || k) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        for (int j = 1; j < kSumLanes; ++j) v[i] += red[j][i][l];
    put<T>(p, p.dw_pre, c, v[0]);
    put<T>(p, p.db_pre, c, v[1]);
    put<T>(p, p.dw_post, c, p.bs * v[2]);
    put<T>(p, p.db_post, c, p.bs * v[3]);
}


// ------------------------------------------------------------------ pipelined rows
constexpr int kPipeThreads = 512, kPipeMaxD = 8192;

struct PipeP {
    int slots, slotB;                     // ring
    int off_dxo, off_dh, off_y, off_gate; // regions of a slot (x at 0); off_gate -1: one gate row for many tokens
    int off_hold, holdB;                  // after the ring: the current gate row
    uint32_t row_bytes;                   // bytes of a row's copies in all
    uint32_t tcols;                       // backward: tensor memory columns
    int clear;                            // some columns or rows of the ring are not copied: zeros
    int *status, *abort_flag;
    unsigned long long wait_ns;
};

__device__ __forceinline__ void bulk(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// Starts the copies of token t's rows into slot s (one thread).
__device__ __forceinline__ void issue_row(const NormP &p, const PipeP &q, uint8_t *ring, uint64_t *full, int s, int64_t t)
{
    const uint32_t dst = smem_addr(ring) + (uint32_t)(s * q.slotB), xB = (uint32_t)p.d * (p.x32 ? 4 : 2), hB = (uint32_t)p.d * 2;
    const int xe = p.x32 ? 4 : 2;
    uint64_t *b = full + s;
    mbar_expect(b, q.row_bytes);
    if (p.x) bulk(dst, (const uint8_t *)p.x + t * p.ldx * xe, xB, b);
    if (p.dxo) bulk(dst + q.off_dxo, (const uint8_t *)p.dxo + t * p.ldxo * xe, xB, b);
    if (p.dh) bulk(dst + q.off_dh, p.dh + t * p.ldh, hB, b);
    if (p.y) bulk(dst + q.off_y, p.y + t * p.ldy, hB, b);
    if (q.off_gate >= 0) bulk(dst + q.off_gate, p.gate + t * p.ldgate, hB, b);
}

template <typename T, bool X32> __device__ __forceinline__ void ring8x(const uint8_t *row, int c, float (&v)[8])
{
    if (X32) load8f(reinterpret_cast<const float *>(row) + c, 8, true, v);
    else load8<T>(reinterpret_cast<const uint16_t *>(row) + c, 8, true, v);
}

// a parameter's 8 elements, packed; 1 or 0 where there is none
template <typename T> __device__ __forceinline__ uint4 param8(const uint16_t *w, int c, int d, float none)
{
    if (w && c < d) return *reinterpret_cast<const uint4 *>(w + c);
    const uint32_t v = C16<T>::round2(none, none);
    return make_uint4(v, v, v, v);
}

template <typename T> __device__ __forceinline__ void ring8(const uint8_t *row, int c, float (&v)[8])
{
    unpack8<T>(*reinterpret_cast<const uint4 *>(row + 2 * c), v);
}

// The columns past the row, and rows that are not there, are zeros that no
// copy ever overwrites: the kernels compute on whole chunks without a test.
__device__ __forceinline__ void clear_ring(uint8_t *ring, int bytes)
{
    for (int i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16) *reinterpret_cast<uint4 *>(ring + i) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); // before the copies write there
}

// The gate row of the tokens to come (ones without a gate), each thread its own columns.
template <typename T, int V> __device__ __forceinline__ void hold_gate(const NormP &p, uint8_t *hold, int group)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c < p.d)
            *reinterpret_cast<uint4 *>(hold + 2 * c) = param8<T>(p.gate ? p.gate + (int64_t)group * p.ldgate : nullptr, c, p.d, 1.f);
    }
}

// The same for the backward pass, as fp32 factors bs gate w_post (zeros past
// the row): a chunk's 8 values in two planes of 16 bytes per thread.
template <typename T, int V> __device__ __forceinline__ void hold_factors(const NormP &p, uint8_t *hold, int group)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        float g[8], w[8];
        unpack8<T>(param8<T>(p.gate ? p.gate + (int64_t)group * p.ldgate : nullptr, c, p.d, 1.f), g);
        unpack8<T>(param8<T>(p.w_post, c, p.d, 1.f), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = c < p.d ? p.bs * g[j] * w[j] : 0.f;
        float4 *o = reinterpret_cast<float4 *>(hold) + 2 * i * blockDim.x + threadIdx.x;
        o[0] = make_float4(g[0], g[1], g[2], g[3]), o[blockDim.x] = make_float4(g[4], g[5], g[6], g[7]);
    }
}

__device__ __forceinline__ void load8f2(const float *a, const float *b, float (&v)[8])
{
    const float4 p = *reinterpret_cast<const float4 *>(a), q = *reinterpret_cast<const float4 *>(b);
    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
}

// sum over 16 lanes (both halves hold the same values)
__device__ __forceinline__ float half_add(float a)
{
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}

// Row statistics in one exchange between the warps: each publishes the sum of
// its n elements and the squares m about its own mean; the row's squares about
// its mean are sum (m_w + n_w (mean_w - mean)^2).
//
// Sums over the warp of several values at once: lanes that have added two
// halves carry on with different values, so that two sums take 6 shuffles
// instead of 10 and four take 6 instead of 20.  (A good part of the backward pass's
// instructions were such sums and what joins them: 8000 x 8192 196 -> 178 us.)
__device__ __forceinline__ float pair_sum(float a, float b, int lane) // a's in lanes 0-15, b's in 16-31
{
    float v = (lane & 16 ? b : a) + __shfl_xor_sync(0xffffffffu, lane & 16 ? a : b, 16);
    return half_add(v);
}
__device__ __forceinline__ float quad_sum(float a, float b, float c, float d, int lane) // in lanes 0-7, 8-15, ...
{
    const float v = (lane & 16 ? c : a) + __shfl_xor_sync(0xffffffffu, lane & 16 ? a : c, 16);
    const float w = (lane & 16 ? d : b) + __shfl_xor_sync(0xffffffffu, lane & 16 ? b : d, 16);
    float u = (lane & 8 ? w : v) + __shfl_xor_sync(0xffffffffu, lane & 8 ? v : w, 8);
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    return u;
}
__device__ __forceinline__ float lane_of(float v, int lane) { return __shfl_sync(0xffffffffu, v, lane); }

__device__ __forceinline__ int row_of(int64_t Tn, int c, int G) { return (int)(Tn * c / G); }

// the CTA of G whose range holds token t
__device__ __forceinline__ int cta_of(const NormP &p, int64_t t, int G) { return (int)(((t + 1) * G + p.Tn - 1) / p.Tn - 1); }

// Elements of this warp within the row (its chunks start every blockDim * 8 columns).
template <int V> __device__ __forceinline__ float warp_elems(int d)
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) n += max(0, min(256, d - (int)((threadIdx.x >> 5) * 256 + i * blockDim.x * 8)));
    return (float)n;
}

// End of a pipelined kernel that gave up: copies in flight land before it leaves.
__device__ __forceinline__ void pipe_settle()
{
    const uint64_t t0 = gtimer();
    while (gtimer() - t0 < 5000000ull) {
    }
}

// One barrier a row: behind it lie all warps' shares of the statistics of x'
// and, computed ahead about each warp's own mean, of the next row's y (4096 x
// 7168 with both norms: 72 us, 84 % of the copy rate; with three barriers 75).
template <typename T, bool X32, int V, bool MX>
__global__ void __launch_bounds__(kPipeThreads, 1) norm_fwd_pipe(const __grid_constant__ NormP p, const __grid_constant__ PipeP q)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[8];
    __shared__ float red[2][16][5]; // a warp's sums of x' and of y, then of the squares about its means
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5, S = q.slots, d = p.d;
    const int r0 = row_of(p.Tn, blockIdx.x, gridDim.x), r1 = row_of(p.Tn, blockIdx.x + 1, gridDim.x);
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init1(full + s);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    uint8_t *hold = ring + q.off_hold;
    if (q.clear) clear_ring(ring, q.off_hold + q.holdB);
    __syncthreads();
    pdl_enter();
    int issued = r0;
    if (tid == 0)
        for (; issued < min(r1, r0 + S); ++issued) issue_row(p, q, ring, full, issued - r0, issued);
    uint4 wp[V], bp[V], wq[V], bq[V];
    int c[V];
    bool on[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        c[i] = (tid + i * blockDim.x) * 8;
        on[i] = c[i] < d;
        wp[i] = param8<T>(p.w_pre, c[i], d, 1.f), bp[i] = param8<T>(p.b_pre, c[i], d, 0.f);
        wq[i] = param8<T>(p.w_post, c[i], d, 1.f), bq[i] = param8<T>(p.b_post, c[i], d, 0.f);
    }
    const bool post = p.y && p.post != PI_NORM_NONE;
    const bool lpre = p.pre == PI_NORM_LAYER, lpost = post && p.post == PI_NORM_LAYER;
    const float nel = warp_elems<V>(d), inv_nel = nel > 0.f ? 1.f / nel : 0.f, inv_d = 1.f / (float)d;
    float nz = 0.f; // elements of warp (lane mod 16), whose share this lane joins
#pragma unroll
    for (int i = 0; i < V; ++i) nz += (float)max(0, min(256, d - (int)((lane & 15) * 256 + i * blockDim.x * 8)));
    if ((lane & 15) >= nw) nz = 0.f;
    const float inv_nz = nz > 0.f ? 1.f / nz : 0.f;
    int group = -1, slot = 0, flip = 0;
    uint32_t par = 0;
    float x[V][8] = {}, z[V][8]; // x' of this row, y of the next, less the warp's means
    float rx = 0.f, cx = 0.f, rz = 0.f, cz = 0.f; // normalised: x rx + cx, z rz + cz
    float wmx = 0.f, wmz = 0.f;
    auto load_y = [&](const uint8_t *row) {
#pragma unroll
        for (int i = 0; i < V; ++i) ring8<T>(row + q.off_y, c[i], z[i]);
    };
    auto publish = [&]() {
        if (lpre || lpost) {
            float sx = 0.f, sz = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) sx += x[i][j], sz += z[i][j];
            const float v = pair_sum(sx, sz, lane);
            if ((lane & 15) == 0) red[flip][warp][lane >> 4] = v;
            if (lpre) wmx = lane_of(v, 0) * inv_nel;
            if (lpost) wmz = lane_of(v, 16) * inv_nel;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (on[i]) x[i][j] -= wmx, z[i][j] -= wmz;
        }
        float qx = 0.f, qz = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) qx = fmaf(x[i][j], x[i][j], qx), qz = fmaf(z[i][j], z[i][j], qz);
        const float v = pair_sum(qx, qz, lane);
        if ((lane & 15) == 0) red[flip][warp][2 + (lane >> 4)] = v;
    };
    // all warps' shares: those of x' in lanes 0-15, of y in lanes 16-31
    auto join = [&]() {
        const int hi = lane >> 4;
        const bool in = (lane & 15) < nw;
        const float *w = red[flip][lane & 15];
        float m = in ? w[2 + hi] : 0.f, mean = 0.f;
        if (lpre || lpost) {
            const float u = in ? w[hi] : 0.f, all = half_add(u);
            if (hi ? lpost : lpre) {
                mean = all * inv_d;
                const float e = u * inv_nz - mean;
                m = fmaf(nz * e, e, m);
            }
        }
        m = half_add(m);
        const float r = (hi ? post : p.h != nullptr) ? 1.f / sqrtf(m * inv_d + p.eps) : 1.f;
        // (the warp's mean lies within sqrt(d / its elements) deviations of the row's: x rx + cx cancels little)
        rx = lane_of(r, 0), rz = lane_of(r, 16);
        cx = (wmx - lane_of(mean, 0)) * rx, cz = (wmz - lane_of(mean, 16)) * rz;
    };
    if (MX) mx_pad_scales(p.mx_scales, p.Tn, p.mx_tiles, (int64_t)blockIdx.x * blockDim.x + tid, (int64_t)gridDim.x * blockDim.x);
    bool ok = true;
    if (r0 < r1) {
        ok = mbar_wait_bounded(full, 0, q);
        load_y(ring);
        publish();
    }
    ok = __syncthreads_and(ok);
    if (ok && r0 < r1) join();
    flip = 1;
    for (int t = r0; ok && t < r1; ++t) {
        const uint8_t *row = ring + slot * q.slotB, *gate = q.off_gate >= 0 ? row + q.off_gate : hold;
        if (q.off_gate < 0 && t / p.gate_rows != group) {
            group = t / p.gate_rows;
            hold_gate<T, V>(p, hold, group);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float g[8];
            if (post) {
                float w8[8], b8[8];
                unpack8<T>(wq[i], w8), unpack8<T>(bq[i], b8);
#pragma unroll
                for (int j = 0; j < 8; ++j) z[i][j] = fmaf(fmaf(z[i][j], rz, cz), w8[j], b8[j]);
            }
            ring8x<T, X32>(row, c[i], x[i]);
            ring8<T>(gate, c[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = fmaf(p.bs * g[j], z[i][j], p.rs * x[i][j]);
            if (p.xo && on[i]) storex8<T>(p.xo, X32, (int64_t)t * p.ldxo + c[i], 8, true, x[i]);
        }
        const int done = slot;
        if (++slot == S) slot = 0, par ^= 1u;
        if (t + 1 < r1) {
            ok = mbar_wait_bounded(full + slot, par, q);
            load_y(ring + slot * q.slotB);
        }
        publish();
        ok = __syncthreads_and(ok); // also: every thread is done with this row's slot
        if (!ok) break;
        if (tid == 0 && issued < r1) issue_row(p, q, ring, full, done, issued), ++issued;
        join();
        if (p.h) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float w8[8], b8[8];
                unpack8<T>(wp[i], w8), unpack8<T>(bp[i], b8);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = fmaf(fmaf(x[i][j], rx, cx), w8[j], b8[j]);
                if (MX) norm_store_mx(p, t, c[i], x[i]);
                else if (on[i]) store8<T>(p.h + (int64_t)t * p.ldh + c[i], 8, true, x[i]);
            }
        }
        flip ^= 1;
    }
    if (!ok || *(volatile int *)q.abort_flag) pipe_settle();
}

// 16 values of this thread's tensor memory lane, written (tm_settle before they are read)
__device__ __forceinline__ void tm_st16(uint32_t at, const float (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
                 "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
                 "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
                 : "memory");
}
// The load of 16 columns starts; tm_have16 before its values are used (they
// are operands there, so that no use moves in front of the wait).
__device__ __forceinline__ void tm_ld16(uint32_t at, float (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
                   "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(at));
}
__device__ __forceinline__ void tm_have16(float (&v)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                   "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
__device__ __forceinline__ void tm_settle() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What a warp publishes of a row in the backward pass: the sums of x' and y,
// then about its own means of x'^2, dh w x', y^2 and dh w.
enum { ST_SX, ST_SY, ST_MX, ST_SQX, ST_MY, ST_SQ, ST_N = 9 }; // (9: no bank conflicts)

// FULL: layer norms, and the plain sums P0 and S0 (biases); else RMS norms
// without them.  Per row two barriers: each warp publishes its share of the
// statistics about its own mean, then of the sums for y's gradient.
// The column sums, 4 fp32 values per column of this CTA's tokens, live in
// tensor memory, where each thread adds to its own columns' values: in
// registers they took half of what 512 threads have (8000 x 8192 layer norms:
// 345 us with 512 threads and spills, 271 us with 256 threads of 32 columns).
// Bound by the latency of one row at a time (4 warps a scheduler, 0.58 issues per
// cycle, HBM 50 %; of a warp's time 21 % waits for shared memory and shuffles, 7 %
// at the barriers, 21 % for warps that are ready at the same moment), so fewer
// instructions still count: what one gate row's tokens share, bs gate
// w_post, is multiplied once, each element's value is kept in the form that its
// next use wants (209 -> 196 us), and sums share shuffles (178 us; 172 with the
// join below; 4.6 TB/s).  (The next row's statistics computed ahead of the same
// barrier took 235 instead of 196 us, the registers being full.)
// RG: a gate row per token, in the ring.
template <typename T, bool X32, int V, bool FULL, bool RG>
__global__ void __launch_bounds__(kPipeThreads, 1) norm_bwd_pipe(const __grid_constant__ NormP p, const __grid_constant__ PipeP q)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[8];
    __shared__ float red[2][16][ST_N], red2[2][16][2];
    __shared__ uint32_t tslot;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5, S = q.slots, d = p.d;
    const int r0 = row_of(p.Tn, blockIdx.x, gridDim.x), r1 = row_of(p.Tn, blockIdx.x + 1, gridDim.x);
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init1(full + s);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    uint8_t *hold = ring + q.off_hold;
    if (q.clear) clear_ring(ring, q.off_hold + q.holdB);
    const uint32_t tmem = tmem_alloc(&tslot, q.tcols);
    pdl_enter();
    int issued = r0;
    if (tid == 0)
        for (; issued < min(r1, r0 + S); ++issued) issue_row(p, q, ring, full, issued - r0, issued);
    constexpr bool row_gate = RG;
    const bool pre = p.dh != nullptr, post = p.y && p.post != PI_NORM_NONE;
    const bool lpre = FULL && p.pre == PI_NORM_LAYER, lpost = FULL && p.post == PI_NORM_LAYER;
    uint4 wp[V], wq[V];
    int c[V];
    bool on[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        c[i] = (tid + i * blockDim.x) * 8;
        on[i] = c[i] < d;
        wp[i] = param8<T>(p.w_pre, c[i], d, 1.f), wq[i] = param8<T>(p.w_post, c[i], d, 1.f);
    }
    // this thread's sums: chunk i at columns 32 i of its warp's: P1, P0, S1, S0 (8 each)
    const uint32_t sums = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(warp >> 2) * 32 * V;
    {
        float z[16] = {};
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) tm_st16(sums + 16 * i, z);
    }
    const float nel = warp_elems<V>(d), inv_nel = nel > 0.f ? 1.f / nel : 0.f, inv_d = 1.f / (float)d;
    // elements of warp (lane mod 16), whose share this lane joins
    float nz = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) nz += (float)max(0, min(256, d - (int)((lane & 15) * 256 + i * blockDim.x * 8)));
    if ((lane & 15) >= nw) nz = 0.f;
    const float inv_nz = nz > 0.f ? 1.f / nz : 0.f;
    int group = -1, slot = 0, flip = 0;
    uint32_t par = 0;
    bool ok = true;
    // S1 and S0 of the rows of one gate row so far -> their partial slot
    auto flush = [&]() {
        float *o = p.part + (2 * (int64_t)gridDim.x + 2 * ((int64_t)blockIdx.x + (p.per_token ? 0 : group))) * d;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v[16];
            tmem_ld16(sums + 32 * i + 16, v);
            if (on[i]) store8f(o + c[i], 8, true, *reinterpret_cast<float(*)[8]>(v));
            if (FULL && on[i]) store8f(o + d + c[i], 8, true, *reinterpret_cast<float(*)[8]>(v + 8));
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.f;
            tm_st16(sums + 32 * i + 16, v);
        }
        tm_settle();
    };
    for (int t = r0; t < r1; ++t) {
        ok = mbar_wait_bounded(full + slot, par, q);
        const uint8_t *row = ring + slot * q.slotB;
        tm_settle(); // (the previous row's sums are in tensor memory)
        if (!row_gate && t / p.gate_rows != group) {
            if (group >= 0 && p.part) flush();
            group = t / p.gate_rows;
            hold_factors<T, V>(p, hold, group);
        }
        // statistics of x' and y, and the sums of dh w and dh w xh, about the warp's means
        float wmx = 0.f, wmy = 0.f, sx = 0.f, sy = 0.f, qx = 0.f, qy = 0.f, sq = 0.f, sqx = 0.f;
        float x[V][8], y[V][8]; // x' and y, then less the warp's means, then normalised
#pragma unroll
        for (int i = 0; i < V; ++i) {
            ring8x<T, X32>(row, c[i], x[i]);
            ring8<T>(row + q.off_y, c[i], y[i]);
            if (FULL) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sx += x[i][j], sy += y[i][j];
            }
        }
        if (FULL) {
            const float v = pair_sum(sx, sy, lane);
            if ((lane & 15) == 0) red[flip][warp][lane ? ST_SY : ST_SX] = v;
            if (lpre) wmx = lane_of(v, 0) * inv_nel;
            if (lpost) wmy = lane_of(v, 16) * inv_nel;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float h[8], w[8];
            ring8<T>(row + q.off_dh, c[i], h);
            unpack8<T>(wp[i], w);
            const float mx = on[i] ? wmx : 0.f, my = on[i] ? wmy : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float k = h[j] * w[j];
                if (FULL) x[i][j] -= mx, y[i][j] -= my;
                qx = fmaf(x[i][j], x[i][j], qx);
                if (FULL) sq += k;
                sqx = fmaf(k, x[i][j], sqx);
                qy = fmaf(y[i][j], y[i][j], qy);
            }
        }
        {
            const float v = quad_sum(qx, sqx, qy, sq, lane);
            if ((lane & 7) == 0) red[flip][warp][ST_MX + (lane >> 3)] = v;
        }
        if (!__syncthreads_and(ok)) break;
        // all warps' shares: those of x' in lanes 0-15, of y in lanes 16-31
        float mx = 0.f, my = 0.f, c1 = 0.f, rx, ry, c2;
        {
            const bool hi = lane & 16, in = (lane & 15) < nw;
            const float *z = red[flip][lane & 15];
            float m = in ? z[hi ? ST_MY : ST_MX] : 0.f, k = in ? z[hi ? ST_SQ : ST_SQX] : 0.f;
            float mean = 0.f;
            if (FULL) {
                const float u = in ? z[hi ? ST_SY : ST_SX] : 0.f, all = half_add(u);
                if (hi ? lpost : lpre) {
                    mean = all * inv_d;
                    const float e = u * inv_nz - mean;
                    m = fmaf(nz * e, e, m);
                    if (!hi && in) k = fmaf(e, z[ST_SQ], k);
                }
                mx = lane_of(mean, 0), my = lane_of(mean, 16);
            }
            m = half_add(m), k = half_add(k);
            const float r = (hi ? post : pre) ? 1.f / sqrtf(m * inv_d + p.eps) : hi ? 1.f : 0.f;
            rx = lane_of(r, 0), ry = lane_of(r, 16);
            c2 = lane_of(k, 0) * rx * inv_d;
            if (lpre) c1 = lane_of(k, 16) * inv_d;
        }
        // (the warp's mean lies within sqrt(d / its elements) deviations of the row's: x rx + cx cancels little)
        const float cx = (wmx - mx) * rx, cy = (wmy - my) * ry;
        // D, dx, the column sums, and the sums for y's gradient
        float D[V][8]; // later D bs gate w_post, the gradient of y's normalised row
        float s1 = 0.f, s2 = 0.f;
        const float k0 = -rx * c1, kx = -rx * c2;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v[8], h[8], w[8], a[16]; // a: P1, P0
            tm_ld16(sums + 32 * i, a);
            ring8x<T, X32>(row + q.off_dxo, c[i], D[i]);
            ring8<T>(row + q.off_dh, c[i], h);
            unpack8<T>(wp[i], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = FULL ? fmaf(x[i][j], rx, cx) : x[i][j] * rx;
                float e = fmaf(rx * h[j], w[j], D[i][j]);
                if (FULL) e += k0;
                D[i][j] = fmaf(kx, xh, e);
                v[j] = p.rs * D[i][j];
                x[i][j] = xh;
            }
            tm_have16(a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] = fmaf(h[j], x[i][j], a[j]);
                if (FULL) a[8 + j] += h[j];
            }
            tm_st16(sums + 32 * i, a);
            if (p.dx && on[i]) storex8<T>(p.dx, X32, (int64_t)t * p.lddx + c[i], 8, true, v);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float g[8], a[16]; // g: the gate, or bs gate w_post; a: S1, S0
            tm_ld16(sums + 32 * i + 16, a);
            if (row_gate) ring8<T>(row + q.off_gate, c[i], g);
            else {
                const float *o = reinterpret_cast<const float *>(hold) + (2 * i * blockDim.x + tid) * 4;
                load8f2(o, o + 4 * blockDim.x, g);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) y[i][j] = FULL ? fmaf(y[i][j], ry, cy) : y[i][j] * ry;
            if (row_gate && p.dgate && on[i]) {
                float b[8], o[8], w[8];
                unpack8<T>(wq[i], w);
                unpack8<T>(param8<T>(p.b_post, c[i], d, 0.f), b);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = p.bs * D[i][j] * fmaf(y[i][j], w[j], b[j]);
                const int64_t at = (int64_t)t * d + c[i];
                if (p.acc) {
                    float old[8];
                    loadx8<T>(p.dgate, p.g32, at, 8, true, old);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] += old[j];
                }
                storex8<T>(p.dgate, p.g32, at, 8, true, o);
            }
            float w[8];
            if (row_gate) unpack8<T>(wq[i], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float k = row_gate ? g[j] * D[i][j] : D[i][j]; // (what S1 and S0 sum)
                D[i][j] = row_gate ? p.bs * k * w[j] : k * g[j];
                if (FULL) s1 += D[i][j];
                s2 = fmaf(D[i][j], y[i][j], s2);
                g[j] = k;
            }
            tm_have16(a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] = fmaf(g[j], y[i][j], a[j]);
                if (FULL) a[8 + j] += g[j];
            }
            tm_st16(sums + 32 * i + 16, a);
        }
        if (post) {
            const float v = pair_sum(s1, s2, lane);
            if ((lane & 15) == 0) red2[flip][warp][lane >> 4] = v;
        }
        __syncthreads(); // also: every thread is done with the row's slot
        if (tid == 0 && issued < r1) issue_row(p, q, ring, full, slot, issued), ++issued;
        if (p.dy) {
            float k1 = 0.f, k2 = 0.f;
            if (post) {
                const float v = half_add((lane & 15) < nw ? red2[flip][lane & 15][lane >> 4] : 0.f);
                if (lpost) k1 = lane_of(v, 0) * inv_d;
                k2 = lane_of(v, 16) * inv_d;
            }
            k1 *= -ry, k2 *= -ry;
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[i][j] = fmaf(k2, y[i][j], FULL ? fmaf(ry, D[i][j], k1) : ry * D[i][j]);
                if (on[i]) store8<T>(p.dy + (int64_t)t * p.ldy + c[i], 8, true, y[i]);
            }
        }
        flip ^= 1;
        if (++slot == S) slot = 0, par ^= 1u;
    }
    tm_settle();
    if (!ok || *(volatile int *)q.abort_flag) pipe_settle();
    if (!__syncthreads_and(ok) || !p.part) {
        tmem_free(tmem, q.tcols);
        return;
    }
    flush();
    float *o = p.part + 2 * (int64_t)blockIdx.x * d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float v[16];
        tmem_ld16(sums + 32 * i, v);
        if (on[i]) store8f(o + c[i], 8, true, *reinterpret_cast<float(*)[8]>(v));
        if (FULL && on[i]) store8f(o + d + c[i], 8, true, *reinterpret_cast<float(*)[8]>(v + 8));
    }
    tmem_free(tmem, q.tcols);
}

// The CTAs' partials in a fixed order: 32 columns a CTA, 16 lanes that share
// the parts (32: one CTA at a time on an SM, 177 instead of 172 us for the
// backward pass of 8000 x 8192 in all).
// Tokens of gate row g lie in CTAs c0 .. c1 of the row kernel; partial slot
// c + g.  blockIdx.y 0: the parameters' gradients; y > 0: gate rows.
constexpr int kJoinLanes = 16;
constexpr int kMaxCtas = 2048; // of the row kernel

template <typename T>
__global__ void __launch_bounds__(32 * kJoinLanes) norm_bwd_join(const __grid_constant__ NormP p, int G, int groups, int sums, int lpg)
{
    __shared__ float red[kJoinLanes][6][32];
    extern __shared__ __align__(128) uint8_t ring[];
    int *first = reinterpret_cast<int *>(ring), *last = first + G; // gate rows of a CTA's tokens
    if (blockIdx.y == 0) {
        for (int i = threadIdx.x; i < G; i += blockDim.x) {
            first[i] = p.per_token ? 0 : row_of(p.Tn, i, G) / p.gate_rows;
            last[i] = p.per_token ? 0 : (row_of(p.Tn, i + 1, G) - 1) / p.gate_rows;
        }
        __syncthreads();
    }
    pdl_enter();
    const int l = threadIdx.x & 31, k = threadIdx.x >> 5, c = blockIdx.x * 32 + l, d = p.d;
    const bool in = c < d;
    const float *S = p.part + (int64_t)G * 2 * d;
    const float w = in && p.w_post ? C16<T>::one(p.w_post[c]) : 1.f, b = in && p.b_post ? C16<T>::one(p.b_post[c]) : 0.f;
    if (blockIdx.y > 0) {
        // lpg lanes to a gate row, kJoinLanes / lpg gate rows at a time
        const int per = kJoinLanes / lpg, sub = k % lpg;
        for (int g0 = ((int)blockIdx.y - 1) * per; g0 < groups; g0 += ((int)gridDim.y - 1) * per) {
            const int g = g0 + k / lpg;
            float a = 0.f, z = 0.f;
            if (in && g < groups) {
                const int c0 = cta_of(p, g * (int64_t)p.gate_rows, G);
                const int c1 = cta_of(p, min((int64_t)p.Tn, (g + 1) * (int64_t)p.gate_rows) - 1, G);
#pragma unroll 4
                for (int i = c0 + sub; i <= c1; i += lpg) {
                    a += S[(int64_t)(i + g) * 2 * d + c];
                    if (sums) z += S[((int64_t)(i + g) * 2 + 1) * d + c];
                }
            }
            red[k][0][l] = a, red[k][1][l] = z;
            __syncthreads();
            if (in && sub == 0 && g < groups) {
                for (int j = 1; j < lpg; ++j) a += red[k + j][0][l], z += red[k + j][1][l];
                put<T>(p, p.dgate, (int64_t)g * d + c, p.bs * fmaf(w, a, b * z));
            }
            __syncthreads();
        }
        return;
    }
    float v[6] = {}; // P1, P0, gate S1, gate S0, S1, S0
    auto add_s = [&](int i, int g) {
        const float gate = p.gate && !p.per_token ? C16<T>::one(p.gate[(int64_t)g * p.ldgate + c]) : 1.f;
        const float a = S[(int64_t)(i + g) * 2 * d + c], z = sums ? S[((int64_t)(i + g) * 2 + 1) * d + c] : 0.f;
        v[2] = fmaf(gate, a, v[2]);
        v[3] = fmaf(gate, z, v[3]);
        v[4] += a;
        v[5] += z;
    };
    if (in) {
#pragma unroll 4
        for (int i = k; i < G; i += kJoinLanes) {
            v[0] += p.part[(int64_t)i * 2 * d + c];
            if (sums) v[1] += p.part[((int64_t)i * 2 + 1) * d + c];
        }
        if (p.y) {
            // most CTAs meet one gate row: their loads first, all in flight
#pragma unroll 4
            for (int i = k; i < G; i += kJoinLanes) add_s(i, first[i]);
            for (int i = k; i < G; i += kJoinLanes)
                for (int g = first[i] + 1; g <= last[i]; ++g) add_s(i, g);
        }
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) red[k][i][l] = v[i];
    __syncthreads();
    if (k < 6) { // a warp each
        float a = red[0][k][l];
#pragma unroll
        for (int j = 1; j < kJoinLanes; ++j) a += red[j][k][l];
        red[0][k][l] = a;
    }
    __syncthreads();
    if (!in || k) return;
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = red[0][i][l];
    put<T>(p, p.dw_pre, c, v[0]);
    put<T>(p, p.db_pre, c, v[1]);
    put<T>(p, p.dw_post, c, p.bs * v[2]);
    put<T>(p, p.db_post, c, p.bs * v[3]);
    if (p.dgate && groups == 1 && !p.per_token) put<T>(p, p.dgate, c, p.bs * fmaf(w, v[4], b * v[5]));
}

template <typename T, int V, bool MX> cudaError_t launch_fwd(const NormP &p, cudaStream_t s)
{
    const int nt = ((p.d + 8 * V - 1) / (8 * V) + 31) / 32 * 32;
    // (16 rows of a tile's scales a CTA more, where a microscaled h leaves some)
    const int pad = MX ? (((128 - (p.Tn & 127)) & 127) + 15) / 16 : 0;
    return launch_pdl(norm_fwd<T, V, MX>, dim3(p.Tn + pad), dim3(nt), 0, s, p);
}

// The ring of a pipelined launch: rows of up to kPipeMaxD elements, all 16-byte
// aligned; false if they are not.  CTAs per SM: as many as 512 threads and
// about 200 KB of ring allow, with two to four slots each.
struct Pipe {
    PipeP q;
    int threads, v, grid, smem;
};

bool plan_pipe(const NormP &p, bool backward, bool row_gate, const CtxView &c, Pipe &o)
{
    if (p.d % 8 || p.d > kPipeMaxD) return false;
    const unsigned need = NV_PAR | (p.x ? NV_X : 0) | (p.y ? NV_Y : 0) | (p.gate ? NV_GATE : 0) |
                          (backward ? (p.dxo ? NV_DXO : 0) | (p.dh ? NV_H : 0) | (p.dx ? NV_DX : 0) | (p.dy ? NV_DY : 0) |
                                          (p.dgate ? NV_DGATE : 0)
                                    : (p.xo ? NV_XO : 0) | (p.h ? NV_H : 0));
    if ((p.vec & need) != need) return false;
    o.v = p.d > 8 * kPipeThreads ? 2 : 1;
    o.threads = (p.d / 8 + 32 * o.v - 1) / (32 * o.v) * 32;
    // regions of whole chunks: a row's own bytes, then zeros
    const int wide = o.threads * 8 * o.v, xB = wide * (p.x32 ? 4 : 2), hB = wide * 2, xe = p.x32 ? 4 : 2;
    PipeP &q = o.q;
    int at = xB;
    auto take = [&](int bytes) { const int r = at; at += bytes; return r; };
    q.off_dxo = backward ? take(xB) : 0;
    q.off_dh = backward ? take(hB) : 0;
    q.off_y = take(hB);
    q.off_gate = row_gate ? take(hB) : -1;
    q.slotB = at;
    q.row_bytes = (uint32_t)p.d * ((p.x ? xe : 0) + (backward && p.dxo ? xe : 0) + (backward && p.dh ? 2 : 0) + (p.y ? 2 : 0) +
                                   (row_gate ? 2 : 0));
    q.clear = wide != p.d || !p.x || !p.y || (backward && (!p.dxo || !p.dh));
    q.holdB = row_gate ? 0 : backward ? 2 * hB : hB; // (16 bits, or factors of 32)
    const int budget = c.smem_optin - 2048 - q.holdB;
    int per_sm = std::min(8, kPipeThreads / o.threads);
    while (per_sm > 1 && per_sm * (2 * q.slotB + q.holdB + 4096) > budget) --per_sm;
    q.slots = std::min(4, (budget / per_sm - (per_sm > 1 ? q.holdB + 4096 : 0)) / q.slotB);
    if (q.slots < 2) return false;
    q.off_hold = q.slots * q.slotB;
    o.smem = q.off_hold + q.holdB;
    // (a power of two from 32 up; at most 256 a CTA of 16 warps, so that the CTAs of an SM fit its 512)
    q.tcols = 32;
    while (q.tcols < (uint32_t)(o.threads / 32 + 3) / 4 * 32 * o.v) q.tcols *= 2;
    o.grid = std::min({p.Tn, c.sms * per_sm, kMaxCtas});
    q.status = c.status, q.abort_flag = c.abort_flag, q.wait_ns = c.wait_ns;
    return true;
}

template <auto KERN> cudaError_t run_pipe(const NormP &p, const Pipe &o, cudaStream_t s)
{
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = raise_limit((const void *)KERN, ready);
    return e != cudaSuccess ? e : launch_pdl(KERN, dim3(o.grid), dim3(o.threads), o.smem, s, p, o.q);
}

// Tokens from which the pipelined forward kernel runs: below two per SM
// nothing is left to overlap, and one CTA per token with the whole row in
// flight at once answers sooner.
constexpr int kPipeRows = 2;

template <typename T, bool MX> cudaError_t fwd_as(const NormP &p, const CtxView &c)
{
    Pipe o;
    const bool row_gate = p.gate && p.gate_rows == 1;
    if (p.Tn >= kPipeRows * c.sms && plan_pipe(p, false, row_gate, c, o)) {
        if (p.x32)
            return o.v == 1 ? run_pipe<norm_fwd_pipe<T, true, 1, MX>>(p, o, c.stream)
                            : run_pipe<norm_fwd_pipe<T, true, 2, MX>>(p, o, c.stream);
        return o.v == 1 ? run_pipe<norm_fwd_pipe<T, false, 1, MX>>(p, o, c.stream)
                        : run_pipe<norm_fwd_pipe<T, false, 2, MX>>(p, o, c.stream);
    }
    return p.d <= 8192 ? launch_fwd<T, 1, MX>(p, c.stream) : launch_fwd<T, 2, MX>(p, c.stream);
}
template <typename T> cudaError_t fwd(const NormP &p, const CtxView &c) { return p.mx ? fwd_as<T, true>(p, c) : fwd_as<T, false>(p, c); }

template <typename T, bool X32, bool FULL> cudaError_t bwd_pipe(const NormP &p, const Pipe &o, cudaStream_t s)
{
    if (o.q.off_gate >= 0)
        return o.v == 1 ? run_pipe<norm_bwd_pipe<T, X32, 1, FULL, true>>(p, o, s)
                        : run_pipe<norm_bwd_pipe<T, X32, 2, FULL, true>>(p, o, s);
    return o.v == 1 ? run_pipe<norm_bwd_pipe<T, X32, 1, FULL, false>>(p, o, s)
                    : run_pipe<norm_bwd_pipe<T, X32, 2, FULL, false>>(p, o, s);
}

template <typename T> cudaError_t bwd(const NormP &p, bool cols, const CtxView &c)
{
    Pipe o;
    const cudaStream_t s = c.stream;
    if (plan_pipe(p, true, p.per_token != 0, c, o)) {
        const bool sums = p.db_pre || p.db_post || (p.dgate && p.b_post);
        const bool full = sums || p.pre == PI_NORM_LAYER || p.post == PI_NORM_LAYER;
        const cudaError_t e = p.x32 ? (full ? bwd_pipe<T, true, true>(p, o, s) : bwd_pipe<T, true, false>(p, o, s))
                                    : (full ? bwd_pipe<T, false, true>(p, o, s) : bwd_pipe<T, false, false>(p, o, s));
        if (e != cudaSuccess || !cols) return e;
        const int groups = p.per_token ? 1 : (int)((p.Tn + (int64_t)p.gate_rows - 1) / p.gate_rows);
        int lpg = 1;
        while (2 * lpg * groups <= kJoinLanes) lpg *= 2;
        const int sets = (groups + kJoinLanes / lpg - 1) / (kJoinLanes / lpg);
        const int gy = p.dgate && !p.per_token && groups > 1 ? std::min(sets, 64) : 0;
        return launch_pdl(norm_bwd_join<T>, dim3((p.d + 31) / 32, 1 + gy), dim3(32 * kJoinLanes), o.grid * 8, s, p, o.grid,
                          groups, (int)full, lpg);
    }
    const int nt = std::min(512, ((p.d + 7) / 8 + 31) / 32 * 32);
    cudaError_t e = launch_pdl(norm_bwd_rows<T>, dim3(p.Tn), dim3(nt), 0, s, p);
    if (e != cudaSuccess || !cols) return e;
    const int64_t blocks = (int64_t)p.units * ((p.d + 1023) / 1024);
    e = launch_pdl(norm_bwd_cols<T>, dim3((unsigned)blocks), dim3(128), 0, s, p);
    if (e != cudaSuccess) return e;
    const int groups = p.units / p.per_group, gy = p.dgate && !p.per_token ? std::min(groups, 64) : 0;
    return launch_pdl(norm_bwd_sum<T>, dim3((p.d + 31) / 32, 1 + gy), dim3(32 * kSumLanes), 0, s, p, groups);
}

bool norm_kind(int k) { return k == PI_NORM_NONE || k == PI_NORM_RMS || k == PI_NORM_LAYER; }

pi_status check(pi_ctx *c, const pi_norm_residual_desc *d, pi_norm_residual_desc &o)
{
    if (!d) return ctx_fail(c, PI_ERR_ARG, "desc is NULL");
    o = *d;
    if (o.dtype != PI_F16 && o.dtype != PI_BF16)
        return ctx_fail(c, PI_ERR_ARG, "dtype %d is not PI_F16 or PI_BF16", o.dtype);
    if (o.x_dtype != o.dtype && o.x_dtype != PI_F32)
        return ctx_fail(c, PI_ERR_ARG, "x_dtype %d is neither dtype nor PI_F32", o.x_dtype);
    if (o.grad_dtype != o.dtype && o.grad_dtype != PI_F32)
        return ctx_fail(c, PI_ERR_ARG, "grad_dtype %d is neither dtype nor PI_F32", o.grad_dtype);
    if (!norm_kind(o.pre) || !norm_kind(o.post)) return ctx_fail(c, PI_ERR_ARG, "pre %d or post %d invalid", o.pre, o.post);
    if (o.gate_rows < 0) return ctx_fail(c, PI_ERR_ARG, "gate_rows %d is negative", o.gate_rows);
    if (!std::isfinite(o.res_scale) || !std::isfinite(o.branch_scale) || !std::isfinite(o.eps) || o.eps < 0.f)
        return ctx_fail(c, PI_ERR_ARG, "res_scale, branch_scale or eps is not finite, or eps is negative");
    if (o.T < 0 || o.T > kMaxT) return ctx_fail(c, PI_ERR_SHAPE, "T %d outside [0, %d]", o.T, kMaxT);
    if (o.d < 1 || o.d > kMaxNormD) return ctx_fail(c, PI_ERR_SHAPE, "d %d outside [1, %d]", o.d, kMaxNormD);
    int64_t *lds[] = {&o.ldx, &o.ldxo, &o.ldy, &o.ldh, &o.ldgate};
    for (int64_t *l : lds) {
        if (!*l) *l = o.d;
        if (*l < o.d) return ctx_fail(c, PI_ERR_SHAPE, "row stride %lld below the row's %d elements", (long long)*l, o.d);
    }
    if (!o.lddxo) o.lddxo = o.ldxo;
    if (o.lddxo < o.d) return ctx_fail(c, PI_ERR_SHAPE, "row stride %lld below the row's %d elements", (long long)o.lddxo, o.d);
    return PI_OK;
}

unsigned vb(const void *p, int64_t ld, int elem, unsigned bit)
{
    return ((uintptr_t)p & 15) == 0 && (ld * elem) % 16 == 0 ? bit : 0;
}

NormP params(const pi_norm_residual_desc &d, const pi_norm_residual_params *q)
{
    NormP p = {};
    p.Tn = d.T, p.d = d.d, p.pre = d.pre, p.post = d.post, p.x32 = d.x_dtype == PI_F32;
    p.gate_rows = d.gate_rows ? d.gate_rows : std::max(1, d.T);
    p.rs = d.res_scale, p.bs = d.branch_scale, p.eps = d.eps;
    p.ldx = d.ldx, p.ldxo = d.ldxo, p.ldy = d.ldy, p.ldh = d.ldh, p.ldgate = d.ldgate;
    if (q) {
        p.w_pre = (const uint16_t *)q->w_pre, p.b_pre = (const uint16_t *)q->b_pre;
        p.w_post = (const uint16_t *)q->w_post, p.b_post = (const uint16_t *)q->b_post;
    }
    if (p.pre == PI_NORM_NONE) p.w_pre = p.b_pre = nullptr;
    if (p.post == PI_NORM_NONE) p.w_post = p.b_post = nullptr;
    const uintptr_t all = (uintptr_t)p.w_pre | (uintptr_t)p.b_pre | (uintptr_t)p.w_post | (uintptr_t)p.b_post;
    if ((all & 15) == 0) p.vec |= NV_PAR;
    return p;
}

// The units of the column sums, and the workspace.
struct Units {
    int units, per_group, unit;
    bool per_token;
    size_t stats, part;
};

Units plan_units(const pi_norm_residual_desc &d, bool gate, int sms)
{
    Units u;
    const int gr = gate && d.gate_rows ? d.gate_rows : std::max(1, d.T);
    u.per_token = gate && gr == 1 && d.T > 1;
    u.unit = unit_rows(d.T, d.d, sms);
    u.per_group = ((u.per_token ? d.T : std::min(gr, std::max(1, d.T))) + u.unit - 1) / u.unit;
    const int64_t groups = u.per_token ? 1 : (d.T + (int64_t)gr - 1) / gr;
    // the last gate row may have fewer tokens, and units without any add zeros
    u.units = (int)(groups * u.per_group);
    u.stats = ((size_t)d.T * 8 * 4 + 255) / 256 * 256;
    u.part = (size_t)u.units * 4 * d.d * 4;
    // the pipelined kernel: [CTAs][2][d], then [CTAs + gate rows][2][d]
    const size_t ctas = std::min<size_t>(d.T, (size_t)8 * sms);
    u.part = std::max(u.part, (2 * ctas + (size_t)groups) * 2 * d.d * 4);
    return u;
}

#define CUN(call)                                                                                          \
    do {                                                                                                   \
        cudaError_t e_ = (call);                                                                           \
        if (e_ != cudaSuccess) return ctx_fail(c, PI_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_));   \
    } while (0)

// A forward call whose h is in place.
pi_status forward(pi_ctx *c, const pi_norm_residual_desc &d, NormP &p, const void *x, const void *y, const void *gate, void *x_out)
{
    if (!x) return ctx_fail(c, PI_ERR_ARG, "x is NULL");
    if (y && !x_out) return ctx_fail(c, PI_ERR_ARG, "x_out is NULL");
    if (!p.h && !x_out) return PI_OK;
    const CtxView v = ctx_view(c);
    const int xe = p.x32 ? 4 : 2;
    if (pi_status st = check_elements(c, xe, {x, x_out})) return st;
    if (pi_status st = check_elements(c, 2, {y, gate, p.w_pre, p.b_pre, p.w_post, p.b_post})) return st;
    p.x = x, p.y = (const uint16_t *)y, p.gate = y ? (const uint16_t *)gate : nullptr, p.xo = x_out;
    p.vec |= vb(x, p.ldx, xe, NV_X) | vb(x_out, p.ldxo, xe, NV_XO) | vb(y, p.ldy, 2, NV_Y) | vb(gate, p.ldgate, 2, NV_GATE);
    DeviceGuard g(v.device);
    CUN(d.dtype == PI_BF16 ? fwd<__nv_bfloat16>(p, v) : fwd<__half>(p, v));
    return PI_OK;
}

} // namespace
} // namespace pi

using namespace pi;

extern "C" {

pi_status pi_norm_residual(pi_ctx *c, const pi_norm_residual_desc *desc, const pi_norm_residual_params *q,
                           const void *x, const void *y, const void *gate, void *x_out, void *h)
{
    if (!c) return PI_ERR_ARG;
    pi_norm_residual_desc d;
    if (pi_status st = check(c, desc, d)) return st;
    if (d.T == 0) return PI_OK;
    if ((h != nullptr) != (d.pre != PI_NORM_NONE)) return ctx_fail(c, PI_ERR_ARG, "h goes with a pre norm, and only with it");
    if (pi_status st = check_elements(c, 2, {h})) return st;
    NormP p = params(d, q);
    p.h = static_cast<uint16_t *>(h);
    p.vec |= vb(h, p.ldh, 2, NV_H);
    return forward(c, d, p, x, y, gate, x_out);
}

pi_status pi_norm_residual_mx(pi_ctx *c, const pi_norm_residual_desc *desc, int32_t kind, const pi_norm_residual_params *q,
                              const void *x, const void *y, const void *gate, void *x_out, const pi_mx *h)
{
    if (!c) return PI_ERR_ARG;
    if (!desc) return ctx_fail(c, PI_ERR_ARG, "desc is NULL");
    if (kind != PI_MX8 && kind != PI_MX4) return ctx_fail(c, PI_ERR_ARG, "kind %d is not PI_MX8 or PI_MX4", kind);
    pi_norm_residual_desc d = *desc;
    d.ldh = 0; // (bytes, not elements)
    if (pi_status st = check(c, &d, d)) return st;
    if (d.pre == PI_NORM_NONE) return ctx_fail(c, PI_ERR_ARG, "h goes with a pre norm");
    const int64_t row = mx_row_bytes(kind, d.d), ldh = desc->ldh ? desc->ldh : row;
    if (ldh < row) return ctx_fail(c, PI_ERR_SHAPE, "h: row stride %lld below the row's %lld bytes", (long long)ldh, (long long)row);
    if (ldh % 32) return ctx_fail(c, PI_ERR_ARG, "h: row stride %lld is not a multiple of 32 bytes", (long long)ldh);
    if (d.T == 0) return PI_OK;
    if (!h || !h->codes || !h->scales) return ctx_fail(c, PI_ERR_ARG, "h: codes or scales are NULL");
    if ((uintptr_t)h->codes % 32 || (uintptr_t)h->scales % 16)
        return ctx_fail(c, PI_ERR_ARG, "h: codes have to start at a multiple of 32 bytes, scales at one of 16");
    NormP p = params(d, q);
    p.h = static_cast<uint16_t *>(h->codes), p.ldh = ldh;
    p.mx = kind, p.mx_tiles = mx_tiles(d.d), p.mx_scales = static_cast<uint8_t *>(h->scales);
    p.vec |= NV_H;
    return forward(c, d, p, x, y, gate, x_out);
}

pi_status pi_norm_residual_bwd_workspace(pi_ctx *c, const pi_norm_residual_desc *desc, size_t *bytes)
{
    if (!c) return PI_ERR_ARG;
    if (!bytes) return ctx_fail(c, PI_ERR_ARG, "bytes is NULL");
    pi_norm_residual_desc d;
    if (pi_status st = check(c, desc, d)) return st;
    const int sms = ctx_view(c).sms;
    const Units a = plan_units(d, true, sms), b = plan_units(d, false, sms);
    *bytes = d.T ? a.stats + std::max(a.part, b.part) : 0;
    return PI_OK;
}

pi_status pi_norm_residual_bwd(pi_ctx *c, const pi_norm_residual_desc *desc, const pi_norm_residual_params *q,
                               const void *dx_out, const void *dh, const void *x_out, const void *y, const void *gate,
                               const pi_norm_residual_grads *gr, int32_t accumulate, void *ws, size_t ws_bytes)
{
    if (!c) return PI_ERR_ARG;
    pi_norm_residual_desc d;
    if (pi_status st = check(c, desc, d)) return st;
    if (!gr) return ctx_fail(c, PI_ERR_ARG, "grads is NULL");
    const bool want = gr->dgate || gr->dw_pre || gr->db_pre || gr->dw_post || gr->db_post;
    const CtxView v = ctx_view(c);
    if (d.pre == PI_NORM_NONE && (gr->dw_pre || gr->db_pre)) return ctx_fail(c, PI_ERR_ARG, "gradients of a pre norm that is not there");
    if (d.post == PI_NORM_NONE && (gr->dw_post || gr->db_post)) return ctx_fail(c, PI_ERR_ARG, "gradients of a post norm that is not there");
    if (d.T == 0) {
        if (accumulate) return PI_OK;
        DeviceGuard g(v.device);
        void *const ps[] = {gr->dw_pre, gr->db_pre, gr->dw_post, gr->db_post};
        for (void *p : ps)
            if (p) CUN(cudaMemsetAsync(p, 0, (size_t)d.d * (d.grad_dtype == PI_F32 ? 4 : 2), v.stream));
        // (no token: the gate has no rows, or one that no token uses)
        if (gr->dgate && !d.gate_rows) CUN(cudaMemsetAsync(gr->dgate, 0, (size_t)d.d * (d.grad_dtype == PI_F32 ? 4 : 2), v.stream));
        return PI_OK;
    }
    if (d.pre != PI_NORM_NONE && !dh) return ctx_fail(c, PI_ERR_ARG, "dh is NULL, but there is a pre norm");
    if (d.pre != PI_NORM_NONE && !x_out) return ctx_fail(c, PI_ERR_ARG, "x_out is NULL");
    if (d.pre == PI_NORM_NONE && dh) return ctx_fail(c, PI_ERR_ARG, "dh given, but there is no pre norm");
    if (!y && (gr->dy || gr->dgate || gr->dw_post || gr->db_post)) return ctx_fail(c, PI_ERR_ARG, "y is NULL but needed");
    if (!gate && gr->dgate) return ctx_fail(c, PI_ERR_ARG, "dgate wanted without a gate");
    NormP p = params(d, q);
    if (pi_status st = check_elements(c, p.x32 ? 4 : 2, {dx_out, x_out, gr->dx})) return st;
    if (pi_status st = check_elements(c, 2, {dh, y, gate, gr->dy, p.w_pre, p.b_pre, p.w_post, p.b_post})) return st;
    if (pi_status st = check_elements(c, d.grad_dtype == PI_F32 ? 4 : 2, {gr->dgate, gr->dw_pre, gr->db_pre, gr->dw_post, gr->db_post}))
        return st;
    p.x = x_out, p.y = (const uint16_t *)y, p.gate = y ? (const uint16_t *)gate : nullptr;
    p.dxo = dx_out, p.dh = (const uint16_t *)dh, p.dx = gr->dx, p.dy = (uint16_t *)gr->dy;
    p.dgate = gr->dgate, p.dw_pre = gr->dw_pre, p.db_pre = gr->db_pre, p.dw_post = gr->dw_post, p.db_post = gr->db_post;
    p.g32 = d.grad_dtype == PI_F32, p.acc = accumulate != 0;
    const Units u = plan_units(d, p.gate != nullptr, v.sms);
    p.units = u.units, p.per_group = u.per_group, p.unit = u.unit, p.per_token = u.per_token;
    if (!p.gate) p.gate_rows = d.T;
    if (want) {
        const size_t need = u.stats + u.part;
        if (!ws || ws_bytes < need)
            return ctx_fail(c, PI_ERR_ARG, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
        if ((uintptr_t)ws & 15) return ctx_fail(c, PI_ERR_ARG, "workspace not 16-byte aligned");
        p.stats = (float *)ws;
        p.part = (float *)((uint8_t *)ws + u.stats);
    }
    p.lddx = d.ldx, p.ldx = d.ldxo, p.ldxo = d.lddxo;
    if (p.pre == PI_NORM_NONE) p.x = nullptr; // (not needed)
    const int xe = p.x32 ? 4 : 2;
    p.vec |= vb(x_out, p.ldx, xe, NV_X) | vb(y, p.ldy, 2, NV_Y) | vb(dh, p.ldh, 2, NV_H) | vb(gate, p.ldgate, 2, NV_GATE) |
             vb(gr->dx, p.lddx, xe, NV_DX) | vb(gr->dy, p.ldy, 2, NV_DY) | vb(dx_out, p.ldxo, xe, NV_DXO) |
             vb(gr->dgate, d.d, p.g32 ? 4 : 2, NV_DGATE);
    DeviceGuard g(v.device);
    CUN(d.dtype == PI_BF16 ? bwd<__nv_bfloat16>(p, want, v) : bwd<__half>(p, want, v));
    return PI_OK;
}

} // extern "C"
