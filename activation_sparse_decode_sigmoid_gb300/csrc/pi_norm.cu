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
// All of it is bound by HBM: a few operations per 16-bit or fp32 element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pi.h"
#include "pi_block.h"
#include "pi_epi.cuh"
#include "pi_kernels.h"

namespace pi {
namespace {

constexpr int kMaxT = 1 << 22, kMaxNormD = 16384;
constexpr int kUnitRows = 64; // tokens whose column sums one unit adds up

struct NormP {
    int Tn, d, pre, post, x32;
    int gate_rows; // tokens per gate row (>= 1)
    float rs, bs, eps;
    const void *x;              // forward: x; backward: x'
    const uint16_t *y, *gate;   // or NULL
    const uint16_t *w_pre, *b_pre, *w_post, *b_post;
    void *xo;                   // forward: x' (or NULL)
    uint16_t *h;                // or NULL
    int64_t ldx, ldxo, ldy, ldh, ldgate, lddx; // (ldx: of `x`)
    unsigned vec;               // 16-byte accesses: 1 x, 2 xo, 4 y, 8 h, 16 gate, 32.. parameters, 64 dx, 128 dy, 256 dxo
    // backward
    const void *dxo;
    const uint16_t *dh;
    void *dx;
    uint16_t *dy;
    float *stats;               // [T][8]: mean_x, r_x, c1, c2, mean_y, r_y
    float *part;                // [units][4][d]: P1, P0, S1, S0
    int units, per_group;       // units in all, and per gate row
    int per_token;              // a gate row per token: S1, S0 carry the gate, dgate is written by the row kernel
    void *dgate, *dw_pre, *db_pre, *dw_post, *db_post;
    int g32, acc;
};

enum : unsigned { NV_X = 1, NV_XO = 2, NV_Y = 4, NV_H = 8, NV_GATE = 16, NV_PAR = 32, NV_DX = 64, NV_DY = 128, NV_DXO = 256 };

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
// buf: 64 floats of shared memory, a different half on alternating calls.
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
// of 8 per thread (two passes over the registers for a layer norm)
template <int V>
__device__ __forceinline__ void row_stats(int kind, const float (&v)[V][8], int d, float eps, float *buf, int &flip,
                                          float &mean, float &r)
{
    mean = 0.f;
    if (kind == PI_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
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

// Forward: one CTA per token, the row in registers.
template <typename T, int V> __global__ void __launch_bounds__(1024) norm_fwd(const __grid_constant__ NormP p)
{
    __shared__ float buf[128];
    int flip = 0;
    pdl_enter();
    const int64_t t = blockIdx.x;
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
    // (chunks past the row hold zeros; a layer norm's statistics skip them)
    row_stats<V>(p.pre, x, p.d, p.eps, buf, flip, mean, r);
    apply_norm<T, V>(p, x, p.w_pre, p.b_pre, mean, r);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8, n = p.d - c;
        if (n > 0) store8<T>(p.h + t * p.ldh + c, n, p.vec & NV_H, x[i]);
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
                    loadx8<T>(p.dgate, p.g32, at, n, false, old);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] += old[j];
                }
                storex8<T>(p.dgate, p.g32, at, n, false, o);
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
__device__ __forceinline__ void unit_rows(const NormP &p, int u, int &t0, int &t1)
{
    const int g = u / p.per_group, k = u % p.per_group;
    const int end = p.per_token ? p.Tn : (int)min((int64_t)p.Tn, (int64_t)(g + 1) * p.gate_rows);
    t0 = (p.per_token ? 0 : g * p.gate_rows) + k * kUnitRows;
    t1 = min(end, t0 + kUnitRows);
}

// Backward, columns: one CTA adds up one unit's tokens over 1024 columns.
template <typename T> __global__ void __launch_bounds__(128) norm_bwd_cols(const __grid_constant__ NormP p)
{
    pdl_enter();
    const int ncb = (p.d + 1023) / 1024;
    const int u = blockIdx.x / ncb, c = (blockIdx.x % ncb) * 1024 + threadIdx.x * 8;
    if (c >= p.d) return;
    int t0, t1;
    unit_rows(p, u, t0, t1);
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

// Backward, the units' partials in order: parameter gradients and dgate.
template <typename T> __global__ void norm_bwd_sum(const __grid_constant__ NormP p)
{
    pdl_enter();
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= p.d) return;
    const float w = p.w_post ? C16<T>::one(p.w_post[c]) : 1.f, b = p.b_post ? C16<T>::one(p.b_post[c]) : 0.f;
    float p1 = 0.f, p0 = 0.f, dw = 0.f, db = 0.f;
    for (int g = 0; g * p.per_group < p.units; ++g) {
        float s1 = 0.f, s0 = 0.f;
        for (int k = 0; k < p.per_group && g * p.per_group + k < p.units; ++k) {
            const float *o = p.part + (int64_t)(g * p.per_group + k) * 4 * p.d + c;
            p1 += o[0];
            p0 += o[p.d];
            s1 += o[2 * (int64_t)p.d];
            s0 += o[3 * (int64_t)p.d];
        }
        const float gate = p.gate && !p.per_token ? C16<T>::one(p.gate[g * p.ldgate + c]) : 1.f;
        dw = fmaf(p.bs * gate, s1, dw);
        db = fmaf(p.bs * gate, s0, db);
        if (p.dgate && !p.per_token) put<T>(p, p.dgate, (int64_t)g * p.d + c, p.bs * fmaf(w, s1, b * s0));
    }
    put<T>(p, p.dw_pre, c, p1);
    put<T>(p, p.db_pre, c, p0);
    put<T>(p, p.dw_post, c, dw);
    put<T>(p, p.db_post, c, db);
}

template <typename T, int V> cudaError_t launch_fwd(const NormP &p, cudaStream_t s)
{
    const int nt = ((p.d + 8 * V - 1) / (8 * V) + 31) / 32 * 32;
    return launch_pdl(norm_fwd<T, V>, dim3(p.Tn), dim3(nt), 0, s, p);
}

template <typename T> cudaError_t fwd(const NormP &p, cudaStream_t s)
{
    return p.d <= 8192 ? launch_fwd<T, 1>(p, s) : launch_fwd<T, 2>(p, s);
}

template <typename T> cudaError_t bwd(const NormP &p, bool cols, cudaStream_t s)
{
    const int nt = std::min(512, ((p.d + 7) / 8 + 31) / 32 * 32);
    cudaError_t e = launch_pdl(norm_bwd_rows<T>, dim3(p.Tn), dim3(nt), 0, s, p);
    if (e != cudaSuccess || !cols) return e;
    const int64_t blocks = (int64_t)p.units * ((p.d + 1023) / 1024);
    e = launch_pdl(norm_bwd_cols<T>, dim3((unsigned)blocks), dim3(128), 0, s, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_bwd_sum<T>, dim3((p.d + 63) / 64), dim3(64), 0, s, p);
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
    int units, per_group;
    bool per_token;
    size_t stats, part;
};

Units plan_units(const pi_norm_residual_desc &d, bool gate)
{
    Units u;
    const int gr = gate && d.gate_rows ? d.gate_rows : std::max(1, d.T);
    u.per_token = gate && gr == 1 && d.T > 1;
    u.per_group = ((u.per_token ? d.T : std::min(gr, std::max(1, d.T))) + kUnitRows - 1) / kUnitRows;
    const int64_t groups = u.per_token ? 1 : (d.T + (int64_t)gr - 1) / gr;
    // the last gate row may have fewer tokens, and units without any add zeros
    u.units = (int)(groups * u.per_group);
    u.stats = ((size_t)d.T * 8 * 4 + 255) / 256 * 256;
    u.part = (size_t)u.units * 4 * d.d * 4;
    return u;
}

#define CUN(call)                                                                                          \
    do {                                                                                                   \
        cudaError_t e_ = (call);                                                                           \
        if (e_ != cudaSuccess) return ctx_fail(c, PI_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_));   \
    } while (0)

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
    if (!x) return ctx_fail(c, PI_ERR_ARG, "x is NULL");
    if (y && !x_out) return ctx_fail(c, PI_ERR_ARG, "x_out is NULL");
    if ((h != nullptr) != (d.pre != PI_NORM_NONE)) return ctx_fail(c, PI_ERR_ARG, "h goes with a pre norm, and only with it");
    if (!h && !x_out) return PI_OK;
    const CtxView v = ctx_view(c);
    NormP p = params(d, q);
    p.x = x, p.y = (const uint16_t *)y, p.gate = y ? (const uint16_t *)gate : nullptr, p.xo = x_out, p.h = (uint16_t *)h;
    const int xe = p.x32 ? 4 : 2;
    p.vec |= vb(x, p.ldx, xe, NV_X) | vb(x_out, p.ldxo, xe, NV_XO) | vb(y, p.ldy, 2, NV_Y) | vb(h, p.ldh, 2, NV_H) |
             vb(gate, p.ldgate, 2, NV_GATE);
    DeviceGuard g(v.device);
    CUN(d.dtype == PI_BF16 ? fwd<__nv_bfloat16>(p, v.stream) : fwd<__half>(p, v.stream));
    return PI_OK;
}

pi_status pi_norm_residual_bwd_workspace(pi_ctx *c, const pi_norm_residual_desc *desc, size_t *bytes)
{
    if (!c) return PI_ERR_ARG;
    if (!bytes) return ctx_fail(c, PI_ERR_ARG, "bytes is NULL");
    pi_norm_residual_desc d;
    if (pi_status st = check(c, desc, d)) return st;
    const Units a = plan_units(d, true), b = plan_units(d, false);
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
    p.x = x_out, p.y = (const uint16_t *)y, p.gate = y ? (const uint16_t *)gate : nullptr;
    p.dxo = dx_out, p.dh = (const uint16_t *)dh, p.dx = gr->dx, p.dy = (uint16_t *)gr->dy;
    p.dgate = gr->dgate, p.dw_pre = gr->dw_pre, p.db_pre = gr->db_pre, p.dw_post = gr->dw_post, p.db_post = gr->db_post;
    p.g32 = d.grad_dtype == PI_F32, p.acc = accumulate != 0;
    const Units u = plan_units(d, p.gate != nullptr);
    p.units = u.units, p.per_group = u.per_group, p.per_token = u.per_token;
    if (!p.gate) p.gate_rows = d.T;
    if (want) {
        const size_t need = u.stats + u.part;
        if (!ws || ws_bytes < need)
            return ctx_fail(c, PI_ERR_ARG, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
        if ((uintptr_t)ws & 15) return ctx_fail(c, PI_ERR_ARG, "workspace not 16-byte aligned");
        p.stats = (float *)ws;
        p.part = (float *)((uint8_t *)ws + u.stats);
    }
    p.lddx = d.ldx, p.ldx = d.ldxo;
    const int xe = p.x32 ? 4 : 2;
    p.vec |= vb(x_out, p.ldx, xe, NV_X) | vb(y, p.ldy, 2, NV_Y) | vb(dh, p.ldh, 2, NV_H) | vb(gate, p.ldgate, 2, NV_GATE) |
             vb(gr->dx, p.lddx, xe, NV_DX) | vb(gr->dy, p.ldy, 2, NV_DY) | vb(dx_out, p.ldxo, xe, NV_DXO);
    DeviceGuard g(v.device);
    CUN(d.dtype == PI_BF16 ? bwd<__nv_bfloat16>(p, want, v.stream) : bwd<__half>(p, want, v.stream));
    return PI_OK;
}

} // extern "C"
