// The block operators' C entry points (linear layer, gated FFN, forward and
// backward): argument checks, the plan of their launches and workspaces, and
// the small kernels around the matrix products (activation gradients, column
// sums, copies of operands whose rows are not 16-byte aligned).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "pi.h"
#include "pi_block.h"
#include "pi_epi.cuh"
#include "pi_kernels.h"

namespace pi {
namespace {

constexpr int kMaxT = 1 << 22, kMaxDim = 1 << 20;

// ------------------------------------------------------------------ kernels
// Rows of 16-bit elements that may start on odd ones, by 32-bit words: a lane
// reads one aligned word of the row, takes the next one's low half from its
// neighbour where the row starts in the middle of a word, and writes one word
// of the (aligned) copy.  Only words that lie inside the row are read whole.
// R rows of 8 x 31 words a CTA: 16 of a large matrix (loads in flight), 4 of a small one (CTAs).
template <int R>
__device__ __forceinline__ void pack_rows(unsigned block, const uint16_t *src, int64_t lds, uint32_t *dst, int64_t ldd, int rows, int cols)
{
    const int nw = (cols + 1) / 2, ncb = (nw + 247) / 248; // (31 words a warp: lane 31 only lends its word)
    const int lane = threadIdx.x & 31, w = (int)(block % ncb) * 248 + (threadIdx.x >> 5) * 31 + lane;
    const int64_t r0 = (int64_t)(block / ncb) * R;
    uint32_t q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        q[i] = 0;
        if (r0 + i >= rows) continue;
        const uint16_t *row = src + (r0 + i) * lds;
        const int c = 2 * w - (((uintptr_t)row & 2) ? 1 : 0); // the word's first column
        if (c >= 0 && c + 1 < cols) q[i] = *reinterpret_cast<const uint32_t *>(row + c);
        else {
            if (c >= 0 && c < cols) q[i] = row[c];
            if (c + 1 >= 0 && c + 1 < cols) q[i] |= (uint32_t)row[c + 1] << 16;
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint32_t next = __shfl_down_sync(0xffffffffu, q[i], 1);
        const bool odd = ((uintptr_t)(src + (r0 + i) * lds) & 2) != 0;
        if (lane < 31 && w < nw && r0 + i < rows) dst[(r0 + i) * (ldd / 2) + w] = odd ? (q[i] >> 16) | (next << 16) : q[i];
    }
}

// The same for rows that are 8-byte aligned (strides of 4 elements): 8 bytes a thread.
template <int R>
__device__ __forceinline__ void pack_rows8(unsigned block, const uint16_t *src, int64_t lds, uint2 *dst, int64_t ldd, int rows, int cols)
{
    const int nq = cols / 4, ncb = (nq + 256) / 256; // (the last, partial 8 bytes included)
    const int w = (int)(block % ncb) * 256 + threadIdx.x;
    const int64_t r0 = (int64_t)(block / ncb) * R;
    if (w > nq) return;
    uint2 q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (r0 + i >= rows) continue;
        const uint16_t *row = src + (r0 + i) * lds;
        if (w < nq) q[i] = *reinterpret_cast<const uint2 *>(row + 4 * w);
        else {
            uint32_t v[2] = {};
            for (int j = 0; j < (cols & 3); ++j) v[j >> 1] |= (uint32_t)row[4 * w + j] << (16 * (j & 1));
            q[i] = make_uint2(v[0], v[1]);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (r0 + i < rows && (w < nq || (cols & 3))) dst[(r0 + i) * (ldd / 4) + w] = q[i];
}

// All copies of a call in one launch: of small operands, each costs more as a launch than as a copy.
constexpr int kMaxCopies = 6;
struct CopySet {
    struct One {
        const uint16_t *src;
        void *dst;
        int64_t lds, ldd;
        int rows, cols;
        unsigned block0; // its first block
        bool large, by8;
    } m[kMaxCopies];
    int n;
};

__global__ void __launch_bounds__(256) pack_set(const __grid_constant__ CopySet s)
{
    pdl_enter();
    int i = 0;
    while (i + 1 < s.n && blockIdx.x >= s.m[i + 1].block0) ++i;
    const CopySet::One &m = s.m[i];
    const unsigned block = blockIdx.x - m.block0;
    if (m.by8) {
        if (m.large) pack_rows8<16>(block, m.src, m.lds, static_cast<uint2 *>(m.dst), m.ldd, m.rows, m.cols);
        else pack_rows8<4>(block, m.src, m.lds, static_cast<uint2 *>(m.dst), m.ldd, m.rows, m.cols);
    } else {
        if (m.large) pack_rows<16>(block, m.src, m.lds, static_cast<uint32_t *>(m.dst), m.ldd, m.rows, m.cols);
        else pack_rows<4>(block, m.src, m.lds, static_cast<uint32_t *>(m.dst), m.ldd, m.rows, m.cols);
    }
}

// Column sums in two launches: a CTA sums some rows of 256 columns (8 per
// thread, 8 row lanes), then the row blocks' partials are added in order.
// Rows per CTA: enough CTAs for four on every SM, at least 8 rows; a
// 4096 x 1024 dz took 52 us with 256 rows each (64 CTAs).
int sum_rows(int T, int N, int sms)
{
    const int64_t ncb = (N + 255) / 256, want = (T * ncb + 4 * sms - 1) / (4 * sms);
    return (int)std::min<int64_t>(256, std::max<int64_t>(8, (want + 7) / 8 * 8));
}

// dz = scale * dy * fn'(z), rounded into dz unless that is NULL, and the
// column sums of the unrounded values over the CTA's rows into part [row
// block][N] unless that is NULL.
template <typename T>
__device__ __forceinline__ void dact_block(unsigned block, const void *dy, int dy32, int64_t ldy, const uint16_t *z, int64_t ldz,
                                           int fn, float scale, uint16_t *dz, int64_t lddz, int Trows, int N, float *part, int vec,
                                           int rpb)
{
    __shared__ float red[8][256];
    const int nb = (N + 255) / 256;
    const int rb = (int)(block / nb), cb = (int)(block % nb);
    const int lane = threadIdx.x & 31, wr = threadIdx.x >> 5;
    const int c = cb * 256 + lane * 8, n = N - c;
    const int r1 = (int)min((int64_t)Trows, (rb + 1) * (int64_t)rpb);
    float sum[8] = {};
    if (n > 0) {
        for (int r = rb * rpb + wr; r < r1; r += 8) {
            float v[8];
            if (dy32) load8f(static_cast<const float *>(dy) + (int64_t)r * ldy + c, n, vec & 1, v);
            else load8<T>(static_cast<const uint16_t *>(dy) + (int64_t)r * ldy + c, n, vec & 1, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= scale;
            if (fn != PI_FN_NONE) {
                float zz[8], f[8], df[8];
                load8<T>(z + (int64_t)r * ldz + c, n, vec & 2, zz);
                both8(fn, zz, f, df);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= df[i];
            }
            if (dz) store8<T>(dz + (int64_t)r * lddz + c, n, vec & 4, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += v[i];
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) red[wr][lane * 8 + i] = sum[i];
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += red[w][threadIdx.x];
    const int cc = cb * 256 + threadIdx.x;
    if (cc < N) part[(int64_t)rb * N + cc] = s;
}

template <typename T>
__global__ void __launch_bounds__(256) dact_rows(const void *dy, int dy32, int64_t ldy, const uint16_t *z, int64_t ldz,
                                                 int fn, float scale, uint16_t *dz, int64_t lddz, int Trows, int N,
                                                 float *part, int vec, int rpb)
{
    pdl_enter();
    dact_block<T>(blockIdx.x, dy, dy32, ldy, z, ldz, fn, scale, dz, lddz, Trows, N, part, vec, rpb);
}

// 32 columns a CTA, 32 lanes that share the parts (8: 1 us more for 128 parts).
constexpr int kSumLanes = 32;
template <typename T>
__device__ __forceinline__ void sum_block(unsigned block, const float *part, int nparts, int N, void *out, int out32, int accumulate)
{
    __shared__ float red[kSumLanes][32];
    const int l = threadIdx.x & 31, k = threadIdx.x >> 5, c = block * 32 + l;
    float s = 0.f;
    if (c < N) {
#pragma unroll 4
        for (int i = k; i < nparts; i += kSumLanes) s += part[(int64_t)i * N + c];
    }
    red[k][l] = s;
    __syncthreads();
    if (k || c >= N) return;
#pragma unroll
    for (int j = 1; j < kSumLanes; ++j) s += red[j][l];
    if (out32) {
        float *o = static_cast<float *>(out);
        o[c] = accumulate ? o[c] + s : s;
    } else {
        uint16_t *o = static_cast<uint16_t *>(out);
        o[c] = C16<T>::round(accumulate ? C16<T>::one(o[c]) + s : s);
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kSumLanes) sum_parts(const float *part, int nparts, int N, void *out, int out32, int accumulate)
{
    pdl_enter();
    sum_block<T>(blockIdx.x, part, nparts, N, out, out32, accumulate);
}

// The column sums of up to three 16-bit matrices of T rows in two launches.
struct SumSet {
    struct One {
        const uint16_t *src;
        void *out;
        float *part;
        int64_t ld;
        int N, rpb, nparts, vec;
        unsigned block0, join0; // its first block of either launch
    } m[3];
    int n, T, out32, accumulate, sms;
};

template <typename T> __global__ void __launch_bounds__(256) col_sums(const __grid_constant__ SumSet s)
{
    pdl_enter();
    int i = 0;
    while (i + 1 < s.n && blockIdx.x >= s.m[i + 1].block0) ++i;
    const SumSet::One &m = s.m[i];
    dact_block<T>(blockIdx.x - m.block0, m.src, 0, m.ld, nullptr, 0, PI_FN_NONE, 1.f, nullptr, 0, s.T, m.N, m.part, m.vec, m.rpb);
}

template <typename T> __global__ void __launch_bounds__(32 * kSumLanes) join_sums(const __grid_constant__ SumSet s)
{
    pdl_enter();
    int i = 0;
    while (i + 1 < s.n && blockIdx.x >= s.m[i + 1].join0) ++i;
    const SumSet::One &m = s.m[i];
    sum_block<T>(blockIdx.x - m.join0, m.part, m.nparts, m.N, m.out, s.out32, s.accumulate);
}

bool aligned16(const void *p, int64_t ld, int elem) { return ((uintptr_t)p & 15) == 0 && (ld * elem) % 16 == 0; }

template <typename T>
cudaError_t dact_t(const void *dy, int dy32, int64_t ldy, const void *z, int64_t ldz, int fn, float scale, void *dz,
                   int64_t lddz, int Trows, int N, void *db, int db32, int accumulate, float *part, const CtxView &v)
{
    const cudaStream_t s = v.stream;
    const int rpb = sum_rows(Trows, N, v.sms), nrb = (Trows + rpb - 1) / rpb;
    const int64_t blocks = (int64_t)nrb * ((N + 255) / 256);
    const int vec = (aligned16(dy, ldy, dy32 ? 4 : 2) ? 1 : 0) | (z && aligned16(z, ldz, 2) ? 2 : 0) |
                    (dz && aligned16(dz, lddz, 2) ? 4 : 0);
    float *pt = db ? part : nullptr;
    cudaError_t e = cudaSuccess;
    if (blocks > 0) {
        e = launch_pdl(dact_rows<T>, dim3((unsigned)blocks), dim3(256), 0, s, dy, dy32, ldy, (const uint16_t *)z, ldz, fn,
                       scale, (uint16_t *)dz, lddz, Trows, N, pt, vec, rpb);
    }
    if (e != cudaSuccess || !db) return e;
    return launch_pdl(sum_parts<T>, dim3((N + 31) / 32), dim3(32 * kSumLanes), 0, s, (const float *)part, nrb, N, db, db32,
                      accumulate);
}

// ------------------------------------------------------------------ workspace
// Walks a workspace: the same code counts the bytes (base NULL) and hands out
// the pieces.
struct Arena {
    uint8_t *base;
    size_t used = 0;
    explicit Arena(void *p) : base(static_cast<uint8_t *>(p)) {}
    void *take(size_t bytes)
    {
        const size_t at = used;
        used += (bytes + 255) / 256 * 256;
        return base ? base + at : nullptr;
    }
};

int64_t pitch8(int n) { return ((int64_t)n + 63) / 64 * 64; } // elements of a workspace row

bool is16(int dt) { return dt == PI_F16 || dt == PI_BF16; }
bool fn_ok(int fn) { return fn >= PI_FN_NONE && fn <= PI_FN_GELU_TANH; }

// A stride of 0 stands for packed rows.
int64_t or_packed(int64_t ld, int cols) { return ld ? ld : cols; }

pi_status bad_ld(pi_ctx *c, const char *what, int64_t ld, int cols)
{
    return ctx_fail(c, PI_ERR_SHAPE, "%s: row stride %lld below the row's %d elements", what, (long long)ld, cols);
}

// One operand of a product as the kernels need it: in place when base and
// stride allow 16-byte accesses, else a copy in the workspace.
struct Staged {
    Mat m;
    bool copy = false;
    const void *src = nullptr;
    int64_t lds = 0;
    int rows = 0, cols = 0;
};

Staged stage(Arena &ws, const void *p, int64_t ld, int rows, int cols, int mn)
{
    Staged s;
    s.m = {p, ld, mn};
    // (a single row has no stride)
    if (((uintptr_t)p & 15) || (rows > 1 && ld % 8)) {
        s.copy = true;
        s.src = p, s.lds = ld, s.rows = rows, s.cols = cols;
        s.m.ld = pitch8(cols);
        s.m.p = ws.take((size_t)rows * s.m.ld * 2);
    } else if (rows == 1)
        s.m.ld = pitch8(cols);
    return s;
}

// The copies of the operands that need one.
cudaError_t run_copies(std::initializer_list<const Staged *> list, cudaStream_t st)
{
    CopySet c = {};
    uint64_t blocks = 0;
    for (const Staged *s : list) {
        if (!s->copy) continue;
        CopySet::One &m = c.m[c.n++];
        m = {(const uint16_t *)s->src, const_cast<void *>(s->m.p), s->lds, s->m.ld, s->rows, s->cols, (unsigned)blocks,
             (int64_t)s->rows * s->cols > (4 << 20), ((uintptr_t)s->src & 7) == 0 && s->lds % 4 == 0};
        const int64_t r = m.large ? 16 : 4;
        blocks += (uint64_t)((m.rows + r - 1) / r) * (m.by8 ? (m.cols / 4 + 256) / 256 : ((m.cols + 1) / 2 + 247) / 248);
    }
    if (!c.n) return cudaSuccess;
    return launch_pdl(pack_set, dim3((unsigned)blocks), dim3(256), 0, st, c);
}

unsigned vbit(const void *p, int64_t ld, int elem, unsigned bit) { return p && aligned16(p, ld, elem) ? bit : 0; }

void set_vec(Epi &e)
{
    const int oe = e.out32 ? 4 : 2;
    e.vec = vbit(e.res, e.ldr, oe, V_RES) | vbit(e.out, e.ldo, oe, V_OUT) | vbit(e.out2, e.ld2, 2, V_OUT2) |
            vbit(e.out3, e.ld3, 2, V_OUT3) | vbit(e.in1, e.ldi1, 2, V_IN1) | vbit(e.in2, e.ldi2, 2, V_IN2) |
            vbit(e.bias, 0, 2, V_BIAS) | vbit(e.bias2, 0, 2, V_BIAS2);
}

#define CUB(call)                                                                                              \
    do {                                                                                                       \
        cudaError_t e_ = (call);                                                                               \
        if (e_ != cudaSuccess)                                                                                 \
            return ctx_fail(c, e_ == cudaErrorMemoryAllocation ? PI_ERR_OOM : PI_ERR_CUDA, "%s: %s", #call,    \
                            cudaGetErrorString(e_));                                                           \
    } while (0)

pi_status check_ws(pi_ctx *c, const void *ws, size_t have, size_t need)
{
    if (need && (!ws || have < need))
        return ctx_fail(c, PI_ERR_ARG, "workspace of %zu bytes needed, %zu given", need, ws ? have : (size_t)0);
    if (((uintptr_t)ws & 15) != 0) return ctx_fail(c, PI_ERR_ARG, "workspace not 16-byte aligned");
    return PI_OK;
}

// Launches follow one another on one stream, so their workspaces share one
// region.
struct Plan {
    Gemm g[5];
    int n = 0;
    size_t bytes = 0;
    Gemm &add()
    {
        g[n] = Gemm{};
        g[n].segs = 1;
        g[n].e.scale = 1.f;
        return g[n++];
    }
    // products [0, first) run alone, the rest in one launch
    void size(const CtxView &v, int first)
    {
        for (int i = 0; i < first; ++i) bytes = std::max(bytes, gemm_workspace(g[i], v));
        if (n > first) bytes = std::max(bytes, gemms_workspace(g + first, n - first, v));
    }
};

// ------------------------------------------------------------------ linear
pi_status check_linear(pi_ctx *c, const pi_linear_desc *d, pi_linear_desc &o)
{
    if (!d) return ctx_fail(c, PI_ERR_ARG, "desc is NULL");
    o = *d;
    if (!is16(o.dtype)) return ctx_fail(c, PI_ERR_ARG, "dtype %d is not PI_F16 or PI_BF16", o.dtype);
    if (o.out_dtype != o.dtype && o.out_dtype != PI_F32)
        return ctx_fail(c, PI_ERR_ARG, "out_dtype %d is neither dtype nor PI_F32", o.out_dtype);
    if (o.grad_dtype != o.dtype && o.grad_dtype != PI_F32)
        return ctx_fail(c, PI_ERR_ARG, "grad_dtype %d is neither dtype nor PI_F32", o.grad_dtype);
    if (!fn_ok(o.fn)) return ctx_fail(c, PI_ERR_ARG, "fn %d invalid", o.fn);
    if (!std::isfinite(o.scale)) return ctx_fail(c, PI_ERR_ARG, "scale is not finite");
    if (o.T < 0 || o.T > kMaxT) return ctx_fail(c, PI_ERR_SHAPE, "T %d outside [0, %d]", o.T, kMaxT);
    if (o.K < 1 || o.K > kMaxDim) return ctx_fail(c, PI_ERR_SHAPE, "K %d outside [1, %d]", o.K, kMaxDim);
    if (o.N < 1 || o.N > kMaxDim) return ctx_fail(c, PI_ERR_SHAPE, "N %d outside [1, %d]", o.N, kMaxDim);
    struct {
        int64_t *ld;
        int cols;
        const char *name;
    } lds[] = {{&o.ldx, o.K, "x"}, {&o.ldw, o.K, "w"}, {&o.ldz, o.N, "z"},   {&o.ldr, o.N, "residual"},
               {&o.ldy, o.N, "y"}, {&o.lddx, o.K, "dx"}, {&o.lddw, o.K, "dw"}};
    for (auto &l : lds) {
        *l.ld = or_packed(*l.ld, l.cols);
        if (*l.ld < l.cols) return bad_ld(c, l.name, *l.ld, l.cols);
    }
    return PI_OK;
}

struct LinearFwd {
    Staged x, w;
    Plan p;
    void *gws;
    size_t bytes;
};

LinearFwd plan_linear(const pi_linear_desc &d, const CtxView &v, const void *x, const void *w, const void *b,
                      const void *r, void *z, void *y, void *ws)
{
    LinearFwd f;
    Arena a(ws);
    f.x = stage(a, x, d.ldx, d.T, d.K, 0);
    f.w = stage(a, w, d.ldw, d.N, d.K, 0);
    Gemm &g = f.p.add();
    g.mode = EPI_LINEAR;
    g.M = d.T, g.N = d.N, g.K[0] = d.K;
    g.a[0] = f.x.m, g.b[0] = f.w.m;
    Epi &e = g.e;
    e.fn = d.fn, e.scale = d.scale, e.out32 = d.out_dtype == PI_F32;
    e.bias = (const uint16_t *)b, e.res = r, e.ldr = d.ldr, e.out = y, e.ldo = d.ldy;
    e.out2 = (uint16_t *)z, e.ld2 = d.ldz;
    set_vec(e);
    f.p.size(v, f.p.n);
    f.gws = a.take(f.p.bytes);
    f.bytes = a.used;
    return f;
}

struct LinearBwd {
    Staged x, w, dz;
    bool direct; // dz is dy itself
    void *dzbuf;
    int64_t lddz;
    void *part;
    Plan p;
    void *gws;
    size_t bytes;
};

LinearBwd plan_linear_bwd(const pi_linear_desc &d, const CtxView &v, const void *dy, const void *x, const void *w,
                          const void *dx, void *dw, const void *db, int acc, void *ws)
{
    LinearBwd f;
    Arena a(ws);
    // dz = dy when nothing changes it, else a 16-bit copy
    f.direct = d.fn == PI_FN_NONE && d.scale == 1.f && d.out_dtype != PI_F32;
    f.dzbuf = nullptr, f.lddz = 0;
    if (f.direct) f.dz = stage(a, dy, d.ldy, d.T, d.N, 0);
    else {
        f.lddz = pitch8(d.N);
        f.dzbuf = dx || dw ? a.take((size_t)d.T * f.lddz * 2) : nullptr;
        f.dz.m = {f.dzbuf, f.lddz, 0};
    }
    if (dw) f.x = stage(a, x, d.ldx, d.T, d.K, 1);
    if (dx) f.w = stage(a, w, d.ldw, d.N, d.K, 1);
    f.part = db ? a.take(colsum_bytes(d.T, d.N, v.sms)) : nullptr;
    if (dx) {
        Gemm &g = f.p.add();
        g.mode = EPI_LINEAR;
        g.M = d.T, g.N = d.K, g.K[0] = d.N;
        g.a[0] = f.dz.m, g.b[0] = f.w.m;
        g.e.out = const_cast<void *>(dx), g.e.ldo = d.lddx;
        set_vec(g.e);
    }
    if (dw) {
        Gemm &g = f.p.add();
        g.mode = EPI_LINEAR;
        g.M = d.N, g.N = d.K, g.K[0] = d.T;
        g.a[0] = f.dz.m, g.a[0].mn = 1, g.b[0] = f.x.m;
        g.e.out32 = d.grad_dtype == PI_F32;
        g.e.out = dw, g.e.ldo = d.lddw;
        if (acc) g.e.res = dw, g.e.ldr = d.lddw;
        set_vec(g.e);
    }
    f.p.size(v, 0);
    f.gws = a.take(f.p.bytes);
    f.bytes = a.used;
    return f;
}

// ------------------------------------------------------------------ gated FFN
pi_status check_ffn(pi_ctx *c, const pi_gated_ffn_desc *d, pi_gated_ffn_desc &o)
{
    if (!d) return ctx_fail(c, PI_ERR_ARG, "desc is NULL");
    o = *d;
    if (!is16(o.dtype)) return ctx_fail(c, PI_ERR_ARG, "dtype %d is not PI_F16 or PI_BF16", o.dtype);
    if (o.grad_dtype != o.dtype && o.grad_dtype != PI_F32)
        return ctx_fail(c, PI_ERR_ARG, "grad_dtype %d is neither dtype nor PI_F32", o.grad_dtype);
    if (!fn_ok(o.fn)) return ctx_fail(c, PI_ERR_ARG, "fn %d invalid", o.fn);
    if (o.gated != 0 && o.gated != 1) return ctx_fail(c, PI_ERR_ARG, "gated %d is not 0 or 1", o.gated);
    if (o.T < 0 || o.T > kMaxT) return ctx_fail(c, PI_ERR_SHAPE, "T %d outside [0, %d]", o.T, kMaxT);
    if (o.d < 1 || o.d > kMaxDim) return ctx_fail(c, PI_ERR_SHAPE, "d %d outside [1, %d]", o.d, kMaxDim);
    if (o.n < 1 || o.n > kMaxDim) return ctx_fail(c, PI_ERR_SHAPE, "n %d outside [1, %d]", o.n, kMaxDim);
    struct {
        int64_t *ld;
        int cols;
        const char *name;
    } lds[] = {{&o.ldx, o.d, "x"},        {&o.ldy, o.d, "y"}, {&o.ld_gate, o.d, "w_gate"}, {&o.ld_up, o.d, "w_up"},
               {&o.ld_down, o.n, "w_down"}, {&o.ldg, o.n, "g"}, {&o.ldu, o.n, "u"},          {&o.lda, o.n, "a"}};
    for (auto &l : lds) {
        *l.ld = or_packed(*l.ld, l.cols);
        if (*l.ld < l.cols) return bad_ld(c, l.name, *l.ld, l.cols);
    }
    return PI_OK;
}

pi_status check_ffn_weights(pi_ctx *c, const pi_gated_ffn_desc &d, const pi_gated_ffn_weights *w)
{
    if (!w) return ctx_fail(c, PI_ERR_ARG, "weights are NULL");
    if (!w->w_up || !w->w_down || (d.gated && !w->w_gate)) return ctx_fail(c, PI_ERR_ARG, "a weight matrix is NULL");
    if (!d.gated && (w->w_gate || w->b_gate)) return ctx_fail(c, PI_ERR_ARG, "gate weights given, but gated is 0");
    return PI_OK;
}

struct FfnFwd {
    Staged x, wg, wu, wd, a;
    Plan p;
    void *gws;
    size_t bytes;
};

FfnFwd plan_ffn(const pi_gated_ffn_desc &d, const CtxView &v, const pi_gated_ffn_weights &w, const void *x,
                const pi_gated_ffn_save &s, void *y, void *ws)
{
    FfnFwd f;
    Arena ar(ws);
    f.x = stage(ar, x, d.ldx, d.T, d.d, 0);
    if (d.gated) f.wg = stage(ar, w.w_gate, d.ld_gate, d.n, d.d, 0);
    f.wu = stage(ar, w.w_up, d.ld_up, d.n, d.d, 0);
    f.wd = stage(ar, w.w_down, d.ld_down, d.d, d.n, 0);
    // the activations: the caller's buffer, or the workspace
    void *a = s.a;
    int64_t lda = d.lda;
    if (!a) {
        lda = pitch8(d.n);
        a = ar.take((size_t)d.T * lda * 2);
        f.a.m = {a, lda, 0};
    } else
        f.a = stage(ar, a, lda, d.T, d.n, 0);
    Gemm &g = f.p.add();
    g.mode = d.gated ? EPI_GATED : EPI_LINEAR;
    g.M = d.T, g.N = d.n, g.K[0] = d.d;
    g.a[0] = f.x.m;
    g.e.fn = d.fn, g.e.out = a, g.e.ldo = lda;
    if (d.gated) {
        g.b[0] = f.wg.m, g.b[1] = f.wu.m;
        g.e.bias = (const uint16_t *)w.b_gate, g.e.bias2 = (const uint16_t *)w.b_up;
        g.e.out2 = (uint16_t *)s.g, g.e.ld2 = d.ldg;
        g.e.out3 = (uint16_t *)s.u, g.e.ld3 = d.ldu;
    } else {
        g.b[0] = f.wu.m;
        g.e.bias = (const uint16_t *)w.b_up;
        g.e.out2 = (uint16_t *)s.u, g.e.ld2 = d.ldu;
    }
    set_vec(g.e);
    Gemm &h = f.p.add();
    h.mode = EPI_LINEAR;
    h.M = d.T, h.N = d.d, h.K[0] = d.n;
    h.a[0] = f.a.m, h.b[0] = f.wd.m;
    h.early = 1;
    h.e.bias = (const uint16_t *)w.b_down;
    h.e.out = y, h.e.ldo = d.ldy;
    set_vec(h.e);
    f.p.size(v, f.p.n);
    f.gws = ar.take(f.p.bytes);
    f.bytes = ar.used;
    return f;
}

struct FfnBwd {
    Staged x, wg, wu, wd, dy, a;
    void *dg, *du;
    int64_t ldd;
    void *part;
    Plan p;
    bool da = false; // the first product is da; the others follow it
    void *gws;
    size_t bytes;
};

FfnBwd plan_ffn_bwd(const pi_gated_ffn_desc &d, const CtxView &v, const pi_gated_ffn_weights &w, const void *x,
                    const void *dy, const pi_gated_ffn_save &s, void *dx, const pi_gated_ffn_grads &gr, int acc,
                    void *ws)
{
    FfnBwd f;
    Arena ar(ws);
    const bool want_d = dx || gr.w_up || gr.w_gate || gr.b_up || gr.b_gate; // dg, du needed
    f.ldd = pitch8(d.n);
    f.dy = stage(ar, dy, d.ldy, d.T, d.d, 0);
    f.dg = want_d && d.gated ? ar.take((size_t)d.T * f.ldd * 2) : nullptr;
    f.du = want_d ? ar.take((size_t)d.T * f.ldd * 2) : nullptr;
    if (want_d) f.wd = stage(ar, w.w_down, d.ld_down, d.d, d.n, 1);
    if (dx) {
        if (d.gated) f.wg = stage(ar, w.w_gate, d.ld_gate, d.n, d.d, 1);
        f.wu = stage(ar, w.w_up, d.ld_up, d.n, d.d, 1);
    }
    if (gr.w_up || gr.w_gate) f.x = stage(ar, x, d.ldx, d.T, d.d, 1);
    if (gr.w_down) f.a = stage(ar, s.a, d.lda, d.T, d.n, 1);
    const size_t part = (gr.b_gate ? colsum_bytes(d.T, d.n, v.sms) : 0) + (gr.b_up ? colsum_bytes(d.T, d.n, v.sms) : 0) +
                        (gr.b_down ? colsum_bytes(d.T, d.d, v.sms) : 0);
    f.part = part ? ar.take(part) : nullptr;
    const int g32 = d.grad_dtype == PI_F32;
    if (want_d) {
        f.da = true;
        Gemm &g = f.p.add();
        g.mode = EPI_DACT;
        g.M = d.T, g.N = d.n, g.K[0] = d.d;
        g.a[0] = f.dy.m, g.b[0] = f.wd.m;
        g.e.fn = d.fn;
        if (d.gated) {
            g.e.in1 = (const uint16_t *)s.g, g.e.ldi1 = d.ldg;
            g.e.in2 = (const uint16_t *)s.u, g.e.ldi2 = d.ldu;
            g.e.out = f.dg, g.e.ldo = f.ldd;
            g.e.out2 = (uint16_t *)f.du, g.e.ld2 = f.ldd;
        } else {
            g.e.in1 = (const uint16_t *)s.u, g.e.ldi1 = d.ldu;
            g.e.out = f.du, g.e.ldo = f.ldd;
        }
        set_vec(g.e);
    }
    if (dx) {
        Gemm &g = f.p.add();
        g.mode = EPI_LINEAR;
        g.M = d.T, g.N = d.d;
        int k = 0;
        if (d.gated) g.K[k] = d.n, g.a[k] = {f.dg, f.ldd, 0}, g.b[k] = f.wg.m, ++k;
        g.K[k] = d.n, g.a[k] = {f.du, f.ldd, 0}, g.b[k] = f.wu.m, ++k;
        g.segs = k;
        g.e.out = dx, g.e.ldo = d.ldx;
        set_vec(g.e);
    }
    auto wgrad = [&](Gemm &g, Mat a, int M, int N, Mat b, void *out) {
        g.mode = EPI_LINEAR;
        g.M = M, g.N = N, g.K[0] = d.T;
        a.mn = 1;
        b.mn = 1;
        g.a[0] = a, g.b[0] = b;
        g.e.out32 = g32;
        g.e.out = out, g.e.ldo = N;
        if (acc) g.e.res = out, g.e.ldr = N;
        set_vec(g.e);
    };
    if (gr.w_gate) wgrad(f.p.add(), {f.dg, f.ldd, 1}, d.n, d.d, f.x.m, gr.w_gate);
    if (gr.w_up) wgrad(f.p.add(), {f.du, f.ldd, 1}, d.n, d.d, f.x.m, gr.w_up);
    if (gr.w_down) wgrad(f.p.add(), f.dy.m, d.d, d.n, f.a.m, gr.w_down);
    f.p.size(v, f.da);
    f.gws = ar.take(f.p.bytes);
    f.bytes = ar.used;
    return f;
}

} // namespace

size_t colsum_bytes(int T, int N, int sms)
{
    const int rpb = sum_rows(T, N, sms);
    return (size_t)((T + rpb - 1) / rpb) * N * sizeof(float);
}

cudaError_t launch_dact(const void *dy, int dy32, int64_t ldy, const void *z, int64_t ldz, int fn, float scale,
                        void *dz, int64_t lddz, int T, int N, void *db, int db32, int accumulate, bool bf16,
                        void *part, const CtxView &v)
{
    return bf16 ? dact_t<__nv_bfloat16>(dy, dy32, ldy, z, ldz, fn, scale, dz, lddz, T, N, db, db32, accumulate,
                                        (float *)part, v)
                : dact_t<__half>(dy, dy32, ldy, z, ldz, fn, scale, dz, lddz, T, N, db, db32, accumulate, (float *)part,
                                 v);
}

// One more matrix whose column sums are wanted (out NULL: not wanted).  part: its partials.
void add_sum(SumSet &s, const void *src, int64_t ld, int N, void *out, void *&part)
{
    if (!out) return;
    SumSet::One &m = s.m[s.n];
    const int rpb = sum_rows(s.T, N, s.sms), nparts = (s.T + rpb - 1) / rpb;
    m = {(const uint16_t *)src, out, (float *)part, ld, N, rpb, nparts, aligned16(src, ld, 2) ? 1 : 0, 0, 0};
    if (s.n) {
        const SumSet::One &l = s.m[s.n - 1];
        m.block0 = l.block0 + (unsigned)l.nparts * ((l.N + 255) / 256), m.join0 = l.join0 + (l.N + 31) / 32;
    }
    part = (uint8_t *)part + colsum_bytes(s.T, N, s.sms);
    ++s.n;
}

cudaError_t launch_sums(const SumSet &s, bool bf16, cudaStream_t st)
{
    if (!s.n) return cudaSuccess;
    const SumSet::One &l = s.m[s.n - 1];
    const dim3 blocks(l.block0 + (unsigned)l.nparts * ((l.N + 255) / 256)), joins(l.join0 + (l.N + 31) / 32);
    cudaError_t e = bf16 ? launch_pdl(col_sums<__nv_bfloat16>, blocks, dim3(256), 0, st, s) : launch_pdl(col_sums<__half>, blocks, dim3(256), 0, st, s);
    if (e != cudaSuccess) return e;
    return bf16 ? launch_pdl(join_sums<__nv_bfloat16>, joins, dim3(32 * kSumLanes), 0, st, s) : launch_pdl(join_sums<__half>, joins, dim3(32 * kSumLanes), 0, st, s);
}

} // namespace pi

using namespace pi;

extern "C" {

pi_status pi_linear_workspace(pi_ctx *c, const pi_linear_desc *desc, int32_t backward, size_t *bytes)
{
    if (!c) return PI_ERR_ARG;
    if (!bytes) return ctx_fail(c, PI_ERR_ARG, "bytes is NULL");
    pi_linear_desc d;
    if (pi_status st = check_linear(c, desc, d)) return st;
    // the most that a call with this desc takes: with `unaligned`, every
    // operand is copied
    const CtxView v = ctx_view(c);
    const void *odd = (const void *)(uintptr_t)(d.unaligned ? 2 : 16);
    if (backward) {
        // (fewer outputs may be cut differently)
        *bytes = 0;
        for (int want = 0; d.T && want < 4; ++want) {
            void *dx = want & 1 ? (void *)odd : nullptr, *dw = want & 2 ? (void *)odd : nullptr;
            *bytes = std::max(*bytes, plan_linear_bwd(d, v, odd, odd, odd, dx, dw, odd, 1, nullptr).bytes);
        }
    } else
        *bytes = d.T ? plan_linear(d, v, odd, odd, odd, odd, (void *)odd, (void *)odd, nullptr).bytes : 0;
    return PI_OK;
}

pi_status pi_linear(pi_ctx *c, const pi_linear_desc *desc, const void *x, const void *w, const void *b,
                    const void *residual, void *z, void *y, void *ws, size_t ws_bytes)
{
    if (!c) return PI_ERR_ARG;
    pi_linear_desc d;
    if (pi_status st = check_linear(c, desc, d)) return st;
    if (d.T == 0) return PI_OK;
    if (!x || !w || !y) return ctx_fail(c, PI_ERR_ARG, "x, w or y is NULL");
    if (pi_status st = check_elements(c, 2, {x, w, b, z})) return st;
    if (pi_status st = check_elements(c, d.out_dtype == PI_F32 ? 4 : 2, {residual, y})) return st;
    const CtxView v = ctx_view(c);
    const LinearFwd f = plan_linear(d, v, x, w, b, residual, z, y, ws);
    if (pi_status st = check_ws(c, ws, ws_bytes, f.bytes)) return st;
    DeviceGuard g(v.device);
    CUB(run_copies({&f.x, &f.w}, v.stream));
    CUB(launch_gemm(f.p.g[0], d.dtype == PI_BF16, v, f.gws));
    return PI_OK;
}

pi_status pi_linear_bwd(pi_ctx *c, const pi_linear_desc *desc, const void *dy, const void *x, const void *w,
                        const void *z, void *dx, void *dw, void *db, int32_t accumulate, void *ws, size_t ws_bytes)
{
    if (!c) return PI_ERR_ARG;
    pi_linear_desc d;
    if (pi_status st = check_linear(c, desc, d)) return st;
    const CtxView v = ctx_view(c);
    const bool bf = d.dtype == PI_BF16;
    const int g32 = d.grad_dtype == PI_F32;
    if (d.T == 0) {
        // an empty sum
        if (accumulate) return PI_OK;
        DeviceGuard g(v.device);
        const size_t eb = g32 ? 4 : 2;
        if (dw) CUB(cudaMemset2DAsync(dw, d.lddw * eb, 0, d.K * eb, d.N, v.stream));
        if (db) CUB(cudaMemsetAsync(db, 0, d.N * eb, v.stream));
        return PI_OK;
    }
    if (!dx && !dw && !db) return PI_OK;
    if (!dy || (dw && !x) || (dx && !w) || (d.fn != PI_FN_NONE && !z))
        return ctx_fail(c, PI_ERR_ARG, "dy, x, w or z is NULL but needed");
    if (pi_status st = check_elements(c, 2, {x, w, z, dx})) return st;
    if (pi_status st = check_elements(c, d.out_dtype == PI_F32 ? 4 : 2, {dy})) return st;
    if (pi_status st = check_elements(c, g32 ? 4 : 2, {dw, db})) return st;
    const LinearBwd f = plan_linear_bwd(d, v, dy, x, w, dx, dw, db, accumulate, ws);
    if (pi_status st = check_ws(c, ws, ws_bytes, f.bytes)) return st;
    DeviceGuard g(v.device);
    const int dy32 = d.out_dtype == PI_F32;
    CUB(run_copies({&f.dz, &f.x, &f.w}, v.stream));
    if (!f.direct) {
        CUB(launch_dact(dy, dy32, d.ldy, z, d.ldz, d.fn, d.scale, f.dzbuf, f.lddz, d.T, d.N, db, g32, accumulate, bf,
                        f.part, v));
    } else {
        SumSet sums = {{}, 0, d.T, g32, accumulate, v.sms};
        void *part = f.part;
        add_sum(sums, dy, d.ldy, d.N, db, part);
        CUB(launch_sums(sums, bf, v.stream));
    }
    if (f.p.n) CUB(launch_gemms(f.p.g, f.p.n, bf, v, f.gws));
    return PI_OK;
}

pi_status pi_gated_ffn_workspace(pi_ctx *c, const pi_gated_ffn_desc *desc, int32_t backward, size_t *bytes)
{
    if (!c) return PI_ERR_ARG;
    if (!bytes) return ctx_fail(c, PI_ERR_ARG, "bytes is NULL");
    pi_gated_ffn_desc d;
    if (pi_status st = check_ffn(c, desc, d)) return st;
    const CtxView v = ctx_view(c);
    void *odd = (void *)(uintptr_t)(d.unaligned ? 2 : 16);
    void *gate = d.gated ? odd : nullptr;
    const pi_gated_ffn_weights w = {gate, odd, odd, gate, odd, odd};
    const pi_gated_ffn_save s = {gate, odd, odd}, none = {nullptr, nullptr, nullptr};
    if (d.T == 0) *bytes = 0;
    else if (backward) {
        *bytes = 0;
        for (int want = 0; want < 16; ++want) {
            const pi_gated_ffn_grads gr = {want & 1 ? gate : nullptr, want & 2 ? odd : nullptr, want & 4 ? odd : nullptr, gate, odd, odd};
            *bytes = std::max(*bytes, plan_ffn_bwd(d, v, w, odd, odd, s, want & 8 ? odd : nullptr, gr, 1, nullptr).bytes);
        }
    } else
        *bytes = std::max(plan_ffn(d, v, w, odd, s, odd, nullptr).bytes, plan_ffn(d, v, w, odd, none, odd, nullptr).bytes);
    return PI_OK;
}

pi_status pi_gated_ffn(pi_ctx *c, const pi_gated_ffn_desc *desc, const pi_gated_ffn_weights *w, const void *x,
                       const pi_gated_ffn_save *save, void *y, void *ws, size_t ws_bytes)
{
    if (!c) return PI_ERR_ARG;
    pi_gated_ffn_desc d;
    if (pi_status st = check_ffn(c, desc, d)) return st;
    if (pi_status st = check_ffn_weights(c, d, w)) return st;
    pi_gated_ffn_save s = {nullptr, nullptr, nullptr};
    if (save) s = *save;
    if (!d.gated && s.g) return ctx_fail(c, PI_ERR_ARG, "save->g given, but gated is 0");
    if (d.T == 0) return PI_OK;
    if (!x || !y) return ctx_fail(c, PI_ERR_ARG, "x or y is NULL");
    if (pi_status st = check_elements(c, 2, {x, w->w_gate, w->w_up, w->w_down, w->b_gate, w->b_up, w->b_down, s.g, s.u, s.a, y}))
        return st;
    const CtxView v = ctx_view(c);
    const bool bf = d.dtype == PI_BF16;
    const FfnFwd f = plan_ffn(d, v, *w, x, s, y, ws);
    if (pi_status st = check_ws(c, ws, ws_bytes, f.bytes)) return st;
    DeviceGuard g(v.device);
    CUB(run_copies({&f.x, &f.wg, &f.wu, &f.wd}, v.stream));
    CUB(launch_gemm(f.p.g[0], bf, v, f.gws));
    CUB(run_copies({&f.a}, v.stream)); // (the caller's a, written by the product above)
    CUB(launch_gemm(f.p.g[1], bf, v, f.gws));
    return PI_OK;
}

pi_status pi_gated_ffn_bwd(pi_ctx *c, const pi_gated_ffn_desc *desc, const pi_gated_ffn_weights *w, const void *x,
                           const void *dy, const pi_gated_ffn_save *save, void *dx, const pi_gated_ffn_grads *grads,
                           int32_t accumulate, void *ws, size_t ws_bytes)
{
    if (!c) return PI_ERR_ARG;
    pi_gated_ffn_desc d;
    if (pi_status st = check_ffn(c, desc, d)) return st;
    pi_gated_ffn_grads gr = {};
    if (grads) gr = *grads;
    if (!d.gated && (gr.w_gate || gr.b_gate)) return ctx_fail(c, PI_ERR_ARG, "gate gradients wanted, but gated is 0");
    const CtxView v = ctx_view(c);
    const bool bf = d.dtype == PI_BF16;
    const int g32 = d.grad_dtype == PI_F32;
    if (d.T == 0) {
        if (accumulate) return PI_OK;
        DeviceGuard g(v.device);
        const size_t eb = g32 ? 4 : 2, nd = (size_t)d.n * d.d * eb;
        void *const ps[] = {gr.w_gate, gr.w_up, gr.w_down, gr.b_gate, gr.b_up, gr.b_down};
        const size_t sz[] = {nd, nd, nd, d.n * eb, d.n * eb, d.d * eb};
        for (int i = 0; i < 6; ++i)
            if (ps[i]) CUB(cudaMemsetAsync(ps[i], 0, sz[i], v.stream));
        return PI_OK;
    }
    const bool want_d = dx || gr.w_up || gr.w_gate || gr.b_up || gr.b_gate;
    if (!want_d && !gr.w_down && !gr.b_down) return PI_OK;
    if (pi_status st = check_ffn_weights(c, d, w)) return st;
    if (!dy || ((gr.w_up || gr.w_gate) && !x)) return ctx_fail(c, PI_ERR_ARG, "dy or x is NULL but needed");
    if (!save || (want_d && (!save->u || (d.gated && !save->g))) || (gr.w_down && !save->a))
        return ctx_fail(c, PI_ERR_ARG, "save, or what is needed of it, is NULL");
    if (pi_status st = check_elements(c, 2, {x, dy, w->w_gate, w->w_up, w->w_down, save->g, save->u, save->a, dx})) return st;
    if (pi_status st = check_elements(c, g32 ? 4 : 2, {gr.w_gate, gr.w_up, gr.w_down, gr.b_gate, gr.b_up, gr.b_down})) return st;
    const FfnBwd f = plan_ffn_bwd(d, v, *w, x, dy, *save, dx, gr, accumulate, ws);
    if (pi_status st = check_ws(c, ws, ws_bytes, f.bytes)) return st;
    DeviceGuard g(v.device);
    CUB(run_copies({&f.dy, &f.wd, &f.wg, &f.wu, &f.x, &f.a}, v.stream));
    if (f.da) CUB(launch_gemm(f.p.g[0], bf, v, f.gws));
    if (f.p.n > f.da) CUB(launch_gemms(f.p.g + f.da, f.p.n - f.da, bf, v, f.gws));
    // (the sums of dg and du as they are stored, rounded: the epilogue that holds
    // them unrounded has a row in each thread, so that sums over rows would cost it
    // a pass through shared memory per tile; each rounding is off by at most half a
    // step either way, and T of them add up to about the sum's own rounding)
    SumSet sums = {{}, 0, d.T, g32, accumulate, v.sms};
    void *part = f.part;
    add_sum(sums, f.dg, f.ldd, d.n, gr.b_gate, part);
    add_sum(sums, f.du, f.ldd, d.n, gr.b_up, part);
    add_sum(sums, dy, d.ldy, d.d, gr.b_down, part);
    CUB(launch_sums(sums, bf, v.stream));
    return PI_OK;
}

} // extern "C"
