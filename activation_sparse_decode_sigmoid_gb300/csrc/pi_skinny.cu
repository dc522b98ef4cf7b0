// The matrix product of the block operators for few tokens (M <= 128 rows of A):
//     D[t][f] = sum_k X[t][k] W[f][k]
//
// Bound by HBM: every weight is read once for 2 M operations.  The weights
// are the MMA's 128-row operand and the tokens its columns (M rounded up to
// 16), so no part of the product is spent on rows that are not there; a CTA
// per SM streams its share of W through a ring of boxes that fills shared
// memory (about 200 KB in flight per SM, whatever the token count).
// The work is cut by bytes, not by tiles: all (128-feature tile, k step) pairs
// end to end, in equal ranges, one per CTA.  Each CTA writes the fp32 partial
// sums of its tiles, [tokens][128], and skinny_join adds the parts of a tile in
// the order of k and runs the epilogue on 8 features at a time.  (Whole rows
// per CTA, without the second launch, lost: an MMA of 128 x 16 x 16 takes about
// 100 cycles however few of its rows count, so 56 rows of K = 28672 took 101 us
// against 80.)
//
// One token, and up to four of a smaller matrix (gemv_takes), take one launch
// of gemv_rows instead: dot products on the CUDA cores, no workspace.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pi_block.h"
#include "pi_epi.cuh"
#include "pi_kernels.h"
#include "pi_tc.cuh"

namespace pi {
namespace {

constexpr int kSkThreads = 192;   // warps 0-3: partial sums out of tensor memory; 4: TMA; 5: MMA
constexpr uint32_t kWTile = 16384; // 128 features x 64 k
constexpr int kMaxRing = 12;

struct SkParams {
    CUtensorMap mw[2], mx;
    int T, Tp, N;         // tokens, rounded up to 16; features of one weight matrix
    int tn, tiles, KT;    // tiles of one matrix, of all; k steps
    int parts, smax;
    int slots;            // ring
    int early;            // the weights are older than the launch before this one: load them ahead of its results
    uint32_t slotB;
    float *part;          // [tiles][smax][T][128]
    int *status, *abort_flag;
    unsigned long long wait_ns;
    Epi e;
};

__host__ __device__ inline int64_t sk_range(int64_t units, int c, int parts) { return units * c / parts; }
__host__ __device__ inline int sk_part_of(int64_t units, int64_t u, int parts)
{
    return (int)(((u + 1) * parts + units - 1) / units - 1);
}

template <typename T> __global__ void __launch_bounds__(kSkThreads, 1) skinny_tc(const __grid_constant__ SkParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using H = H16<T>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t S = (uint32_t)p.slots;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * p.slotB);
    uint64_t *empty = full + kMaxRing;
    uint64_t *acc_full = empty + kMaxRing, *acc_empty = acc_full + 2;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    if (tid == 128) prefetch_map(&p.mw[0]), prefetch_map(&p.mx);
    if (tid == 0) {
        for (uint32_t s = 0; s < S; ++s) mbar_init1(full + s), mbar_init1(empty + s);
        for (int s = 0; s < 2; ++s) mbar_init1(acc_full + s), mbar_init(acc_empty + s, 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const uint32_t tmem = tmem_alloc(tslot, 256); // two accumulators of up to 128 columns
    if (!(p.early && warp == 4)) pdl_enter();
    const int64_t units = (int64_t)p.tiles * p.KT;
    int64_t u = sk_range(units, (int)blockIdx.x, p.parts);
    const int64_t u1 = sk_range(units, (int)blockIdx.x + 1, p.parts);
    const uint32_t base = smem_addr(smem);
    bool ok = true;
    if (warp == 4) {
        Cur cur(0, S);
        uint32_t round = 0;
        const uint32_t bytes = kWTile + (uint32_t)p.Tp * 128u;
        int tile = (int)(u / p.KT), k = (int)(u - (int64_t)tile * p.KT);
        auto load_w = [&](uint32_t s) {
            const int m = tile >= p.tn ? 1 : 0;
            mbar_expect(full + s, bytes);
            tile_load(base + s * p.slotB, &p.mw[m], k * kBK, (tile - m * p.tn) * 128, full + s);
        };
        if (p.early) {
            // fill the ring's weights while the launch before finishes, then their tokens
            int kx = k;
            for (; u < u1 && round < S; ++u, ++round) {
                if (elect_one()) load_w(round);
                __syncwarp();
                if (++k == p.KT) k = 0, ++tile;
            }
            pdl_enter();
            for (uint32_t s = 0; s < round; ++s) {
                if (elect_one()) tile_load(base + s * p.slotB + kWTile, &p.mx, kx * kBK, 0, full + s);
                __syncwarp();
                if (++kx == p.KT) kx = 0;
            }
            cur = Cur(round, S);
        }
        for (; u < u1; ++u) {
            if (round >= S && !mbar_wait_all(empty + cur.s, cur.ph ^ 1u, p)) {
                ok = false;
                break;
            }
            if (elect_one()) {
                load_w(cur.s);
                tile_load(base + cur.s * p.slotB + kWTile, &p.mx, k * kBK, 0, full + cur.s);
            }
            __syncwarp();
            cur.next(S);
            ++round;
            if (++k == p.KT) k = 0, ++tile;
        }
        for (uint32_t i = round < S ? round : S; ok && i > 0; --i) { // nothing of its own is left in flight
            const Cur last(round - i, S);
            ok = mbar_wait_all(empty + last.s, last.ph, p);
        }
    } else if (warp == 5) {
        const uint32_t id = idesc(H::fmt, 0, 0, 128, (uint32_t)p.Tp);
        const uint64_t d0 = sdesc(base, 16, 1024);
        Cur cur(0, S);
        for (uint32_t it = 0; ok && u < u1; ++it) {
            const uint32_t buf = it & 1, ph = (it >> 1) & 1;
            if (it >= 2 && !mbar_wait_all(acc_empty + buf, ph ^ 1u, p)) break;
            tc_after();
            const int64_t end = min(u1, (u / p.KT + 1) * p.KT);
            for (bool first = true; u < end; ++u, first = false) {
                if (!mbar_wait_all(full + cur.s, cur.ph, p)) {
                    ok = false;
                    break;
                }
                tc_after();
                if (elect_one()) {
                    const uint64_t a = d0 + ((cur.s * p.slotB) >> 4), b = a + (kWTile >> 4);
#pragma unroll
                    for (int j = 0; j < kBK / 16; ++j) mma(tmem + buf * 128u, a + 2 * j, b + 2 * j, id, (!first || j > 0) ? 1u : 0u);
                    mma_commit(empty + cur.s);
                }
                __syncwarp();
                cur.next(S);
            }
            if (ok && elect_one()) mma_commit(acc_full + buf);
            __syncwarp();
        }
    } else {
        for (uint32_t it = 0; ok && u < u1; ++it) {
            const uint32_t buf = it & 1, ph = (it >> 1) & 1;
            ok = warp_wait(acc_full + buf, ph, p, lane);
            if (!ok) break;
            tc_after();
            const int tile = (int)(u / p.KT);
            const int slot = (int)blockIdx.x - sk_part_of(units, (int64_t)tile * p.KT, p.parts);
            float *dst = p.part + ((size_t)tile * p.smax + slot) * (size_t)p.T * 128 + warp * 32 + lane;
            const uint32_t ta = tmem + ((uint32_t)(warp * 32) << 16) + buf * 128u;
            for (int t0 = 0; t0 < p.T; t0 += 16) {
                float v[16];
                tmem_ld16(ta + t0, v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (t0 + i < p.T) dst[(size_t)(t0 + i) * 128] = v[i];
            }
            tc_before();
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(acc_empty + buf)) : "memory");
            u = min(u1, (int64_t)(tile + 1) * p.KT);
        }
    }
    __syncwarp();
    if (*(volatile int *)p.abort_flag) { // copies and MMAs in flight finish before the CTA leaves
        const uint64_t t0 = gtimer();
        while (gtimer() - t0 < 5000000ull) {
        }
    }
    tmem_free(tmem, 256);
}

template <typename T, int MODE> __global__ void __launch_bounds__(128) skinny_join(const __grid_constant__ SkParams p)
{
    pdl_enter();
    const int per = p.tn * 16; // groups of 8 features of a token
    const int i = blockIdx.x * 128 + threadIdx.x;
    const int t = i / per, f = (i - t * per) * 8;
    if (t >= p.T || f >= p.N) return;
    const int64_t units = (int64_t)p.tiles * p.KT;
    float v[2][8] = {};
#pragma unroll
    for (int m = 0; m < (MODE == EPI_GATED ? 2 : 1); ++m) {
        const int tile = f / 128 + m * p.tn;
        const int cnt = sk_part_of(units, (int64_t)(tile + 1) * p.KT - 1, p.parts) - sk_part_of(units, (int64_t)tile * p.KT, p.parts) + 1;
        const float *src = p.part + ((size_t)tile * p.smax * p.T + t) * 128 + (f & 127);
#pragma unroll 8
        for (int s = 0; s < cnt; ++s) {
            float w[8];
            load8f(src + (size_t)s * p.T * 128, 8, true, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[m][j] += w[j];
        }
    }
    epilogue8<T, MODE>(p.e, p.N, t, f, v[0], v[1]);
}

// ------------------------------------------------------------------ one token, or few and a smaller matrix
// A group of `wpr` warps of a CTA computes R features (gated: their g and u)
// for all tokens: lanes take chunks of 8 elements of the rows, 4 loads or
// more in flight each, and the warps' sums are added in order.  With 2 to 4
// tokens two rows share each chunk of x read (four rows, with half the loads
// in flight, took 95 us instead of 85 for 8192 x 28672 at 4 tokens).
constexpr int kGvWarps = 8, kGvTokens = 4;

struct GvParams {
    int T, N, K, wpr;
    const uint16_t *x, *w[2];
    int64_t ldx, ldw[2];
    Epi e;
};

template <typename T, int MODE, int TT, int R>
__global__ void __launch_bounds__(32 * kGvWarps) gemv_rows(const __grid_constant__ GvParams p)
{
    constexpr int NM = MODE == EPI_GATED ? 2 : 1, NR = NM * R, U = NR > 2 ? 2 : 4;
    __shared__ float red[kGvWarps][NR][TT];
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % p.wpr, f0 = ((int)blockIdx.x * (kGvWarps / p.wpr) + warp / p.wpr) * R;
    float acc[NR][TT] = {};
    if (f0 < p.N) {
        const uint4 *w[NR], *x = reinterpret_cast<const uint4 *>(p.x);
#pragma unroll
        for (int i = 0; i < NR; ++i) // (past the last feature: the last again, not kept)
            w[i] = reinterpret_cast<const uint4 *>(p.w[i / R] + (int64_t)min(f0 + i % R, p.N - 1) * p.ldw[i / R]);
        const int nch = p.K >> 3, step = 32 * p.wpr;
        const int64_t ldx = p.ldx >> 3;
        int c = part * 32 + lane;
        for (; c + (U - 1) * step < nch; c += U * step) {
            uint4 q[NR][U];
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int j = 0; j < U; ++j) q[i][j] = __ldg(w[i] + c + j * step);
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const uint4 v = x[t * ldx + c + j * step];
#pragma unroll
                    for (int i = 0; i < NR; ++i) acc[i][t] = fma8<T>(q[i][j], v, acc[i][t]);
                }
        }
        for (; c < nch; c += step)
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const uint4 q = __ldg(w[i] + c);
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[i][t] = fma8<T>(q, x[t * ldx + c], acc[i][t]);
            }
        const int k = nch * 8 + lane; // the last K mod 8 elements
        if (part == 0 && k < p.K)
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    acc[i][t] = fmaf(C16<T>::one(reinterpret_cast<const uint16_t *>(w[i])[k]), C16<T>::one(p.x[t * p.ldx + k]), acc[i][t]);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) acc[i][t] += __shfl_xor_sync(0xffffffffu, acc[i][t], o);
            if (lane == 0) red[warp][i][t] = acc[i][t];
        }
    if (p.wpr > 1) __syncthreads();
    else __syncwarp();
    const int t = lane % TT, r = lane / TT;
    if (part || r >= R || f0 + r >= p.N) return;
    float v[2] = {};
    for (int w = 0; w < p.wpr; ++w)
#pragma unroll
        for (int m = 0; m < NM; ++m) v[m] += red[warp + w][m * R + r][t];
    epilogue1<T, MODE>(p.e, t, f0 + r, v[0], v[1]);
}

template <typename T, int MODE, int TT, int R> cudaError_t run_gemv(const GvParams &p, cudaStream_t s)
{
    const int per = kGvWarps / p.wpr * R;
    return launch_pdl(gemv_rows<T, MODE, TT, R>, dim3((p.N + per - 1) / per), dim3(32 * kGvWarps), 0, s, p);
}

template <typename T, int MODE> cudaError_t pick_gemv(const GvParams &p, cudaStream_t s)
{
    constexpr int NM = MODE == EPI_GATED ? 2 : 1;
    return p.T == 1   ? run_gemv<T, MODE, 1, 1>(p, s)
           : p.T == 2 ? run_gemv<T, MODE, 2, 2 / NM>(p, s)
           : p.T == 3 ? run_gemv<T, MODE, 3, 2 / NM>(p, s)
                      : run_gemv<T, MODE, 4, 2 / NM>(p, s);
}

template <typename T> cudaError_t gemv(const Gemm &g, const CtxView &v)
{
    GvParams p = {};
    p.T = g.M, p.N = g.N, p.K = g.K[0];
    p.x = static_cast<const uint16_t *>(g.a[0].p), p.ldx = g.a[0].ld;
    const int nm = g.mode == EPI_GATED ? 2 : 1;
    for (int m = 0; m < nm; ++m) p.w[m] = static_cast<const uint16_t *>(g.b[m].p), p.ldw[m] = g.b[m].ld;
    // warps to a group of rows: one, unless there are too few rows for about
    // 54 warps' work per SM (8192 x K at one token: 1, 2, 4 and 8 warps
    // 70, 70, 69, 70 us at K = 28672; 2048 rows 32, 23, 20, 21 us; 28672 rows of 1024 13, 18, 26, 41 us)
    const int rows = p.T == 1 ? nm : 2; // rows of a group
    const int64_t groups = (int64_t)p.N * nm / rows;
    p.wpr = 1;
    while (p.wpr < kGvWarps && groups * p.wpr < 54 * (int64_t)v.sms && p.K >= 2048 * p.wpr) p.wpr *= 2;
    p.e = g.e;
    return g.mode == EPI_GATED ? pick_gemv<T, EPI_GATED>(p, v.stream) : pick_gemv<T, EPI_LINEAR>(p, v.stream);
}

// One token: always (8192 x 28672: 70 us, 6.7 TB/s; skinny_tc 80 us).  Two to
// four: matrices of up to this many bytes; beyond, the reads of x through L1
// cost more than skinny_tc's second launch (4 tokens, 8.4, 34, 134 and 268 MB:
// 4.4, 9, 27 and 52 us, skinny_tc 8, 13, 29 and 49 us).
constexpr int64_t kGemvBytes = 128 << 20;

bool gemv_takes(const Gemm &g)
{
    const int64_t bytes = (int64_t)g.N * g.K[0] * 2 * (g.mode == EPI_GATED ? 2 : 1);
    return g.M == 1 || (g.M <= kGvTokens && bytes <= kGemvBytes);
}

SkParams plan(const Gemm &g, const CtxView &v)
{
    SkParams p = {};
    p.T = g.M, p.Tp = (g.M + 15) / 16 * 16, p.N = g.N;
    p.tn = (g.N + 127) / 128;
    p.tiles = p.tn * (g.mode == EPI_GATED ? 2 : 1);
    p.KT = (g.K[0] + kBK - 1) / kBK;
    const int64_t units = (int64_t)p.tiles * p.KT;
    p.parts = (int)std::min<int64_t>(v.sms, std::max<int64_t>(1, units / 6)); // at least six k steps each
    p.smax = (int)std::min<int64_t>(p.parts, p.KT / (units / p.parts) + 2);
    p.slotB = kWTile + (uint32_t)p.Tp * 128u;
    p.slots = std::min(kMaxRing, (v.smem_optin - 1024) / (int)p.slotB);
    p.status = v.status, p.abort_flag = v.abort_flag, p.wait_ns = v.wait_ns;
    p.early = g.early;
    p.e = g.e;
    return p;
}

template <typename T, int MODE> cudaError_t run(const SkParams &p, cudaStream_t s)
{
    auto kern = skinny_tc<T>;
    const int smem = p.slots * (int)p.slotB + (2 * kMaxRing + 4) * 8 + 16;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = raise_limit((const void *)kern, ready);
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(p.parts), dim3(kSkThreads), smem, s, p);
    if (e != cudaSuccess) return e;
    const int64_t threads = (int64_t)p.T * p.tn * 16;
    return launch_pdl(skinny_join<T, MODE>, dim3((unsigned)((threads + 127) / 128)), dim3(128), 0, s, p);
}

template <typename T> cudaError_t run_mode(const Gemm &g, const SkParams &p, cudaStream_t s)
{
    return g.mode == EPI_GATED ? run<T, EPI_GATED>(p, s) : run<T, EPI_LINEAR>(p, s);
}

} // namespace

bool skinny_takes(const Gemm &g)
{
    return g.M <= kSkinnyRows && g.segs == 1 && g.mode != EPI_DACT && !g.a[0].mn && !g.b[0].mn;
}

size_t skinny_workspace(const Gemm &g, const CtxView &v)
{
    if (gemv_takes(g)) return 0;
    const SkParams p = plan(g, v);
    return (size_t)p.tiles * p.smax * p.T * 128 * sizeof(float);
}

cudaError_t launch_skinny(const Gemm &g, bool bf16, const CtxView &v, void *ws)
{
    if (gemv_takes(g)) return bf16 ? gemv<__nv_bfloat16>(g, v) : gemv<__half>(g, v);
    SkParams p = plan(g, v);
    p.part = static_cast<float *>(ws);
    const int nm = g.mode == EPI_GATED ? 2 : 1;
    cudaError_t e = encode_map(&p.mx, g.a[0].p, (uint64_t)g.K[0], (uint64_t)g.M, (uint64_t)g.a[0].ld * 2, (uint32_t)p.Tp);
    for (int i = 0; i < nm && e == cudaSuccess; ++i)
        e = encode_map(&p.mw[i], g.b[i].p, (uint64_t)g.K[0], (uint64_t)g.N, (uint64_t)g.b[i].ld * 2, 128);
    if (e != cudaSuccess) return e;
    return bf16 ? run_mode<__nv_bfloat16>(g, p, v.stream) : run_mode<__half>(g, p, v.stream);
}

} // namespace pi
