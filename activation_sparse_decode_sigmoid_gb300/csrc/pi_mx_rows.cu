// The product of 8-bit x and 4-bit W, both microscaled, for very few tokens and
// large matrices (mx_rows_takes), with its epilogue:
//     D[t][f] = sum_k X[t][k] W[f][k]
//
// Bound by HBM: every weight is read once.  Here the tokens are the MMA's 128
// rows (those behind the last are whatever lies behind them in shared memory;
// their sums are not read) and 256 features its columns.  An MMA of mixed types
// takes 32 of k and about 130 cycles, with 256 columns as with 16: as in
// pi_mx_skinny.cu, with the weights as rows, 8192 -> 28672 takes 377 of them an
// SM, 27 us, where reading it takes 18; so, it takes half as many, and streams at
// 6.3 TB/s instead of 5.5.  (One token 27.3 us, there 30.9; 28672 -> 8192 27.2 and 34.1.)
//
// A cluster of CTAs shares a tile of 256 features (gated: of 128 in both
// matrices), each CTA a part of k.  At a tile's end two warps take the sums out
// of tensor memory, a token to a lane, into shared memory; four others send
// them on, slice by slice of the features, whole lines at a time, to the CTA that owns the slice
// (distributed shared memory; straight from the lanes, a row to each, took 10 us),
// which adds them in a fixed order and runs the epilogue, a feature to a thread.
//
// Every wait is bounded, as in pi_tc.cuh.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "pi_block.h"
#include "pi_epi.cuh"
#include "pi_kernels.h"
#include "pi_mx_cluster.cuh"
#include "pi_mx_tc.cuh"
#include "pi_pair.cuh"
#include "pi_tc.cuh"

namespace pi {
namespace {

constexpr int kMrOps = OPS_MX84;
constexpr int kMrThreads = 288;              // warps 0, 8: sums out of tensor memory; 1: TMA; 2: MMA; 4-7: epilogue
constexpr uint32_t kMrX = 4096, kMrW = 32768; // a step's tokens, its 256 features
constexpr uint32_t kMrSlot = kMrX + kMrW + 2048;
constexpr int kMrRing = 5;
// Tensor memory behind the accumulator: four sets of scales, of W from a set's column 8
constexpr uint32_t kMrScales = 256, kMrSet = 32, kMrSetW = 8;

struct MrParams {
    CUtensorMap mw[2], mx, msw[2], msx;
    int T, Tp, N;         // tokens, rounded up to 16; features of one weight matrix
    int tn, KT, cs;       // tiles of features, k steps, CTAs to a cluster
    int slots, early;     // ring; the weights are older than the launch before this one
    int slice;            // features (of a matrix) that a CTA owns
    uint32_t sumsB, partB, resB;
    int *status, *abort_flag;
    unsigned long long wait_ns;
    Epi e;
};

__device__ __forceinline__ void st_cluster4(uint32_t at, float a, float b, float c, float d)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// Calls f with the call's activation and output type as types (a microscaled output has x's kind).
template <int V> struct Const {
    static constexpr int value = V;
};
template <typename T, int MODE, typename F> __device__ __forceinline__ void finish(const MrParams &p, F f)
{
    auto by_out = [&](auto fn) {
        if constexpr (MODE == EPI_GATED) f(fn, Const<Ops<kMrOps>::xkind>{});
        else if (p.e.mx) f(fn, Const<Ops<kMrOps>::xkind>{});
        else if (p.e.out32) f(fn, Const<PI_F32>{});
        else f(fn, Const<PI_F16>{}); // (either 16-bit type)
    };
    switch (p.e.fn) {
    case PI_FN_RELU: return by_out(Const<PI_FN_RELU>{});
    case PI_FN_SQRELU: return by_out(Const<PI_FN_SQRELU>{});
    case PI_FN_SIGMOID: return by_out(Const<PI_FN_SIGMOID>{});
    case PI_FN_SILU: return by_out(Const<PI_FN_SILU>{});
    case PI_FN_GELU: return by_out(Const<PI_FN_GELU>{});
    case PI_FN_GELU_TANH: return by_out(Const<PI_FN_GELU_TANH>{});
    default: return by_out(Const<PI_FN_NONE>{});
    }
}

template <typename T, int MODE> __global__ void __launch_bounds__(kMrThreads, 1) mx_rows(const __grid_constant__ MrParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using O = Ops<kMrOps>;
    constexpr int NM = MODE == EPI_GATED ? 2 : 1, kTileN = 256 / NM; // features of a tile
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t S = (uint32_t)p.slots;
    const int rank = (int)cta_rank(), cluster = (int)blockIdx.x / p.cs, clusters = (int)gridDim.x / p.cs;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * kMrSlot + p.sumsB + p.partB + p.resB);
    uint64_t *empty = full + kMrRing;
    uint64_t *acc_full = empty + kMrRing, *acc_empty = acc_full + 1, *sums_full = acc_empty + 1, *sums_free = sums_full + 1;
    uint64_t *part_full = sums_free + 1, *part_free = part_full + 1;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(part_free + 1);
    if (tid == 32) prefetch_map(&p.mw[0]), prefetch_map(&p.mx), prefetch_map(&p.msw[0]), prefetch_map(&p.msx);
    if (tid == 0) {
        for (uint32_t s = 0; s < S; ++s) mbar_init1(full + s), mbar_init1(empty + s);
        mbar_init1(acc_full), mbar_init(acc_empty, 2), mbar_init(sums_full, 2), mbar_init(sums_free, 4);
        const uint32_t others = 4u * (uint32_t)max(1, p.cs - 1); // four warps of each other CTA
        mbar_init(part_full, others), mbar_init(part_free, others); // have sent, have read
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const uint32_t tmem = tmem_alloc(tslot, 512);
    // The code behind the products runs once or a few times a launch, and the first
    // time it comes from memory: the weights have passed through L2 since the
    // launch before.  Its warps go through it once ahead, with nothing to wait for,
    // send to another CTA or store (8192 -> 28672 at one token 29.6, so 27.4 us, 28672 -> 8192
    // at eight 30.1, so 28.2).  Others send sums only when that is over.
    const bool rehearses = (warp & 7) == 0 || warp >= 4;
    if (p.cs > 1 && !rehearses) cluster_arrive(); // all barriers are set up
    if (!rehearses && !(p.early && warp == 1)) pdl_enter();
    const uint32_t base = smem_addr(smem);
    MxWalk w(p.tn, 1, p.KT, p.cs, cluster, clusters, rank);
    // this CTA's sums, [token][256 and a pad: rows start in different banks], and the
    // others' of its slice: [CTA][matrix][token][feature]
    constexpr uint32_t kSumRow = 260 * 4;
    const uint32_t sums = base + S * kMrSlot, part = sums + p.sumsB, res = part + p.partB;
    const uint32_t rowB = (uint32_t)p.slice * 4u, matB = rowB * (uint32_t)p.T, srcB = matB * NM;
    bool ok = true;
    if (warp == 1) {
        Cur cur(0, S);
        uint32_t round = 0;
        const uint32_t bytes = 256u * mx_row_tx(true) + (uint32_t)p.Tp * 128u + 512u + 1024u;
        auto load_w = [&](uint32_t s) {
            const uint32_t at = base + s * kMrSlot, sf = at + kMrX + kMrW + 512;
            mbar_expect(full + s, bytes);
            if (NM == 2) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    tile_load(at + kMrX + m * (kMrW / 2), &p.mw[m], w.k * 128, w.tile * 128, full + s);
                    tile_load(sf + 512 * m, &p.msw[m], w.k * 128, w.tile, full + s);
                }
            } else {
                tile_load(at + kMrX, &p.mw[0], w.k * 128, w.tile * 256, full + s);
                tile_load(sf, &p.msw[0], w.k * 128, w.tile * 2, full + s);
            }
        };
        auto load_x = [&](uint32_t s, int k) {
            const uint32_t at = base + s * kMrSlot;
            tile_load(at, &p.mx, k * 128, 0, full + s);
            tile_load(at + kMrX + kMrW, &p.msx, k * 128, 0, full + s);
        };
        if (p.early) {
            // fill the ring's weights while the launch before finishes, then their tokens
            MxWalk x = w;
            for (; w.more() && round < S; w.next(), ++round) {
                if (elect_one()) load_w(round);
                __syncwarp();
            }
            pdl_enter();
            for (uint32_t s = 0; s < round; ++s, x.next()) {
                if (elect_one()) load_x(s, x.k);
                __syncwarp();
            }
            cur = Cur(round, S);
        }
        for (; w.more(); w.next()) {
            if (round >= S && !mbar_wait_all(empty + cur.s, cur.ph ^ 1u, p)) {
                ok = false;
                break;
            }
            if (elect_one()) {
                load_w(cur.s);
                load_x(cur.s, w.k);
            }
            __syncwarp();
            cur.next(S);
            ++round;
        }
        for (uint32_t i = round < S ? round : S; ok && i > 0; --i) { // nothing of its own is left in flight
            const Cur last(round - i, S);
            ok = mbar_wait_all(empty + last.s, last.ph, p);
        }
    } else if (warp == 2) {
        const uint32_t id = idesc_mx(O::xfmt, O::wfmt, 128, 256);
        const uint64_t d0 = sdesc(base, 16, 1024);
        uint32_t set = 0;
        Cur cur(0, S);
        for (uint32_t it = 0; ok && w.more(); ++it) {
            if (it >= 1 && !mbar_wait_all(acc_empty, (it - 1) & 1, p)) break;
            tc_after();
            const int tile = w.tile;
            for (; w.more() && w.tile == tile; w.next()) {
                if (!mbar_wait_all(full + cur.s, cur.ph, p)) {
                    ok = false;
                    break;
                }
                tc_after();
                if (elect_one()) {
                    const uint64_t a = d0 + ((cur.s * kMrSlot) >> 4), b = a + (kMrX >> 4);
                    const uint32_t ts = tmem + kMrScales + set * kMrSet, sf = base + cur.s * kMrSlot + kMrX + kMrW;
                    cp_scales(ts, sf);
                    cp_scales(ts + kMrSetW, sf + 512), cp_scales(ts + kMrSetW + 4, sf + 1024);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_mx<kMrOps>(tmem, a + 2 * j, b + 2 * j, id | sf_id<kMrOps>(j), ts, ts + kMrSetW, (w.k > w.k0 || j > 0) ? 1u : 0u);
                    mma_commit(empty + cur.s);
                }
                set = (set + 1) & 3;
                __syncwarp();
                cur.next(S);
            }
            if (ok && elect_one()) mma_commit(acc_full);
            __syncwarp();
        }
    } else if ((warp & 7) == 0) { // the tokens lie in these warps' lanes of tensor memory; half of the columns each
        const int half = warp >> 3;
        bool dry = true;
        uint32_t it = 0;
        for (int tile = cluster; tile < p.tn;) {
            if (!dry) {
                ok = warp_wait(acc_full, it & 1, p, lane);
                if (ok && it > 0) ok = warp_wait(sums_free, (it - 1) & 1, p, lane);
                if (!ok) break;
                tc_after();
            }
#pragma unroll 1
            for (int c = 128 * half; c < 128 * half + 128; c += 64) {
                uint32_t v[2][32];
                tmem_ld32_async(tmem + (uint32_t)c, v[0]);
                tmem_ld32_async(tmem + (uint32_t)c + 32, v[1]);
                tmem_wait32(v[0]);
                tmem_wait32(v[1]);
                const uint32_t at = sums + (uint32_t)lane * kSumRow + (uint32_t)c * 4u;
                if (lane < p.T) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 128 * h + 4 * i), "r"(v[h][i]), "r"(v[h][i + 1]), "r"(v[h][i + 2]), "r"(v[h][i + 3]) : "memory");
                }
                __syncwarp(); // (some lanes stored: loads from tensor memory take whole warps)
            }
            tc_before();
            __syncwarp();
            if (dry) {
                if (p.cs > 1) cluster_arrive();
                pdl_enter();
                dry = false;
                continue;
            }
            if (lane == 0) {
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(acc_empty)) : "memory");
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(sums_full)) : "memory");
            }
            tile += clusters, ++it;
        }
    } else if (warp >= 4) { // (4 to 7)
        // A feature to a thread (two, where a CTA owns all 256); where a slice has
        // fewer than 128, the other warps take other tokens.  The code of the call's
        // own activation and output type only: it runs once or a few times a launch, so that every
        // line of it comes from memory (all of them, unrolled over 8 tokens, took 5 to 7 us instead of 1).
        const int e = tid - 128, shift = 31 - __clz(p.slice), i0 = e & (p.slice - 1), tg = e >> shift, ng = max(1, 128 >> shift);
        bool dry = true;
        uint32_t it = 0;
        for (int tile = cluster; tile < p.tn;) {
            const int fs = tile * kTileN + rank * p.slice; // the slice's first feature
            // biases and the residual, on their way while the products run; a thread reads back what it put
            float bias[2][2] = {}; // [matrix][i0, i0 + 128]
            if (!dry)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int f = fs + i0 + 128 * h;
                    if (128 * h >= p.slice || f >= p.N) continue;
                    if (p.e.bias) bias[0][h] = C16<T>::one(p.e.bias[f]);
                    if (NM == 2 && p.e.bias2) bias[1][h] = C16<T>::one(p.e.bias2[f]);
                }
            if (MODE == EPI_LINEAR && p.e.res && !dry) {
#pragma unroll 1
                for (int i = i0; i < p.slice; i += 128) {
                    const int f = fs + i;
                    if (f >= p.N) break;
#pragma unroll 4
                    for (int t = tg; t < p.T; t += ng) {
                        const float r = p.e.out32 ? static_cast<const float *>(p.e.res)[t * p.e.ldr + f]
                                                  : C16<T>::one(static_cast<const uint16_t *>(p.e.res)[t * p.e.ldr + f]);
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(res + (uint32_t)(t * p.slice + i) * 4u), "f"(r) : "memory");
                    }
                }
            }
            if (!dry) {
                ok = warp_wait(sums_full, it & 1, p, lane);
                if (ok && p.cs > 1 && it > 0) ok = warp_wait_cluster(part_free, (it - 1) & 1, p, lane);
                if (!ok) break;
            }
            if (p.cs > 1) {
                // 16 bytes a thread; at the owner [matrix][token][slice]
                const int qs = shift - 2, c4 = e & ((1 << qs) - 1);
#pragma unroll 1
                for (int r = 1; r < p.cs; ++r) {
                    const int q = (rank + r) & (p.cs - 1);
                    const uint32_t dst = (dry ? part : in_cta(part, (uint32_t)q) + (uint32_t)(rank - (rank > q ? 1 : 0)) * srcB) + 16u * (uint32_t)c4;
                    const uint32_t src = sums + (uint32_t)(q * p.slice + 4 * c4) * 4u;
#pragma unroll 2
                    for (int row = e >> qs; row < NM * p.T; row += 128 >> qs) {
                        const int m = NM == 2 && row >= p.T ? 1 : 0;
                        float a, b, c, d;
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a), "=f"(b), "=f"(c), "=f"(d)
                                     : "r"(src + (uint32_t)(row - m * p.T) * kSumRow + (uint32_t)(m * kTileN) * 4u) : "memory");
                        st_cluster4(dst + (uint32_t)row * rowB, a, b, c, d);
                    }
                }
                __syncwarp(); // (the arrivals release what the whole warp wrote)
                if (!dry) {
                    if (lane < p.cs && lane != rank) arrive_cluster(in_cta(smem_addr(part_full), (uint32_t)lane));
                    ok = warp_wait_cluster(part_full, it & 1, p, lane);
                    if (!ok) break;
                }
            }
            finish<T, MODE>(p, [&](auto fn, auto out) {
#pragma unroll 1
                for (int i = i0; i < p.slice; i += 128) {
                    const int f = dry ? INT_MAX : fs + i;
                    const float b[2] = {i < 128 ? bias[0][0] : bias[0][1], i < 128 ? bias[1][0] : bias[1][1]};
#pragma unroll 4
                    for (int t = tg; t < p.T; t += ng) {
                        float v[2], r = 0.f;
#pragma unroll
                        for (int m = 0; m < NM; ++m) {
                            uint32_t at = part + (uint32_t)m * matB + (uint32_t)(t * p.slice + i) * 4u;
                            float s;
                            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(sums + (uint32_t)t * kSumRow + (uint32_t)(m * kTileN + rank * p.slice + i) * 4u));
#pragma unroll 1
                            for (int k = 1; k < p.cs; ++k, at += srcB) { // (this CTA's own first, then the others' in order)
                                float x;
                                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
                                s += x;
                            }
                            v[m] = s + b[m];
                        }
                        v[0] = act_one<decltype(fn)::value>(v[0]);
                        if (NM == 2) v[0] *= v[1];
                        if (MODE == EPI_LINEAR && p.e.res && f < p.N) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(res + (uint32_t)(t * p.slice + i) * 4u));
                        put32<T, decltype(out)::value>(p.e, t, f, p.N, v[0], r);
                    }
                }
            });
            __syncwarp();
            if (dry) {
                if (p.cs > 1) cluster_arrive();
                pdl_enter();
                if (p.cs > 1) cluster_wait();
                dry = false;
                continue;
            }
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(sums_free)) : "memory");
            if (lane < p.cs && lane != rank) arrive_cluster(in_cta(smem_addr(part_free), (uint32_t)lane));
            tile += clusters, ++it;
        }
    }
    settle(p); // copies and MMAs in flight finish before the CTA leaves
    if (p.cs > 1) {
        if (warp < 4 || warp == 8) cluster_wait(); // (of the first arrival)
        __syncthreads();
        cluster_sync(); // no CTA leaves while another still writes to it
    }
    tmem_free(tmem, 512);
}

constexpr int kMrExchange = 8; // steps

MrParams plan(const Gemm &g, const CtxView &v, const int (&n)[4], int &grid)
{
    MrParams p = {};
    const int nm = g.mode == EPI_GATED ? 2 : 1, tileN = 256 / nm;
    p.T = g.M, p.Tp = (g.M + 15) / 16 * 16, p.N = g.N;
    p.tn = (g.N + tileN - 1) / tileN, p.KT = mx_tiles(g.K[0]);
    int clusters = 1;
    p.cs = mx_cluster(p.tn, 1, p.KT, n, tileN / 32, kMrExchange, clusters);
    p.slice = tileN / p.cs;
    p.sumsB = ((uint32_t)p.T * 1040u + 127u) / 128u * 128u;
    p.partB = (uint32_t)(p.cs - 1) * nm * p.T * p.slice * 4u;
    p.resB = g.e.res ? (uint32_t)p.T * p.slice * 4u : 0u;
    p.slots = std::min(kMrRing, (v.smem_optin - 1024 - (int)(p.sumsB + p.partB + p.resB)) / (int)kMrSlot);
    p.status = v.status, p.abort_flag = v.abort_flag, p.wait_ns = v.wait_ns;
    p.early = g.early;
    p.e = g.e;
    grid = clusters * p.cs;
    return p;
}

template <typename T, int MODE> cudaError_t run(const Gemm &g, const CtxView &v)
{
    static std::atomic<uint64_t> ready{0};
    static ClusterCounts known;
    auto kern = mx_rows<T, MODE>;
    int n[4], grid = 0;
    cudaError_t e = raise_limit((const void *)kern, ready);
    if (e == cudaSuccess) e = cluster_counts(kern, known, kMrThreads, v, n);
    if (e != cudaSuccess) return e;
    MrParams p = plan(g, v, n, grid);
    const int tiles = mx_tiles(g.K[0]), nm = MODE == EPI_GATED ? 2 : 1;
    e = encode_map_bytes(&p.mx, g.a[0].p, (uint64_t)mx_row_bytes(PI_MX8, g.K[0]), (uint64_t)g.M, (uint64_t)g.a[0].ld, (uint32_t)p.Tp);
    if (e == cudaSuccess) e = encode_map_scales(&p.msx, g.sa, tiles, 1, 1, 1);
    for (int i = 0; i < nm && e == cudaSuccess; ++i) {
        e = encode_map_nibbles(&p.mw[i], g.b[i].p, (uint64_t)tiles * 128, (uint64_t)g.N, (uint64_t)g.b[i].ld, 256 / nm);
        if (e == cudaSuccess) e = encode_map_scales(&p.msw[i], g.sb[i], tiles, mx_tiles(g.N), 1, 2 / nm);
    }
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, grid, p.cs, kMrThreads, (size_t)p.slots * kMrSlot + p.sumsB + p.partB + p.resB + (2 * kMrRing + 6) * 8 + 16, v.stream, p);
}

} // namespace

// The sums' way from lanes to columns, and a whole SM for a CTA, so that no launch
// waits beside the one before it, cost about a microsecond at one token and 0.15 more for
// each further one, and again at each tile where k is too short to hide them: worth it
// from 20 MB of weights on (2 more a token) and 2048 values of k, to 16 tokens.  us, here and in pi_mx_skinny.cu:
//   1024 -> 28672, 16 MB:    8.7,  8.4 at one token,  9.6,  8.5 at 8, 10.6,  8.5 at 16
//   2048 -> 28672, 31 MB:   11.3, 12.5               12.4, 12.5       13.4, 12.5
//   4096 -> 28672, 62 MB:   17.4, 19.8               18.2, 19.9       19.4, 20.1
//   8192 -> 28672, 125 MB:  27.3, 30.9               28.5, 31.3       29.7, 31.6
//   1024 -> 128256, 70 MB:  21.2, 19.6               22.3, 19.7       24.5, 19.9
bool mx_rows_takes(const Gemm &g)
{
    const int64_t bytes = (int64_t)g.N * mx_tiles(g.K[0]) * 68 * (g.mode == EPI_GATED ? 2 : 1);
    return g.ops == kMrOps && g.M <= 16 && g.K[0] >= 2048 && bytes >= (int64_t)(18 + 2 * g.M) << 20;
}

cudaError_t launch_mx_rows(const Gemm &g, bool bf16, const CtxView &v)
{
    if (g.mode == EPI_GATED) return bf16 ? run<__nv_bfloat16, EPI_GATED>(g, v) : run<__half, EPI_GATED>(g, v);
    return bf16 ? run<__nv_bfloat16, EPI_LINEAR>(g, v) : run<__half, EPI_LINEAR>(g, v);
}

} // namespace pi
