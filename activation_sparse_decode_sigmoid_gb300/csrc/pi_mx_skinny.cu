// The product of microscaled operands for few tokens (M <= 128 rows of A), with
// its epilogue:
//     D[t][f] = sum_k X[t][k] W[f][k]
//
// Bound by HBM: every weight is read once.  The weights are the MMA's 128-row
// operand and the tokens its columns (M rounded up to 16); a CTA per SM streams
// its share of W through a ring of boxes in half of the SM's shared memory (more
// in flight gained nothing), so that the next launch's CTAs can start beside
// them.  8192 -> 28672, one token: both of 4 bits 24.0 us (5.2 TB/s of weights), of 8
// 42.6 (5.7 TB/s; a copy reaches 6.8), 4-bit weights under 8-bit x 30.9 (4.0 TB/s: bound by the
// MMAs' number, see pi_mx_rows.cu).
//
// A cluster of CTAs takes a tile of 128 features at a time, each CTA a part of
// k: as many CTAs to a cluster as deal the tiles' steps most evenly.  At a
// tile's end every CTA sends the sums of a token to the CTA of the cluster that
// owns the token (distributed shared memory), which adds them in a fixed
// order and runs the epilogue: one launch, no workspace.  (Work cut by bytes
// over all CTAs, partial sums through memory and a second launch that joins
// them, as in pi_skinny.cu: both of 4 bits 26.3 us at 8192 -> 28672.)
//
// Every wait is bounded, as in pi_tc.cuh.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pi_block.h"
#include "pi_epi.cuh"
#include "pi_kernels.h"
#include "pi_mx_cluster.cuh"
#include "pi_mx_tc.cuh"
#include "pi_pair.cuh"
#include "pi_tc.cuh"

namespace pi {
namespace {

constexpr int kMsThreads = 192;    // warps 0-3: epilogue; 4: TMA; 5: MMA
constexpr uint32_t kMsW = 16384;   // 128 features of a step
constexpr int kMsRing = 12;
// Tensor memory: four sets of scales, of W in the first 8 columns of a set; then the accumulators
constexpr uint32_t kMsSet = 16, kMsSetX = 8, kMsAcc = 64;

struct MsParams {
    CUtensorMap mw[2], mx, msw[2], msx;
    int T, Tp, N;         // tokens, rounded up to 16; features of one weight matrix
    int tn, KT;           // tiles of features; k steps
    int cs, own, owners;  // CTAs to a cluster; tokens that one owns (a multiple of 16); CTAs that own some
    int nbuf;             // tiles in flight
    uint32_t tcols;       // tensor memory
    int slots;            // ring
    int early;            // the weights are older than the launch before this one: load them ahead of its results
    uint32_t slotB, partB;
    int *status, *abort_flag;
    unsigned long long wait_ns;
    Epi e;
};

__device__ __forceinline__ void st_cluster(uint32_t at, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// The outputs of tokens t0 .. t0 + n - 1 (n <= 16) in a warp's 32 features, one a lane.
template <int KIND> __device__ __forceinline__ void put_mx(const Epi &e, int t0, int n, int f, int N, const float (&v)[16])
{
    uint8_t *row = static_cast<uint8_t *>(e.out) + (int64_t)t0 * e.ldo + (KIND == PI_MX8 ? f : f >> 1);
#pragma unroll
    for (int i = 0; i < 16; ++i, row += e.ldo) { // (the warp holds a block)
        if (i >= n) break;
        const float x = f < N ? v[i] : 0.f;
        const uint32_t code = mx_scale<KIND>(__reduce_max_sync(0xffffffffu, mag(x)));
        float q[8] = {x * mx_inverse(code)};
        if (KIND == PI_MX4) q[1] = __shfl_xor_sync(0xffffffffu, q[0], 1);
        const uint8_t byte = KIND == PI_MX4 && code == 255u ? 0 : (uint8_t)mx_pack8<KIND>(q).x;
        if (KIND == PI_MX8 || !(f & 1)) *row = byte;
        if (!(f & 31)) e.mx_scales[mx_scale_at(t0 + i, f >> 7, e.mx_tiles) + ((f >> 5) & 3)] = (uint8_t)code;
    }
}
template <typename U, typename F> __device__ __forceinline__ void put_rows(const Epi &e, int t0, int n, int f, const float (&v)[16], F conv)
{
    U *o = static_cast<U *>(e.out) + (int64_t)t0 * e.ldo + f;
    if (e.res) {
        const U *r = static_cast<const U *>(e.res) + (int64_t)t0 * e.ldr + f;
        U x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i, r += e.ldr)
            if (i < n) x[i] = *r;
#pragma unroll
        for (int i = 0; i < 16; ++i, o += e.ldo)
            if (i < n) *o = conv(v[i] * e.scale, &x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i, o += e.ldo)
            if (i < n) *o = conv(v[i] * e.scale, (const U *)nullptr);
    }
}
// (gated: a, which has x's kind; so has what an ungated block's first product leaves)
template <typename T, int MODE, int OPS> __device__ __forceinline__ void put16(const Epi &e, int t0, int n, int f, int N, const float (&v)[16])
{
    if constexpr (MODE == EPI_GATED) put_mx<Ops<OPS>::xkind>(e, t0, n, f, N, v);
    else {
        if (e.mx) return put_mx<Ops<OPS>::xkind>(e, t0, n, f, N, v);
        if (f >= N) return;
        if (e.out32) put_rows<float>(e, t0, n, f, v, [](float a, const float *r) { return r ? a + *r : a; });
        else put_rows<uint16_t>(e, t0, n, f, v, [](float a, const uint16_t *r) { return C16<T>::round(r ? a + C16<T>::one(*r) : a); });
    }
}

template <typename T, int MODE, int OPS> __global__ void __launch_bounds__(kMsThreads, 2) mx_skinny(const __grid_constant__ MsParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using O = Ops<OPS>;
    constexpr int NM = MODE == EPI_GATED ? 2 : 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t S = (uint32_t)p.slots;
    const int rank = (int)cta_rank(), cluster = (int)blockIdx.x / p.cs, clusters = (int)gridDim.x / p.cs;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * p.slotB + p.partB);
    uint64_t *empty = full + kMsRing;
    uint64_t *acc_full = empty + kMsRing, *acc_empty = acc_full + 2;
    uint64_t *part_full = acc_empty + 2, *part_free = part_full + 1;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(part_free + 1);
    MxWalk w(p.tn, NM, p.KT, p.cs, cluster, clusters, rank);
    if (tid == 128) prefetch_map(&p.mw[0]), prefetch_map(&p.mx), prefetch_map(&p.msw[0]), prefetch_map(&p.msx);
    if (tid == 0) {
        for (uint32_t s = 0; s < S; ++s) mbar_init1(full + s), mbar_init1(empty + s);
        for (int s = 0; s < 2; ++s) mbar_init1(acc_full + s), mbar_init(acc_empty + s, 4);
        mbar_init(part_full, max(1, 4 * (p.cs - 1)));                            // each other CTA's warps have sent
        mbar_init(part_free, max(1, 4 * (p.owners - (rank < p.owners ? 1 : 0)))); // each other owner's warps have read
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const uint32_t tmem = tmem_alloc(tslot, p.tcols);
    if (p.cs > 1) cluster_sync(); // all barriers are set up
    if (!(p.early && warp == 4)) pdl_enter();
    const uint32_t base = smem_addr(smem);
    bool ok = true;
    if (warp == 4) {
        Cur cur(0, S);
        uint32_t round = 0;
        constexpr uint32_t sfB = 512u * O::words; // scales of W, and of x, to a step
        const uint32_t bytes = 128u * mx_row_tx(O::nibbles) + (uint32_t)p.Tp * 128u + 2 * sfB, sf = kMsW + (uint32_t)p.Tp * 128u;
        auto load_w = [&](uint32_t s) {
            const uint32_t at = base + s * p.slotB;
            mbar_expect(full + s, bytes);
            tile_load(at, &p.mw[w.m], w.k * 128, w.tile * 128, full + s); // (column: bytes, or codes that are spread)
            tile_load(at + sf, &p.msw[w.m], w.k * 128 * O::words, w.tile, full + s);
        };
        auto load_x = [&](uint32_t s, int k) {
            const uint32_t at = base + s * p.slotB;
            tile_load(at + kMsW, &p.mx, k * 128, 0, full + s);
            tile_load(at + sf + sfB, &p.msx, k * 128 * O::words, 0, full + s);
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
    } else if (warp == 5) {
        const uint32_t id = idesc_mx(O::wfmt, O::xfmt, 128, (uint32_t)p.Tp), sf = base + kMsW + (uint32_t)p.Tp * 128u;
        const uint64_t d0 = sdesc(base, 16, 1024);
        uint32_t set = 0;
        Cur cur(0, S), buf(0, (uint32_t)p.nbuf);
        for (uint32_t it = 0; ok && w.more(); ++it) {
            if (it >= (uint32_t)p.nbuf && !mbar_wait_all(acc_empty + buf.s, buf.ph ^ 1u, p)) break;
            tc_after();
            const int tile = w.tile;
            for (; w.more() && w.tile == tile; w.next()) {
                if (!mbar_wait_all(full + cur.s, cur.ph, p)) {
                    ok = false;
                    break;
                }
                tc_after();
                if (elect_one()) {
                    const uint64_t a = d0 + ((cur.s * p.slotB) >> 4), b = a + (kMsW >> 4);
                    const uint32_t ts = tmem + set * kMsSet, d = tmem + kMsAcc + (uint32_t)((buf.s * NM + w.m) * p.Tp);
#pragma unroll
                    for (int v = 0; v < O::words; ++v) {
                        cp_scales(ts + 4 * v, sf + cur.s * p.slotB + 512 * v);
                        cp_scales(ts + kMsSetX + 4 * v, sf + cur.s * p.slotB + 512 * (O::words + v));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_mx<OPS>(d, a + 2 * j, b + 2 * j, id | sf_id<OPS>(j), ts + 4 * sf_word<OPS>(j),
                                    ts + kMsSetX + 4 * sf_word<OPS>(j), (w.k > w.k0 || j > 0) ? 1u : 0u);
                    mma_commit(empty + cur.s);
                }
                set = (set + 1) & 3;
                __syncwarp();
                cur.next(S);
            }
            if (ok && elect_one()) mma_commit(acc_full + buf.s);
            __syncwarp();
            buf.next((uint32_t)p.nbuf);
        }
    } else {
        const uint32_t part = base + S * p.slotB;
        const int f0 = warp * 32 + lane;
        Cur buf(0, (uint32_t)p.nbuf);
        // this lane's sums of 16 tokens from t0 on
        auto sums = [&](uint32_t b, int m, int t0, float(&v)[16]) {
            tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + kMsAcc + (uint32_t)((b * NM + m) * p.Tp + t0), v);
        };
        // where CTA q keeps what CTA s sends of matrix m, token t (q's own): [s, q left out][m][token][128]
        auto place = [&](int q, int s, int m, int t) {
            return (uint32_t)((((s - (s > q ? 1 : 0)) * NM + m) * p.own + (t - q * p.own)) * 128 + f0) * 4u;
        };
        uint32_t it = 0;
        for (int tile = cluster; tile < p.tn; tile += clusters, ++it) {
            const int f = tile * 128 + f0;
            float bias = 0.f, bias2 = 0.f;
            if (rank < p.owners && f < p.N) {
                if (p.e.bias) bias = C16<T>::one(p.e.bias[f]);
                if (NM == 2 && p.e.bias2) bias2 = C16<T>::one(p.e.bias2[f]);
            }
            ok = warp_wait(acc_full + buf.s, buf.ph, p, lane);
            if (!ok) break;
            tc_after();
            if (p.cs > 1) {
                if (it > 0 && p.owners > (rank < p.owners ? 1 : 0)) {
                    ok = warp_wait_cluster(part_free, (it - 1) & 1, p, lane);
                    if (!ok) break;
                }
                for (int t0 = 0; t0 < p.T; t0 += 16) {
                    const int q = t0 / p.own;
                    if (q == rank) continue;
                    const uint32_t dst = in_cta(part, (uint32_t)q);
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        float v[16];
                        sums(buf.s, m, t0, v);
                        const uint32_t at = dst + place(q, rank, m, t0);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (t0 + i < p.T) st_cluster(at + 512 * i, v[i]);
                    }
                }
                __syncwarp(); // (the arrivals below release what the whole warp wrote)
                if (lane < p.owners && lane != rank) arrive_cluster(in_cta(smem_addr(part_full), (uint32_t)lane));
                if (rank < p.owners) {
                    ok = warp_wait_cluster(part_full, it & 1, p, lane);
                    if (!ok) break;
                }
            }
            const int t1 = min(p.T, (rank + 1) * p.own);
            for (int t0 = rank * p.own; t0 < t1; t0 += 16) {
                float v[NM][16];
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    sums(buf.s, m, t0, v[m]);
                    for (int s = 0; s < p.cs; ++s) {
                        if (s == rank) continue;
                        const uint32_t at = part + place(rank, s, m, t0);
                        float x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (t0 + i < t1) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[i]) : "r"(at + 512 * i) : "memory");
                            else x[i] = 0.f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[m][i] += x[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) v[0][i] += bias;
                acts(p.e.fn, v[0]);
                if (NM == 2) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[0][i] *= v[NM - 1][i] + bias2;
                }
                put16<T, MODE, OPS>(p.e, t0, min(16, t1 - t0), f, p.N, v[0]);
                __syncwarp(); // (some lanes stored: loads from tensor memory take whole warps)
            }
            tc_before();
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(acc_empty + buf.s)) : "memory");
            if (rank < p.owners && lane < p.cs && lane != rank) arrive_cluster(in_cta(smem_addr(part_free), (uint32_t)lane));
            buf.next((uint32_t)p.nbuf);
        }
    }
    settle(p); // copies and MMAs in flight finish before the CTA leaves
    if (p.cs > 1) {
        __syncthreads();
        cluster_sync(); // no CTA leaves while another still writes to it
    }
    tmem_free(tmem, p.tcols);
}

// ------------------------------------------------------------------ host
constexpr int kMsExchange = 12; // steps: 2 to 3 us at about 0.2 us a step of 16 KB

MsParams plan(const Gemm &g, const CtxView &v, const int (&n)[4], int &grid)
{
    MsParams p = {};
    const int words = g.ops == OPS_MX44 ? 2 : 1, nm = g.mode == EPI_GATED ? 2 : 1;
    p.T = g.M, p.Tp = (g.M + 15) / 16 * 16, p.N = g.N;
    p.tn = mx_tiles(g.N), p.KT = (mx_tiles(g.K[0]) + words - 1) / words;
    int clusters = 1;
    p.cs = mx_cluster(p.tn, nm, p.KT, n, 8, kMsExchange, clusters);
    p.own = ((p.T + p.cs - 1) / p.cs + 15) / 16 * 16;
    p.owners = (p.T + p.own - 1) / p.own;
    // half of an SM's shared and tensor memory where that gives a ring of four
    // steps: the next launch's CTAs then wait beside these for their end, their
    // barriers set up (and, with `early`, their first weights loaded)
    const int acc = nm * p.Tp;
    p.slotB = kMsW + (uint32_t)p.Tp * 128u + 1024u * words;
    p.partB = (uint32_t)(p.cs - 1) * nm * p.own * 512u;
    const int half = (v.smem_optin + 1024) / 2 - 2048 - (int)p.partB;
    const bool two = half >= 4 * (int)p.slotB && (int)kMsAcc + acc <= 256;
    p.tcols = two ? 256 : 512;
    p.nbuf = (int)kMsAcc + 2 * acc <= (int)p.tcols ? 2 : 1;
    p.slots = std::min(kMsRing, (two ? half : v.smem_optin - 1024 - (int)p.partB) / (int)p.slotB);
    p.status = v.status, p.abort_flag = v.abort_flag, p.wait_ns = v.wait_ns;
    p.early = g.early;
    p.e = g.e;
    grid = clusters * p.cs;
    return p;
}

// The operands' maps.
cudaError_t maps(const Gemm &g, MsParams &p)
{
    const int xk = g.ops == OPS_MX44 ? PI_MX4 : PI_MX8, wk = g.ops == OPS_MX88 ? PI_MX8 : PI_MX4;
    const int tiles = mx_tiles(g.K[0]), words = g.ops == OPS_MX44 ? 2 : 1;
    cudaError_t e = encode_map_bytes(&p.mx, g.a[0].p, (uint64_t)mx_row_bytes(xk, g.K[0]), (uint64_t)g.M, (uint64_t)g.a[0].ld, (uint32_t)p.Tp);
    if (e == cudaSuccess) e = encode_map_scales(&p.msx, g.sa, tiles, 1, words, 1);
    for (int i = 0; i < (g.mode == EPI_GATED ? 2 : 1) && e == cudaSuccess; ++i) {
        e = g.ops == OPS_MX84 ? encode_map_nibbles(&p.mw[i], g.b[i].p, (uint64_t)tiles * 128, (uint64_t)g.N, (uint64_t)g.b[i].ld, 128)
                              : encode_map_bytes(&p.mw[i], g.b[i].p, (uint64_t)mx_row_bytes(wk, g.K[0]), (uint64_t)g.N, (uint64_t)g.b[i].ld, 128);
        if (e == cudaSuccess) e = encode_map_scales(&p.msw[i], g.sb[i], tiles, p.tn, words, 1);
    }
    return e;
}

template <typename T, int MODE, int OPS> cudaError_t run(const Gemm &g, const CtxView &v)
{
    static std::atomic<uint64_t> ready{0};
    static ClusterCounts known;
    auto kern = mx_skinny<T, MODE, OPS>;
    int n[4], grid = 0;
    cudaError_t e = raise_limit((const void *)kern, ready);
    if (e == cudaSuccess) e = cluster_counts(kern, known, kMsThreads, v, n);
    if (e != cudaSuccess) return e;
    MsParams p = plan(g, v, n, grid);
    e = maps(g, p);
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, grid, p.cs, kMsThreads, (size_t)p.slots * p.slotB + p.partB + (2 * kMsRing + 6) * 8 + 16, v.stream, p);
}

template <int OPS> cudaError_t run_ops(const Gemm &g, bool bf16, const CtxView &v)
{
    if (g.mode == EPI_GATED) return bf16 ? run<__nv_bfloat16, EPI_GATED, OPS>(g, v) : run<__half, EPI_GATED, OPS>(g, v);
    return bf16 ? run<__nv_bfloat16, EPI_LINEAR, OPS>(g, v) : run<__half, EPI_LINEAR, OPS>(g, v);
}

} // namespace

cudaError_t launch_mx_skinny(const Gemm &g, bool bf16, const CtxView &v)
{
    return g.ops == OPS_MX84   ? run_ops<OPS_MX84>(g, bf16, v)
           : g.ops == OPS_MX88 ? run_ops<OPS_MX88>(g, bf16, v)
                               : run_ops<OPS_MX44>(g, bf16, v);
}

} // namespace pi
