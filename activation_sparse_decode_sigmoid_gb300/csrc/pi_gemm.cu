// The matrix product of the block operators with its fused epilogue, on the
// tcgen05 tensor cores:
//     D[m][n] = sum_k A(m, k) B(n, k)   (one or two segments of k)
//
// Bound by the tensor cores for more than about 300 rows of A and of B (2 M N
// K operations on (M K + N K) 2 bytes), by HBM below.  One tile is 256 x 256,
// computed by a pair of CTAs on two SMs (cta_group::2): each holds 128 rows of
// A and 128 of B per 64-element step of k in shared memory, so a step costs
// each SM 32 KB of loads for 256 x 256 x 64 products - half of what a CTA of
// its own with 128 x 256 tiles would load per product.  The gated FFN's pair
// holds 128 rows of Wg in one CTA and of Wu in the other: one accumulator of
// 256 columns carries g and u of the same 128 neurons to the epilogue.
//
// Persistent CTA pairs with fixed roles: warp 8 issues the TMA loads (both
// CTAs), warp 9 of the pair's first CTA the MMAs, warps 0-7 run the epilogue
// of the previous tile out of the other half of tensor memory (2 x 256
// columns).  Six stages of 32 KB.
//
// Tiles past the last whole wave are split along k: their steps, put end to
// end, are cut into equal ranges, one per pair; each pair writes its fp32
// partial tile(s), and gemm_fixup adds them in order and runs the epilogue.
// So a few rows with a long k still use every SM.
//
// Operands may be stored along k or along their rows (the MMA's K-major and
// MN-major forms, 128-byte swizzle), so the backward products read dz, W and
// x as they lie.
//
// A thread of the epilogue holds one row of the accumulator; outputs, and the
// inputs that the epilogue needs (the residual, or g and u), pass through
// shared memory in boxes of 32 x 32 per warp, so that memory sees 64
// consecutive bytes per row.  (Straight from the registers, 16 bytes in each
// of 32 rows at a time, or by TMA stores of such boxes, a 256 x 256 tile took
// 6.5 us or more; its products take 4.3 us at 1024 values of k.)
//
// Every wait is bounded; after one that ran out a pair stops issuing, waits
// for what it has in flight, frees its tensor memory and returns.
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

constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 32 * (kEpiWarps + 2);
constexpr int kStages = 6;
constexpr uint32_t kOpBytes = 16384;            // one operand of one CTA's stage: 128 rows x 64 k
constexpr uint32_t kStageBytes = 2 * kOpBytes;
constexpr uint32_t kAtom = 8192;                // MN-major: 64 rows x 64 k
constexpr int kTile = 256;
constexpr uint32_t kBox = 2048;                 // 32 rows x 32 columns of an epilogue warp
constexpr uint32_t kBoxes = kEpiWarps * 2 * kBox;
constexpr uint32_t kBiasB = 256;                // a warp's 128 bias values (gated: 64 of each)

struct TcParams {
    CUtensorMap ma[2], mb[2];
    int M, N, tm, tn;     // tiles along M and N
    int kt0, KT;          // k steps of the first segment, and of all
    int a_mn, b_mn;
    int nfull;            // tiles computed whole (the first ones)
    int nsplit, parts;    // tiles split along k, and pairs that share them
    int smax;             // partial tiles kept per split tile
    float *part;          // [nsplit][smax][256][256]
    int *status, *abort_flag;
    unsigned long long wait_ns;
    Epi e;
};

// ------------------------------------------------------------------ schedule
// Tile t -> its place: groups of 8 tile rows, down the rows first, so that
// the tiles in flight share operands in L2.
__device__ __forceinline__ void tile_at(int t, int tm, int tn, int &mi, int &ni)
{
    constexpr int kGroup = 8;
    const int per = kGroup * tn, g = t / per, r = t - g * per;
    const int rows = min(kGroup, tm - g * kGroup);
    ni = r / rows;
    mi = g * kGroup + (r - ni * rows);
}

__host__ __device__ inline int range_at(int64_t units, int c, int parts) { return (int)(units * c / parts); }
// the part whose range holds unit u
__host__ __device__ inline int part_of(int64_t units, int64_t u, int parts)
{
    return (int)(((u + 1) * parts + units - 1) / units - 1);
}

struct Work {
    int tile, k0, k1, slot; // slot < 0: a whole tile
};

// The work of pair c of n, in order; every role of both CTAs walks it alike.
struct Walk {
    const TcParams &p;
    int t, n, u, u1, c;
    __device__ __forceinline__ Walk(const TcParams &q, int c_, int n_) : p(q), t(c_), n(n_), u(0), u1(0), c(c_)
    {
        if (c < p.parts) {
            const int64_t units = (int64_t)p.nsplit * p.KT;
            u = range_at(units, c, p.parts);
            u1 = range_at(units, c + 1, p.parts);
        }
    }
    __device__ __forceinline__ bool next(Work &w)
    {
        if (t < p.nfull) {
            w = {t, 0, p.KT, -1};
            t += n;
            return true;
        }
        if (u >= u1) return false;
        const int r = u / p.KT, k0 = u - r * p.KT;
        const int k1 = min(p.KT, k0 + u1 - u);
        const int first = part_of((int64_t)p.nsplit * p.KT, (int64_t)r * p.KT, p.parts);
        w = {p.nfull + r, k0, k1, r * p.smax + (c - first)};
        u += k1 - k0;
        return true;
    }
};

// ------------------------------------------------------------------ pair helpers
__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// address of the first CTA's copy of a shared-memory object
__device__ __forceinline__ uint32_t in_first(uint32_t addr)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// a box of 64 columns into this CTA's shared memory; the bytes count on `bar`, which may be the first CTA's
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap *tm, int col, int row, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                 " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(tm), "r"(bar), "r"(col), "r"(row)
                 : "memory");
}

__device__ __forceinline__ void mma2(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{ .reg .pred q; setp.ne.b32 q, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, q; }" ::"r"(
                     d_tmem),
                 "l"(a), "l"(b), "r"(id), "r"(acc));
}

// arrives on the same barrier of both CTAs once the MMAs issued so far are done
__device__ __forceinline__ void commit2(uint64_t *b)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_addr(b)),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
                   "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                   "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// After a failure: copies and MMAs in flight finish within microseconds; the
// CTA stays for a bounded time that covers them.
__device__ __forceinline__ void linger()
{
    const uint64_t t0 = gtimer();
    while (gtimer() - t0 < 5000000ull) {
    }
}

// ------------------------------------------------------------------ boxes of the epilogue
// A warp's box: row r at 64 r, 16-byte chunk j at j ^ ((r >> 1) & 3): 8 lanes'
// chunks fall into different banks, by rows and by chunks of a row.
__device__ __forceinline__ uint32_t box_at(uint32_t box, int r, int j) { return box + r * 64 + ((j ^ ((r >> 1) & 3)) << 4); }

__device__ __forceinline__ void sts16(uint32_t at, const uint4 &q)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 q;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}

// 32 columns of this thread's row into the box
template <typename T> __device__ __forceinline__ void box_put(uint32_t box, int lane, const float (&v)[32])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) sts16(box_at(box, lane, j), pack8<T>(*reinterpret_cast<const float(*)[8]>(v + 8 * j)));
}

// A matrix that the epilogue reads or writes, seen from a warp: lane l moves
// chunk l mod 4 of rows l / 4, l / 4 + 8, ...; rows that are not 16-byte
// aligned, and the last columns of others, element by element.
struct Strip {
    uint16_t *p;
    int64_t ld;
    bool vec;
};

// 32 x 32 values at (row, col) on their way into the box: loads now, box later
__device__ __forceinline__ void strip_load(const Strip &s, int lane, int row, int col, int M, int N, uint4 (&q)[4])
{
    const int c = col + (lane & 3) * 8, n = N - c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = row + i * 8 + (lane >> 2);
        q[i] = make_uint4(0, 0, 0, 0);
        if (r >= M || n <= 0) continue;
        const uint16_t *p = s.p + r * s.ld + c;
        if (s.vec && n >= 8) q[i] = *reinterpret_cast<const uint4 *>(p);
        else {
            uint32_t w[4] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
            q[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

__device__ __forceinline__ void strip_to_box(uint32_t box, int lane, const uint4 (&q)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) sts16(box_at(box, i * 8 + (lane >> 2), lane & 3), q[i]);
}

// The box into rows [row, row + 32), columns [col, col + 32); what lies
// outside is left out.  inside: nothing does.
__device__ __forceinline__ void box_send(uint32_t box, const Strip &s, int lane, int row, int col, int M, int N, bool inside)
{
    __syncwarp();
    const int c = col + (lane & 3) * 8, n = N - c;
    if (s.vec && inside) {
        // (rows 8 apart lie 512 bytes apart in the box, their chunks alike)
        const uint32_t at = box_at(box, lane >> 2, lane & 3);
        uint16_t *p = s.p + (int64_t)(row + (lane >> 2)) * s.ld + c;
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = lds16(at + 512 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i, p += 8 * s.ld) *reinterpret_cast<uint4 *>(p) = q[i];
    } else if (s.vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row + i * 8 + (lane >> 2);
            if (r >= M || n <= 0) continue;
            const uint4 q = lds16(box_at(box, i * 8 + (lane >> 2), lane & 3));
            uint16_t *p = s.p + r * s.ld + c;
            if (n >= 8) *reinterpret_cast<uint4 *>(p) = q;
            else {
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
            }
        }
    } else if (col + lane < N) {
        uint16_t *o = s.p + row * s.ld + col + lane;
        const int rows = min(32, M - row);
#pragma unroll 8
        for (int r = 0; r < rows; ++r, o += s.ld) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(box_at(box, r, lane >> 3) + (lane & 7) * 2) : "memory");
            *o = v;
        }
    }
    __syncwarp();
}

// ------------------------------------------------------------------ the kernel
template <typename T, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1) gemm_tc(const __grid_constant__ TcParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using H = H16<T>;
    constexpr int kOutN = MODE == EPI_GATED ? 128 : kTile; // output columns of a tile
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cta_rank();
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes + kBoxes + kEpiWarps * kBiasB); // used in the first CTA
    uint64_t *empty = full + kStages;
    uint64_t *acc_full = empty + kStages;  // [2]
    uint64_t *acc_empty = acc_full + 2;    // [2], used in the first CTA
    uint32_t *tslot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    if (warp == kEpiWarps && lane == 0) {
        // the maps are on their way while the rest is set up
        prefetch_map(&p.ma[0]), prefetch_map(&p.mb[0]);
        if (p.kt0 < p.KT || MODE == EPI_GATED) prefetch_map(&p.ma[1]), prefetch_map(&p.mb[1]);
    }
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init1(full + s), mbar_init1(empty + s);
        for (int s = 0; s < 2; ++s) mbar_init1(acc_full + s), mbar_init(acc_empty + s, 2 * kEpiWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_before();
    __syncthreads();
    cluster_sync(); // both CTAs' barriers are set up
    tc_after();
    const uint32_t tmem = *(volatile uint32_t *)tslot;
    pdl_enter();

    const uint32_t base = smem_addr(smem);
    Walk walk(p, (int)blockIdx.x >> 1, (int)gridDim.x >> 1);
    Work w;
    bool ok = true;
    if (warp == kEpiWarps) {
        const uint32_t full0 = in_first(smem_addr(full));
        Cur cur(0, kStages);
        uint32_t round = 0;
        while (ok && walk.next(w)) {
            int mi, ni;
            tile_at(w.tile, p.tm, p.tn, mi, ni);
            const int m0 = mi * kTile + (int)rank * 128;
            const int n0 = ni * kOutN + (MODE == EPI_GATED ? 0 : (int)rank * 128);
            for (int seg = 0; seg < 2; ++seg) {
                const int lo = seg ? p.kt0 : 0, ka = max(w.k0, lo), kb = min(w.k1, seg ? p.KT : p.kt0);
                const CUtensorMap *ma = &p.ma[seg], *mb = &p.mb[MODE == EPI_GATED ? (int)rank : seg];
                for (int k = ka; k < kb; ++k) {
                    if (round >= kStages && !mbar_wait_all(empty + cur.s, cur.ph ^ 1u, p)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t bar = full0 + cur.s * 8, sa = base + cur.s * kStageBytes, sb = sa + kOpBytes;
                        const int kc = (k - lo) * kBK;
                        if (rank == 0) mbar_expect(full + cur.s, 2 * kStageBytes);
                        if (p.a_mn) {
                            pair_load(sa, ma, m0, kc, bar);
                            pair_load(sa + kAtom, ma, m0 + 64, kc, bar);
                        } else
                            pair_load(sa, ma, kc, m0, bar);
                        if (p.b_mn) {
                            pair_load(sb, mb, n0, kc, bar);
                            pair_load(sb + kAtom, mb, n0 + 64, kc, bar);
                        } else
                            pair_load(sb, mb, kc, n0, bar);
                    }
                    __syncwarp();
                    cur.next(kStages);
                    ++round;
                }
            }
        }
        // the MMAs' arrivals on this CTA's barriers land before it leaves
        for (uint32_t i = min(round, (uint32_t)kStages); ok && i > 0; --i) {
            const Cur last(round - i, kStages);
            ok = mbar_wait_all(empty + last.s, last.ph, p);
        }
    } else if (warp == kEpiWarps + 1) {
        if (rank == 0) {
            const uint32_t id = idesc(H::fmt, (uint32_t)p.a_mn, (uint32_t)p.b_mn, 256, 256);
            // descriptors of stage 0; a byte offset o adds o / 16 (the start address field)
            const uint64_t da = p.a_mn ? sdesc(base, kAtom, 1024) : sdesc(base, 16, 1024);
            const uint64_t db = p.b_mn ? sdesc(base + kOpBytes, kAtom, 1024) : sdesc(base + kOpBytes, 16, 1024);
            const uint32_t ka = p.a_mn ? 128 : 2, kb = p.b_mn ? 128 : 2; // 16 elements of k
            Cur cur(0, kStages);
            for (uint32_t it = 0; ok && walk.next(w); ++it) {
                const uint32_t buf = it & 1, ph = (it >> 1) & 1;
                if (it >= 2 && !mbar_wait_all(acc_empty + buf, ph ^ 1u, p)) {
                    ok = false;
                    break;
                }
                tc_after();
                const uint32_t d = tmem + buf * 256u;
                for (int k = w.k0; k < w.k1; ++k) {
                    if (!mbar_wait_all(full + cur.s, cur.ph, p)) {
                        ok = false;
                        break;
                    }
                    tc_after();
                    if (elect_one()) {
                        const uint32_t so = (cur.s * kStageBytes) >> 4;
#pragma unroll
                        for (int j = 0; j < kBK / 16; ++j)
                            mma2(d, da + so + j * ka, db + so + j * kb, id, (k > w.k0 || j > 0) ? 1u : 0u);
                        commit2(empty + cur.s);
                    }
                    __syncwarp();
                    cur.next(kStages);
                }
                if (ok && elect_one()) commit2(acc_full + buf);
                __syncwarp();
            }
        }
    } else {
        // epilogue: warp w reads TMEM lanes 32 (w mod 4) .., the first or second half of the columns
        const int q = warp & 3, half = warp >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t box0 = base + kStages * kStageBytes + (uint32_t)warp * 2 * kBox, box1 = box0 + kBox;
        const Epi &e = p.e;
        const bool two = MODE == EPI_DACT && e.in2, out32 = MODE == EPI_LINEAR && e.out32;
        const bool has_in = MODE == EPI_DACT || (MODE == EPI_LINEAR && e.res && !out32);
        const Strip out = {static_cast<uint16_t *>(e.out), e.ldo, (e.vec & V_OUT) != 0};
        const Strip out2 = {e.out2, e.ld2, (e.vec & V_OUT2) != 0}, out3 = {e.out3, e.ld3, (e.vec & V_OUT3) != 0};
        const Strip in1 = MODE == EPI_DACT ? Strip{const_cast<uint16_t *>(e.in1), e.ldi1, (e.vec & V_IN1) != 0}
                                           : Strip{static_cast<uint16_t *>(const_cast<void *>(e.res)), e.ldr, (e.vec & V_RES) != 0};
        const Strip in2 = {const_cast<uint16_t *>(e.in2), e.ldi2, (e.vec & V_IN2) != 0};
        constexpr int kCols = kOutN / 2; // of this warp
        const uint32_t bias = base + kStages * kStageBytes + kBoxes + (uint32_t)warp * kBiasB;
        const bool biased = MODE != EPI_DACT && (e.bias || e.bias2);
        for (uint32_t it = 0; ok && walk.next(w); ++it) {
            const uint32_t buf = it & 1, ph = (it >> 1) & 1;
            int mi, ni;
            tile_at(w.tile, p.tm, p.tn, mi, ni);
            const int row0 = mi * kTile + (int)rank * 128 + q * 32, col0 = ni * kOutN + half * kCols;
            const bool whole = w.slot < 0;
            uint4 q1[4], q2[4]; // the next chunk's inputs
            if (whole && has_in) { // in flight while the products finish
                strip_load(in1, lane, row0, col0, p.M, p.N, q1);
                if (two) strip_load(in2, lane, row0, col0, p.M, p.N, q2);
            }
            if (whole && biased) { // 4 values a lane
                const int h = MODE == EPI_GATED ? lane >> 4 : 0, k = (MODE == EPI_GATED ? lane & 15 : lane) * 4;
                const uint16_t *src = h ? e.bias2 : e.bias;
                uint32_t b[2] = {};
                if (src) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (col0 + k + i < p.N) b[i >> 1] |= (uint32_t)src[col0 + k + i] << (16 * (i & 1));
                }
                __syncwarp();
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(bias + lane * 8), "r"(b[0]), "r"(b[1]) : "memory");
                __syncwarp();
            }
            ok = warp_wait(acc_full + buf, ph, p, lane);
            if (!ok) break;
            tc_after();
            const uint32_t ta = lane_addr + buf * 256u;
            bool released = false;
            if (!whole) {
                const int r = (int)rank * 128 + q * 32 + lane; // row within the tile
                float *dst = p.part + ((size_t)w.slot * kTile + r) * kTile;
#pragma unroll 1
                for (int c = half * 128; c < half * 128 + 128; c += 32) {
                    float v[32];
                    tmem_ld32(ta + c, v);
                    if (row0 + lane < p.M) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(dst + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                }
            } else if (row0 < p.M) {
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    const int col = col0 + c;
                    if (col >= p.N) break;
                    const bool inside = row0 + 32 <= p.M && col + 32 <= p.N;
                    float v[32], u[MODE == EPI_GATED ? 32 : 1];
                    tmem_ld32(ta + half * kCols + c, v);
                    if (MODE == EPI_GATED) tmem_ld32(ta + 128 + half * kCols + c, *reinterpret_cast<float(*)[32]>(u));
                    if (c + 32 >= kCols || col + 32 >= p.N) {
                        // the accumulator is in registers: the next tile's products may begin
                        tc_before();
                        __syncwarp();
                        if (lane == 0) arrive_cluster(in_first(smem_addr(acc_empty + buf)));
                        released = true;
                    }
                    if (has_in) {
                        strip_to_box(box0, lane, q1);
                        if (two) strip_to_box(box1, lane, q2);
                        if (!released) {
                            strip_load(in1, lane, row0, col + 32, p.M, p.N, q1);
                            if (two) strip_load(in2, lane, row0, col + 32, p.M, p.N, q2);
                        }
                        __syncwarp();
                    }
                    if (biased) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float b[8];
                            unpack8<T>(lds16(bias + 2 * (c + 8 * j)), b);
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[8 * j + i] += b[i];
                            if (MODE == EPI_GATED) {
                                unpack8<T>(lds16(bias + 128 + 2 * (c + 8 * j)), b);
#pragma unroll
                                for (int i = 0; i < 8; ++i) u[(8 * j + i) % (MODE == EPI_GATED ? 32 : 1)] += b[i];
                            }
                        }
                    }
                    if (MODE != EPI_DACT && e.out2) {
                        box_put<T>(box1, lane, v);
                        box_send(box1, out2, lane, row0, col, p.M, p.N, inside);
                    }
                    if (MODE == EPI_GATED && e.out3) {
                        box_put<T>(box1, lane, *reinterpret_cast<float(*)[32]>(u));
                        box_send(box1, out3, lane, row0, col, p.M, p.N, inside);
                    }
                    if (MODE == EPI_DACT) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float g[8], f[8], df[8];
                            unpack8<T>(lds16(box_at(box0, lane, j)), g);
                            both8(e.fn, g, f, df);
                            if (two) {
                                float s[8];
                                unpack8<T>(lds16(box_at(box1, lane, j)), s);
#pragma unroll
                                for (int i = 0; i < 8; ++i) f[i] *= v[8 * j + i], v[8 * j + i] *= s[i] * df[i];
                                sts16(box_at(box1, lane, j), pack8<T>(f)); // du
                            } else {
#pragma unroll
                                for (int i = 0; i < 8; ++i) v[8 * j + i] *= e.scale * df[i];
                            }
                        }
                        if (two) box_send(box1, out2, lane, row0, col, p.M, p.N, inside);
                    } else {
                        if (e.fn != PI_FN_NONE) acts(e.fn, v);
                        if (MODE == EPI_GATED) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= u[i % (MODE == EPI_GATED ? 32 : 1)];
                        } else {
                            if (e.scale != 1.f) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] *= e.scale;
                            }
                            if (out32) {
                                if (row0 + lane < p.M)
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        const int cj = col + 8 * j;
                                        if (cj >= p.N) break;
                                        float(&x)[8] = *reinterpret_cast<float(*)[8]>(v + 8 * j);
                                        if (e.res) {
                                            float r[8];
                                            load8f(static_cast<const float *>(e.res) + (int64_t)(row0 + lane) * e.ldr + cj, p.N - cj, e.vec & V_RES, r);
#pragma unroll
                                            for (int i = 0; i < 8; ++i) x[i] += r[i];
                                        }
                                        store8f(static_cast<float *>(e.out) + (int64_t)(row0 + lane) * e.ldo + cj, p.N - cj, e.vec & V_OUT, x);
                                    }
                                continue;
                            }
                            if (has_in) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    float r[8];
                                    unpack8<T>(lds16(box_at(box0, lane, j)), r);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) v[8 * j + i] += r[i];
                                }
                            }
                        }
                    }
                    box_put<T>(box0, lane, v);
                    box_send(box0, out, lane, row0, col, p.M, p.N, inside);
                }
            }
            if (!released) {
                tc_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(in_first(smem_addr(acc_empty + buf)));
            }
        }
    }
    __syncwarp();
    if (*(volatile int *)p.abort_flag) linger();
    tc_before();
    __syncthreads();
    cluster_sync(); // neither CTA leaves while the other still reads its shared or tensor memory
    tc_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// The split tiles: partials added in the order of k, then the epilogue.
// 256 threads take 8 columns each of 8 (gated: 16) rows.
template <typename T, int MODE> __global__ void __launch_bounds__(256) gemm_fixup(const __grid_constant__ TcParams p)
{
    pdl_enter();
    constexpr int kOutN = MODE == EPI_GATED ? 128 : kTile, kCols = kOutN / 8, kRows = 256 / kCols;
    const int per = kTile / kRows, r = (int)blockIdx.x / per;
    const int row = ((int)blockIdx.x % per) * kRows + threadIdx.x / kCols, c = (threadIdx.x % kCols) * 8;
    int mi, ni;
    tile_at(p.nfull + r, p.tm, p.tn, mi, ni);
    const int grow = mi * kTile + row, gcol = ni * kOutN + c;
    if (grow >= p.M || gcol >= p.N) return;
    const int64_t units = (int64_t)p.nsplit * p.KT;
    const int cnt = part_of(units, (int64_t)(r + 1) * p.KT - 1, p.parts) - part_of(units, (int64_t)r * p.KT, p.parts) + 1;
    float v[8] = {}, u[8] = {};
    const float *src = p.part + ((size_t)r * p.smax * kTile + row) * kTile + c;
    for (int s = 0; s < cnt; ++s, src += kTile * kTile) {
        float t[8];
        load8f(src, 8, true, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
        if (MODE == EPI_GATED) {
            load8f(src + 128, 8, true, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] += t[i];
        }
    }
    epilogue8<T, MODE>(p.e, p.N, grow, gcol, v, u);
}

// ------------------------------------------------------------------ host
// The tiles that are split along k, and over how many pairs.  A last wave of
// `rem` tiles on n pairs would take KT steps; split, it takes rem KT / n and
// the fixup launch with its traffic, worth about kFixupSteps steps.
constexpr int kFixupSteps = 32;
constexpr int kMinShare = 4; // k steps per pair, at least

struct Split {
    int tm, tn, KT, kt0, nfull, nsplit, parts, smax;
    size_t bytes;
};

Split plan_split(const Gemm &g, int sms)
{
    Split s = {};
    const int n = sms / 2, outn = g.mode == EPI_GATED ? 128 : kTile;
    s.tm = (g.M + kTile - 1) / kTile;
    s.tn = (g.N + outn - 1) / outn;
    s.kt0 = (g.K[0] + kBK - 1) / kBK;
    s.KT = s.kt0 + (g.segs > 1 ? (g.K[1] + kBK - 1) / kBK : 0);
    const int tiles = s.tm * s.tn, rem = tiles % n;
    s.nfull = tiles;
    s.smax = 1;
    if (rem && (int64_t)s.KT * (n - rem) > (int64_t)kFixupSteps * n) {
        s.nfull = tiles - rem;
        s.nsplit = rem;
        const int64_t units = (int64_t)rem * s.KT;
        s.parts = (int)std::min<int64_t>(n, std::max<int64_t>(1, units / kMinShare));
        const int share = (int)(units / s.parts); // the smallest range
        s.smax = s.KT / share + 2;
        s.bytes = (size_t)rem * s.smax * kTile * kTile * sizeof(float);
    }
    return s;
}

cudaError_t map_of(CUtensorMap *m, const Mat &a, int rows, int K)
{
    return a.mn ? encode_map(m, a.p, (uint64_t)rows, (uint64_t)K, (uint64_t)a.ld * 2, 64)
                : encode_map(m, a.p, (uint64_t)K, (uint64_t)rows, (uint64_t)a.ld * 2, 128);
}

template <typename T, int MODE> cudaError_t run(const TcParams &p, int pairs, cudaStream_t s)
{
    constexpr int smem = kStages * kStageBytes + kBoxes + kEpiWarps * kBiasB + (2 * kStages + 4) * 8 + 16;
    auto kern = gemm_tc<T, MODE>;
    static std::atomic<uint64_t> ready{0}; // devices whose limit has been raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1))) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev);
    }
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(2 * pairs), dim3(kGemmThreads), smem, s, p);
    if (e != cudaSuccess || !p.nsplit) return e;
    constexpr int kCols = (MODE == EPI_GATED ? 128 : kTile) / 8;
    return launch_pdl(gemm_fixup<T, MODE>, dim3(p.nsplit * kTile / (256 / kCols)), dim3(256), 0, s, p);
}

template <typename T> cudaError_t run_mode(const Gemm &g, const TcParams &p, int pairs, cudaStream_t s)
{
    return g.mode == EPI_LINEAR ? run<T, EPI_LINEAR>(p, pairs, s)
           : g.mode == EPI_GATED ? run<T, EPI_GATED>(p, pairs, s)
                                 : run<T, EPI_DACT>(p, pairs, s);
}

} // namespace

size_t gemm_workspace(const Gemm &g, const CtxView &v)
{
    return skinny_takes(g) ? skinny_workspace(g, v) : plan_split(g, v.sms).bytes;
}

cudaError_t launch_gemm(const Gemm &g, bool bf16, const CtxView &v, void *ws)
{
    if (skinny_takes(g)) return launch_skinny(g, bf16, v, ws);
    const Split s = plan_split(g, v.sms);
    TcParams p = {};
    p.M = g.M, p.N = g.N, p.tm = s.tm, p.tn = s.tn, p.kt0 = s.kt0, p.KT = s.KT;
    p.a_mn = g.a[0].mn, p.b_mn = g.b[0].mn;
    p.nfull = s.nfull, p.nsplit = s.nsplit, p.parts = s.parts, p.smax = s.smax;
    p.part = static_cast<float *>(ws);
    p.status = v.status, p.abort_flag = v.abort_flag, p.wait_ns = v.wait_ns;
    p.e = g.e;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < g.segs && e == cudaSuccess; ++i) e = map_of(&p.ma[i], g.a[i], g.M, g.K[i]);
    const int nb = g.mode == EPI_GATED ? 2 : g.segs;
    for (int i = 0; i < nb && e == cudaSuccess; ++i)
        e = map_of(&p.mb[i], g.b[i], g.N, g.K[g.mode == EPI_GATED ? 0 : i]);
    if (e != cudaSuccess) return e;
    const int pairs = std::min(v.sms / 2, std::max(std::min(p.nfull, v.sms / 2), p.parts));
    return bf16 ? run_mode<__nv_bfloat16>(g, p, pairs, v.stream) : run_mode<__half>(g, p, pairs, v.stream);
}

} // namespace pi
