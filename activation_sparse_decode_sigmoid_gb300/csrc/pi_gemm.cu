// The matrix product of the block operators with its fused epilogue, on the
// tcgen05 tensor cores:
//     D[m][n] = sum_k A(m, k) B(n, k)   (one or two segments of k)
//
// Bound by the tensor cores for more than about 300 rows of A and of B (2 M N
// K operations on (M K + N K) 2 bytes), by HBM below.  One tile is 256 x 256
// (256 x 128 where those would leave half of the SMs idle, see plan_group),
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
// One launch takes up to four products that do not wait for one another (a
// backward pass's gradients of x and of the weights): their tiles are dealt to
// the pairs longest first, so that one product's last, partly filled wave is
// filled by the next.
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
// A thread of the epilogue holds one row of the accumulator.  Plain outputs
// leave through shared memory by TMA stores of 32 x 64 boxes; the others, and
// the inputs that the epilogue needs (the residual, or g and u), pass through
// boxes of 32 x 32 per warp, so that memory sees 64 consecutive bytes per row.
// (Straight from the registers, 16 bytes in each of 32 rows at a time, or by
// TMA stores of 32 x 32 boxes, a 256 x 256 tile took 6.5 us or more; its
// products take 4.3 us at 1024 values of k.)  fp32 outputs, and the fp32 stream
// they are added to, still go straight from the registers: 4096 x 1024 -> 8192
// takes 162 us into an fp32 stream, 56 in 16 bits; 2048 x 28672 -> 8192, whose
// products hide it, 545 and 525.
//
// Every wait is bounded; after one that ran out a pair stops issuing, waits
// for what it has in flight, frees its tensor memory and returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <numeric>

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

constexpr int kMaxProbs = 4;

struct Prob {
    CUtensorMap ma[2], mb[2];
    CUtensorMap mo;       // the output, for tiles that are only rounded (16-byte aligned rows)
    int M, N, tm, tn;     // tiles along M and N
    int kt0, KT;          // k steps of the first segment, and of all
    int a_mn, b_mn;
    Epi e;
};

// Tiles tile0 + i, i < count, of a product, computed whole: by pair (pair0 + i mod npairs) mod all pairs.
struct Deal {
    int prob, tile0, count, pair0, npairs;
};

// How a group of products is cut.
struct Sched {
    Deal deal[2 * kMaxProbs];
    int ndeal, pairs;     // pairs that tiles are dealt to
    int sprob, stile0;    // the product whose last tiles are split along k, the first of them
    int nsplit, parts;    // how many, and pairs that share them (each lane's)
    int lanes;            // split tiles in a row that are cut alike, each by pairs of its own
    int smax;             // partial tiles kept per split tile
};

template <int NP> struct TcParams {
    Prob prob[NP];
    Sched s;
    float *part;          // [nsplit][smax][256 / 4 columns][256 rows][4]: a warp's 32 rows write 512 bytes in a row
    int *status, *abort_flag;
    unsigned long long wait_ns;
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
    int prob, tile, k0, k1, slot; // slot < 0: a whole tile
};

// The work of pair c, in order; every role of both CTAs walks it alike.
template <int NP> struct Walk {
    const TcParams<NP> &p;
    int c, d, i, u, u1;
    __device__ __forceinline__ Walk(const TcParams<NP> &q, int c_) : p(q), c(c_), d(0), u(0), u1(0)
    {
        i = first(0);
        if (c < p.s.parts * p.s.lanes) {
            const int64_t units = (int64_t)(p.s.nsplit / p.s.lanes) * p.prob[NP == 1 ? 0 : p.s.sprob].KT;
            u = range_at(units, c / p.s.lanes, p.s.parts);
            u1 = range_at(units, c / p.s.lanes + 1, p.s.parts);
        }
    }
    // this pair's first index in deal d
    __device__ __forceinline__ int first(int d_) const
    {
        const Deal &e = p.s.deal[d_];
        int pos = c - e.pair0;
        pos += pos < 0 ? p.s.pairs : 0;
        return pos < e.npairs ? pos : 0x7fffffff;
    }
    __device__ __forceinline__ bool next(Work &w)
    {
        while (d < p.s.ndeal) {
            const Deal &e = p.s.deal[d];
            if (i < e.count) {
                w = {NP == 1 ? 0 : e.prob, e.tile0 + i, 0, p.prob[NP == 1 ? 0 : e.prob].KT, -1};
                i += e.npairs;
                return true;
            }
            if (++d < p.s.ndeal) i = first(d);
        }
        if (u >= u1) return false;
        const int KT = p.prob[NP == 1 ? 0 : p.s.sprob].KT;
        const int q = u / KT, k0 = u - q * KT, lane = c % p.s.lanes;
        const int k1 = min(KT, k0 + u1 - u), r = q * p.s.lanes + lane;
        const int lead = part_of((int64_t)(p.s.nsplit / p.s.lanes) * KT, (int64_t)q * KT, p.s.parts);
        w = {p.s.sprob, p.s.stile0 + r, k0, k1, r * p.s.smax + (c / p.s.lanes - lead)};
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

// The same without the wait: tmem_wait32 before the values are used.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
                   "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                   "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
// (the registers are operands, so that no use of them moves in front of the wait)
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
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

// what TMA stores still read from the warp's box
__device__ __forceinline__ void box_settle(int lane)
{
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// A warp's 32 x COLS values, rounded and nothing else, all inside the output:
// 64 columns at a time through the warp's 4 KB (128-byte swizzle) and out by a
// TMA store, the next 32 columns on their way out of tensor memory meanwhile.
// (By the warps' own stores, 64 bytes a row, a tile took 2.7 us.)  `last` runs
// once the accumulator has been read.
template <typename T, int COLS, typename F>
__device__ __forceinline__ void plain_strip(uint32_t ta, uint32_t box, const CUtensorMap *mo, int lane, int row, int col, F last)
{
    uint32_t r[2][32];
    tmem_ld32_async(ta, r[0]);
    box_settle(lane);
    tmem_wait32(r[0]);
#pragma unroll
    for (int c = 0; c < COLS / 32; ++c) {
        uint32_t(&v)[32] = r[c & 1];
        if (c < COLS / 32 - 1) tmem_ld32_async(ta + 32 * (c + 1), r[(c + 1) & 1]);
        else last();
        if (c && !(c & 1)) box_settle(lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[8 * j + i]);
            sts16(box + lane * 128 + ((((c & 1) * 4 + j) ^ (lane & 7)) << 4), pack8<T>(x));
        }
        if (c & 1) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(mo), "r"(box),
                             "r"(col + 64 * (c >> 1)), "r"(row)
                             : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        }
        if (c < COLS / 32 - 1) tmem_wait32(r[(c + 1) & 1]);
    }
    __syncwarp();
}

// ------------------------------------------------------------------ the kernel
// WIDE: columns of a tile's accumulator, 256 or 128.
template <typename T, int MODE, int NP, int WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1) gemm_tc(const __grid_constant__ TcParams<NP> p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using H = H16<T>;
    constexpr int kOutN = MODE == EPI_GATED ? 128 : WIDE; // output columns of a tile
    constexpr bool kPlain = NP > 1; // a backward pass's products: no bias, activation, scale or z
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cta_rank();
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes + kBoxes + kEpiWarps * kBiasB); // used in the first CTA
    uint64_t *empty = full + kStages;
    uint64_t *acc_full = empty + kStages;  // [2]
    uint64_t *acc_empty = acc_full + 2;    // [2], used in the first CTA
    uint32_t *tslot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    if (warp == kEpiWarps && lane == 0) {
        // the maps are on their way while the rest is set up
        const Prob &pr = p.prob[NP == 1 ? 0 : p.s.ndeal ? p.s.deal[0].prob : p.s.sprob];
        prefetch_map(&pr.ma[0]), prefetch_map(&pr.mb[0]);
        if (MODE == EPI_GATED) prefetch_map(&pr.mb[1]);
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
    Walk<NP> walk(p, (int)blockIdx.x >> 1);
    Work w;
    bool ok = true;
    if (warp == kEpiWarps) {
        const uint32_t full0 = in_first(smem_addr(full));
        Cur cur(0, kStages);
        uint32_t round = 0;
        while (ok && walk.next(w)) {
            const Prob &pr = p.prob[NP == 1 ? 0 : w.prob];
            int mi, ni;
            tile_at(w.tile, pr.tm, pr.tn, mi, ni);
            const int m0 = mi * kTile + (int)rank * 128;
            const int n0 = ni * kOutN + (MODE == EPI_GATED ? 0 : (int)rank * (WIDE / 2));
            for (int seg = 0; seg < 2 && ok; ++seg) {
                const int lo = seg ? pr.kt0 : 0, ka = max(w.k0, lo), kb = min(w.k1, seg ? pr.KT : pr.kt0);
                const CUtensorMap *ma = &pr.ma[seg], *mb = &pr.mb[MODE == EPI_GATED ? (int)rank : seg];
                for (int k = ka; k < kb; ++k) {
                    if (round >= kStages && !mbar_wait_all(empty + cur.s, cur.ph ^ 1u, p)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t bar = full0 + cur.s * 8, sa = base + cur.s * kStageBytes, sb = sa + kOpBytes;
                        const int kc = (k - lo) * kBK;
                        if (rank == 0) mbar_expect(full + cur.s, 2 * kOpBytes + WIDE * kBK * 2);
                        if (pr.a_mn) {
                            pair_load(sa, ma, m0, kc, bar);
                            pair_load(sa + kAtom, ma, m0 + 64, kc, bar);
                        } else
                            pair_load(sa, ma, kc, m0, bar);
                        if (pr.b_mn) {
                            pair_load(sb, mb, n0, kc, bar);
                            if (WIDE == kTile) pair_load(sb + kAtom, mb, n0 + 64, kc, bar);
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
            Cur cur(0, kStages);
            for (uint32_t it = 0; ok && walk.next(w); ++it) {
                const Prob &pr = p.prob[NP == 1 ? 0 : w.prob];
                const uint32_t id = idesc(H::fmt, (uint32_t)pr.a_mn, (uint32_t)pr.b_mn, 256, WIDE);
                // descriptors of stage 0; a byte offset o adds o / 16 (the start address field)
                const uint64_t da = pr.a_mn ? sdesc(base, kAtom, 1024) : sdesc(base, 16, 1024);
                const uint64_t db = pr.b_mn ? sdesc(base + kOpBytes, kAtom, 1024) : sdesc(base + kOpBytes, 16, 1024);
                const uint32_t ka = pr.a_mn ? 128 : 2, kb = pr.b_mn ? 128 : 2; // 16 elements of k
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
        constexpr int kCols = kOutN / 2; // of this warp
        const uint32_t bias = base + kStages * kStageBytes + kBoxes + (uint32_t)warp * kBiasB;
        for (uint32_t it = 0; ok && walk.next(w); ++it) {
            const Prob &pr = p.prob[NP == 1 ? 0 : w.prob];
            const int M = pr.M, N = pr.N;
            const Epi &e = pr.e;
            const bool two = MODE == EPI_DACT && e.in2, out32 = MODE == EPI_LINEAR && e.out32;
            const bool has_in = MODE == EPI_DACT || (MODE == EPI_LINEAR && e.res && !out32);
            const Strip out = {static_cast<uint16_t *>(e.out), e.ldo, (e.vec & V_OUT) != 0};
            const Strip out2 = {e.out2, e.ld2, (e.vec & V_OUT2) != 0}, out3 = {e.out3, e.ld3, (e.vec & V_OUT3) != 0};
            const Strip in1 = MODE == EPI_DACT ? Strip{const_cast<uint16_t *>(e.in1), e.ldi1, (e.vec & V_IN1) != 0}
                                               : Strip{static_cast<uint16_t *>(const_cast<void *>(e.res)), e.ldr, (e.vec & V_RES) != 0};
            const Strip in2 = {const_cast<uint16_t *>(e.in2), e.ldi2, (e.vec & V_IN2) != 0};
            const bool biased = !kPlain && MODE != EPI_DACT && (e.bias || e.bias2);
            const bool simple = MODE == EPI_LINEAR && !has_in && !out32 && out.vec &&
                                (kPlain || (!biased && !e.out2 && e.fn == PI_FN_NONE && e.scale == 1.f));
            const uint32_t buf = it & 1, ph = (it >> 1) & 1;
            int mi, ni;
            tile_at(w.tile, pr.tm, pr.tn, mi, ni);
            const int row0 = mi * kTile + (int)rank * 128 + q * 32, col0 = ni * kOutN + half * kCols;
            const bool whole = w.slot < 0;
            uint4 q1[4], q2[4]; // the next chunk's inputs
            if (whole && has_in) { // in flight while the products finish
                strip_load(in1, lane, row0, col0, M, N, q1);
                if (two) strip_load(in2, lane, row0, col0, M, N, q2);
            }
            if (whole && biased) { // 4 values a lane
                const int h = MODE == EPI_GATED ? lane >> 4 : 0, k = (MODE == EPI_GATED ? lane & 15 : lane) * 4;
                const uint16_t *src = h ? e.bias2 : e.bias;
                uint32_t b[2] = {};
                if (src) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (col0 + k + i < N) b[i >> 1] |= (uint32_t)src[col0 + k + i] << (16 * (i & 1));
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
                float4 *dst = reinterpret_cast<float4 *>(p.part) + (size_t)w.slot * (kTile * kTile / 4) + r;
#pragma unroll 1
                for (int c = half * (WIDE / 2); c < (half + 1) * (WIDE / 2); c += 32) {
                    float v[32];
                    tmem_ld32(ta + c, v);
                    if (row0 + lane < M) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            dst[(c + i) / 4 * kTile] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                }
            } else if (simple && row0 + 32 <= M && col0 + kCols <= N) {
                plain_strip<T, kCols>(ta + half * kCols, box0, &pr.mo, lane, row0, col0, [&]() {
                    tc_before();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(in_first(smem_addr(acc_empty + buf)));
                });
                released = true;
            } else if (row0 < M) {
                if (MODE == EPI_LINEAR) box_settle(lane);
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    const int col = col0 + c;
                    if (col >= N) break;
                    const bool inside = row0 + 32 <= M && col + 32 <= N;
                    float v[32], u[MODE == EPI_GATED ? 32 : 1];
                    tmem_ld32(ta + half * kCols + c, v);
                    if (MODE == EPI_GATED) tmem_ld32(ta + 128 + half * kCols + c, *reinterpret_cast<float(*)[32]>(u));
                    if (c + 32 >= kCols || col + 32 >= N) {
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
                            strip_load(in1, lane, row0, col + 32, M, N, q1);
                            if (two) strip_load(in2, lane, row0, col + 32, M, N, q2);
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
                    if (!kPlain && MODE != EPI_DACT && e.out2) {
                        box_put<T>(box1, lane, v);
                        box_send(box1, out2, lane, row0, col, M, N, inside);
                    }
                    if (MODE == EPI_GATED && e.out3) {
                        box_put<T>(box1, lane, *reinterpret_cast<float(*)[32]>(u));
                        box_send(box1, out3, lane, row0, col, M, N, inside);
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
                        if (two) box_send(box1, out2, lane, row0, col, M, N, inside);
                    } else {
                        if (!kPlain && e.fn != PI_FN_NONE) acts(e.fn, v);
                        if (MODE == EPI_GATED) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= u[i % (MODE == EPI_GATED ? 32 : 1)];
                        } else {
                            if (!kPlain && e.scale != 1.f) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] *= e.scale;
                            }
                            if (out32) {
                                if (row0 + lane < M)
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        const int cj = col + 8 * j;
                                        if (cj >= N) break;
                                        float(&x)[8] = *reinterpret_cast<float(*)[8]>(v + 8 * j);
                                        if (e.res) {
                                            float r[8];
                                            load8f(static_cast<const float *>(e.res) + (int64_t)(row0 + lane) * e.ldr + cj, N - cj, e.vec & V_RES, r);
#pragma unroll
                                            for (int i = 0; i < 8; ++i) x[i] += r[i];
                                        }
                                        store8f(static_cast<float *>(e.out) + (int64_t)(row0 + lane) * e.ldo + cj, N - cj, e.vec & V_OUT, x);
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
                    box_send(box0, out, lane, row0, col, M, N, inside);
                }
            }
            if (!released) {
                tc_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(in_first(smem_addr(acc_empty + buf)));
            }
        }
        if (MODE == EPI_LINEAR && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); // written
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

__device__ __forceinline__ void load4x2(const float4 *a, const float4 *b, float (&v)[8])
{
    const float4 p = *a, q = *b;
    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
}

// The split tiles: partials added in the order of k, then the epilogue.
// 256 threads take 8 columns each of 8 (gated: 16) rows; a warp's 8 rows x 32
// columns are 128 bytes in a row of the partials, 64 of the output.
template <typename T, int MODE, int NP>
__global__ void __launch_bounds__(256) gemm_fixup(const __grid_constant__ TcParams<NP> p, int wide)
{
    pdl_enter();
    const Prob &pr = p.prob[NP == 1 ? 0 : p.s.sprob];
    constexpr int kOutN = MODE == EPI_GATED ? 128 : kTile, kCols = kOutN / 8, kRows = 256 / kCols;
    const int outn = MODE == EPI_GATED ? 128 : wide;
    const int per = kTile / kRows, r = (int)blockIdx.x / per;
    constexpr int kWarps = kOutN / 32; // that share 8 rows
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = ((int)blockIdx.x % per) * kRows + warp / kWarps * 8 + (lane & 7), c = warp % kWarps * 32 + (lane >> 3) * 8;
    int mi, ni;
    tile_at(p.s.stile0 + r, pr.tm, pr.tn, mi, ni);
    const int grow = mi * kTile + row, gcol = ni * outn + c;
    if (grow >= pr.M || gcol >= pr.N || c >= outn) return;
    const int64_t units = (int64_t)(p.s.nsplit / p.s.lanes) * pr.KT, u0 = (int64_t)(r / p.s.lanes) * pr.KT;
    const int cnt = part_of(units, u0 + pr.KT - 1, p.s.parts) - part_of(units, u0, p.s.parts) + 1;
    float v[8] = {}, u[8] = {};
    const float4 *src = reinterpret_cast<const float4 *>(p.part) + (size_t)r * p.s.smax * (kTile * kTile / 4) + c / 4 * kTile + row;
    for (int s = 0; s < cnt; ++s, src += kTile * kTile / 4) {
        float t[8];
        load4x2(src, src + kTile, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
        if (MODE == EPI_GATED) {
            load4x2(src + 32 * kTile, src + 33 * kTile, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] += t[i];
        }
    }
    epilogue8<T, MODE>(pr.e, pr.N, grow, gcol, v, u);
}

// ------------------------------------------------------------------ host
// A last wave of `rem` tiles on n pairs takes KT steps; split along k, it takes
// rem KT / n and the fixup launch with its traffic, worth about kFixupSteps steps.
// One product of a group may be split: the longest that the others do not fill up.
constexpr int kFixupSteps = 32;
constexpr int kMinShare = 4; // k steps per pair, at least
constexpr int kTileSteps = 8; // a tile's epilogue takes as long as about this many steps, which it hides behind

struct Plan {
    Sched s;
    int order[kMaxProbs]; // products by falling k steps
    int tm[kMaxProbs], tn[kMaxProbs], kt0[kMaxProbs], KT[kMaxProbs]; // in that order
    int launched;         // pairs
    int wide;             // columns of a tile
    size_t bytes;
};

Plan plan_group(const Gemm *g, int n, int sms)
{
    Plan q = {};
    const int P = sms / 2;
    int KT[kMaxProbs];
    for (int i = 0; i < n; ++i) {
        KT[i] = (g[i].K[0] + kBK - 1) / kBK + (g[i].segs > 1 ? (g[i].K[1] + kBK - 1) / kBK : 0);
        q.order[i] = i;
    }
    std::stable_sort(q.order, q.order + n, [&](int a, int b) { return KT[a] > KT[b]; });
    // Where tiles of 256 x 256 would leave half of the pairs idle, ones of 256
    // x 128 use them: a step of k takes about 2 / 3 as long (24 instead of 32 KB
    // of loads, which bound it, and half of the epilogue).  512 x 4096 x 4096:
    // 20 us, 256 wide 24; 300 rows, K 1024, N 4096: 9.1, 10.9.  A long k is
    // better split (129 x 28672 x 8192: 256 wide and split 89 us, 128 wide 108).
    // Outputs of up to 128 columns fill no wider tile.
    int64_t tiles = 0, steps = 0, longest = 0;
    bool thin = true;
    for (int i = 0; i < n; ++i) {
        thin = thin && g[i].N <= 128;
        const int64_t t = (int64_t)((g[i].M + kTile - 1) / kTile) * ((g[i].N + kTile - 1) / kTile);
        tiles += t, steps += t * KT[i], longest = std::max<int64_t>(longest, KT[i]);
    }
    const bool idle = tiles <= P / 2 && 2 * longest < 3 * (steps / P + kFixupSteps);
    q.wide = g[0].mode != EPI_GATED && (thin || idle) ? 128 : kTile;
    const int fixup = q.wide == kTile ? kFixupSteps : 2 * kFixupSteps;
    Sched &s = q.s;
    s.pairs = P;
    s.smax = 1, s.lanes = 1;
    int64_t later = 0; // steps of the products that follow
    int cost[kMaxProbs];
    for (int j = 0; j < n; ++j) {
        const Gemm &x = g[q.order[j]];
        const int outn = x.mode == EPI_GATED ? 128 : q.wide;
        q.tm[j] = (x.M + kTile - 1) / kTile;
        q.tn[j] = (x.N + outn - 1) / outn;
        q.kt0[j] = (x.K[0] + kBK - 1) / kBK;
        q.KT[j] = KT[q.order[j]];
        cost[j] = std::max(q.KT[j], kTileSteps);
        later += (int64_t)q.tm[j] * q.tn[j] * cost[j];
    }
    // Pairs base .. base + high - 1 (mod P) are ahead of the others by `gap` steps.
    int base = 0, high = 0, gap = 0, used = 0;
    for (int j = 0; j < n; ++j) {
        later -= (int64_t)q.tm[j] * q.tn[j] * cost[j];
        int t0 = 0, m = q.tm[j] * q.tn[j];
        if (high && gap >= cost[j]) { // the pairs behind catch up first
            const int lo = P - high;
            const int cnt = (int)std::min<int64_t>(m, (int64_t)(gap / cost[j]) * lo);
            s.deal[s.ndeal++] = {j, t0, cnt, (base + high) % P, lo};
            used = P;
            t0 += cnt, m -= cnt;
            gap -= (cnt + lo - 1) / lo * cost[j];
        }
        if (!m) continue;
        int rem = m % P;
        const int from = (base + high) % P;
        // (what follows fills the pairs that the last wave leaves idle, as far as it goes)
        if (!s.nsplit && rem && (int64_t)q.KT[j] * (P - rem) - later > (int64_t)fixup * P) {
            s.sprob = j, s.stile0 = t0 + m - rem, s.nsplit = rem;
            // the split tiles of a column (they lie together, see tile_at) are
            // cut alike, where they come in whole groups: pairs that work on
            // one column then read the same of B at a time.  (512 x 8192 x
            // 28672: cut end to end, its two rows read B twice, 194 us instead of 149)
            const int rows = q.tm[j] <= 8 ? q.tm[j] : q.tm[j] % 8 ? 1 : 8;
            s.lanes = std::gcd(std::gcd(rows, s.stile0), rem);
            while (s.lanes % 2 == 0 && P % s.lanes) s.lanes /= 2; // (no pair left over)
            const int64_t units = (int64_t)(rem / s.lanes) * q.KT[j];
            s.parts = (int)std::min<int64_t>(P / s.lanes, std::max<int64_t>(1, units / kMinShare));
            s.smax = q.KT[j] / (int)(units / s.parts) + 2;
            q.bytes = (size_t)rem * s.smax * kTile * kTile * sizeof(float);
            m -= rem;
            rem = 0;
            used = std::max(used, s.parts * s.lanes);
        }
        if (m) {
            s.deal[s.ndeal++] = {j, t0, m, from, P};
            used = from ? P : std::max(used, std::min(m, P));
        }
        base = from, high = rem, gap = cost[j];
    }
    q.launched = used;
    return q;
}

// box: rows of a stage
cudaError_t map_of(CUtensorMap *m, const Mat &a, int rows, int K, int box)
{
    return a.mn ? encode_map(m, a.p, (uint64_t)rows, (uint64_t)K, (uint64_t)a.ld * 2, 64)
                : encode_map(m, a.p, (uint64_t)K, (uint64_t)rows, (uint64_t)a.ld * 2, box);
}

template <typename T, int MODE, int NP, int WIDE> cudaError_t run_plan(const Gemm *g, int n, const Plan &q, const CtxView &v, void *ws)
{
    TcParams<NP> p = {};
    p.s = q.s;
    cudaError_t e = cudaSuccess;
    for (int j = 0; j < n; ++j) {
        const Gemm &x = g[q.order[j]];
        Prob &pr = p.prob[j];
        pr.M = x.M, pr.N = x.N, pr.tm = q.tm[j], pr.tn = q.tn[j], pr.kt0 = q.kt0[j], pr.KT = q.KT[j];
        pr.a_mn = x.a[0].mn, pr.b_mn = x.b[0].mn;
        pr.e = x.e;
        for (int i = 0; i < x.segs && e == cudaSuccess; ++i) e = map_of(&pr.ma[i], x.a[i], x.M, x.K[i], 128);
        const int nb = MODE == EPI_GATED ? 2 : x.segs;
        if (MODE == EPI_LINEAR && !x.e.out32 && (x.e.vec & V_OUT) && e == cudaSuccess)
            e = encode_map(&pr.mo, x.e.out, (uint64_t)x.N, (uint64_t)x.M, (uint64_t)x.e.ldo * 2, 32);
        for (int i = 0; i < nb && e == cudaSuccess; ++i) e = map_of(&pr.mb[i], x.b[i], x.N, x.K[MODE == EPI_GATED ? 0 : i], MODE == EPI_GATED ? 128 : WIDE / 2);
    }
    if (e != cudaSuccess) return e;
    p.part = static_cast<float *>(ws);
    p.status = v.status, p.abort_flag = v.abort_flag, p.wait_ns = v.wait_ns;

    constexpr int smem = kStages * kStageBytes + kBoxes + kEpiWarps * kBiasB + (2 * kStages + 4) * 8 + 16;
    auto kern = gemm_tc<T, MODE, NP, WIDE>;
    static std::atomic<uint64_t> ready{0}; // devices whose limit has been raised
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1))) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev);
    }
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(2 * q.launched), dim3(kGemmThreads), smem, v.stream, p);
    if (e != cudaSuccess || !p.s.nsplit) return e;
    constexpr int kCols = (MODE == EPI_GATED ? 128 : kTile) / 8;
    return launch_pdl(gemm_fixup<T, MODE, NP>, dim3(p.s.nsplit * kTile / (256 / kCols)), dim3(256), 0, v.stream, p, WIDE);
}

template <typename T, int MODE, int NP> cudaError_t run(const Gemm *g, int n, const CtxView &v, void *ws)
{
    const Plan q = plan_group(g, n, v.sms);
    if constexpr (MODE != EPI_GATED)
        if (q.wide != kTile) return run_plan<T, MODE, NP, 128>(g, n, q, v, ws);
    return run_plan<T, MODE, NP, kTile>(g, n, q, v, ws);
}

template <typename T> cudaError_t run_mode(const Gemm *g, int n, const CtxView &v, void *ws)
{
    if (n > 1) return run<T, EPI_LINEAR, kMaxProbs>(g, n, v, ws);
    return g->mode == EPI_LINEAR  ? run<T, EPI_LINEAR, 1>(g, 1, v, ws)
           : g->mode == EPI_GATED ? run<T, EPI_GATED, 1>(g, 1, v, ws)
                                  : run<T, EPI_DACT, 1>(g, 1, v, ws);
}

} // namespace

size_t gemm_workspace(const Gemm &g, const CtxView &v)
{
    return skinny_takes(g) ? skinny_workspace(g, v) : plan_group(&g, 1, v.sms).bytes;
}

cudaError_t launch_gemm(const Gemm &g, bool bf16, const CtxView &v, void *ws)
{
    if (skinny_takes(g)) return launch_skinny(g, bf16, v, ws);
    return bf16 ? run_mode<__nv_bfloat16>(&g, 1, v, ws) : run_mode<__half>(&g, 1, v, ws);
}

size_t gemms_workspace(const Gemm *g, int n, const CtxView &v)
{
    return n == 1 ? gemm_workspace(*g, v) : plan_group(g, n, v.sms).bytes;
}

cudaError_t launch_gemms(const Gemm *g, int n, bool bf16, const CtxView &v, void *ws)
{
    if (n == 1) return launch_gemm(*g, bf16, v, ws);
    return bf16 ? run_mode<__nv_bfloat16>(g, n, v, ws) : run_mode<__half>(g, n, v, ws);
}

} // namespace pi
