// What the products of microscaled operands for few tokens share: clusters of
// CTAs that split k, their exchange, and outputs a feature to a lane.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pi_block.h"
#include "pi_epi.cuh"
#include "pi_mx.cuh"
#include "pi_pair.cuh"
#include "pi_tc.cuh"

namespace pi {
namespace {

// address of a shared-memory object in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// a warp's wait for arrivals from other CTAs, after which it sees what they wrote before them
__device__ __forceinline__ bool mbar_try_cluster(uint64_t *b, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred q; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 q, [%1], %2; "
                 "selp.u32 %0, 1, 0, q; }"
                 : "=r"(ok)
                 : "r"(smem_addr(b)), "r"(parity)
                 : "memory");
    return ok != 0;
}
template <typename P> __device__ __forceinline__ bool warp_wait_cluster(uint64_t *b, uint32_t parity, const P &p, int lane)
{
    bool ok = true;
    if (lane == 0) ok = mbar_wait_bounded(b, parity, p) && mbar_try_cluster(b, parity); // (the second returns at once)
    return __shfl_sync(0xffffffffu, ok, 0);
}

// The steps of a CTA in order: tiles, the matrices of each, this CTA's part of k.
struct MxWalk {
    int tile, m, k, k0, k1, nm, step, tn;
    __device__ __forceinline__ MxWalk(int tn_, int nm_, int KT, int cs, int cluster, int clusters, int rank)
        : tile(cluster), m(0), nm(nm_), step(clusters), tn(tn_)
    {
        k0 = (int)((int64_t)KT * rank / cs), k1 = (int)((int64_t)KT * (rank + 1) / cs);
        k = k0;
    }
    __device__ __forceinline__ bool more() const { return tile < tn; }
    __device__ __forceinline__ void next()
    {
        if (++k < k1) return;
        k = k0;
        if (++m < nm) return;
        m = 0, tile += step;
    }
};

// One token's outputs of a warp's 32 features, one a lane (microscaled: a
// block), as OUT says: PI_MX8, PI_MX4, PI_F32, or 16 bits.  res: the residual's element, or 0.
template <typename T, int OUT> __device__ __forceinline__ void put32(const Epi &e, int64_t t, int f, int N, float v, float res)
{
    if constexpr (OUT == PI_MX8 || OUT == PI_MX4) {
        const float x = f < N ? v : 0.f;
        const uint32_t code = mx_scale<OUT>(__reduce_max_sync(0xffffffffu, mag(x)));
        if (f >= e.mx_tiles * 128) return; // (behind the padded row, all of a warp)
        float q[8] = {x * mx_inverse(code)};
        uint8_t *row = static_cast<uint8_t *>(e.out) + t * e.ldo;
        if (OUT == PI_MX8) row[f] = (uint8_t)mx_pack8<PI_MX8>(q).x;
        else {
            q[1] = __shfl_xor_sync(0xffffffffu, q[0], 1);
            if (!(f & 1)) row[f >> 1] = code == 255u ? 0 : (uint8_t)mx_pack8<PI_MX4>(q).x;
        }
        if (!(f & 31)) e.mx_scales[mx_scale_at(t, f >> 7, e.mx_tiles) + ((f >> 5) & 3)] = (uint8_t)code;
    } else {
        if (f >= N) return;
        v = e.res ? v * e.scale + res : v * e.scale;
        if (OUT == PI_F32) static_cast<float *>(e.out)[t * e.ldo + f] = v;
        else static_cast<uint16_t *>(e.out)[t * e.ldo + f] = C16<T>::round(v);
    }
}

// How many clusters of 1, 2, 4 and 8 CTAs run at a time, a CTA to an SM (an SM
// that its neighbours leave alone takes no part: fewer than SMs / CTAs); asked
// once per kernel and device.
struct ClusterCounts {
    std::atomic<int> n[64][4];
};
template <typename P> cudaError_t cluster_counts(void (*kern)(P), ClusterCounts &known, int threads, const CtxView &v, int (&n)[4])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
        n[i] = dev < 64 ? known.n[dev][i].load(std::memory_order_relaxed) : 0;
        if (n[i]) continue;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(v.sms / 8 * 8), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = (size_t)v.smem_optin - 1024;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 1u << i, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
        cfg.attrs = at, cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n[i], kern, &cfg);
        if (e == cudaSuccess && dev < 64) known.n[dev][i].store(n[i], std::memory_order_relaxed);
    }
    return e;
}

// CTAs to a cluster, at most `most`: the number that leaves the fewest steps to
// the busiest CTA, the last tile's exchange (2 to 3 us; the others' lie behind
// the next tile's products) counted as `exchange` steps; of numbers as good, the
// smallest.  clusters: of which that many are launched.
inline int mx_cluster(int tn, int nm, int KT, const int (&n)[4], int most, int exchange, int &clusters)
{
    int64_t best = INT64_MAX;
    int got = 1;
    for (int i = 0; i < 4 && (1 << i) <= most && (1 << i) <= KT; ++i) {
        const int cs = 1 << i;
        if (n[i] < 1) continue;
        const int64_t cost = (int64_t)((tn + n[i] - 1) / n[i]) * nm * ((KT + cs - 1) / cs) + (cs > 1 ? exchange : 0);
        if (cost < best) best = cost, got = cs, clusters = std::min(tn, n[i]);
    }
    return got;
}

// A launch of clusters of cs CTAs that may be scheduled while the launch before it finishes.
template <typename P> cudaError_t launch_cluster(void (*kern)(P), int grid, int cs, int threads, size_t smem, cudaStream_t s, const P &p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(threads), cfg.stream = s, cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cs, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
    cfg.attrs = at, cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

} // namespace
} // namespace pi
