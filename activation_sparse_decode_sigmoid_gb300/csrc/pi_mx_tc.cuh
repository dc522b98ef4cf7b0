// Block-scaled products on the tcgen05 tensor cores: operand types, instruction
// descriptors, MMAs and the copies of scales, for the kernels of pi_gemm.cuh,
// pi_mx_skinny.cu and pi_mx_rows.cu.
//
// A step of k is 128 bytes of an operand's row in shared memory, whatever its
// type: 128 elements of 8 bits (of 4, spread to bytes by the TMA, where the
// other operand has 8), or 256 of 4.  Its scales come as whole tiles of 512
// bytes (128 rows x 4 blocks), which one tcgen05.cp each spreads over four
// columns of tensor memory, a word with a row's four scales in each lane; the
// instruction descriptor says which of a word's bytes an MMA takes.
//
// Each step's copies are issued right before its MMAs, into the next of a few
// sets of columns, by the same warp.  There they cost nothing (left out but for a tile's
// first two steps, 2048 x 28672 -> 8192 in 4 bits took the same time); for two or up to four
// steps at a time (157 -> 160, 166 us), in the middle of the step before's MMAs (173) and from
// a warp of their own (184) they did.
#pragma once

#include <stdint.h>

#include "pi_block.h"
#include "pi_mx.cuh"
#include "pi_tc.cuh"

namespace pi {

// bytes of 128 rows of a step on their way (4 bits spread to bytes count as they lie in memory)
constexpr uint32_t mx_row_tx(bool nibbles) { return nibbles ? 64 : 128; }

namespace {

// WORDS: tiles of scales (128 of k) to a step
template <int OPS> struct Ops {
    static constexpr bool mx = OPS != OPS_16;
    static constexpr int words = OPS == OPS_MX44 ? 2 : 1;
    static constexpr int xkind = OPS == OPS_MX44 ? PI_MX4 : PI_MX8; // also a microscaled output's
    static constexpr int wkind = OPS == OPS_MX88 ? PI_MX8 : PI_MX4;
    static constexpr bool nibbles = OPS == OPS_MX84;          // W's codes are spread to bytes
    static constexpr uint32_t xfmt = OPS == OPS_MX44 ? 1 : 0; // operand formats: e4m3 0; e2m1 5, or 1 where both have 4 bits
    static constexpr uint32_t wfmt = OPS == OPS_MX44 ? 1 : OPS == OPS_MX84 ? 5 : 0;
};

// instruction descriptor: formats, sizes, scales that are powers of two; scale ids are added per MMA
__device__ __forceinline__ uint32_t idesc_mx(uint32_t fa, uint32_t fb, uint32_t M, uint32_t N)
{
    return (fa << 7) | (fb << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24);
}
// MMA j of a step: which byte(s) of the scales' words it takes, and of which word
template <int OPS> __device__ __forceinline__ uint32_t sf_id(int j)
{
    const uint32_t s = Ops<OPS>::words == 2 ? (j & 1) * 2 : j;
    return (s << 29) | (s << 4);
}
template <int OPS> __device__ __forceinline__ uint32_t sf_word(int j) { return Ops<OPS>::words == 2 ? j >> 1 : 0; }

// 512 bytes: 32 rows of 16, 8 rows to a group of 128 bytes (no swizzle)
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (8ull << 16) | (8ull << 32) | (1ull << 46);
}

template <int OPS> __device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb, uint32_t acc)
{
    if (OPS == OPS_MX44)
        asm volatile("{ .reg .pred q; setp.ne.b32 q, %4, 0; "
                     "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], q; }" ::"r"(d),
                     "l"(a), "l"(b), "r"(id), "r"(acc), "r"(sa), "r"(sb));
    else
        asm volatile("{ .reg .pred q; setp.ne.b32 q, %4, 0; "
                     "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], q; }" ::"r"(d),
                     "l"(a), "l"(b), "r"(id), "r"(acc), "r"(sa), "r"(sb));
}
template <int OPS> __device__ __forceinline__ void mma2_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb, uint32_t acc)
{
    if (OPS == OPS_MX44)
        asm volatile("{ .reg .pred q; setp.ne.b32 q, %4, 0; "
                     "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], q; }" ::"r"(d),
                     "l"(a), "l"(b), "r"(id), "r"(acc), "r"(sa), "r"(sb));
    else
        asm volatile("{ .reg .pred q; setp.ne.b32 q, %4, 0; "
                     "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], q; }" ::"r"(d),
                     "l"(a), "l"(b), "r"(id), "r"(acc), "r"(sa), "r"(sb));
}

// a tile of scales to tensor memory, the same in all four quarters of its lanes; in order with the MMAs around it
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint32_t saddr)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc_scales(saddr)));
}
// the same in both CTAs of a pair, each from its own shared memory
__device__ __forceinline__ void cp2_scales(uint32_t taddr, uint32_t saddr)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc_scales(saddr)));
}

} // namespace
} // namespace pi
