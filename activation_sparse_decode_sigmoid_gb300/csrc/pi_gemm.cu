// The matrix product of the block operators with its fused epilogue:
//     D[m][n] = sum_k A(m, k) B(n, k)   (one or two segments of k)
// A first, plain version: 64 x 64 tiles through shared memory, fp32 fma on
// the CUDA cores, any strides and either order of each operand.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pi_block.h"
#include "pi_epi.cuh"

namespace pi {
namespace {

constexpr int kT = 64, kK = 16;

template <typename T, int MODE> __global__ void __launch_bounds__(256) gemm_plain(const __grid_constant__ Gemm g)
{
    __shared__ float sa[kK][kT + 1], sb[MODE == EPI_GATED ? 2 : 1][kK][kT + 1];
    const int tid = threadIdx.x, ntn = (g.N + kT - 1) / kT;
    const int m0 = (int)(blockIdx.x / ntn) * kT, n0 = (int)(blockIdx.x % ntn) * kT;
    const int r = tid >> 3, c = (tid & 7) * 8; // rows r, r + 32; columns c .. c + 7
    float acc[2][8] = {}, acc2[2][8] = {};
    for (int s = 0; s < g.segs; ++s) {
        const uint16_t *A = static_cast<const uint16_t *>(g.a[s].p);
        for (int k0 = 0; k0 < g.K[s]; k0 += kK) {
            for (int i = tid; i < kK * kT; i += 256) {
                // neighbouring threads read along the contiguous direction
                const int row = g.a[s].mn ? i % kT : i / kK, k = g.a[s].mn ? i / kT : i % kK;
                const int64_t m = m0 + row, kk = k0 + k;
                sa[k][row] = m < g.M && kk < g.K[s]
                                 ? C16<T>::one(A[g.a[s].mn ? kk * g.a[s].ld + m : m * g.a[s].ld + kk])
                                 : 0.f;
            }
            for (int j = 0; j < (MODE == EPI_GATED ? 2 : 1); ++j) {
                const Mat &b = g.b[MODE == EPI_GATED ? j : s];
                const uint16_t *B = static_cast<const uint16_t *>(b.p);
                for (int i = tid; i < kK * kT; i += 256) {
                    const int row = b.mn ? i % kT : i / kK, k = b.mn ? i / kT : i % kK;
                    const int64_t n = n0 + row, kk = k0 + k;
                    sb[j][k][row] =
                        n < g.N && kk < g.K[s] ? C16<T>::one(B[b.mn ? kk * b.ld + n : n * b.ld + kk]) : 0.f;
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                const float a0 = sa[k][r], a1 = sa[k][r + 32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[0][i] = fmaf(a0, sb[0][k][c + i], acc[0][i]);
                    acc[1][i] = fmaf(a1, sb[0][k][c + i], acc[1][i]);
                    if (MODE == EPI_GATED) {
                        acc2[0][i] = fmaf(a0, sb[1 % (MODE == EPI_GATED ? 2 : 1)][k][c + i], acc2[0][i]);
                        acc2[1][i] = fmaf(a1, sb[1 % (MODE == EPI_GATED ? 2 : 1)][k][c + i], acc2[1][i]);
                    }
                }
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = m0 + r + 32 * h;
        if (m < g.M && n0 + c < g.N) epilogue8<T, MODE>(g.e, g.N, m, n0 + c, acc[h], acc2[h]);
    }
}

template <typename T> cudaError_t launch(const Gemm &g, cudaStream_t s)
{
    const long long tiles = (long long)((g.M + kT - 1) / kT) * ((g.N + kT - 1) / kT);
    const dim3 grid((unsigned)tiles);
    if (g.mode == EPI_LINEAR) gemm_plain<T, EPI_LINEAR><<<grid, 256, 0, s>>>(g);
    else if (g.mode == EPI_GATED) gemm_plain<T, EPI_GATED><<<grid, 256, 0, s>>>(g);
    else gemm_plain<T, EPI_DACT><<<grid, 256, 0, s>>>(g);
    return cudaGetLastError();
}

} // namespace

size_t gemm_workspace(const Gemm &, const CtxView &) { return 0; }

cudaError_t launch_gemm(const Gemm &g, bool bf16, const CtxView &v, void *)
{
    return bf16 ? launch<__nv_bfloat16>(g, v.stream) : launch<__half>(g, v.stream);
}

} // namespace pi
