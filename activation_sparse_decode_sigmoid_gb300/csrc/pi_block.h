// Structures shared by the block operators (linear, gated FFN, norms): the
// matrix product with its epilogue, as the host plans it and the kernels run it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pi_host.h"

namespace pi {

// What follows a product.  Every mode works on the fp32 accumulator(s) of one
// output element and rounds once.
//   EPI_LINEAR  z = acc + bias;  out = res + scale * fn(z);  out2 = z
//   EPI_GATED   g = acc + bias, u = acc' + bias2 (the product with the second
//               weight matrix);  out = fn(g) * u;  out2 = g, out3 = u
//   EPI_DACT    in1, in2 given:  in2: out = acc * in2 * fn'(in1), out2 = acc * fn(in1)
//               else out = scale * acc * fn'(in1)
enum : int { EPI_LINEAR = 0, EPI_GATED = 1, EPI_DACT = 2 };

// bits of Epi::vec: this pointer's rows allow 16-byte accesses at every
// multiple of 8 elements
enum : unsigned { V_RES = 1, V_OUT = 2, V_OUT2 = 4, V_OUT3 = 8, V_IN1 = 16, V_IN2 = 32, V_BIAS = 64, V_BIAS2 = 128 };

struct Epi {
    int fn;       // pi_fn
    int out32;    // res and out are fp32 (EPI_LINEAR), else 16-bit
    float scale;
    unsigned vec;
    const uint16_t *bias, *bias2; // [N] or NULL
    const void *res;              // or NULL
    void *out;
    uint16_t *out2, *out3;        // or NULL
    const uint16_t *in1, *in2;
    int64_t ldr, ldo, ld2, ld3, ldi1, ldi2;
};

// One operand: element (row r, reduction index k) is p[r * ld + k] (mn = 0)
// or p[k * ld + r] (mn = 1).
struct Mat {
    const void *p;
    int64_t ld;
    int mn;
};

// D[M][N] = sum over segments of A_s[M][K_s] B_s[N][K_s]^T, then the
// epilogue; dual (EPI_GATED): one segment, B_0 and B_1 give two accumulators.
struct Gemm {
    int mode;
    int M, N;
    int segs;
    int K[2];
    Mat a[2], b[2];
    // B is complete before the launch in front of this one starts: it may be
    // read before that launch has finished (launches wait for their
    // predecessor before they let their successor start)
    int early;
    Epi e;
};

// Workspace of a launch (bytes), and the launch.
size_t gemm_workspace(const Gemm &g, const CtxView &v);
cudaError_t launch_gemm(const Gemm &g, bool bf16, const CtxView &v, void *ws);

// The same for up to four products that are independent of one another, in one
// launch; their epilogues are EPI_LINEAR without bias, activation, scale or z.
size_t gemms_workspace(const Gemm *g, int n, const CtxView &v);
cudaError_t launch_gemms(const Gemm *g, int n, bool bf16, const CtxView &v, void *ws);

// Products of up to this many rows of A go to skinny_tc (pi_skinny.cu) where
// both operands lie along k.
constexpr int kSkinnyRows = 128;
bool skinny_takes(const Gemm &g);
size_t skinny_workspace(const Gemm &g, const CtxView &v);
cudaError_t launch_skinny(const Gemm &g, bool bf16, const CtxView &v, void *ws);

// Bytes of the partial column sums of a matrix [T][N].
size_t colsum_bytes(int T, int N, int sms);

// dz = scale * dy * fn'(z) [T][N], 16-bit, and its column sums into db (NULL:
// none; the fp32 values before their rounding are summed)
cudaError_t launch_dact(const void *dy, int dy32, int64_t ldy, const void *z, int64_t ldz, int fn, float scale,
                        void *dz, int64_t lddz, int T, int N, void *db, int db32, int accumulate, bool bf16,
                        void *part, const CtxView &v);

} // namespace pi
