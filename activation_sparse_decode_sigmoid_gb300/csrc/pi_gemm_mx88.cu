// Products of microscaled operands (pi_gemm.cuh): both of 8 bits.
#include "pi_gemm.cuh"
#include "pi_gemm_mx.cuh"

namespace pi {

cudaError_t launch_gemm_mx88(const Gemm &g, bool bf16, const CtxView &v, void *ws) { return run_mx<OPS_MX88>(g, bf16, v, ws); }

} // namespace pi
