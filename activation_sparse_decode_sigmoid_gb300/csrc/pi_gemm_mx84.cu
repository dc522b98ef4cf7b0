// Products of microscaled operands (pi_gemm.cuh): 8-bit activations, 4-bit weights.
#include "pi_gemm.cuh"
#include "pi_gemm_mx.cuh"

namespace pi {

cudaError_t launch_gemm_mx84(const Gemm &g, bool bf16, const CtxView &v, void *ws) { return run_mx<OPS_MX84>(g, bf16, v, ws); }

} // namespace pi
