// The products of 16-bit operands (pi_gemm.cuh), and which path a product takes.
#include "pi_gemm.cuh"

namespace pi {
namespace {

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
    if (g.ops != OPS_16 && g.M <= kSkinnyRows) return 0;
    return skinny_takes(g) ? skinny_workspace(g, v) : plan_group(&g, 1, v.sms).bytes;
}

cudaError_t launch_gemm(const Gemm &g, bool bf16, const CtxView &v, void *ws)
{
    if (g.ops != OPS_16)
        return mx_rows_takes(g)     ? launch_mx_rows(g, bf16, v)
               : g.M <= kSkinnyRows ? launch_mx_skinny(g, bf16, v)
               : g.ops == OPS_MX88   ? launch_gemm_mx88(g, bf16, v, ws)
               : g.ops == OPS_MX84 ? launch_gemm_mx84(g, bf16, v, ws)
                                   : launch_gemm_mx44(g, bf16, v, ws);
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
