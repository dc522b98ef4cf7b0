// Which kernel a product of microscaled operands runs (one translation unit for each pair of types).
#pragma once

#include "pi_gemm.cuh"

namespace pi {
namespace {

template <typename T, int OPS> cudaError_t run_mx_as(const Gemm &g, const CtxView &v, void *ws)
{
    const Plan q = plan_group(&g, 1, v.sms);
    if (g.mode == EPI_GATED) return run_plan<T, EPI_GATED, 1, kTile, OPS>(&g, 1, q, v, ws);
    return q.wide != kTile ? run_plan<T, EPI_LINEAR, 1, 128, OPS>(&g, 1, q, v, ws) : run_plan<T, EPI_LINEAR, 1, kTile, OPS>(&g, 1, q, v, ws);
}

template <int OPS> cudaError_t run_mx(const Gemm &g, bool bf16, const CtxView &v, void *ws)
{
    return bf16 ? run_mx_as<__nv_bfloat16, OPS>(g, v, ws) : run_mx_as<__half, OPS>(g, v, ws);
}

} // namespace
} // namespace pi
