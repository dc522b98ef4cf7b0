"""Microscaled matrices without a GPU: the reference's own arithmetic at known
values, the sizes that the library states, and the binding's refusals."""
from __future__ import annotations

import ctypes

import pytest
import torch

from activation_sparse_decode_sigmoid_gb300 import build as B
from activation_sparse_decode_sigmoid_gb300 import pi
from tests import _mx as X


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pi.load_library()


def one_block(*v):
    return torch.tensor([list(v) + [0.0] * (32 - len(v))], dtype=torch.float64)


def test_reference_rounds_to_nearest_even():
    # amax 6: scale 1; every border between two values, and beside it
    a = [6.0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, -0.25, -5.01]
    c, s, v = X.quantize(X.MX4, one_block(*a))
    assert s[0, 0] == 127
    assert v[0, :16].tolist() == [6, 0, 0.5, 1, 0.5, 1, 1.5, 2, 2, 3, 4, 3, 4, 6, 0, -6]
    assert c[0, :4].tolist() == [7, 0, 1, 2] and c[0, 14] == 8 and c[0, 15] == 15
    # e4m3 against torch's own conversion, over its range and below it
    g = torch.Generator().manual_seed(0)
    x = torch.randn(64, 32, generator=g) * torch.exp(6 * torch.randn(64, 32, generator=g))
    x[:, 0] = 448.0
    x = x.clamp(-448, 448)
    c, s, v = X.quantize(X.MX8, x.double())
    assert bool((s[:, 0] == 127).all())
    assert torch.equal(v, x.to(torch.float8_e4m3fn).double())
    assert torch.equal(c[:, :32], x.to(torch.float8_e4m3fn).view(torch.uint8).long())


def test_reference_takes_the_least_scale_that_fits():
    for kind, most in ((X.MX8, 448.0), (X.MX4, 6.0)):
        for k in (-100, -3, 0, 5, 90):
            up = torch.tensor(most, dtype=torch.float64)
            for amax, want in ((up, k), (up * (1 + 2.0 ** -20), k + 1), (up / 2, k - 1), (up / 2 * (1 + 2.0 ** -20), k)):
                assert X.quantize(kind, one_block(amax.item() * 2.0 ** k))[1][0, 0] == want + 127
        assert X.quantize(kind, one_block(0.0))[1][0, 0] == 0        # zeros
        assert X.quantize(kind, one_block(2.0 ** -149))[1][0, 0] == 0  # below the least scale
        assert X.quantize(kind, one_block(float("inf"), 1.0))[1][0, 0] == 255
        assert bool(X.quantize(kind, one_block(float("nan"), 1.0))[2][0].isnan().all())


def test_bytes_of_a_matrix(lib):
    assert pi.pi_mx_bytes(300, 1000, pi.PI_MX8) == (300 * 1024, 3 * 8 * 512)
    assert pi.pi_mx_bytes(128, 128, pi.PI_MX4) == (128 * 64, 512)
    assert pi.pi_mx_bytes(0, 1, pi.PI_MX4) == (0, 0)
    a = ctypes.c_size_t()
    for args, code in (((-1, 1, pi.PI_MX8), pi.PI_ERR_SHAPE), ((1, 0, pi.PI_MX8), pi.PI_ERR_SHAPE),
                       ((1, (1 << 20) + 1, pi.PI_MX8), pi.PI_ERR_SHAPE), (((1 << 22) + 1, 1, pi.PI_MX8), pi.PI_ERR_SHAPE),
                       ((1, 1, pi.PI_F16), pi.PI_ERR_ARG)):
        assert lib.pi_mx_bytes(*args, ctypes.byref(a), ctypes.byref(a)) == code
    assert lib.pi_mx_bytes(1, 1, pi.PI_MX8, None, ctypes.byref(a)) == pi.PI_ERR_ARG


def test_null_context_is_an_error(lib):
    for f, n in ((lib.pi_mx_quantize, 3), (lib.pi_mx_dequantize, 3), (lib.pi_mx_linear_workspace, 2),
                 (lib.pi_mx_gated_ffn_workspace, 2)):
        assert f(None, *[None] * n) == pi.PI_ERR_ARG
    assert lib.pi_mx_linear(None, *[None] * 7, 0) == pi.PI_ERR_ARG
    assert lib.pi_mx_gated_ffn(None, *[None] * 5, 0) == pi.PI_ERR_ARG
    assert lib.pi_norm_residual_mx(None, None, pi.PI_MX8, *[None] * 6) == pi.PI_ERR_ARG


@pytest.fixture
def ctx(lib):
    """A context without a device: the binding's checks come before any call into the library."""
    c = object.__new__(pi.Context)
    c.torch_device, c.handle, c._plans = torch.device("cpu"), None, {}
    return c


def refused(code, f, *a, **k):
    with pytest.raises(pi.PiError) as e:
        f(*a, **k)
    assert e.value.status == code, e.value


def test_binding_refuses(ctx):
    x, w = ctx.mx_empty(4, 64, pi.PI_MX8), ctx.mx_empty(8, 64, pi.PI_MX4)
    assert x.shape == (4, 64) and w.codes.shape == (8, 64) and w.scales.shape == (1, 1, 32, 4, 4)
    refused(pi.PI_ERR_ARG, ctx.mx_empty, 4, 64, pi.PI_F16)
    refused(pi.PI_ERR_ARG, pi.MxMatrix, x.codes, x.scales, 64, pi.PI_Q4_0)
    refused(pi.PI_ERR_ARG, ctx.mx_quantize, torch.zeros(4, 64, dtype=torch.int32))
    refused(pi.PI_ERR_SHAPE, ctx.mx_quantize, torch.zeros(4))
    refused(pi.PI_ERR_ARG, ctx.mx_quantize, torch.zeros(64, 4).t())
    refused(pi.PI_ERR_ARG, ctx.mx_quantize, torch.zeros(4, 64), pi.PI_MX4, out=x)          # another kind
    refused(pi.PI_ERR_SHAPE, ctx.mx_quantize, torch.zeros(4, 65), pi.PI_MX8, out=x)
    refused(pi.PI_ERR_ARG, ctx.mx_quantize, torch.zeros(4, 64, device="meta"))
    refused(pi.PI_ERR_ARG, ctx.mx_dequantize, x, torch.int8)
    refused(pi.PI_ERR_ARG, ctx.mx_dequantize, torch.zeros(4, 64))
    refused(pi.PI_ERR_ARG, ctx.mx_dequantize, x, torch.float16, out=torch.zeros(4, 64))
    refused(pi.PI_ERR_SHAPE, ctx.mx_linear, x, ctx.mx_empty(8, 96, pi.PI_MX4))
    refused(pi.PI_ERR_SHAPE, ctx.mx_linear, x, w, torch.zeros(9, dtype=torch.bfloat16))
    refused(pi.PI_ERR_ARG, ctx.mx_linear, x, w, torch.zeros(8), dtype=torch.float16)
    refused(pi.PI_ERR_ARG, ctx.mx_linear, x, w, dtype=torch.float32)
    refused(pi.PI_ERR_SHAPE, ctx.mx_linear, pi.MxMatrix(x.codes[:, :64], x.scales, 64, pi.PI_MX8), w)
    refused(pi.PI_ERR_SHAPE, ctx.mx_linear, pi.MxMatrix(x.codes, x.scales[:0], 64, pi.PI_MX8), w)
    refused(pi.PI_ERR_ARG, ctx.mx_linear, pi.MxMatrix(x.codes, x.scales.permute(0, 1, 2, 4, 3), 64, pi.PI_MX8), w)
    refused(pi.PI_ERR_ARG, ctx.mx_linear, pi.MxMatrix(x.codes.to(torch.int8), x.scales, 64, pi.PI_MX8), w)
    up, down = ctx.mx_empty(100, 64, pi.PI_MX4), ctx.mx_empty(64, 100, pi.PI_MX4)
    refused(pi.PI_ERR_ARG, ctx.mx_gated_ffn, x, ctx.mx_empty(100, 64, pi.PI_MX8), up, down)  # kinds differ
    refused(pi.PI_ERR_SHAPE, ctx.mx_gated_ffn, x, ctx.mx_empty(99, 64, pi.PI_MX4), up, down)
    refused(pi.PI_ERR_SHAPE, ctx.mx_gated_ffn, x, None, up, ctx.mx_empty(64, 99, pi.PI_MX4))
    refused(pi.PI_ERR_SHAPE, ctx.mx_gated_ffn, x, None, up, down, None, torch.zeros(99, dtype=torch.bfloat16))
    refused(pi.PI_ERR_ARG, ctx.norm_residual_mx, torch.zeros(4, 64), kind=pi.PI_MX4, h=x)
    refused(pi.PI_ERR_SHAPE, ctx.norm_residual_mx, torch.zeros(5, 64), h=x)
