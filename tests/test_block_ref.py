"""The 64-bit references of the block operators against differences, and the
refusals of the binding.  No GPU needed."""
from __future__ import annotations

import ctypes

import pytest
import torch

from activation_sparse_decode_sigmoid_gb300 import build as B
from activation_sparse_decode_sigmoid_gb300 import pi
from tests import _block as R


def diff(fun, t, step=1e-5):
    """Gradient of the scalar fun() with respect to t by central differences."""
    g = torch.zeros_like(t)
    for i in range(t.numel()):
        v = t.view(-1)[i].item()
        t.view(-1)[i] = v + step
        hi = fun()
        t.view(-1)[i] = v - step
        lo = fun()
        t.view(-1)[i] = v
        g.view(-1)[i] = (hi - lo) / (2 * step)
    return g


def rn(g, *s):
    return torch.randn(*s, generator=g, dtype=torch.float64)


def close(a, b):
    assert torch.allclose(a, b, rtol=1e-6, atol=1e-7), (a - b).abs().max()


R.U[torch.float64], R.TINY[torch.float64] = 2.0 ** -53, 0.0


@pytest.mark.parametrize("fn", R.FNS)
def test_linear_gradients_are_differences(fn):
    g = torch.Generator().manual_seed(1)
    x, w, b, dy = rn(g, 3, 4), rn(g, 5, 4), rn(g, 5), rn(g, 3, 5)
    loss = lambda: float((R.linear(x, w, b, fn, 0.7, None, torch.float64)["y"][0] * dy).sum())
    z = R.linear(x, w, b, fn, 0.7, None, torch.float64)["z"][0]
    got = R.linear_bwd(dy, x, w, z, fn, 0.7, torch.float64)
    for k, t in (("dx", x), ("dw", w), ("db", b)):
        close(got[k][0], diff(loss, t))


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("fn", R.FNS[1:])
def test_ffn_gradients_are_differences(fn, gated):
    g = torch.Generator().manual_seed(2)
    x, wu, wd, bu, bd, dy = rn(g, 3, 4), rn(g, 5, 4), rn(g, 4, 5), rn(g, 5), rn(g, 4), rn(g, 3, 4)
    wg, bg = (rn(g, 5, 4), rn(g, 5)) if gated else (None, None)
    run = lambda: R.ffn(x, wg, wu, wd, bg, bu, bd, fn)
    loss = lambda: float((run()["y"][0] * dy).sum())
    s = run()
    got = R.ffn_bwd(dy, x, wg, wu, wd, s["g"][0] if gated else None, s["u"][0], s["a"][0], fn, torch.float64)
    for k, t in (("dx", x), ("w_gate", wg), ("w_up", wu), ("w_down", wd), ("b_gate", bg), ("b_up", bu), ("b_down", bd)):
        if t is not None:
            close(got[k][0], diff(loss, t))


@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("rows", [0, 1, 2])
def test_norm_gradients_are_differences(pre, post, rows):
    g = torch.Generator().manual_seed(3)
    T, d, f64 = 3, 6, torch.float64
    x, y, gate = rn(g, T, d), rn(g, T, d), rn(g, 1 if rows == 0 else -(-T // rows), d)
    wp, bp, wq, bq = (rn(g, d) for _ in range(4))
    dxo, dh = rn(g, T, d), rn(g, T, d)
    run = lambda: R.norm_fwd(x, y, gate, rows, pre, post, wp, bp, wq, bq, 0.8, 1.3, 1e-5, f64)

    def loss():
        o = run()
        return float((o["x"][0] * dxo).sum() + ((o["h"][0] * dh).sum() if pre != "none" else 0))

    got = R.norm_bwd(dxo, dh, run()["x"][0], y, gate, rows, pre, post, wp, wq, bq, 0.8, 1.3, 1e-5, f64, f64)
    for k, t in (("dx", x), ("dy", y), ("gate", gate), ("w_pre", wp), ("b_pre", bp), ("w_post", wq), ("b_post", bq)):
        if k in got:
            close(got[k][0], diff(loss, t))


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def lib():
    B.build()
    return pi.load_library()


def test_null_context(lib):
    n = ctypes.c_size_t()
    assert lib.pi_linear_workspace(None, None, 0, ctypes.addressof(n)) == pi.PI_ERR_ARG
    assert lib.pi_linear(*[None] * 9, 0) == pi.PI_ERR_ARG
    assert lib.pi_linear_bwd(*[None] * 9, 0, None, 0) == pi.PI_ERR_ARG
    assert lib.pi_gated_ffn_workspace(None, None, 0, ctypes.addressof(n)) == pi.PI_ERR_ARG
    assert lib.pi_gated_ffn(*[None] * 7, 0) == pi.PI_ERR_ARG
    assert lib.pi_gated_ffn_bwd(*[None] * 8, 0, None, 0) == pi.PI_ERR_ARG
    assert lib.pi_norm_residual(*[None] * 8) == pi.PI_ERR_ARG
    assert lib.pi_norm_residual_bwd_workspace(None, None, ctypes.addressof(n)) == pi.PI_ERR_ARG
    assert lib.pi_norm_residual_bwd(*[None] * 9, 0, None, 0) == pi.PI_ERR_ARG


def host_context():
    """A context without a library handle: every call below is refused before it would be used."""
    c = object.__new__(pi.Context)
    c.handle, c.device, c.torch_device = None, 0, torch.device("cpu")
    return c


def refused(status, call, *a, **kw):
    with pytest.raises(pi.PiError) as e:
        call(*a, **kw)
    assert e.value.status == status, e.value


def test_binding_refuses_bad_tensors():
    c = host_context()
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    ARG, SHAPE = pi.PI_ERR_ARG, pi.PI_ERR_SHAPE
    refused(ARG, c.linear, h(2, 8).float(), h(4, 8).float())                   # no fp32 product
    refused(ARG, c.linear, h(2, 8), h(4, 8).bfloat16())                        # two types
    refused(SHAPE, c.linear, h(2, 8), h(4, 9))                                 # K differs
    refused(SHAPE, c.linear, h(2, 8), h(4, 8), h(5))
    refused(SHAPE, c.linear, h(2, 8), h(4, 8), residual=h(2, 5))
    refused(ARG, c.linear, h(2, 8), h(4, 8), residual=h(2, 4), y=h(2, 4).float())
    refused(ARG, c.linear, h(8, 2).T, h(4, 8))                                 # rows not consecutive
    refused(SHAPE, c.linear, h(1, 8).expand(2, 8), h(4, 8))                    # overlapping rows
    refused(ARG, c.linear_bwd, h(2, 4), h(2, 8), h(4, 8), accumulate=True)     # nothing to add to
    refused(ARG, c.linear_bwd, h(2, 4), h(2, 8), h(4, 8), dw=h(4, 8).float(), db=h(4))
    refused(SHAPE, c.gated_ffn, h(2, 8), h(6, 8), h(6, 8), h(6, 8))
    refused(SHAPE, c.gated_ffn, h(2, 8), h(5, 8), h(6, 8), h(8, 6))
    refused(SHAPE, c.gated_ffn, h(2, 8), None, h(6, 8), h(8, 6), save=(None, h(2, 6), h(2, 5)))
    refused(ARG, c.gated_ffn_bwd, h(2, 8), h(2, 8), None, h(6, 8), h(8, 6), (None, h(2, 6), h(2, 6)),
            grads={"w_up": h(6, 9)[:, :8]})                                    # not packed
    refused(ARG, c.gated_ffn_bwd, h(2, 8), h(2, 8), None, h(6, 8), h(8, 6), (None, h(2, 6), h(2, 6)),
            grads={"w_up": h(6, 8), "b_up": h(6).float()})
    refused(SHAPE, c.norm_residual, h(2, 8), h(2, 7))
    refused(SHAPE, c.norm_residual, h(5, 8), h(5, 8), h(2, 8), gate_rows=2)    # three gate rows needed
    refused(ARG, c.norm_residual, h(2, 8).float(), h(2, 8), x_out=h(2, 8))
    refused(ARG, c.norm_residual_bwd, None, None, h(2, 8))
    refused(ARG, c.norm_residual_bwd, h(2, 8).float(), h(2, 8), h(2, 8))
    refused(ARG, c.norm_residual_bwd, None, h(2, 8), h(2, 8), w_pre=h(8), accumulate=True)
