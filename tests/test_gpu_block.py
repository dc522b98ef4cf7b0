"""The block operators (linear, gated FFN, norms around a block; forward and
backward) against their 64-bit references, within the bounds that
tests/_block.py derives from the arithmetic."""
from __future__ import annotations

import ctypes
import math
import threading

import numpy as np
import pytest
import torch

from activation_sparse_decode_sigmoid_gb300 import pi
from activation_sparse_decode_sigmoid_gb300 import workload as W
from tests import _block as R
from tests import _gpu as G
from tests._helpers import max_rel_err

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
KIND = {"none": pi.PI_NORM_NONE, "rms": pi.PI_NORM_RMS, "layer": pi.PI_NORM_LAYER}


def FN(fn):
    return getattr(pi, "PI_FN_" + fn.upper())


@pytest.fixture(scope="module")
def c():
    ctx = G.ctx()
    yield ctx
    ctx.check()  # no kernel raised a device error
    ctx.close()


class Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def __call__(self, *shape, dt=F16, std=1.0, pad=0, off=0):
        """Normal values; rows start `off` elements into ones `pad` wider."""
        wide = (*shape[:-1], shape[-1] + pad + off)
        v = (torch.randn(wide, generator=self.g, device="cuda") * std).to(dt)
        return v[..., off: off + shape[-1]]


def outside_untouched(buf, view):
    """A wider buffer filled with a marker, and a check that only `view` of it changed."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[: view[0], : view[1]] = False
    return lambda: bool((buf[mask] == 7).all())


# ------------------------------------------------------------------ linear
# one token to several row tiles; features below, at and past tile borders;
# odd features and slices of wider rows (copied operands)
LINEAR = [(1, 8, 1, 0, 0), (1, 1024, 4096, 0, 0), (2, 64, 128, 0, 0), (3, 257, 31, 0, 0), (8, 512, 129, 8, 0),
          (16, 640, 384, 0, 0), (17, 1000, 515, 0, 0), (33, 72, 1000, 3, 0), (64, 2048, 256, 0, 8), (65, 128, 264, 0, 0),
          (128, 130, 256, 0, 1), (130, 320, 520, 0, 0), (257, 1, 3, 0, 0), (300, 1001, 257, 5, 3), (513, 192, 777, 0, 0),
          (1100, 96, 640, 0, 0)]


@pytest.mark.parametrize("T,K,N,pad,off", LINEAR)
@pytest.mark.parametrize("dt", [F16, BF16])
def test_linear(c, T, K, N, pad, off, dt):
    m = Maker(T * 7 + K)
    fn = R.FNS[(T + K + N) % 7]
    x, w = m(T, K, dt=dt, pad=pad, off=off), m(N, K, dt=dt, std=K ** -0.5, pad=pad, off=off)
    b, r = m(N, dt=dt), m(T, N, dt=dt, pad=pad)
    y = c.linear(x, w, b, fn=FN(fn), residual=r, scale=0.5)
    R.check(y, R.linear(x, w, b, fn, 0.5, r, dt)["y"], "bias, residual")
    assert c.linear(x, w, b, fn=FN(fn), residual=r, scale=0.5).equal(y)  # fixed order
    # no bias, no residual; z kept; rows of a wider output
    buf = torch.full((T + 1, N + 5), 7.0, dtype=dt, device="cuda")
    z = torch.empty(T, N, dtype=dt, device="cuda")
    want = R.linear(x, w, None, fn, 1.0, None, dt)
    c.linear(x, w, fn=FN(fn), z=z, y=buf[:T, :N])
    R.check(buf[:T, :N], want["y"], "plain")
    R.check(z, want["z"], "z")
    assert outside_untouched(buf, (T, N))()


@pytest.mark.parametrize("T,K,N", [(1, 256, 512), (40, 1000, 130), (300, 512, 384)])
def test_linear_adds_into_an_fp32_stream(c, T, K, N):
    m = Maker(5)
    x, w, b = m(T, K, dt=BF16), m(N, K, dt=BF16, std=K ** -0.5), m(N, dt=BF16)
    r = m(T, N, dt=F32, std=3.0)
    want = R.linear(x, w, b, "none", 2.0, r, F32)["y"]
    y = c.linear(x, w, b, residual=r, scale=2.0)
    assert y.dtype == F32
    R.check(y, want)
    c.linear(x, w, b, residual=r, scale=2.0, y=r)  # in place
    assert r.equal(y)


@pytest.mark.parametrize("T,K,N", [(1, 72, 40), (3, 264, 130), (40, 72, 130), (128, 264, 515), (300, 136, 264)])
def test_linear_adds_into_its_residual(c, T, K, N):
    m = Maker(6)
    x, w, r = m(T, K), m(N, K, std=K ** -0.5), m(T, N)
    want = c.linear(x, w, residual=r, fn=pi.PI_FN_SILU)
    c.linear(x, w, residual=r, fn=pi.PI_FN_SILU, y=r)
    assert r.equal(want)


# more tiles than CTA pairs: one round and a bit, several rounds, and a split
# last wave behind whole ones; odd edges
@pytest.mark.parametrize("T,K,N", [(2600, 136, 2056), (5200, 72, 2049), (2600, 4096, 2056)])
def test_linear_of_many_tiles(c, T, K, N):
    m = Maker(7)
    x, w, b, r = m(T, K, dt=BF16), m(N, K, dt=BF16, std=K ** -0.5), m(N, dt=BF16), m(T, N, dt=BF16)
    z = torch.empty(T, N, dtype=BF16, device="cuda")
    want = R.linear(x, w, b, "gelu_tanh", 1.0, r, BF16)
    y = c.linear(x, w, b, fn=pi.PI_FN_GELU_TANH, residual=r, z=z)
    R.check(y, want["y"], "y")
    R.check(z, want["z"], "z")
    R.check(c.linear(x, w), R.linear(x, w, None, "none", 1.0, None, BF16)["y"], "plain")


# backward passes whose products fill up each other's waves, or are split
@pytest.mark.parametrize("T,K,N", [(2304, 1544, 4104), (300, 4104, 2056), (4100, 520, 2056), (200, 264, 9000)])
def test_linear_bwd_of_many_tiles(c, T, K, N):
    m = Maker(8)
    x, w, z, dy = m(T, K), m(N, K, std=K ** -0.5), m(T, N), m(T, N)
    want = R.linear_bwd(dy, x, w, z, "silu", 1.0, F16)
    got = c.linear_bwd(dy, x, w, z, fn=pi.PI_FN_SILU)
    for k, v in zip(("dx", "dw", "db"), got):
        R.check(v, want[k], k)
    for need in ((True, False, False), (False, True, False)):  # alone, each is cut differently
        part = c.linear_bwd(dy, x, w, z, fn=pi.PI_FN_SILU, need=need)
        for k, v in zip(("dx", "dw", "db"), part):
            if v is not None:
                R.check(v, want[k], k + " alone")


# fewer tiles than half of the CTA pairs: narrower ones; thin outputs, whose
# tiles are narrow and split; few tiles of a long k, wide and split
@pytest.mark.parametrize("T,K,N", [(300, 640, 1000), (140, 2056, 300), (9728, 9600, 100), (30000, 136, 128), (200, 12296, 520)])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_linear_and_backward_of_few_or_thin_tiles(c, T, K, N, dt):
    m = Maker(9)
    x, w, b, r = m(T, K, dt=dt), m(N, K, dt=dt, std=K ** -0.5), m(N, dt=dt), m(T, N, dt=dt)
    z, dy = m(T, N, dt=dt), m(T, N, dt=dt)
    R.check(c.linear(x, w), R.linear(x, w, None, "none", 1.0, None, dt)["y"], "plain")
    R.check(c.linear(x, w, b, fn=pi.PI_FN_SILU, residual=r), R.linear(x, w, b, "silu", 1.0, r, dt)["y"], "y")
    want = R.linear_bwd(dy, x, w, z, "relu", 1.0, dt)
    for need in ((True, True, True), (True, False, False), (False, True, False)):
        got = c.linear_bwd(dy, x, w, z, fn=pi.PI_FN_RELU, need=need)
        for k, v in zip(("dx", "dw", "db"), got):
            if v is not None:
                R.check(v, want[k], k)


@pytest.mark.parametrize("fn", R.FNS)
def test_linear_activations_at_their_ends(c, fn):
    """Pre-activations from 0 over the type's range, infinities and NaN:
    an identity product hands x over exactly."""
    v = torch.tensor([0.0, -0.0, 1e-7, -1e-7, 0.5, -0.5, 4.0, -4.0, 12.0, -12.0, 60.0, -60.0, 88.0, -88.0, 200.0, -200.0],
                     device="cuda").to(BF16)
    w = torch.eye(16, device="cuda").to(BF16)
    x = torch.diag(v.float()).to(BF16)
    y = c.linear(x, w, fn=FN(fn)).diagonal()
    want = R.f(fn, v.double())
    # the activation's own bound, plus its relative rounding
    assert bool(((y.double() - want).abs() <= R.act_err(fn, v.double()) * (1 + want.abs()) + R.rnd(want, BF16) + 1e-30).all()), (y, want)
    bad = torch.zeros(3, 16, dtype=BF16, device="cuda")
    bad[0, 0], bad[1, 0] = float("nan"), 1.0
    y = c.linear(bad, torch.ones(8, 16, dtype=BF16, device="cuda"), fn=FN(fn))
    assert bool(y[0].isnan().all()) and bool(y[1:].isfinite().all())  # a NaN stays in its row
    big = torch.full((1, 16), 3e38, dtype=BF16, device="cuda")
    y = c.linear(-big, torch.ones(8, 16, dtype=BF16, device="cuda"), fn=FN(fn))  # z = -inf
    assert bool((y == (0.0 if fn != "none" else float("-inf"))).all()), y


@pytest.mark.parametrize("fn", R.FNS)
@pytest.mark.parametrize("T", [1, 18, 300])
def test_activations_of_infinities(c, fn, T):
    """f and f' at z = inf and -inf are their limits, on every path (few
    tokens, tiles); sums that overflow hand the infinities over."""
    inf = float("inf")
    top = {"none": (inf, -inf), "relu": (inf, 0), "sqrelu": (inf, 0), "sigmoid": (1, 0)}.get(fn, (inf, 0))
    slope = {"none": (1, 1), "relu": (1, 0), "sqrelu": (inf, 0), "sigmoid": (0, 0)}.get(fn, (1, 0))
    w = torch.ones(8, 16, dtype=BF16, device="cuda")
    x = torch.full((T, 16), 3e38, dtype=BF16, device="cuda")
    for k, sign in enumerate((1, -1)):
        assert bool((c.linear(sign * x, w, fn=FN(fn)) == top[k]).all())
        z = torch.full((T, 8), sign * inf, dtype=BF16, device="cuda")
        dy = torch.zeros(T, 8, dtype=BF16, device="cuda")
        dy[0] = 1
        db = torch.empty(8, device="cuda")
        if slope[k] < inf:  # (0 times an infinite slope in the other rows)
            c.linear_bwd(dy, x, w, z, fn=FN(fn), need=(False, False, True), db=db)
            assert bool(((db - slope[k]).abs() < 1e-30).all()), db


def test_sigmoid_derivative_on_both_sides(c):
    """p (1 - p) to within its rounding, however near p is to 0 or 1.  The
    exponential is off by at most 2 + 1.173 |z| steps of 2^-23, 1 / (1 + e) by
    2.5, and three products round: below (1.2 |z| + 10) 2^-23 of the value."""
    z = torch.tensor([0.0, 0.5, 4.0, 8.0, 12.0, 16.0, 20.0, 40.0, 80.0], device="cuda")
    z = torch.cat([z, -z]).to(BF16)[None]
    n = z.shape[1]
    dy, x, w = torch.ones(1, n, dtype=BF16, device="cuda"), torch.zeros(1, n, dtype=BF16, device="cuda"), torch.eye(n, device="cuda").to(BF16)
    db = torch.empty(n, device="cuda")
    kw = dict(fn=pi.PI_FN_SIGMOID)
    c.linear_bwd(dy, x, w, z, need=(False, False, True), db=db, **kw)       # dz itself
    dx = c.linear_bwd(dy, x, w, z, need=(True, False, False), **kw)[0][0]   # dz rounded
    e = torch.exp(-z[0].double().abs())
    want = e / (1 + e) ** 2
    rel = (1.2 * z[0].double().abs() + 10) * 2.0 ** -23
    R.check(db, (want, rel * want), "dz")
    R.check(dx, (want, (rel + R.U[BF16]) * want), "dz rounded")


@pytest.mark.parametrize("T", [1, 18, 300])
@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_gelu_keeps_its_precision_in_the_tail(c, T, dt):
    """z Phi(z) and its derivative Phi(z) + z phi(z), term by term within
    (8 + 4 z^2) 2^-23: the exponential's argument z^2 / 2 rounds twice, the
    exponential is off by 2 + 1.173 z^2 / 2 steps and the factor behind it by
    1.1 (1 + 0.6 z^2), then two products and a division.  An identity product
    hands z over exactly."""
    v = [0.125, 0.5, 1.0, 2.0, 3.0, 3.5, 4.0] + ([] if dt == F16 else [4.5, 5.0, 6.0, 7.5, 9.0, 11.0, 12.5])  # (f16: normal values)
    v = torch.tensor(v + [-a for a in v], device="cuda")
    n, t16 = v.numel(), F16 if dt == F16 else BF16
    x = v.expand(T, n).to(t16)
    w = torch.eye(n, device="cuda").to(t16)
    y = c.linear(x.contiguous(), w, fn=pi.PI_FN_GELU, y=torch.empty(T, n, dtype=dt, device="cuda"))
    z = v.double()
    phi, Phi = torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5, torch.special.erfc(-z / 2 ** 0.5) / 2
    rel = (8 + 4 * z * z) * 2.0 ** -23
    want = z * Phi
    R.check(y, (want.expand(T, n), ((rel + R.U[dt]) * want.abs()).expand(T, n)), "y")
    db = torch.empty(n, device="cuda")
    dy = torch.zeros(T, n, dtype=t16, device="cuda")
    dy[0] = 1
    c.linear_bwd(dy, x.contiguous(), w, x.contiguous(), fn=pi.PI_FN_GELU, need=(False, False, True), db=db)
    R.check(db, (Phi + z * phi, rel * (Phi + z.abs() * phi)), "derivative")


@pytest.mark.parametrize("T,K,N,pad,off", LINEAR)
@pytest.mark.parametrize("dt", [F16, BF16])
def test_linear_bwd(c, T, K, N, pad, off, dt):
    m = Maker(T + K)
    fn = R.FNS[(T + 2 * K + N) % 7]
    x, w = m(T, K, dt=dt, pad=pad, off=off), m(N, K, dt=dt, std=K ** -0.5, pad=pad, off=off)
    z, dy = m(T, N, dt=dt, pad=pad), m(T, N, dt=dt, pad=pad, off=off)
    got = c.linear_bwd(dy, x, w, z, fn=FN(fn))
    want = R.linear_bwd(dy, x, w, z, fn, 1.0, dt)
    for k, v in zip(("dx", "dw", "db"), got):
        R.check(v, want[k], k)
    for v, again in zip(got, c.linear_bwd(dy, x, w, z, fn=FN(fn))):
        assert v.equal(again)
    # fp32 gradients added up; the gradient of an fp32 stream; one output at a time
    dy32 = dy.float() * 1.25
    want = R.linear_bwd(dy32, x, w, z, fn, 0.5, F32)
    dw, db = torch.ones(N, K, device="cuda"), torch.ones(N, device="cuda")
    dx = torch.empty(T, K + 3, dtype=dt, device="cuda")[:, :K]
    c.linear_bwd(dy32, x, w, z, fn=FN(fn), scale=0.5, dx=dx, dw=dw, db=db, accumulate=True)
    R.check(dx, (want["dx"][0], want["dx"][1] + R.rnd(want["dx"][0], dt)), "dx")
    for k, v in (("dw", dw), ("db", db)):
        val, e = want[k]
        R.check(v, (val + 1, e + 2.0 ** -22 * (1 + val.abs())), k)
    only = c.linear_bwd(dy32, x, w, z, fn=FN(fn), scale=0.5, need=(False, False, True))
    assert only[0] is None and only[1] is None
    R.check(only[2], (want["db"][0], want["db"][1] + R.rnd(want["db"][0], dt)), "db alone")


@pytest.mark.parametrize("T,K,N", [(1, 63, 9), (20, 1001, 515), (70, 130, 261), (300, 75, 1029)])
def test_what_lies_beside_the_rows_does_not_matter(c, T, K, N):
    """Rows that end inside a 16-byte chunk, with NaN behind them: none of it
    is read into a result, and none of it is written."""
    m = Maker(15)

    def beside_nan(rows, cols, std=1.0):
        buf = torch.full((rows + 1, (cols + 15) // 8 * 8), float("nan"), dtype=F16, device="cuda")
        buf[:rows, :cols] = m(rows, cols, std=std)
        return buf, buf[:rows, :cols]

    (xb, x), (wb, w), (rb, r) = beside_nan(T, K), beside_nan(N, K, K ** -0.5), beside_nan(T, N)
    (yb, y), (zb, z), (dyb, dy), (dxb, dx) = beside_nan(T, N), beside_nan(T, N), beside_nan(T, N), beside_nan(T, K)
    want = R.linear(x, w, None, "gelu", 1.0, r, F16)
    c.linear(x, w, fn=pi.PI_FN_GELU, residual=r, z=z, y=y)
    R.check(y, want["y"], "y")
    R.check(z, want["z"], "z")
    want = R.linear_bwd(dy, x, w, z, "gelu", 1.0, F16)
    got = c.linear_bwd(dy, x, w, z, fn=pi.PI_FN_GELU, dx=dx)
    for k, v in zip(("dx", "dw", "db"), got):
        R.check(v, want[k], k)
    for buf, cols in ((xb, K), (wb, K), (rb, N), (yb, N), (zb, N), (dyb, N), (dxb, K)):
        assert bool(buf[-1].isnan().all()) and bool(buf[:, cols:].isnan().all())
    (ub, u), (ab, a) = beside_nan(T, N), beside_nan(T, N)
    wd = m(K, N, std=N ** -0.5)
    y = c.gated_ffn(x, None, w, wd, fn=pi.PI_FN_SILU, save=(None, u, a))
    want = R.ffn(x, None, w, wd, None, None, None, "silu")
    R.check(y, want["y"], "ffn y")
    R.check(a, want["a"], "a")
    dy = m(T, K)
    want = R.ffn_bwd(dy, x, None, w, wd, None, u, a, "silu", F16)
    got = c.gated_ffn_bwd(dy, x, None, w, wd, (None, u, a), fn=pi.PI_FN_SILU)
    for k in want:
        R.check(got[k], want[k], k)
    for buf in (ub, ab):
        assert bool(buf[-1].isnan().all()) and bool(buf[:, N:].isnan().all())


def test_linear_bwd_without_activation_takes_dy_itself(c):
    m = Maker(8)
    for T, K, N in ((1, 40, 24), (70, 264, 33)):
        x, w, dy = m(T, K), m(N, K, std=0.1), m(T, N)
        got = c.linear_bwd(dy, x, w)
        want = R.linear_bwd(dy, x, w, None, "none", 1.0, F16)
        for k, v in zip(("dx", "dw", "db"), got):
            R.check(v, want[k], k)


# ------------------------------------------------------------------ gated FFN
FFN = [(1, 64, 200), (1, 1024, 2736), (3, 100, 257), (20, 264, 777), (64, 512, 1000), (65, 130, 384), (200, 192, 515),
       (300, 520, 1025)]


def ffn_weights(m, d, n, dt, gated, bias):
    wg = m(n, d, dt=dt, std=d ** -0.5) if gated else None
    wu, wd = m(n, d, dt=dt, std=d ** -0.5), m(d, n, dt=dt, std=n ** -0.5)
    b = [m(k, dt=dt, std=0.3) if bias and (gated or i) else None for i, k in enumerate((n, n, d))]
    return wg, wu, wd, *b


@pytest.mark.parametrize("T,d,n", FFN)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_gated_ffn_and_backward(c, T, d, n, gated, dt):
    m = Maker(T * 3 + d)
    fn = R.FNS[1 + (T + d + n + gated) % 6]
    wts = ffn_weights(m, d, n, dt, gated, True)
    x, dy = m(T, d, dt=dt), m(T, d, dt=dt)
    want = R.ffn(x, *wts, fn)
    y = c.gated_ffn(x, *wts, fn=FN(fn))
    R.check(y, want["y"], "y")
    save = c.gated_ffn_save(x, wts[0], wts[1])
    assert c.gated_ffn(x, *wts, fn=FN(fn), save=save).equal(y)
    for k, v in zip("gua", save):
        if v is not None:
            R.check(v, want[k], k)
    # packed buffers of odd rows serve as well
    if n % 8:
        packed = tuple(None if v is None else torch.empty(T, n, dtype=dt, device="cuda") for v in save)
        assert c.gated_ffn(x, *wts, fn=FN(fn), save=packed).equal(y)
        assert all(v is None or v.equal(p) for v, p in zip(save, packed))
        save = packed
    want = R.ffn_bwd(dy, x, *wts[:3], *save, fn, dt)
    got = c.gated_ffn_bwd(dy, x, *wts[:3], save, fn=FN(fn))
    assert set(k for k in got if got[k] is not None) == set(want)
    for k in want:
        R.check(got[k], want[k], k)
    again = c.gated_ffn_bwd(dy, x, *wts[:3], save, fn=FN(fn))
    assert all(got[k].equal(again[k]) for k in want)
    # fp32 gradients, added to what is there
    want = R.ffn_bwd(dy, x, *wts[:3], *save, fn, F32)
    gr = {k: torch.full_like(want[k][0], 2.0, dtype=F32) for k in want if k != "dx"}
    got = c.gated_ffn_bwd(dy, x, *wts[:3], save, fn=FN(fn), grads=gr, accumulate=True, need_dx=False)
    assert got["dx"] is None
    for k in gr:
        val, e = want[k]
        R.check(gr[k], (val + 2, e + 2.0 ** -22 * (2 + val.abs())), k)


def test_gated_ffn_of_many_tiles(c):
    m = Maker(19)
    T, d, n = 700, 776, 3080
    wts = ffn_weights(m, d, n, BF16, True, True)
    x, dy = m(T, d, dt=BF16), m(T, d, dt=BF16)
    save = c.gated_ffn_save(x, wts[0], wts[1])
    want = R.ffn(x, *wts, "none")
    R.check(c.gated_ffn(x, *wts, fn=pi.PI_FN_NONE, save=save), want["y"], "y")
    want = R.ffn_bwd(dy, x, *wts[:3], *save, "none", BF16)
    got = c.gated_ffn_bwd(dy, x, *wts[:3], save, fn=pi.PI_FN_NONE)
    for k in want:
        R.check(got[k], want[k], k)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_gradients_accumulate_in_16_bits(c, T):
    m = Maker(20)
    d, n = 136, 264
    wts = ffn_weights(m, d, n, F16, True, True)
    x, dy = m(T, d), m(T, d)
    save = c.gated_ffn_save(x, wts[0], wts[1])
    c.gated_ffn(x, *wts, fn=pi.PI_FN_GELU, save=save)
    want = R.ffn_bwd(dy, x, *wts[:3], *save, "gelu", F32)
    gr = {k: torch.full_like(want[k][0], 2.0, dtype=F16) for k in want if k != "dx"}
    c.gated_ffn_bwd(dy, x, *wts[:3], save, fn=pi.PI_FN_GELU, grads=gr, accumulate=True)
    for k in gr:
        val, e = want[k][0] + 2, want[k][1]
        R.check(gr[k], (val, e + 2.0 ** -22 * (2 + val.abs()) + R.rnd(val, F16)), k)


def test_gated_ffn_partial_gradients(c):
    m = Maker(9)
    wts = ffn_weights(m, 72, 130, BF16, True, False)
    x, dy = m(10, 72, dt=BF16, pad=8), m(10, 72, dt=BF16)
    save = c.gated_ffn_save(x, wts[0], wts[1])
    c.gated_ffn(x, *wts, fn=pi.PI_FN_SILU, save=save)
    want = R.ffn_bwd(dy, x, *wts[:3], *save, "silu", BF16)
    for keys in (["w_down"], ["b_down"], ["b_gate"], ["w_up"], ["w_gate", "b_up"]):
        gr = {k: torch.empty(want[k][0].shape, dtype=BF16, device="cuda") for k in keys}
        got = c.gated_ffn_bwd(dy, x, *wts[:3], save, fn=pi.PI_FN_SILU, grads=gr, need_dx=False)
        for k in keys:
            R.check(got[k], want[k], k)
    R.check(c.gated_ffn_bwd(dy, x, *wts[:3], save, fn=pi.PI_FN_SILU, weight_grads=False, bias_grads=False)["dx"],
            want["dx"], "dx")


# ------------------------------------------------------------------ norms
NORM = [(1, 8, 0), (1, 8192, 0), (1, 16384, 1), (3, 1, 2), (5, 33, 1), (64, 1000, 0), (65, 256, 7), (130, 1001, 64),
        (200, 2048, 70), (33, 8200, 5), (5, 64, 100)]
# rows that follow one another through the rings of the pipelined kernels: many
# per CTA, gate rows that end inside a CTA's tokens and that span several CTAs,
# more gate rows than lanes that join them
NORM_LONG = [(310, 8192, 0), (400, 4104, 100), (620, 1000, 7), (1000, 2048, 70), (700, 8192, 1), (2000, 72, 3),
             (5000, 8, 0), (1400, 4096, 701)]


@pytest.mark.parametrize("T,d,rows", NORM)
@pytest.mark.parametrize("pre,post", [("rms", "none"), ("rms", "rms"), ("layer", "layer"), ("none", "rms"),
                                      ("layer", "none"), ("none", "none")])
@pytest.mark.parametrize("xdt,dt", [(F32, BF16), (F16, F16), (F32, F16)])
def test_norm_residual_and_backward(c, T, d, rows, pre, post, xdt, dt):
    norm_case(c, T, d, rows, pre, post, xdt, dt)


@pytest.mark.parametrize("T,d,rows", NORM_LONG)
@pytest.mark.parametrize("pre,post,xdt,dt", [("rms", "rms", F32, BF16), ("layer", "layer", BF16, BF16), ("rms", "none", F16, F16),
                                             ("layer", "none", F32, F16), ("none", "layer", F32, BF16)])
def test_norm_of_many_rows(c, T, d, rows, pre, post, xdt, dt):
    norm_case(c, T, d, rows, pre, post, xdt, dt)


def norm_case(c, T, d, rows, pre, post, xdt, dt):
    m = Maker(T + d)
    eps = 1e-3  # (a row of one element has no variance)
    x, y = m(T, d, dt=xdt, std=2.0), m(T, d, dt=dt)
    gate = m(1 if rows == 0 else -(-T // rows), d, dt=dt)
    wp, bp = (m(d, dt=dt), m(d, dt=dt)) if pre != "none" else (None, None)
    wq, bq = (m(d, dt=dt), m(d, dt=dt)) if post != "none" else (None, None)
    kw = dict(pre=KIND[pre], post=KIND[post], w_pre=wp, b_pre=bp, w_post=wq, b_post=bq, res_scale=0.75,
              branch_scale=1.5, gate_rows=rows, eps=eps)
    want = R.norm_fwd(x, y, gate, rows, pre, post, wp, bp, wq, bq, 0.75, 1.5, eps, dt)
    xo, h = c.norm_residual(x, y, gate, **kw)
    R.check(xo, want["x"], "x")
    assert (h is None) == (pre == "none")
    if h is not None:
        R.check(h, want["h"], "h")
    xin = x.clone()
    c.norm_residual(xin, y, gate, x_out=xin, **kw)  # in place
    assert xin.equal(xo)

    dxo, dh = m(T, d, dt=xdt), (m(T, d, dt=dt) if pre != "none" else None)
    want = R.norm_bwd(dxo, dh, xo, y, gate, rows, pre, post, wp, wq, bq, 0.75, 1.5, eps, dt, dt)
    got = c.norm_residual_bwd(dxo, dh, xo, y, gate, **kw)
    assert set(k for k in got if got[k] is not None) == set(want)
    for k in want:
        R.check(got[k], want[k], k)
    again = c.norm_residual_bwd(dxo, dh, xo, y, gate, **kw)
    assert all(got[k].equal(again[k]) for k in want)
    # fp32 gradients, added to what is there; no gradient of the stream itself
    if dh is not None:
        want = R.norm_bwd(None, dh, xo, y, gate, rows, pre, post, wp, wq, bq, 0.75, 1.5, eps, dt, F32)
        gr = {k: torch.full_like(want[k][0], 2.0, dtype=F32) for k in want if k not in ("dx", "dy")}
        got = c.norm_residual_bwd(None, dh, xo, y, gate, grads=gr, accumulate=True, **kw)
        for k in want:
            val, e = want[k]
            R.check(got[k], (val + 2, e + 2.0 ** -22 * (2 + val.abs())) if k in gr else (val, e), k)


@pytest.mark.parametrize("T,d", [(1, 40), (7, 1000)])
def test_norm_without_a_block_and_without_parameters(c, T, d):
    m = Maker(11)
    x = m(T, d, dt=F32, pad=4)
    want = R.norm_fwd(x, None, None, 0, "rms", "none", None, None, None, None, 1.0, 1.0, 1e-5, BF16)
    xo, h = c.norm_residual(x, dtype=BF16)
    R.check(xo, want["x"], "x")
    R.check(h, want["h"], "h")
    dh = m(T, d, dt=BF16, pad=8)
    got = c.norm_residual_bwd(None, dh, xo)
    R.check(got["dx"], R.norm_bwd(None, dh, xo, None, None, 0, "rms", "none", None, None, None, 1.0, 1.0, 1e-5, BF16,
                                  BF16)["dx"], "dx")


@pytest.mark.parametrize("T,d", [(5, 1), (9, 33), (9, 65), (7, 1001), (3, 8200), (400, 33), (400, 1000), (310, 4104)])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("given", ["", "w", "b"])
def test_norm_around_a_block_without_gate_and_without_parameters(c, T, d, pre, post, given):
    """Weights, biases and gate that are not there stand for 1, 0 and 1; y
    has a mean, so that what a layer norm takes away shows wherever it stays."""
    m = Maker(T + d)
    x, y = m(T, d, dt=F32, std=2.0), m(T, d, dt=BF16) + 3
    par = lambda kind, which: m(d, dt=BF16) if kind != "none" and given == which else None
    wp, wq, bp, bq = par(pre, "w"), par(post, "w"), par(pre, "b"), par(post, "b")
    kw = dict(pre=KIND[pre], post=KIND[post], w_pre=wp, b_pre=bp, w_post=wq, b_post=bq, eps=1e-3)
    want = R.norm_fwd(x, y, None, 0, pre, post, wp, bp, wq, bq, 1.0, 1.0, 1e-3, BF16)
    xo, h = c.norm_residual(x, y, **kw)
    R.check(xo, want["x"], "x")
    if h is not None:
        R.check(h, want["h"], "h")
    dxo, dh = m(T, d, dt=F32), (m(T, d, dt=BF16) if pre != "none" else None)
    want = R.norm_bwd(dxo, dh, xo, y, None, 0, pre, post, wp, wq, bq, 1.0, 1.0, 1e-3, BF16, BF16)
    got = c.norm_residual_bwd(dxo, dh, xo, y, **kw)
    assert set(k for k in got if got[k] is not None) == \
        {"dx", "dy"} | {k for k, v in dict(w_pre=wp, b_pre=bp, w_post=wq, b_post=bq).items() if v is not None}
    for k in want:
        if got[k] is not None:
            R.check(got[k], want[k], k)


@pytest.mark.parametrize("off,pad", [(1, 2), (8, 8)])
def test_norm_of_slices(c, off, pad):
    """Rows that start anywhere in wider ones, and outputs that leave the rest alone."""
    m = Maker(12)
    T, d = 9, 120
    x, y, gate = m(T, d, dt=F32, off=off, pad=pad), m(T, d, off=off, pad=pad), m(1, d, off=off)
    w = m(d, off=off)
    bx, bh = torch.full((T, d + 6), 7.0, device="cuda"), torch.full((T, d + 6), 7.0, dtype=F16, device="cuda")
    c.norm_residual(x, y, gate, w_pre=w, x_out=bx[:, :d], h=bh[:, :d])
    want = R.norm_fwd(x, y, gate, 0, "rms", "none", w, None, None, None, 1.0, 1.0, 1e-5, F16)
    R.check(bx[:, :d], want["x"], "x")
    R.check(bh[:, :d], want["h"], "h")
    assert bool((bx[:, d:] == 7).all()) and bool((bh[:, d:] == 7).all())
    dh = m(T, d, off=off, pad=pad)
    want = R.norm_bwd(bx[:, :d], dh, bx[:, :d], y, gate, 0, "rms", "none", w, None, None, 1.0, 1.0, 1e-5, F16, F16)
    got = c.norm_residual_bwd(bx[:, :d], dh, bx[:, :d], y, gate, w_pre=w)
    assert set(want) - set(k for k in got if got[k] is not None) == {"b_pre"}  # (there is no b_pre)
    for k in set(want) - {"b_pre"}:
        R.check(got[k], want[k], k)


@pytest.mark.parametrize("T,d", [(1, 40), (9, 120), (400, 1000), (400, 33)])
@pytest.mark.parametrize("wide", ["x_out", "dx_out"])
def test_norm_bwd_of_a_stream_and_a_gradient_with_their_own_strides(c, T, d, wide):
    m = Maker(23)
    x, dxo = m(T, d, dt=F32, pad=8 * (wide == "x_out")), m(T, d, dt=F32, pad=4 * (wide == "dx_out"))
    y, dh, w = m(T, d), m(T, d), m(d)
    want = R.norm_bwd(dxo, dh, x, y, None, 0, "rms", "none", w, None, None, 1.0, 1.0, 1e-5, F16, F16)
    got = c.norm_residual_bwd(dxo, dh, x, y, w_pre=w)
    for k in ("dx", "dy", "w_pre"):
        R.check(got[k], want[k], k)


def test_norm_bwd_refuses_a_stride_below_the_row(c):
    t = torch.zeros(64, dtype=F16, device="cuda")
    lib, p = pi.load_library(), t.data_ptr()
    par, g = pi.pi_norm_residual_params(), pi.pi_norm_residual_grads(p)
    for ld in (7, -8):
        d = pi.pi_norm_residual_desc(2, 8, 0, 0, 0, 1, 0, 0, 1.0, 1.0, 1e-5, 0, 0, 0, 0, 0, ld)
        assert lib.pi_norm_residual_bwd(c.handle, pi._ref(d), pi._ref(par), p, p, p, None, None, pi._ref(g), 0, None, 0) == pi.PI_ERR_SHAPE
    c.check()


def test_norm_parameters_that_nothing_uses_have_no_gradient(c):
    """The forward pass ignores the parameters of a norm that is not there, and
    the gate and the norm of a block that is not there; so does the backward pass."""
    m = Maker(24)
    T, d = 6, 40
    x, y, dxo, dh, w, b, gate = m(T, d, dt=F32), m(T, d), m(T, d, dt=F32), m(T, d), m(d), m(d), m(1, d)
    par = dict(w_pre=w, b_pre=b, w_post=w, b_post=b)
    # no post norm
    xo, h = c.norm_residual(x, y, gate, **par)
    want = R.norm_bwd(dxo, dh, xo, y, gate, 0, "rms", "none", w, w, b, 1.0, 1.0, 1e-5, F16, F16)
    got = c.norm_residual_bwd(dxo, dh, xo, y, gate, **par)
    assert set(k for k in got if got[k] is not None) == {"dx", "dy", "gate", "w_pre", "b_pre"} == set(want)
    for k in want:
        R.check(got[k], want[k], k)
    # no pre norm
    kw = dict(pre=pi.PI_NORM_NONE, post=pi.PI_NORM_LAYER)
    xo, h = c.norm_residual(x, y, gate, **par, **kw)
    want = R.norm_bwd(dxo, None, xo, y, gate, 0, "none", "layer", None, w, b, 1.0, 1.0, 1e-5, F16, F16)
    got = c.norm_residual_bwd(dxo, None, xo, y, gate, **par, **kw)
    assert h is None and set(k for k in got if got[k] is not None) == {"dx", "dy", "gate", "w_post", "b_post"} == set(want)
    for k in want:
        R.check(got[k], want[k], k)
    # no block
    kw = dict(post=pi.PI_NORM_RMS)
    xo, h = c.norm_residual(x, None, gate, dtype=F16, **par, **kw)
    want = R.norm_bwd(dxo, dh, xo, None, None, 0, "rms", "none", w, None, None, 1.0, 1.0, 1e-5, F16, F16)
    got = c.norm_residual_bwd(dxo, dh, xo, None, gate, **par, **kw)
    assert set(k for k in got if got[k] is not None) == {"dx", "w_pre", "b_pre"} == set(want)
    for k in want:
        R.check(got[k], want[k], k)


def test_norm_rows_of_zeros_and_of_nan(c):
    x = torch.zeros(4, 64, device="cuda")
    x[1] = float("nan")
    x[2, 3] = float("inf")
    x[3] = 1.0
    _, h = c.norm_residual(x, dtype=F16, eps=1e-5)
    assert bool((h[0] == 0).all()) and bool(h[1].isnan().all()) and not bool(h[2].isfinite().all())
    assert bool((h[3] == 1).all())
    _, h = c.norm_residual(x, dtype=F16, pre=pi.PI_NORM_LAYER)
    assert bool((h[0] == 0).all()) and bool((h[3] == 0).all())


# ------------------------------------------------------------------ no tokens, refusals, streams, graphs
def test_no_tokens(c):
    e = lambda *s, dt=F16: torch.empty(*s, dtype=dt, device="cuda")
    assert c.linear(e(0, 16), e(8, 16)).shape == (0, 8)
    dx, dw, db = c.linear_bwd(e(0, 8), e(0, 16), e(8, 16))
    assert dx.shape == (0, 16) and not dw.any() and not db.any()
    dw = torch.ones(8, 16, dtype=F16, device="cuda")
    c.linear_bwd(e(0, 8), e(0, 16), e(8, 16), dw=dw, need=(False, True, False), accumulate=True)
    assert bool((dw == 1).all())
    save = c.gated_ffn_save(e(0, 16), e(24, 16), e(24, 16))
    assert c.gated_ffn(e(0, 16), e(24, 16), e(24, 16), e(16, 24), save=save).shape == (0, 16)
    got = c.gated_ffn_bwd(e(0, 16), e(0, 16), e(24, 16), e(24, 16), e(16, 24), save)
    assert all(not v.any() for v in got.values())
    xo, h = c.norm_residual(e(0, 16), e(0, 16), e(1, 16))
    assert xo.shape == h.shape == (0, 16)
    got = c.norm_residual_bwd(None, e(0, 16), e(0, 16), e(0, 16), e(1, 16), w_pre=e(16))
    assert not got["w_pre"].any() and not got["gate"].any()


def test_library_refuses_bad_arguments(c):
    """Host-side checks of the C entry points: nothing is launched."""
    t = torch.zeros(64, dtype=F16, device="cuda")
    ok = lambda **k: pi.pi_linear_desc(*[k.get(n, v) for n, v in
                                         (("T", 2), ("K", 8), ("N", 4), ("dtype", 0), ("out_dtype", 0), ("grad_dtype", 0),
                                          ("fn", 0), ("scale", 1.0), ("unaligned", 0), ("ldx", 0), ("ldw", 0),
                                          ("ldz", 0), ("ldr", 0), ("ldy", 0), ("lddx", 0), ("lddw", 0))])
    lib, h = pi.load_library(), c.handle

    def status(fun, *a):
        n = ctypes.c_size_t()
        return fun(h, *a, ctypes.addressof(n))

    assert status(lib.pi_linear_workspace, pi._ref(ok()), 0) == pi.PI_OK
    for bad, want in ((dict(T=-1), pi.PI_ERR_SHAPE), (dict(K=0), pi.PI_ERR_SHAPE), (dict(N=(1 << 20) + 1), pi.PI_ERR_SHAPE),
                      (dict(dtype=2), pi.PI_ERR_ARG), (dict(out_dtype=1), pi.PI_ERR_ARG), (dict(fn=7), pi.PI_ERR_ARG),
                      (dict(scale=float("nan")), pi.PI_ERR_ARG), (dict(ldx=7), pi.PI_ERR_SHAPE),
                      (dict(lddw=1), pi.PI_ERR_SHAPE)):
        assert status(lib.pi_linear_workspace, pi._ref(ok(**bad)), 1) == want, bad
    assert pi.pi_last_error(h)
    p = t.data_ptr()
    d = ok()
    assert lib.pi_linear(h, pi._ref(d), p, None, None, None, None, p, None, 0) == pi.PI_ERR_ARG
    # a misaligned operand needs a workspace, which is checked before any launch
    assert lib.pi_linear(h, pi._ref(d), p + 2, p, None, None, None, p, None, 0) == pi.PI_ERR_ARG
    assert "workspace" in pi.pi_last_error(h)
    assert lib.pi_linear_bwd(h, pi._ref(ok(fn=1)), p, p, p, None, p, p, p, 0, None, 0) == pi.PI_ERR_ARG  # z
    f = pi.pi_gated_ffn_desc(2, 8, 16, 0, 0, 1, 1, 0, *[0] * 8)
    wts = pi.pi_gated_ffn_weights(p, p, p, None, None, None)
    none = pi.pi_gated_ffn_weights(None, p, p, None, None, None)
    assert lib.pi_gated_ffn(h, pi._ref(f), pi._ref(none), p, None, p, None, 0) == pi.PI_ERR_ARG
    assert lib.pi_gated_ffn(h, pi._ref(f), pi._ref(wts), p, None, p, None, 0) == pi.PI_ERR_ARG  # workspace
    f.gated = 0
    assert lib.pi_gated_ffn(h, pi._ref(f), pi._ref(wts), p, None, p, None, 0) == pi.PI_ERR_ARG
    nd = pi.pi_norm_residual_desc(2, 8, 0, 0, 0, 1, 0, 0, 1.0, 1.0, 1e-5, *[0] * 5)
    assert lib.pi_norm_residual(h, pi._ref(nd), None, p, None, None, p, None) == pi.PI_ERR_ARG  # h
    nd.pre = 3
    assert lib.pi_norm_residual(h, pi._ref(nd), None, p, None, None, p, p) == pi.PI_ERR_ARG
    nd.pre, nd.d = 1, 16385
    assert lib.pi_norm_residual(h, pi._ref(nd), None, p, None, None, p, p) == pi.PI_ERR_SHAPE
    nd.d, nd.eps = 8, -1.0
    assert lib.pi_norm_residual(h, pi._ref(nd), None, p, None, None, p, p) == pi.PI_ERR_ARG
    c.check()


def test_library_refuses_addresses_between_two_elements(c):
    """Every buffer of every call, moved by one byte (16-bit elements) or by
    two (fp32): refused before anything is planned or launched."""
    t = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    lib, h, p = pi.load_library(), c.handle, t.data_ptr()

    def each(fun, args, at):
        """fun with args, moved in one place at a time; at: {index in args: bytes}"""
        for i, by in at.items():
            moved = list(args)
            moved[i] += by
            assert fun(*moved) == pi.PI_ERR_ARG, i
            assert "element" in pi.pi_last_error(h), i

    lin = pi.pi_linear_desc(2, 8, 8, 0, pi.PI_F32, pi.PI_F32, pi.PI_FN_RELU, 1.0, 1, *[0] * 7)
    each(lambda *a: lib.pi_linear(h, pi._ref(lin), *a, p, 1 << 16), [p] * 6, {0: 1, 1: 1, 2: 1, 3: 2, 4: 1, 5: 2})
    each(lambda *a: lib.pi_linear_bwd(h, pi._ref(lin), *a, 0, p, 1 << 16), [p] * 7, {0: 2, 1: 1, 2: 1, 3: 1, 4: 1, 5: 2, 6: 2})
    ffn = pi.pi_gated_ffn_desc(2, 8, 8, 0, pi.PI_F32, pi.PI_FN_RELU, 1, 1, *[0] * 8)

    def ffn_fwd(*a):
        w, s = pi.pi_gated_ffn_weights(*a[:6]), pi.pi_gated_ffn_save(*a[6:9])
        return lib.pi_gated_ffn(h, pi._ref(ffn), pi._ref(w), a[9], pi._ref(s), a[10], p, 1 << 16)

    def ffn_bwd(*a):
        w, s, g = pi.pi_gated_ffn_weights(*a[:3], None, None, None), pi.pi_gated_ffn_save(*a[3:6]), pi.pi_gated_ffn_grads(*a[6:12])
        return lib.pi_gated_ffn_bwd(h, pi._ref(ffn), pi._ref(w), a[12], a[13], pi._ref(s), a[14], pi._ref(g), 0, p, 1 << 16)

    each(ffn_fwd, [p] * 11, {i: 1 for i in range(11)})
    each(ffn_bwd, [p] * 15, {i: 2 if 6 <= i < 12 else 1 for i in range(15)})
    nd = pi.pi_norm_residual_desc(2, 8, pi.PI_F32, 0, pi.PI_F32, 1, 1, 0, 1.0, 1.0, 1e-5, *[0] * 5)

    def norm(*a):
        par = pi.pi_norm_residual_params(*a[:4])
        return lib.pi_norm_residual(h, pi._ref(nd), pi._ref(par), *a[4:])

    def norm_bwd(*a):
        par, g = pi.pi_norm_residual_params(*a[:4]), pi.pi_norm_residual_grads(*a[9:])
        return lib.pi_norm_residual_bwd(h, pi._ref(nd), pi._ref(par), *a[4:9], pi._ref(g), 0, p, 1 << 16)

    each(norm, [p] * 9, {**{i: 1 for i in range(9)}, 4: 2, 7: 2})
    each(norm_bwd, [p] * 16, {**{i: 1 for i in range(9)}, 4: 2, 6: 2, 9: 2, 10: 1, **{i: 2 for i in range(11, 16)}})
    c.check()


def block(c, x, y0, gate, wts, w, fn):
    """x' and h after the norm, the FFN of h, and the next norm's outputs."""
    x1, h1 = c.norm_residual(x, y0, gate, w_pre=w)
    save = c.gated_ffn_save(h1, wts[0], wts[1])
    y1 = c.gated_ffn(h1, *wts, fn=fn, save=save)
    x2, h2 = c.norm_residual(x1, y1, gate, w_pre=w, post=pi.PI_NORM_RMS)
    return x1, h1, save, y1, x2, h2


def block_bwd(c, dx2, dh2, x1, h1, save, y1, x2, y0, gate, wts, w, fn):
    g2 = c.norm_residual_bwd(dx2, dh2, x2, y1, gate, w_pre=w, post=pi.PI_NORM_RMS)
    gf = c.gated_ffn_bwd(g2["dy"], h1, *wts[:3], save, fn=fn)
    g1 = c.norm_residual_bwd(g2["dx"], gf["dx"], x1, y0, gate, w_pre=w)
    return g1, gf, g2


@pytest.mark.parametrize("T,d,n", [(1, 256, 640), (70, 264, 515), (300, 512, 1024)])
def test_a_block_forward_and_backward(c, T, d, n):
    """norm -> gated FFN -> norm and its backward pass as a training step
    runs them, against autograd in 64 bits.  Every hand-over is rounded to 16
    bits (8 roundings in all): the 2-norm of the error stays below 8 half
    steps of the type times 2 for their spread through the norms."""
    m = Maker(13)
    dt = BF16
    wts = ffn_weights(m, d, n, dt, True, True)
    w = m(d, dt=dt, std=0.2) + 1
    x, y0, gate = m(T, d, dt=F32, std=2.0), m(T, d, dt=dt), m(1, d, dt=dt)
    dx2, dh2 = m(T, d, dt=F32), m(T, d, dt=dt)
    x1, h1, save, y1, x2, h2 = block(c, x, y0, gate, wts, w, pi.PI_FN_SILU)
    g1, gf, g2 = block_bwd(c, dx2, dh2, x1, h1, save, y1, x2, y0, gate, wts, w, pi.PI_FN_SILU)

    leaf = {k: v.double().requires_grad_(True) for k, v in
            dict(x=x, y0=y0, gate=gate, w=w, wg=wts[0], wu=wts[1], wd=wts[2], bg=wts[3], bu=wts[4], bd=wts[5]).items()}
    rms = lambda v: v / (v.pow(2).mean(1, keepdim=True) + 1e-5).sqrt()
    X1 = leaf["x"] + leaf["gate"] * leaf["y0"]
    H1 = rms(X1) * leaf["w"]
    A = torch.nn.functional.silu(H1 @ leaf["wg"].T + leaf["bg"]) * (H1 @ leaf["wu"].T + leaf["bu"])
    Y1 = A @ leaf["wd"].T + leaf["bd"]
    X2 = X1 + leaf["gate"] * rms(Y1)
    H2 = rms(X2) * leaf["w"]
    ((X2 * dx2.double()).sum() + (H2 * dh2.double()).sum()).backward()
    tol = 16 * R.U[dt]

    def near(got, want, what):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= tol, (what, rel)

    near(x2, X2.detach(), "x2")
    near(h2, H2.detach(), "h2")
    near(g1["dx"], leaf["x"].grad, "dx")
    near(g1["dy"], leaf["y0"].grad, "dy0")
    near(g1["gate"].float() + g2["gate"].float(), leaf["gate"].grad, "gate")
    near(g1["w_pre"].float() + g2["w_pre"].float(), leaf["w"].grad, "w")
    for k, name in (("w_gate", "wg"), ("w_up", "wu"), ("w_down", "wd"), ("b_gate", "bg"), ("b_up", "bu"), ("b_down", "bd")):
        near(gf[k], leaf[name].grad, k)


def test_captured_and_replayed_beside_eager_calls(c):
    """A training step in a graph, replayed on new inputs while another graph
    and eager calls use the same context: each has its own workspace."""
    dt, T, d, n = BF16, 40, 136, 264
    m = Maker(14)
    wts = ffn_weights(m, d, n, dt, True, True)
    w, gate = m(d, dt=dt), m(1, d, dt=dt)
    bufs = [dict(x=m(T, d, dt=F32), y0=m(T, d, dt=dt), dx2=m(T, d, dt=F32), dh2=m(T, d, dt=dt)) for _ in range(2)]

    def step(b):
        f = block(c, b["x"], b["y0"], gate, wts, w, pi.PI_FN_SILU)
        g1, gf, g2 = block_bwd(c, b["dx2"], b["dh2"], f[0], f[1], f[2], f[3], f[4], b["y0"], gate, wts, w, pi.PI_FN_SILU)
        return [f[4], f[5], g1["dx"], gf["w_up"], gf["b_gate"], g2["w_pre"]]

    step(bufs[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(b))
        graphs.append(g)
    for b in bufs:
        for k, v in b.items():
            b[k].copy_(m(*v.shape, dt=v.dtype))
    eager = [step(b) for b in bufs]
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    with torch.cuda.stream(s2):
        other = step(bufs[0])
    torch.cuda.current_stream().wait_stream(s2)
    torch.cuda.synchronize()
    for want, got in zip(eager + [eager[0]], outs + [other]):
        for a, b in zip(want, got):
            assert a.equal(b)


@pytest.mark.parametrize("T", [40, 300])
def test_a_wait_that_runs_out_is_reported(T):
    """With a wait limit of a nanosecond the products' waits run out: the
    kernels return, the status says so, and the context goes on working."""
    ctx = G.ctx()
    try:
        m = Maker(21)
        x, w = m(T, 2048), m(512, 2048, std=0.02)
        want = ctx.linear(x, w)
        ctx.check()
        pi.pi_debug_set_wait_limit(ctx.handle, 1)
        status = 0
        for _ in range(5):  # (a wait may be over before the clock is read)
            ctx.linear(x, w)
            status = ctx.sync_status() or status  # (which also clears it)
        assert status == pi.PI_ERR_TIMEOUT
        pi.pi_debug_set_wait_limit(ctx.handle, 2_000_000_000)
        assert ctx.linear(x, w).equal(want)
        ctx.check()
    finally:
        ctx.close()


def test_two_threads_with_a_context_each():
    """A context belongs to one thread, two contexts of a device need not: calls
    of one size do not disturb the launches of another (a kernel's
    shared-memory limit belongs to the function, not to the call).  The C entry
    point itself is called, so that the threads spend their time in the library."""
    lib, sizes, T = pi.load_library(), (64, 4096), 400
    ctxs = [G.ctx() for _ in sizes]
    failed = []
    m = Maker(22)
    bufs = {d: [m(T, d), m(T, d), torch.empty(T, d, dtype=F16, device="cuda"), torch.empty(T, d, dtype=F16, device="cuda")]
            for d in sizes}
    torch.cuda.synchronize()

    def work(ctx, d):
        desc = pi.pi_norm_residual_desc(T, d, 0, 0, 0, pi.PI_NORM_RMS, 0, 0, 1.0, 1.0, 1e-5, *[0] * 5)
        par = pi.pi_norm_residual_params()
        x, y, xo, h = (t.data_ptr() for t in bufs[d])
        call = (ctx.handle, pi._ref(desc), pi._ref(par), x, y, None, xo, h)
        failed.extend(d for _ in range(5000) if lib.pi_norm_residual(*call))

    try:
        threads = [threading.Thread(target=work, args=a) for a in zip(ctxs, sizes)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        for ctx in ctxs:
            ctx.check()
        assert not failed, (len(failed), pi.pi_last_error(ctxs[1].handle))
        for x, y, xo, h in bufs.values():
            want = R.norm_fwd(x, y, None, 0, "rms", "none", None, None, None, None, 1.0, 1.0, 1e-5, F16)
            R.check(xo, want["x"], "x")
            R.check(h, want["h"], "h")
    finally:
        for ctx in ctxs:
            ctx.close()


def test_same_block_as_the_loaded_layer(c):
    """The dense path of a loaded ReGLU layer and the block operators agree
    (the loaded layer's own tolerance), norm and residual included."""
    cfg = W.LayerConfig("reglu_bf16", 264, 777, 32, 1, W.REGLU, W.BF16, W.BF16, alpha=0.7, cfg_id=202)
    layer = W.make_layer(cfg, 0, 0, random_b1=True, random_bdown=True)
    ctx = G.ctx(max_layers=1, max_batch=64)
    try:
        ctx.load_layer(0, layer)
        t = lambda k: torch.from_numpy(np.ascontiguousarray(layer[k]).view(np.int16)).cuda().view(BF16)
        for B in (1, 5, 64):
            x = torch.from_numpy(W.decode_inputs(cfg, B, 3).copy()).cuda()
            _, xh = ctx.norm_residual(x, dtype=BF16)
            want = ctx.dense_ffn(0, xh.view(torch.int16))
            got = ctx.gated_ffn(xh, t("w_gate"), t("w_up"), t("w_down"), t("b"), None, t("b_down"))
            assert max_rel_err(got.double().cpu().numpy(), want.double().cpu().numpy()) <= 2e-2
            x2, _ = ctx.norm_residual(x, got, pre=pi.PI_NORM_NONE)
            ctx.dense_step(x)
            assert max_rel_err(x2.double().cpu().numpy(), x.double().cpu().numpy()) <= 1e-2
        ctx.check()
    finally:
        ctx.close()
