"""The microscaled operators (quantisation, linear layer, gated FFN, norms with
a microscaled output) against their 64-bit references, within the bounds that
tests/_mx.py derives from the arithmetic."""
from __future__ import annotations

import ctypes
import math
import threading

import pytest
import torch

from activation_sparse_decode_sigmoid_gb300 import pi
from tests import _block as R
from tests import _gpu as G
from tests import _mx as X

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
MX8, MX4 = pi.PI_MX8, pi.PI_MX4
KINDS = [(MX8, MX4), (MX8, MX8), (MX4, MX4)]
NORM = {"none": pi.PI_NORM_NONE, "rms": pi.PI_NORM_RMS, "layer": pi.PI_NORM_LAYER}


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

    def mx(self, c, rows, cols, kind, std=1.0):
        return c.mx_quantize(self(rows, cols, dt=F32, std=std), kind)


def same(q, want):
    """An MxMatrix against quantize()'s codes and scales; what pads it is 0."""
    codes, scales, pad = X.unpack(q)
    assert pad
    assert torch.equal(scales, want[1])
    bad = (codes != want[0]).nonzero()
    assert not len(bad), (len(bad), bad[0], codes[tuple(bad[0])], want[0][tuple(bad[0])])


# ------------------------------------------------------------------ quantisation
SIZES = [(1, 1), (1, 32), (2, 31), (3, 33), (5, 128), (31, 129), (33, 100), (127, 257), (128, 256), (129, 1000), (300, 1001),
         (1, 8192), (1000, 520)]


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("kind", [MX8, MX4])
def test_quantize(c, T, K, dt, kind):
    m = Maker(T + K)
    for pad, off in ((0, 0), (8, 0), (3, 1)):
        x = m(T, K, dt=dt, pad=pad, off=off).mul_(torch.exp(2 * torch.randn(T, 1, generator=m.g, device="cuda")).to(dt))
        x[T // 2, : K // 2] = 0
        q = c.mx_quantize(x, kind)
        want = X.quantize(kind, x.double())
        same(q, want)
        for out in (F32, BF16):
            assert torch.equal(c.mx_dequantize(q, out).double(), want[2])
        assert torch.equal(c.mx_dequantize(q, F16), want[2].to(F16))
    # a wider matrix's rows, rows of a wider output: nothing beside them changes
    ld = q.codes.shape[1] + 64
    codes = torch.full((T + 1, ld), 7, dtype=torch.uint8, device="cuda")
    w = pi.MxMatrix(codes[:T, : ld - 64], torch.full_like(q.scales, 9), K, kind)
    c.mx_quantize(x, kind, out=w)
    same(w, want)
    assert bool((codes[T] == 7).all()) and bool((codes[:, ld - 64:] == 7).all())
    y = torch.full((T + 1, K + 5), 7.0, device="cuda")
    c.mx_dequantize(w, out=y[:T, :K])
    assert torch.equal(y[:T, :K].double(), want[2]) and bool((y[T] == 7).all()) and bool((y[:, K:] == 7).all())


@pytest.mark.parametrize("kind", [MX8, MX4])
def test_quantize_at_the_borders(c, kind):
    """Every border between two neighbours and the values beside it, at scales
    from the least to the largest; infinities, NaN, zeros of either sign."""
    t = X.table(kind)
    mid = ((t[1:] + t[:-1]) / 2).float()
    v = torch.cat([t.float(), mid, torch.nextafter(mid, torch.tensor(0.0)), torch.nextafter(mid, torch.tensor(1e9))])
    v = torch.cat([v, -v])
    v = torch.nn.functional.pad(v, (0, -v.numel() % 31)).reshape(-1, 31)
    top = torch.full((v.shape[0], 1), t[-1].item())
    rows = torch.cat([v, top], 1)                       # a block each, with the largest value in it: scale 1
    scaled = [rows * 2.0 ** k for k in (-120, -60, -1, 0, 1, 60, 118)]
    x = torch.cat(scaled + [torch.zeros(1, 32), -torch.zeros(1, 32)]).cuda()
    x = torch.cat([x, torch.full((1, 32), 2.0 ** -149).cuda(), torch.full((1, 32), 1e-40).cuda(), torch.full((1, 32), 3.3e38).cuda()])
    same(c.mx_quantize(x, kind), X.quantize(kind, x.double()))
    bad = torch.ones(4, 96, device="cuda")
    bad[0, 3], bad[1, 40], bad[2, 95] = math.nan, math.inf, -math.inf
    q = c.mx_quantize(bad, kind)
    same(q, X.quantize(kind, bad.double()))
    nan = torch.zeros(4, 96, dtype=torch.bool, device="cuda")
    nan[0, :32], nan[1, 32:64], nan[2, 64:] = True, True, True
    assert torch.equal(c.mx_dequantize(q, F32).isnan(), nan)
    assert torch.equal(c.mx_dequantize(q, F16).isnan(), nan)


def test_quantize_of_nothing(c):
    for kind in (MX8, MX4):
        q = c.mx_quantize(torch.empty(0, 40, device="cuda"), kind)
        assert q.shape == (0, 40) and c.mx_dequantize(q).shape == (0, 40)
        w = Maker(0).mx(c, 24, 40, kind)
        assert c.mx_linear(q, w).shape == (0, 24)
        assert c.mx_gated_ffn(q, None, w, Maker(1).mx(c, 40, 24, kind)).shape == (0, 40)
    x, h = c.norm_residual_mx(torch.empty(0, 40, device="cuda"))
    assert x.shape == h.shape == (0, 40)


# ------------------------------------------------------------------ linear
# one token to several row tiles; features below, at and past tile borders; odd
# sizes; few tiles of a long k; many tiles; thin outputs
LINEAR = [(1, 8, 1), (1, 1024, 4096), (2, 64, 128), (3, 257, 31), (4, 3000, 70), (5, 300, 33), (6, 1024, 200), (7, 90, 4000), (8, 512, 129),
          (9, 512, 129), (16, 640, 384), (17, 1000, 515), (33, 72, 1000),
          (64, 2048, 256), (65, 128, 264), (128, 130, 256), (129, 33, 128), (130, 320, 520), (257, 1, 3), (300, 1001, 257),
          (513, 192, 777), (1100, 96, 640), (200, 12296, 520), (2600, 136, 2056), (3000, 264, 100), (40, 4104, 2500)]


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("xk,wk", KINDS)
def test_linear(c, T, K, N, xk, wk):
    m = Maker(T * 7 + K)
    fn = R.FNS[(T + K + N) % 7]
    dt = BF16 if (T + N) % 2 else F16
    x, w = m.mx(c, T, K, xk), m.mx(c, N, K, wk, K ** -0.5)
    b, r = m(N, dt=dt), m(T, N, dt=dt, pad=3)
    y = c.mx_linear(x, w, b, fn=FN(fn), residual=r, scale=0.5)
    assert y.dtype == dt
    R.check(y, X.linear(x, w, b, fn, 0.5, r, dt), "bias, residual")
    assert c.mx_linear(x, w, b, fn=FN(fn), residual=r, scale=0.5).equal(y)  # fixed order
    buf = torch.full((T + 1, N + 5), 7.0, dtype=dt, device="cuda")
    c.mx_linear(x, w, dtype=dt, y=buf[:T, :N])
    R.check(buf[:T, :N], X.linear(x, w, None, "none", 1.0, None, dt), "plain")
    assert bool((buf[T] == 7).all()) and bool((buf[:, N:] == 7).all())
    want = c.mx_linear(x, w, b, fn=FN(fn), residual=r)
    c.mx_linear(x, w, b, fn=FN(fn), residual=r, y=r)  # in place
    assert r.equal(want)


# matrices of 20 MB and more, whose few tokens are the rows of the products, and just below
LARGE = [(1, 16400, 6200), (2, 8192, 12288), (5, 8200, 12500), (8, 28672, 4100), (9, 8200, 12500), (1, 2048, 19300), (16, 8200, 12500),
         (16, 2050, 50000), (13, 30000, 2900), (17, 8200, 12500), (4, 1920, 40000)]


@pytest.mark.parametrize("T,K,N", LARGE)
def test_linear_of_a_large_matrix(c, T, K, N):
    m = Maker(T)
    x, w = m.mx(c, T, K, MX8), m.mx(c, N, K, MX4, K ** -0.5)
    b, r = m(N, dt=BF16), m(T, N, dt=BF16, pad=3)
    for fn in R.FNS:
        y = c.mx_linear(x, w, b, fn=FN(fn), residual=r, scale=0.5)
        R.check(y, X.linear(x, w, b, fn, 0.5, r, BF16), fn)
        assert c.mx_linear(x, w, b, fn=FN(fn), residual=r, scale=0.5).equal(y)
    buf = torch.full((T + 1, N + 5), 7.0, dtype=F16, device="cuda")
    c.mx_linear(x, w, dtype=F16, y=buf[:T, :N])
    R.check(buf[:T, :N], X.linear(x, w, None, "none", 1.0, None, F16), "plain")
    assert bool((buf[T] == 7).all()) and bool((buf[:, N:] == 7).all())
    r32 = m(T, N, dt=F32)
    want = X.linear(x, w, b, "silu", 2.0, r32, F32)
    c.mx_linear(x, w, b, fn=pi.PI_FN_SILU, scale=2.0, residual=r32, y=r32)
    R.check(r32, want, "fp32, in place")
    # a block's scale meets its block; a NaN stays in its row
    for k in (0, 33, (K - 1) // 32):
        xs, ws = torch.zeros(T, K, device="cuda"), torch.zeros(N, K, device="cuda")
        xs[:, 32 * k] = 2.0 ** (torch.arange(T, device="cuda") * 5 % 23 - 11)
        ws[:, 32 * k] = 2.0 ** (torch.arange(N, device="cuda") * 3 % 19 - 9)
        y = c.mx_linear(c.mx_quantize(xs, MX8), c.mx_quantize(ws, MX4), y=torch.empty(T, N, device="cuda"))
        assert torch.equal(y, xs @ ws.t()), k
    ws[N // 2, K - 1] = math.nan
    xs[T // 2, 5] = math.inf
    y = c.mx_linear(c.mx_quantize(xs, MX8), c.mx_quantize(ws, MX4))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[T // 2], bad[:, N // 2] = True, True
    assert torch.equal(y.isnan(), bad)


@pytest.mark.parametrize("T,d,n", [(1, 8192, 6400), (3, 4100, 12500), (8, 8200, 6300), (16, 8200, 6300), (11, 2060, 20500)])
@pytest.mark.parametrize("gated", [True, False])
def test_gated_ffn_of_large_matrices(c, T, d, n, gated):
    m = Maker(T)
    n = n if gated else 2 * n
    x = m.mx(c, T, d, MX8)
    w = ffn_weights(m, c, d, n, MX4, BF16, gated, T != 3)
    for fn in ("relu", "silu", "gelu"):
        y = c.mx_gated_ffn(x, *w, fn=FN(fn), dtype=BF16)
        R.check(y, X.ffn(x, *w, fn, BF16), fn)


@pytest.mark.parametrize("T,K,N", [(1, 256, 512), (40, 1000, 130), (300, 512, 384)])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_linear_adds_into_an_fp32_stream(c, T, K, N, xk, wk):
    m = Maker(5)
    x, w, b, r = m.mx(c, T, K, xk), m.mx(c, N, K, wk, K ** -0.5), m(N, dt=BF16), m(T, N, dt=F32, std=3.0)
    y = c.mx_linear(x, w, b, residual=r, scale=2.0)
    assert y.dtype == F32
    R.check(y, X.linear(x, w, b, "none", 2.0, r, F32))
    c.mx_linear(x, w, b, residual=r, scale=2.0, y=r)
    assert r.equal(y)


@pytest.mark.parametrize("T", [1, 3, 8, 20, 128, 300])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_each_scale_meets_its_block(c, T, xk, wk):
    """One block of x and of W at a time is not zero, with a scale of its own:
    the product is that block's, exactly (powers of two)."""
    K, N = 520, 300
    blocks = (K + 31) // 32
    for k in range(blocks):
        x, w = torch.zeros(T, K, device="cuda"), torch.zeros(N, K, device="cuda")
        x[:, 32 * k] = 2.0 ** ((torch.arange(T, device="cuda") * 5 + k) % 23 - 11)
        w[:, 32 * k] = 2.0 ** ((torch.arange(N, device="cuda") * 3 + k) % 19 - 9)
        y = c.mx_linear(c.mx_quantize(x, xk), c.mx_quantize(w, wk), y=torch.empty(T, N, device="cuda"))
        assert torch.equal(y, x @ w.t()), k


@pytest.mark.parametrize("T", [1, 3, 8, 20, 128, 300])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_scales_of_the_whole_range(c, T, xk, wk):
    """Values of 2^-60 times ones of 2^60; a product past fp32's range is not finite."""
    m = Maker(3)
    x, w = m(T, 256, dt=F32), m(130, 256, dt=F32, std=1 / 16)
    y = c.mx_linear(c.mx_quantize(x * 2.0 ** -60, xk), c.mx_quantize(w * 2.0 ** 60, wk))
    assert y.equal(c.mx_linear(c.mx_quantize(x, xk), c.mx_quantize(w, wk)))
    big = torch.full((T, 256), 2.0 ** 100, device="cuda")
    y = c.mx_linear(c.mx_quantize(big, xk), c.mx_quantize(big[:1].expand(40, -1).contiguous(), wk))
    assert not bool(y.isfinite().any())


@pytest.mark.parametrize("T", [1, 3, 8, 20, 128, 300])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_a_nan_block_stays_in_its_row(c, T, xk, wk):
    m = Maker(4)
    x, w = m(T, 300, dt=F32), m(140, 300, dt=F32)
    x[T // 2, 290] = math.inf
    w[77, 40] = math.nan
    y = c.mx_linear(c.mx_quantize(x, xk), c.mx_quantize(w, wk))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[T // 2], bad[:, 77] = True, True
    assert torch.equal(y.isnan(), bad)


# ------------------------------------------------------------------ gated FFN
FFN = [(1, 64, 200), (1, 1024, 2736), (2, 264, 777), (3, 100, 257), (4, 520, 130), (7, 264, 1000), (8, 100, 257), (20, 264, 777), (64, 512, 1000), (65, 130, 384), (128, 192, 96), (200, 192, 515),
       (300, 520, 1025), (700, 1000, 2600)]


def ffn_weights(m, c, d, n, wk, dt, gated, bias):
    wg = m.mx(c, n, d, wk, d ** -0.5) if gated else None
    wu, wd = m.mx(c, n, d, wk, d ** -0.5), m.mx(c, d, n, wk, n ** -0.5)
    b = [m(k, dt=dt, std=0.3) if bias and (gated or i) else None for i, k in enumerate((n, n, d))]
    return wg, wu, wd, *b


@pytest.mark.parametrize("T,d,n", FFN)
@pytest.mark.parametrize("xk,wk", KINDS)
@pytest.mark.parametrize("gated", [True, False])
def test_gated_ffn(c, T, d, n, xk, wk, gated):
    m = Maker(T + d)
    fn = R.FNS[1 + (T + d + n + gated) % 6]
    dt = BF16 if T % 2 else F16
    x = m.mx(c, T, d, xk)
    w = ffn_weights(m, c, d, n, wk, dt, gated, (T + n) % 3 > 0)
    buf = torch.full((T + 1, d + 3), 7.0, dtype=dt, device="cuda")
    y = c.mx_gated_ffn(x, *w, fn=FN(fn), dtype=dt, y=buf[:T, :d])
    R.check(y, X.ffn(x, *w, fn, dt), fn)
    assert bool((buf[T] == 7).all()) and bool((buf[:, d:] == 7).all())
    assert c.mx_gated_ffn(x, *w, fn=FN(fn), dtype=dt).equal(y)


# ------------------------------------------------------------------ norms
NORMS = [(1, 64), (1, 8192), (3, 100), (5, 1000), (130, 257), (40, 2048), (129, 8200), (310, 512), (400, 1000), (320, 7168), (700, 96),
         (7, 16384)]


@pytest.mark.parametrize("T,d", NORMS)
@pytest.mark.parametrize("kind", [MX8, MX4])
def test_norm_residual_mx(c, T, d, kind):
    m = Maker(T + d)
    for pre, post, rows, xdt, dt in (("rms", "none", 0, F32, BF16), ("layer", "rms", 1, F16, F16), ("rms", "layer", 7, F32, F16)):
        x, y = m(T, d, dt=xdt, std=2.0), m(T, d, dt=dt)
        gate = m(1 if rows == 0 else -(-T // rows), d, dt=dt)
        wp, bp = m(d, dt=dt), m(d, dt=dt) if pre == "layer" else None
        wq, bq = (m(d, dt=dt), m(d, dt=dt)) if post != "none" else (None, None)
        kw = dict(pre=NORM[pre], post=NORM[post], w_pre=wp, b_pre=bp, w_post=wq, b_post=bq, res_scale=0.5, branch_scale=1.5,
                  gate_rows=rows)
        xo, h = c.norm_residual_mx(x, y, gate, kind=kind, **kw)
        want = R.norm_fwd(x, y, gate, rows, pre, post, wp, bp, wq, bq, 0.5, 1.5, 1e-5, F32)
        R.check(xo, want["x"], "x")
        assert X.unpack(h)[2]
        R.check(X.values(h), X.requantized(kind, *want["h"]), "h")
        codes, scales, _ = X.unpack(h)
        assert bool((codes[:, d:] == 0).all())
        assert bool((scales[:, (d + 31) // 32:] == 0).all())
        # what the 16-bit call leaves of x', and the same matrix again, over what was there
        assert xo.equal(c.norm_residual(x, y, gate, **kw)[0])
        h.codes.fill_(0x55), h.scales.fill_(0x55)
        again = c.norm_residual_mx(x, y, gate, kind=kind, h=h, x_out=xo, **kw)
        assert again[1] is h and torch.equal(X.unpack(h)[0], codes) and torch.equal(X.unpack(h)[1], scales) and X.unpack(h)[2]


def test_norm_without_a_block(c):
    m = Maker(2)
    for T in (3, 400):
        x, w = m(T, 320, dt=F32), m(320, dt=BF16)
        xo, h = c.norm_residual_mx(x, w_pre=w)
        assert xo.equal(x)
        want = R.norm_fwd(x, None, None, 0, "rms", "none", w, None, None, None, 1.0, 1.0, 1e-5, F32)
        R.check(X.values(h), X.requantized(MX8, *want["h"]), "h")
        x[T // 2, 5] = math.inf  # a row's NaN stays in it
        h = c.norm_residual_mx(x, w_pre=w)[1]
        bad = X.values(h).isnan()
        assert bool(bad[T // 2].any()) and int(bad.any(1).sum()) == 1


# ------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("T", [1, 33, 400])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_a_block_as_a_model_runs_it(c, T, xk, wk):
    """Norm, FFN, residual stream, next norm: with 16-bit weights that the
    library quantises; and the same captured into a graph, replayed on new input."""
    d, n = 264, 700
    m = Maker(T)
    wg, wu, wd = (m(*s, dt=BF16, std=s[1] ** -0.5) for s in ((n, d), (n, d), (d, n)))
    wn, b = m(d, dt=BF16), m(n, dt=BF16)
    q = [c.mx_quantize(w, wk) for w in (wg, wu, wd)]
    x0, x1 = m(T, d, dt=F32, std=2.0), m(T, d, dt=F32, std=2.0)
    xs = x0.clone()

    def block(x):
        x, h = c.norm_residual_mx(x, w_pre=wn, kind=xk)
        y = c.mx_gated_ffn(h, *q, b, fn=pi.PI_FN_SILU)
        return (*c.norm_residual_mx(x, y, w_pre=wn, kind=xk), h, y)

    x, h2, h, y = block(xs)
    want = R.norm_fwd(x0, None, None, 0, "rms", "none", wn, None, None, None, 1.0, 1.0, 1e-5, F32)
    R.check(X.values(h), X.requantized(xk, *want["h"]), "h")
    R.check(y, X.ffn(h, *q, b, None, None, "silu", BF16), "y")
    want = R.norm_fwd(x0, y, None, 0, "rms", "none", wn, None, None, None, 1.0, 1.0, 1e-5, F32)
    R.check(x, want["x"], "x")
    R.check(X.values(h2), X.requantized(xk, *want["h"]), "next h")
    other = block(x1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block(xs)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block(xs)
    for inp, res in ((x1, other), (x0, (x, h2, h, y))):
        xs.copy_(inp)
        g.replay()
        assert out[0].equal(res[0]) and out[3].equal(res[3])
        assert out[1].codes.equal(res[1].codes) and out[1].scales.equal(res[1].scales)


def test_calls_on_two_streams_at_once(c):
    m = Maker(9)
    x, w, wd = m.mx(c, 200, 1024, MX8), m.mx(c, 2048, 1024, MX4, 1 / 32), m.mx(c, 1024, 2048, MX4, 1 / 45)
    x1 = m.mx(c, 5, 1024, MX8)
    want, want1 = c.mx_gated_ffn(x, None, w, wd), c.mx_gated_ffn(x1, None, w, wd)
    torch.cuda.synchronize()
    bad = []

    def work(xx, res):
        ctx = G.ctx()
        with torch.cuda.stream(torch.cuda.Stream()):
            outs = [ctx.mx_gated_ffn(xx, None, w, wd) for _ in range(30)]
            torch.cuda.current_stream().synchronize()
        ctx.check()
        bad.extend(1 for o in outs if not o.equal(res))
        ctx.close()

    ts = [threading.Thread(target=work, args=a) for a in ((x, want), (x1, want1))]
    [t.start() for t in ts], [t.join() for t in ts]
    assert not bad


def wider(q, extra=64, off=32):
    """The same matrix as rows of wider ones."""
    rows, n = q.codes.shape
    buf = torch.full((rows + 1, off + n + extra - off), 0x7f, dtype=torch.uint8, device="cuda")
    buf[:rows, off: off + n] = q.codes
    return pi.MxMatrix(buf[:rows, off: off + n], q.scales, q.cols, q.kind)


@pytest.mark.parametrize("T", [1, 8, 40, 300])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_rows_of_wider_buffers(c, T, xk, wk):
    m = Maker(12)
    d, n = 300, 520
    x, w = m.mx(c, T, d, xk), ffn_weights(m, c, d, n, wk, BF16, True, True)
    assert c.mx_linear(wider(x), wider(w[0])).equal(c.mx_linear(x, w[0]))
    assert c.mx_gated_ffn(wider(x), *map(wider, w[:3]), *w[3:]).equal(c.mx_gated_ffn(x, *w))


@pytest.mark.parametrize("T", [1, 8])
def test_rows_of_wider_large_matrices(c, T):
    m = Maker(13)
    x, w = m.mx(c, T, 8200, MX8), m.mx(c, 12500, 8200, MX4)
    assert c.mx_linear(wider(x), wider(w)).equal(c.mx_linear(x, w))


def test_tokens_from_a_row_tile_on(c):
    """Rows from a multiple of 128 on are a matrix of their own."""
    m = Maker(14)
    x, w = m.mx(c, 400, 300, MX8), m.mx(c, 200, 300, MX4)
    y = c.mx_linear(x, w)
    for a in (128, 256, 384):
        part = pi.MxMatrix(x.codes[a:], x.scales[a // 128:], 300, MX8)
        want = X.linear(part, w, None, "none", 1.0, None, BF16)
        R.check(c.mx_linear(part, w), want)
        R.check(y[a:], want)


@pytest.mark.parametrize("kind", [MX8, MX4])
def test_more_than_2_31_elements(c, kind):
    """Offsets past 32 bits: the last rows as they are by themselves."""
    T, K = 270000, 8000
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    x[-300:] = Maker(15)(300, K, dt=BF16)
    q = c.mx_quantize(x, kind)
    y = c.mx_dequantize(q)
    same(c.mx_quantize(x[-300:], kind), X.quantize(kind, x[-300:].double()))
    assert torch.equal(y[-300:].double(), X.quantize(kind, x[-300:].double())[2])
    assert not bool(y[:-300].any())
    w = Maker(16).mx(c, 16, K, kind)
    out = c.mx_linear(q, w)
    R.check(out[-300:], X.linear(c.mx_quantize(x[-300:], kind), w, None, "none", 1.0, None, BF16))
    assert not bool(out[:-300].any())


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_weights_written_right_before_their_use(c, T, xk, wk):
    """Launches may begin before those in front of them end: no load is ahead of what writes its data."""
    m = Maker(17)
    d, n = 1000, 2700
    raw = [[m(*s, dt=BF16, std=s[1] ** -0.5) for s in ((n, d), (n, d), (d, n))] for _ in range(3)]
    xs = [m(T, d, dt=F32) for _ in range(3)]
    want = []
    for r, x in zip(raw, xs):
        q = [c.mx_quantize(w, wk) for w in r]
        h = c.norm_residual_mx(x, kind=xk)[1]
        torch.cuda.synchronize()
        want.append(c.mx_gated_ffn(h, *q))
        torch.cuda.synchronize()
    q = [c.mx_empty(*w.shape, wk) for w in raw[0]]
    h, xo = c.mx_empty(T, d, xk), torch.empty(T, d, device="cuda")
    got = []
    for i in range(30):
        for w, o in zip(raw[i % 3], q):
            c.mx_quantize(w, wk, out=o)
        c.norm_residual_mx(xs[i % 3], kind=xk, h=h, x_out=xo)
        got.append(c.mx_gated_ffn(h, *q))
    assert all(y.equal(want[i % 3]) for i, y in enumerate(got))


def test_norm_in_place(c):
    m = Maker(18)
    for T in (3, 400):
        x, y = m(T, 520, dt=F32), m(T, 520, dt=BF16)
        want, h = c.norm_residual_mx(x, y)
        xo, h2 = c.norm_residual_mx(x, y, x_out=x)
        assert xo is x and x.equal(want) and h2.codes.equal(h.codes) and h2.scales.equal(h.scales)


@pytest.mark.parametrize("T,K,N", [(1, 2048, 512), (100, 2048, 512), (300, 2048, 512), (4, 8200, 12500)])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_a_wait_that_runs_out_is_reported(T, K, N, xk, wk):
    """With a wait limit of a nanosecond the products' waits run out: the
    kernels return, the status says so, and the context goes on working."""
    ctx = G.ctx()
    try:
        m = Maker(21)
        x, w = m.mx(ctx, T, K, xk), m.mx(ctx, N, K, wk, 0.02)
        want = ctx.mx_linear(x, w)
        ctx.check()
        pi.pi_debug_set_wait_limit(ctx.handle, 1)
        status = 0
        for _ in range(5):  # (a wait may be over before the clock is read)
            ctx.mx_linear(x, w)
            status = ctx.sync_status() or status  # (which also clears it)
        assert status == pi.PI_ERR_TIMEOUT
        pi.pi_debug_set_wait_limit(ctx.handle, 2_000_000_000)
        assert ctx.mx_linear(x, w).equal(want)
        ctx.check()
    finally:
        ctx.close()


@pytest.mark.parametrize("T,d,n", [(3, 8192, 6400), (40, 520, 2600), (300, 520, 2600)])
@pytest.mark.parametrize("gated", [True, False])
def test_waits_that_run_out_in_a_block(T, d, n, gated):
    """The same in both products of a block, the second of which loads ahead of
    the first one's end: every warp comes to the end of its launch, clusters too."""
    ctx = G.ctx()
    try:
        m = Maker(22)
        n = n if gated else 2 * n
        x, w = m.mx(ctx, T, d, MX8), ffn_weights(m, ctx, d, n, MX4, F16, gated, True)
        run = lambda: ctx.mx_gated_ffn(x, *w, fn=pi.PI_FN_SILU, dtype=F16)
        want = run()
        ctx.check()
        pi.pi_debug_set_wait_limit(ctx.handle, 1)
        status = 0
        for _ in range(5):
            run()
            status = ctx.sync_status() or status
        assert status == pi.PI_ERR_TIMEOUT
        pi.pi_debug_set_wait_limit(ctx.handle, 2_000_000_000)
        assert run().equal(want)
        ctx.check()
    finally:
        ctx.close()


def test_refusals(c):
    lib = pi.load_library()
    dev = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    p = dev.data_ptr()

    def mx(codes=p, scales=p):
        return ctypes.byref(pi.pi_mx(codes, scales))

    def desc(struct, good, **bad):
        return ctypes.byref(struct(**{**good, **bad}))

    Q = dict(rows=4, cols=40, kind=MX8, dtype=pi.PI_F16)
    for f, args in ((lib.pi_mx_quantize, lambda x, q: (x, q)), (lib.pi_mx_dequantize, lambda x, q: (q, x))):
        for bad, code in ((dict(kind=pi.PI_F16), pi.PI_ERR_ARG), (dict(dtype=MX8), pi.PI_ERR_ARG), (dict(rows=-1), pi.PI_ERR_SHAPE),
                          (dict(cols=0), pi.PI_ERR_SHAPE), (dict(cols=(1 << 20) + 1), pi.PI_ERR_SHAPE),
                          (dict(rows=(1 << 22) + 1), pi.PI_ERR_SHAPE), (dict(ldx=39), pi.PI_ERR_SHAPE),
                          (dict(ldq=96), pi.PI_ERR_SHAPE), (dict(ldq=136), pi.PI_ERR_ARG)):
            assert f(c.handle, desc(pi.pi_mx_desc, Q, **bad), *args(p, mx())) == code, bad
        assert f(c.handle, None, *args(p, mx())) == pi.PI_ERR_ARG
        good = desc(pi.pi_mx_desc, Q)
        for x, q in ((None, mx()), (p + 1, mx()), (p, None), (p, mx(0)), (p, mx(p, 0)), (p, mx(p + 16)), (p, mx(p, p + 8))):
            assert f(c.handle, good, *args(x, q)) == pi.PI_ERR_ARG
    L = dict(T=4, K=40, N=24, x_kind=MX8, w_kind=MX4, dtype=pi.PI_BF16, out_dtype=pi.PI_BF16, fn=0, scale=1.0)
    n = ctypes.c_size_t()
    call = lambda d, x=None, w=None, b=None, r=None, y=p, ws=p, wsn=1 << 16: lib.pi_mx_linear(
        c.handle, d, x or mx(), w or mx(), b, r, y, ws, wsn)
    for bad, code in ((dict(x_kind=0), pi.PI_ERR_ARG), (dict(x_kind=MX4, w_kind=MX8), pi.PI_ERR_UNSUPPORTED),
                      (dict(dtype=pi.PI_F32), pi.PI_ERR_ARG), (dict(out_dtype=pi.PI_F16), pi.PI_ERR_ARG), (dict(fn=7), pi.PI_ERR_ARG),
                      (dict(scale=math.nan), pi.PI_ERR_ARG), (dict(T=-1), pi.PI_ERR_SHAPE), (dict(K=0), pi.PI_ERR_SHAPE),
                      (dict(N=0), pi.PI_ERR_SHAPE), (dict(ldy=23), pi.PI_ERR_SHAPE), (dict(ldr=23), pi.PI_ERR_SHAPE)):
        d = desc(pi.pi_mx_linear_desc, L, **bad)
        assert call(d) == code, bad
        assert lib.pi_mx_linear_workspace(c.handle, d, ctypes.byref(n)) == code
    for bad, code in ((dict(ldx=96), pi.PI_ERR_SHAPE), (dict(ldx=130), pi.PI_ERR_ARG), (dict(ldw=32), pi.PI_ERR_SHAPE)):
        assert call(desc(pi.pi_mx_linear_desc, L, **bad)) == code, bad
    good = desc(pi.pi_mx_linear_desc, L)
    assert lib.pi_mx_linear_workspace(c.handle, good, None) == pi.PI_ERR_ARG
    assert call(good, x=mx(p + 8)) == call(good, w=mx(p, p + 4)) == call(good, b=p + 1) == call(good, y=None) == pi.PI_ERR_ARG
    assert call(good, y=p + 1) == call(good, r=p + 1) == pi.PI_ERR_ARG
    F = dict(T=200, d=40, n=24, x_kind=MX8, w_kind=MX4, dtype=pi.PI_BF16, fn=1, gated=0)
    wts = pi.pi_mx_gated_ffn_weights(0, 0, p, p, p, p, 0, 0, 0)
    ffn = lambda d, w=wts, y=p, ws=p, wsn=1 << 16: lib.pi_mx_gated_ffn(c.handle, d, w and ctypes.byref(w), mx(), y, ws, wsn)
    for bad, code in ((dict(x_kind=MX4, w_kind=MX8), pi.PI_ERR_UNSUPPORTED), (dict(w_kind=2), pi.PI_ERR_ARG), (dict(gated=2), pi.PI_ERR_ARG),
                      (dict(fn=-1), pi.PI_ERR_ARG), (dict(n=0), pi.PI_ERR_SHAPE), (dict(d=0), pi.PI_ERR_SHAPE), (dict(ldy=39), pi.PI_ERR_SHAPE),
                      (dict(dtype=MX8), pi.PI_ERR_ARG)):
        d = desc(pi.pi_mx_gated_ffn_desc, F, **bad)
        assert ffn(d) == code, bad
        assert lib.pi_mx_gated_ffn_workspace(c.handle, d, ctypes.byref(n)) == code
    good = desc(pi.pi_mx_gated_ffn_desc, F)
    assert lib.pi_mx_gated_ffn_workspace(c.handle, good, ctypes.byref(n)) == 0 and n.value > 0
    assert ffn(good, wsn=n.value - 1) == ffn(good, ws=None) == ffn(good, ws=p + 8) == ffn(good, w=None) == ffn(good, y=None) == pi.PI_ERR_ARG
    assert ffn(good, w=pi.pi_mx_gated_ffn_weights(p, p, p, p, p, p, 0, 0, 0)) == pi.PI_ERR_ARG  # a gate, but gated is 0
    assert ffn(desc(pi.pi_mx_gated_ffn_desc, F, gated=1)) == pi.PI_ERR_ARG                      # none, but gated is 1
    N = dict(T=4, d=40, x_dtype=pi.PI_F32, dtype=pi.PI_BF16, grad_dtype=pi.PI_BF16, pre=1, post=0, res_scale=1.0, branch_scale=1.0)
    norm = lambda d, k=MX8, x=p, h=mx(): lib.pi_norm_residual_mx(c.handle, d, k, None, x, None, None, p, h)
    for bad, code in ((dict(pre=0), pi.PI_ERR_ARG), (dict(ldh=96), pi.PI_ERR_SHAPE), (dict(ldh=136), pi.PI_ERR_ARG),
                      (dict(d=16385), pi.PI_ERR_SHAPE), (dict(eps=-1.0), pi.PI_ERR_ARG)):
        assert norm(desc(pi.pi_norm_residual_desc, N, **bad)) == code, bad
    good = desc(pi.pi_norm_residual_desc, N)
    assert norm(good, k=pi.PI_Q4_0) == norm(good, x=None) == norm(good, h=None) == norm(good, h=mx(0)) == norm(good, h=mx(p + 16)) == pi.PI_ERR_ARG
    torch.cuda.synchronize()
    c.check()
