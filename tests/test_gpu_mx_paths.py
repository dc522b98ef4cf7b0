"""Paths of the microscaled products that small matrices do not take: several
tiles to a pair of CTAs, whose accumulators share columns of tensor memory, and
few tokens through large 4-bit matrices with launches that overlap."""
from __future__ import annotations

import threading

import pytest
import torch

from activation_sparse_decode_sigmoid_gb300 import pi
from tests import _block as R
from tests import _gpu as G
from tests import _mx as X
from tests.test_gpu_mx import BF16, F16, F32, FN, KINDS, MX4, MX8, Maker, ffn_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c():
    ctx = G.ctx()
    yield ctx
    ctx.check()
    ctx.close()


# ------------------------------------------------------------------ many tiles
# With 76 pairs of CTAs: tiles of 256 rows x 256 columns (gated: 128).  The first
# sizes are all whole tiles, three or four to a pair; the others end inside one.
@pytest.mark.parametrize("T,K,N", [(5120, 136, 3328), (4999, 520, 3001), (2700, 264, 5500)])
@pytest.mark.parametrize("xk,wk", KINDS)
def test_linear_of_many_tiles(c, T, K, N, xk, wk):
    m = Maker(T + N)
    x, w = m.mx(c, T, K, xk), m.mx(c, N, K, wk, K ** -0.5)
    for dt, fn, bias, scale, out in ((BF16, "silu", True, 0.5, BF16), (F16, "none", False, 1.0, F16), (BF16, "relu", True, 1.0, F32)):
        b, r = m(N, dt=dt) if bias else None, m(T, N, dt=out, pad=T % 2)
        y = c.mx_linear(x, w, b, fn=FN(fn), residual=r, scale=scale, dtype=dt)
        R.check(y, X.linear(x, w, b, fn, scale, r, out), (fn, out))
        y = c.mx_linear(x, w, b, fn=FN(fn), scale=scale, dtype=dt, y=torch.empty(T, N, dtype=out, device="cuda"))
        R.check(y, X.linear(x, w, b, fn, scale, None, out), (fn, out, "no residual"))


@pytest.mark.parametrize("T,d,n", [(5120, 136, 1664), (4999, 264, 1500), (2700, 520, 3001)])
@pytest.mark.parametrize("xk,wk", KINDS)
@pytest.mark.parametrize("gated", [True, False])
def test_gated_ffn_of_many_tiles(c, T, d, n, xk, wk, gated):
    m = Maker(T + n)
    n = n if gated else 2 * n
    x = m.mx(c, T, d, xk)
    for dt, fn, bias in ((BF16, "silu", True), (F16, "relu", False)):
        w = ffn_weights(m, c, d, n, wk, dt, gated, bias)
        y = c.mx_gated_ffn(x, *w, fn=FN(fn), dtype=dt)
        R.check(y, X.ffn(x, *w, fn, dt), (fn, dt))
        assert c.mx_gated_ffn(x, *w, fn=FN(fn), dtype=dt).equal(y)


@pytest.mark.parametrize("T,d,n", [(300, 512, 1000), (2700, 520, 3001), (4999, 264, 1500)])
@pytest.mark.parametrize("xk,wk", KINDS)
@pytest.mark.parametrize("gated", [True, False])
def test_a_block_equals_its_parts(c, T, d, n, xk, wk, gated):
    """The block is its two products and the quantisation between them, to the
    bit: what differs from another evaluation's a differs by the order of its sums.

    Up to 32 steps of k no product is cut along k, so an element is one
    accumulator's sum over k in order, in either kernel; ReLU and the gate's
    product are each one operation in fp32, which torch rounds alike."""
    m = Maker(T)
    n = n if gated else 2 * n
    x = m.mx(c, T, d, xk)
    wg, wu, wd, *_ = ffn_weights(m, c, d, n, wk, BF16, gated, False)
    new = lambda: torch.empty(T, n, device="cuda")
    if gated:
        a = c.mx_linear(x, wg, fn=pi.PI_FN_RELU, y=new()) * c.mx_linear(x, wu, y=new())
    else:
        a = c.mx_linear(x, wu, fn=pi.PI_FN_RELU, y=new())
    assert c.mx_gated_ffn(x, wg, wu, wd, fn=pi.PI_FN_RELU).equal(c.mx_linear(c.mx_quantize(a, xk), wd))


# ------------------------------------------------------------------ few tokens, large matrices
# Both products of a block through the kernel that takes the tokens as rows.
FEW = [(1, 8192, 6400), (3, 8192, 6400), (16, 8200, 8000)]


@pytest.mark.parametrize("T,d,n", FEW)
@pytest.mark.parametrize("gated", [True, False])
def test_large_weights_written_right_before_their_use(c, T, d, n, gated):
    """The second product loads its weights while the first one still runs, and
    a launch's warps go through their last code ahead of all results: neither
    sees what a launch before the block has yet to write."""
    m = Maker(30 + T)
    n = n if gated else 2 * n
    shapes = ((n, d), (n, d), (d, n)) if gated else ((n, d), (d, n))
    raw = [[m(*s, dt=BF16, std=s[1] ** -0.5) for s in shapes] for _ in range(3)]
    xs = [m(T, d, dt=F32) for _ in range(3)]
    call = lambda h, q: c.mx_gated_ffn(h, *(q if gated else [None, *q]))
    want = []
    for r, x in zip(raw, xs):
        q = [c.mx_quantize(w, MX4) for w in r]
        h = c.norm_residual_mx(x, kind=MX8)[1]
        torch.cuda.synchronize()
        want.append(call(h, q))
        torch.cuda.synchronize()
    q = [c.mx_empty(*w.shape, MX4) for w in raw[0]]
    h, xo = c.mx_empty(T, d, MX8), torch.empty(T, d, device="cuda")
    got = []
    for i in range(30):
        order = list(zip(raw[i % 3], q))
        for w, o in order if i % 2 else order[::-1]:  # (the down-projection's last, or first)
            c.mx_quantize(w, MX4, out=o)
        c.norm_residual_mx(xs[i % 3], kind=MX8, h=h, x_out=xo)
        got.append(call(h, q))
    assert all(y.equal(want[i % 3]) for i, y in enumerate(got))


@pytest.mark.parametrize("T,d,n", FEW)
def test_blocks_of_large_matrices_in_a_row(c, T, d, n):
    """Launch behind launch with nothing between, eagerly and replayed: y is the next block's x."""
    m = Maker(40 + T)
    w = ffn_weights(m, c, d, n, MX4, F16, True, True)
    x0, x1 = m(T, d, dt=F16), m(T, d, dt=F16)
    xs = x0.clone()

    def layers():
        x, out = xs, []
        for _ in range(4):
            y = c.mx_gated_ffn(c.mx_quantize(x, MX8), *w, fn=pi.PI_FN_GELU, dtype=F16)
            x = y
            out.append(y)
        return out

    def apart(x):
        out = []
        xs.copy_(x)
        x = xs
        for _ in range(4):
            q = c.mx_quantize(x, MX8)
            torch.cuda.synchronize()
            y = c.mx_gated_ffn(q, *w, fn=pi.PI_FN_GELU, dtype=F16)
            torch.cuda.synchronize()
            x = y
            out.append(y)
        return out

    want1, want0 = apart(x1), apart(x0)
    R.check(want0[0], X.ffn(c.mx_quantize(x0, MX8), *w, "gelu", F16), "first block")
    assert all(a.equal(b) for a, b in zip(layers(), want0))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layers()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layers()
    for x, want in ((x1, want1), (x0, want0), (x1, want1)):
        xs.copy_(x)
        g.replay()
        assert all(a.equal(b) for a, b in zip(out, want))


def test_large_matrices_on_two_streams_at_once(c):
    m = Maker(50)
    d, n = 8192, 6400
    w = ffn_weights(m, c, d, n, MX4, BF16, True, True)
    xs = [m.mx(c, T, d, MX8) for T in (1, 5)]
    want = [c.mx_gated_ffn(x, *w) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(x, res):
        ctx = G.ctx()
        with torch.cuda.stream(torch.cuda.Stream()):
            outs = [ctx.mx_gated_ffn(x, *w) for _ in range(30)]
            torch.cuda.current_stream().synchronize()
        ctx.check()
        bad.extend(1 for o in outs if not o.equal(res))
        ctx.close()

    ts = [threading.Thread(target=work, args=a) for a in zip(xs, want)]
    [t.start() for t in ts], [t.join() for t in ts]
    assert not bad


@pytest.mark.parametrize("T,d,n", FEW)
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("gated", [True, False])
def test_gated_ffn_of_large_matrices_in_either_type(c, T, d, n, dt, gated):
    m = Maker(60 + T)
    n = n if gated else 2 * n
    x, w = m.mx(c, T, d, MX8), ffn_weights(m, c, d, n, MX4, dt, gated, True)
    for fn in R.FNS:
        buf = torch.full((T + 1, d + 5), 7.0, dtype=dt, device="cuda")
        y = c.mx_gated_ffn(x, *w, fn=FN(fn), dtype=dt, y=buf[:T, :d])
        R.check(y, X.ffn(x, *w, fn, dt), fn)
        assert bool((buf[T] == 7).all()) and bool((buf[:, d:] == 7).all())


@pytest.mark.parametrize("T,K,N", [(1, 8192, 12288), (7, 8200, 12500), (16, 28672, 4100)])
def test_linear_of_a_large_matrix_in_f16(c, T, K, N):
    m = Maker(70 + T)
    x, w = m.mx(c, T, K, MX8), m.mx(c, N, K, MX4, K ** -0.5)
    b, r = m(N, dt=F16), m(T, N, dt=F16, pad=3)
    for fn in R.FNS:
        y = c.mx_linear(x, w, b, fn=FN(fn), residual=r, scale=0.5)
        assert y.dtype == F16
        R.check(y, X.linear(x, w, b, fn, 0.5, r, F16), fn)
    want = c.mx_linear(x, w, b, residual=r)
    c.mx_linear(x, w, b, residual=r, y=r)
    assert r.equal(want)
    r32 = m(T, N, dt=F32)
    R.check(c.mx_linear(x, w, b, residual=r32, dtype=F16), X.linear(x, w, b, "none", 1.0, r32, F32), "fp32")


# ------------------------------------------------------------------ ends of the range
@pytest.mark.parametrize("kind", [MX8, MX4])
def test_values_at_the_ends_of_the_range(c, kind):
    """Values next to fp32's largest may round up to 2^128, which fp32 and bf16
    hold as infinity; the least ones are below bf16's subnormals.  What a NaN block
    holds behind the row's end is NaN, and nothing else that pads is."""
    g = torch.Generator(device="cuda").manual_seed(80)
    u = torch.rand(64, 70, generator=g, device="cuda") * 2 - 1
    for s in (torch.finfo(F32).max, 2.0 ** -118, 2.0 ** -126, 2.0 ** -140):
        x = u * s
        x[:, 3] = s
        q = c.mx_quantize(x, kind)
        codes, scales, want = X.quantize(kind, x.double())
        got = X.unpack(q)
        assert torch.equal(got[0], codes) and torch.equal(got[1], scales) and got[2]
        for dt in (F32, BF16):
            assert torch.equal(c.mx_dequantize(q, dt), want.float().to(dt)), (s, dt)
    x = u.clone()
    x[5, 69] = float("nan")
    codes, scales, pad = X.unpack(c.mx_quantize(x, kind))
    assert pad and int(scales[5, 2]) == 255 and not bool(scales[:, 3].any())
    assert bool((codes[5, 64:96] == (0x7f if kind == MX8 else 0)).all()) and not bool(codes[:, 96:].any())
    codes[5] = 0
    assert not bool(codes[:, 70:].any())
