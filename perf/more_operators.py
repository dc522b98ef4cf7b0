"""The FFN block in microscaled 8- and 4-bit floating point, as measured cases.

A matrix of this kind has blocks of 32 along its rows that share a scale
2^(c - 127), c a byte (255: the block is NaN).  mx8: elements e4m3; mx4: e2m1,
two to a byte, the even column in the low half.  Rows of codes are padded to
128 columns; the scales lie in tiles of 128 rows x 4 blocks:
scales[row / 128][block / 4][row % 32][row % 128 / 32][block % 4].  What pads
is 0.  A block's scale is the smallest at which no element passes the largest
value of the type (448, 6); elements are rounded to the nearest, ties to even.

Four operators, serving's side of a linear layer, a gated FFN and a norm:
  quantize    q = Q(x), and the values back
  linear      y = r + f(x W^T + b), x and W of these kinds
  ffn         y = Q(f(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd
  norm        x' = rs x + bs gate * norm_post(y),  h = Q(norm_pre(x'))

`run` computes them in their plain form (elementary torch operations in 32
bits), or, with `own`, through the library's calls.  `exact` evaluates the
definitions in 64 bits.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FNS = ("none", "relu", "sqrelu", "sigmoid", "silu", "gelu", "gelu_tanh")
EPS = 1e-5


def listed():
    return [
        # a LLaMA-70B-shaped up-projection to 4 bits, and the values back (what its rounding costs)
        dict(name="quantize_weights", op="quantize", T=28672, K=8192, dt="bf16", kind="mx4", pad=0),
        # a prompt's activations to 8 bits
        dict(name="quantize_prompt", op="quantize", T=2048, K=8192, dt="f16", kind="mx8", pad=0),
        # a small odd matrix, rows that are slices of wider ones, from 32 bits
        dict(name="quantize_ragged", op="quantize", T=333, K=1001, dt="f32", kind="mx8", pad=7),
        # one token through the LLaMA-70B-shaped up-projection, 4-bit weights: a latency case
        dict(name="linear_token", op="linear", T=1, K=8192, N=28672, dt="bf16", xk="mx8", wk="mx4", fn="relu", bias=True,
             res=False),
        # 8 decode tokens through the down-projection, added to the residual
        dict(name="linear_tokens8", op="linear", T=8, K=28672, N=8192, dt="bf16", xk="mx8", wk="mx4", fn="none", bias=False,
             res=True),
        # a long prompt through the OPT-30B-shaped up-projection, squared ReLU
        dict(name="linear_prompt", op="linear", T=2048, K=7168, N=28672, dt="f16", xk="mx8", wk="mx4", fn="sqrelu", bias=True,
             res=False),
        # the same with activations of 4 bits, and the down-projection's direction
        dict(name="linear_prompt4", op="linear", T=2048, K=28672, N=8192, dt="bf16", xk="mx4", wk="mx4", fn="none", bias=False,
             res=True),
        # one decode token through the LLaMA-70B-shaped ReGLU block
        dict(name="ffn_token", op="ffn", T=1, d=8192, n=28672, dt="bf16", xk="mx8", wk="mx4", fn="relu", gated=True, bias=True),
        # a prompt through the SwiGLU block
        dict(name="ffn_prompt", op="ffn", T=2048, d=8192, n=28672, dt="bf16", xk="mx8", wk="mx4", fn="silu", gated=True,
             bias=False),
        # a ragged batch of a small gated layer with 8-bit weights
        dict(name="ffn_ragged", op="ffn", T=45, d=1000, n=2731, dt="f16", xk="mx8", wk="mx8", fn="gelu", gated=True, bias=True),
        # the norm between two blocks for one decode token, fp32 residual stream
        dict(name="norm_token", op="norm", T=1, d=8192, xdt="f32", dt="bf16", pre="rms", post="none", gate=0, rs=1.0),
        # norms before and after a block on a prompt, fp32 residual stream
        dict(name="norm_prompt", op="norm", T=4096, d=7168, xdt="f32", dt="f16", pre="rms", post="rms", gate=1, rs=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "ffn", "ffn", "norm"])
    dt = rng.choice(["f16", "bf16"])
    # half of the time tens of tokens or fewer (decode batches), else prompts
    T = _log(rng, 1, 80) if rng.random() < 0.5 else _log(rng, 80, 4096)
    kinds = rng.choice([("mx8", "mx4"), ("mx8", "mx4"), ("mx8", "mx8"), ("mx4", "mx4")])
    if op == "quantize":
        K = _log(rng, 16, 32768)
        # the values back in bf16: 16-bit floats of the other kind lack its range
        return dict(op=op, T=min(T * 8, (1 << 27) // K), K=K if rng.random() < 0.4 else -(-K // 32) * 32,
                    dt=rng.choice(["f16", "bf16", "f32"]), kind=rng.choice(["mx8", "mx4"]), pad=rng.choice([0, 0, 8, 3]))
    if op == "linear":
        K, N = _log(rng, 64, 28672), _log(rng, 64, 28672)
        if rng.random() < 0.7:  # most models keep their widths multiples of 32
            K, N = K // 32 * 32, N // 32 * 32
        return dict(op=op, T=T, K=K, N=N, dt=dt, xk=kinds[0], wk=kinds[1], fn=rng.choice(FNS), bias=rng.random() < 0.5,
                    res=rng.random() < 0.5)
    if op == "ffn":
        d = _log(rng, 128, 8192)
        n = _log(rng, 2 * d, 4 * d)
        if rng.random() < 0.7:
            d, n = d // 32 * 32, n // 32 * 32
        while 6 * T * d * n > 2.8e12:
            T //= 2
        return dict(op=op, T=T, d=d, n=n, dt=dt, xk=kinds[0], wk=kinds[1], fn=rng.choice(FNS[1:]), gated=rng.random() < 0.7,
                    bias=rng.random() < 0.5)
    d = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        d = -(-d // 32) * 32
    return dict(op=op, T=T, d=d, xdt=rng.choice(["f32", "f32", dt]), dt=dt, pre=rng.choice(["rms", "layer"]),
                post=rng.choice(["none", "rms", "layer"]), gate=rng.choice([0, 1, _log(rng, 2, 1024)]),
                rs=rng.choice([1.0, 0.5]))


# ------------------------------------------------------------------ the format, in torch
MOST = {"mx8": (8, 448.0), "mx4": (2, 6.0)}  # exponent of the largest value, and that value


def _scale_codes(amax, kind):
    """the scale byte of each block, from its largest magnitude (32-bit)"""
    emax, most = MOST[kind]
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    c = e - 1 - emax + (2 * m > most / 2 ** emax).int() + 127
    c = torch.where(amax > 0, c, 0).clamp(0, 254)
    return torch.where(torch.isfinite(amax), c, 255)


def _blocked(codes, rows):
    """[rows][blocks] -> tiles of 128 rows x 4 blocks (blocks: a multiple of 4)"""
    R = -(-rows // 128)
    full = torch.zeros(R * 128, codes.shape[1], dtype=torch.uint8, device=codes.device)
    full[:rows] = codes
    return full.view(R, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous()


def _e2m1(v):
    """codes of the nearest values, ties to even"""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c + (torch.signbit(v).to(torch.uint8) << 3)


def _power(c):
    """2^(c - 127) in 32 bits, exactly, for c from 0 to 254"""
    return torch.where(c == 0, 1 << 22, c << 23).int().view(torch.float32)


def _quantize(v, kind):
    """(codes as the matrix holds them, scales) of 32- or 64-bit values"""
    T, K = v.shape
    Kp = -(-K // 128) * 128
    p = torch.zeros(T, Kp, dtype=v.dtype, device=v.device)
    p[:, :K] = v
    b = p.view(T, -1, 32)
    c = _scale_codes(b.abs().amax(2), kind)
    q = b * _power(254 - c.clamp(max=254))[:, :, None]  # (exact: a power of two)
    bad = (c == 255)[:, :, None]
    if kind == "mx8":
        codes = torch.where(bad, 127, q.to(torch.float8_e4m3fn).view(torch.uint8)).view(T, Kp)
    else:
        n = torch.where(bad, 0, _e2m1(q)).view(T, Kp)
        codes = n[:, 0::2] | (n[:, 1::2] << 4)
    return codes, _blocked(c.to(torch.uint8), T)


def _values(codes, scales, K, kind, dtype=torch.float32):
    """what a matrix stands for"""
    T = codes.shape[0]
    if kind == "mx8":
        v = codes.view(torch.float8_e4m3fn).to(dtype)
    else:
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=codes.device)
        v = table[torch.stack((codes & 15, codes >> 4), 2).view(T, -1).int()]
    c = scales.permute(0, 3, 2, 1, 4).reshape(scales.shape[0] * 128, -1)[:T]
    s = torch.where(c == 255, math.nan, _power(c.int()).to(dtype))
    return (v.view(T, -1, 32) * s[:, :, None]).view(T, -1)[:, :K]


def _held(codes, scales, K):
    """an mx8 matrix as an output: elements and scales, as the values they stand for"""
    return {"q": codes.view(torch.float8_e4m3fn)[:, :K], "s": scales.view(torch.float8_e8m0fnu)}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[case["dt"]]

    def normal(*shape, std=1.0, t=dt, pad=0):
        # (pad: the rows are the first columns of wider ones)
        wide = shape[:-1] + (shape[-1] + pad,)
        v = torch.randn(wide, generator=gen, device=dev, dtype=dt if t == torch.float32 and len(shape) < 2 else t)
        return v.mul_(std).to(t)[..., : shape[-1]]

    def matrix(rows, cols, kind, std=1.0):
        return _quantize(normal(rows, cols, std=std, t=torch.bfloat16).float(), kind)

    def relu_bias(n):
        # the bias of a neuron that fires with probability p, p spread over its logarithm
        p = torch.exp(torch.rand(n, generator=gen, device=dev) * math.log(0.9 / 0.02) + math.log(0.02))
        return torch.special.ndtri(p).to(dt)

    s, op, T = {"case": case}, case["op"], case["T"]
    if op == "quantize":
        # rows of different sizes, as weights and activations have them
        size = torch.exp(torch.randn(T, 1, generator=gen, device=dev))
        s["x"] = normal(T, case["K"], pad=case["pad"]).mul_(size.to(dt))
    elif op == "linear":
        K, N = case["K"], case["N"]
        s["x"], s["w"] = matrix(T, K, case["xk"]), matrix(N, K, case["wk"], K ** -0.5)
        s["b"] = normal(N, std=0.5) if case["bias"] else None
        s["r"] = normal(T, N) if case["res"] else None
    elif op == "ffn":
        d, n, wk, gated = case["d"], case["n"], case["wk"], case["gated"]
        s["x"] = matrix(T, d, case["xk"])
        s["wg"] = matrix(n, d, wk, d ** -0.5) if gated else None
        s["wu"], s["wd"] = matrix(n, d, wk, d ** -0.5), matrix(d, n, wk, n ** -0.5)
        # (the first: of the projection that the activation takes)
        first, second = relu_bias(n) if case["fn"] in ("relu", "sqrelu") else normal(n, std=0.1), normal(n, std=0.1)
        bg, bu = (first, second) if gated else (None, first)
        s["bg"], s["bu"] = (bg, bu) if case["bias"] else (None, None)
        s["bd"] = normal(d, std=0.1) if case["bias"] else None
    else:
        d = case["d"]
        s["x"], s["y"] = normal(T, d, std=2.0, t=DT[case["xdt"]]), normal(T, d)
        for k in ("pre", "post"):
            s["w_" + k] = normal(d, std=0.2).add_(1.0) if case[k] != "none" else None
            s["b_" + k] = normal(d, std=0.2) if case[k] == "layer" else None
        s["gate"] = normal(1 if case["gate"] == 0 else -(-T // case["gate"]), d, std=0.5)
    return s


# ------------------------------------------------------------------ plain forms
def _f(fn, z):
    if fn == "none":
        return z
    if fn == "relu":
        return torch.clamp(z, min=0)
    if fn == "sqrelu":
        return torch.clamp(z, min=0) ** 2
    if fn == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if fn == "silu":
        return z / (1 + torch.exp(-z))
    if fn == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))


def _plain_quantize(s):
    c = s["case"]
    codes, scales = _quantize(s["x"].float(), c["kind"])
    if c["kind"] == "mx8":
        return _held(codes, scales, c["K"])
    return _values(codes, scales, c["K"], "mx4").to(torch.bfloat16)


def _proj(x, w, K, kind, b):
    z = x @ _values(*w, K, kind).t()
    return z if b is None else z + b.float()


def _plain_linear(s):
    c = s["case"]
    y = _f(c["fn"], _proj(_values(*s["x"], c["K"], c["xk"]), s["w"], c["K"], c["wk"], s["b"]))
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(DT[c["dt"]])


def _plain_ffn(s):
    c = s["case"]
    d, n, wk = c["d"], c["n"], c["wk"]
    x = _values(*s["x"], d, c["xk"])
    u = _proj(x, s["wu"], d, wk, s["bu"])
    a = _f(c["fn"], _proj(x, s["wg"], d, wk, s["bg"])) * u if c["gated"] else _f(c["fn"], u)
    a = _values(*_quantize(a, c["xk"]), n, c["xk"])
    return _proj(a, s["wd"], n, wk, s["bd"]).to(DT[c["dt"]])


def _hat(kind, v):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _scaled(v, w, b):
    v = v if w is None else v * w.float()
    return v if b is None else v + b.float()


def _plain_norm(s):
    c, gate = s["case"], s["gate"].float()
    if c["gate"]:
        gate = gate[torch.arange(c["T"], device=gate.device) // c["gate"]]
    v = s["y"].float()
    if c["post"] != "none":
        v = _scaled(_hat(c["post"], v), s["w_post"], s["b_post"])
    xo = c["rs"] * s["x"].float() + gate * v
    h = _scaled(_hat(c["pre"], xo), s["w_pre"], s["b_pre"])
    return {"x": xo.to(s["x"].dtype), **_held(*_quantize(h, "mx8"), c["d"])}


# ------------------------------------------------------------------ the library's calls
_ctx = None


def _library():
    """The context a program keeps for its whole run."""
    global _ctx
    from activation_sparse_decode_sigmoid_gb300 import pi
    if _ctx is None:
        _ctx = pi.Context(0)
    return pi, _ctx


def _own(s):
    pi, c = _library()
    case, op = s["case"], s["case"]["op"]
    kinds = {"mx8": pi.PI_MX8, "mx4": pi.PI_MX4}

    def mx(m, cols, kind):
        return None if m is None else pi.MxMatrix(m[0], m[1], cols, kinds[kind])

    if op == "quantize":
        q = c.mx_quantize(s["x"], kinds[case["kind"]])
        return _held(q.codes, q.scales, case["K"]) if case["kind"] == "mx8" else c.mx_dequantize(q, torch.bfloat16)
    if op == "norm":
        norms = {"none": pi.PI_NORM_NONE, "rms": pi.PI_NORM_RMS, "layer": pi.PI_NORM_LAYER}
        x, h = c.norm_residual_mx(s["x"], s["y"], s["gate"], kind=pi.PI_MX8, pre=norms[case["pre"]], post=norms[case["post"]],
                                  w_pre=s["w_pre"], b_pre=s["b_pre"], w_post=s["w_post"], b_post=s["b_post"],
                                  res_scale=case["rs"], gate_rows=case["gate"], eps=EPS)
        return {"x": x, **_held(h.codes, h.scales, case["d"])}
    fn, dt = getattr(pi, "PI_FN_" + case["fn"].upper()), DT[case["dt"]]
    if op == "linear":
        K = case["K"]
        return c.mx_linear(mx(s["x"], K, case["xk"]), mx(s["w"], K, case["wk"]), s["b"], fn=fn, residual=s["r"], dtype=dt)
    d, n, wk = case["d"], case["n"], case["wk"]
    return c.mx_gated_ffn(mx(s["x"], d, case["xk"]), mx(s["wg"], d, wk), mx(s["wu"], d, wk), mx(s["wd"], n, wk), s["bg"], s["bu"],
                          s["bd"], fn=fn, dtype=dt)


def run(state):
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "linear": _plain_linear, "ffn": _plain_ffn, "norm": _plain_norm}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def _bytes(rows, cols, kind):
    return rows * cols * (1 if kind == "mx8" else 0.5) + rows * cols / 32


def work(case):
    op, T = case["op"], case["T"]
    if op == "quantize":
        K, e = case["K"], 4 if case["dt"] == "f32" else 2
        # (4 bits: the matrix is written, and read again for its values)
        q = _bytes(T, K, case["kind"]) * (1 if case["kind"] == "mx8" else 2)
        return {"bytes": T * K * e + q + (0 if case["kind"] == "mx8" else 2 * T * K), "flops": 4 * T * K}
    if op == "linear":
        K, N = case["K"], case["N"]
        return {"bytes": _bytes(T, K, case["xk"]) + _bytes(N, K, case["wk"]) + 2 * (T * N * (2 if case["res"] else 1) +
                                                                                (N if case["bias"] else 0)),
                "flops": 2 * T * K * N}
    if op == "ffn":
        d, n, k = case["d"], case["n"], 3 if case["gated"] else 2
        return {"bytes": _bytes(T, d, case["xk"]) + k * _bytes(n, d, case["wk"]) + 2 * T * d, "flops": 2 * k * T * d * n}
    d, ex = case["d"], 4 if case["xdt"] == "f32" else 2
    gate = d * (1 if case["gate"] == 0 else -(-T // case["gate"]))
    return {"bytes": T * d * (2 * ex + 2) + _bytes(T, d, "mx8") + 2 * gate, "flops": 14 * T * d}


# ------------------------------------------------------------------ definitions in 64 bits
def _exact_quantize(v, kind):
    """(elements, scales per block) of 64-bit values, by the definitions: the
    least power of two s with amax / s <= the type's largest value, and the
    type's value nearest to v / s, of two as near the one with an even last bit"""
    T, K = v.shape
    Kp = -(-K // 128) * 128
    b = torch.nn.functional.pad(v, (0, Kp - K)).reshape(T, Kp // 32, 32)
    emax, most = MOST[kind]
    s = torch.exp2(torch.ceil(torch.log2(b.abs().amax(2) / most)).clamp(-127, 127))
    s = torch.where(b.abs().amax(2) > s * most, 2 * s, s)
    s = torch.where((b.abs().amax(2) <= s / 2 * most) & (s > 2.0 ** -127), s / 2, s)
    x = b / s[:, :, None]
    mant, least = (3, -6) if kind == "mx8" else (1, 0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** least))) - mant)
    return torch.round(x / step) * step, s  # (round: ties to even)


def _exact_values(v, kind):
    q, s = _exact_quantize(v, kind)
    return (q * s[:, :, None]).reshape(v.shape[0], -1)[:, : v.shape[1]]


def _exact_held(v):
    q, s = _exact_quantize(v, "mx8")
    T, R = v.shape[0], -(-v.shape[0] // 128) * 128
    s = torch.nn.functional.pad(s, (0, 0, 0, R - T), value=2.0 ** -127)
    return {"q": q.reshape(T, -1)[:, : v.shape[1]], "s": s.reshape(R // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous()}


def _exact_f(fn, z):
    if fn == "none":
        return z
    if fn in ("relu", "sqrelu"):
        f = torch.where(z > 0, z, torch.zeros_like(z))
        return f * f if fn == "sqrelu" else f
    if fn == "sigmoid":
        return torch.sigmoid(z)
    if fn == "silu":
        return z * torch.sigmoid(z)
    if fn == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def D(k):
        return None if s.get(k) is None else s[k].double()

    def M(k, cols, kind):
        return _values(*s[k], cols, kind, torch.float64)

    def layer(x, w, b):
        z = torch.einsum("tk,nk->tn", x, w)
        return z if b is None else z + b

    if op == "quantize":
        return _exact_held(D("x")) if case["kind"] == "mx8" else _exact_values(D("x"), "mx4")
    if op == "linear":
        K = case["K"]
        y = _exact_f(case["fn"], layer(M("x", K, case["xk"]), M("w", K, case["wk"]), D("b")))
        return y if s["r"] is None else y + D("r")
    if op == "ffn":
        d, n, wk = case["d"], case["n"], case["wk"]
        x = M("x", d, case["xk"])
        a = layer(x, M("wu", d, wk), D("bu"))
        a = _exact_f(case["fn"], layer(x, M("wg", d, wk), D("bg"))) * a if case["gated"] else _exact_f(case["fn"], a)
        return layer(_exact_values(a, case["xk"]), M("wd", n, wk), D("bd"))

    def normed(kind, v, w, b):
        if kind == "rms":
            out = v / ((v ** 2).mean(1, keepdim=True) + EPS).sqrt()
        else:
            out = (v - v.mean(1, keepdim=True)) / (v.var(1, keepdim=True, unbiased=False) + EPS).sqrt()
        out = out if w is None else out * w
        return out if b is None else out + b

    v = D("y") if case["post"] == "none" else normed(case["post"], D("y"), D("w_post"), D("b_post"))
    gate = D("gate")
    gate = gate if case["gate"] == 0 else gate.repeat_interleave(case["gate"], 0)[: case["T"]]
    xo = case["rs"] * D("x") + gate * v
    return {"x": xo, **_exact_held(normed(case["pre"], xo, D("w_pre"), D("b_pre")))}
