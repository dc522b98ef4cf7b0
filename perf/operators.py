"""The operators of an FFN block outside the sparse decode path, as measured cases.

Three operators, each forward and backward:
  linear          y = r + s f(x W^T + b)
  gated_ffn       y = (f(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd
  norm_residual   x' = rs x + bs gate * norm_post(y),  h = norm_pre(x')

`run` computes them in their plain form (elementary torch operations in 32
bits, rounded once at the end) or, with `own`, through the library's calls.
`exact` evaluates the definitions in 64 bits.  Backward cases take what the
forward pass left in 16 bits (z; g, u and a; x') as inputs, as a training
program has it in hand.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FNS = ("none", "relu", "sqrelu", "sigmoid", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one token through the up-projection of the small OPT-shaped layer: a latency case
        dict(name="linear_token", op="linear", T=1, K=1024, N=4096, dt="f16", fn="relu", bias=True, res=False, pad=0),
        # 8 decode tokens through the LLaMA-70B-shaped down-projection, added to the residual
        dict(name="linear_tokens8", op="linear", T=8, K=28672, N=8192, dt="bf16", fn="none", bias=False, res=True, pad=0),
        # a long prompt through the OPT-30B-shaped up-projection, squared ReLU
        dict(name="linear_prompt", op="linear", T=2048, K=7168, N=28672, dt="f16", fn="sqrelu", bias=True, res=False,
             pad=0),
        # training the predictor's hidden layer (rank 1024) on 4096 inputs: gradients of x, W and b
        dict(name="linear_bwd", op="linear_bwd", T=4096, K=8192, N=1024, dt="bf16", fn="relu", pad=0),
        # a small ragged layer: odd features, rows that are slices of wider ones
        dict(name="linear_bwd_ragged", op="linear_bwd", T=333, K=1001, N=515, dt="f16", fn="gelu", pad=7),
        # one decode token through the LLaMA-70B-shaped ReGLU block, dense
        dict(name="ffn_token", op="ffn", T=1, d=8192, n=28672, dt="bf16", fn="relu", gated=True, bias=True, save=False),
        # the same block on a prompt
        dict(name="ffn_prompt", op="ffn", T=2048, d=8192, n=28672, dt="bf16", fn="relu", gated=True, bias=True,
             save=False),
        # a ragged batch of a small gated layer, saving what its backward pass needs
        dict(name="ffn_ragged", op="ffn", T=45, d=1000, n=2731, dt="f16", fn="gelu", gated=True, bias=True, save=True),
        # the backward pass of a LLaMA-70B-shaped SwiGLU block over 2048 tokens
        dict(name="ffn_bwd", op="ffn_bwd", T=2048, d=8192, n=28672, dt="bf16", fn="silu", gated=True, bias=False),
        # the norm between two blocks for one decode token, fp32 residual stream
        dict(name="norm_token", op="norm", T=1, d=8192, xdt="f32", dt="bf16", pre="rms", post="none", gate=0, rs=1.0),
        # norms before and after a block on a prompt, fp32 residual stream
        dict(name="norm_prompt", op="norm", T=4096, d=7168, xdt="f32", dt="f16", pre="rms", post="rms", gate=1,
             rs=1.0),
        # training: layer norms with weights and biases, a gate per sequence of 1000 tokens, 16-bit stream
        dict(name="norm_bwd", op="norm_bwd", T=8000, d=8192, xdt="bf16", dt="bf16", pre="layer", post="layer",
             gate=1000, rs=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "ffn", "ffn", "ffn_bwd", "norm", "norm_bwd"])
    dt = rng.choice(["f16", "bf16"])
    # half of the time tens of tokens or fewer (decode batches), else prompts and training batches
    T = _log(rng, 1, 80) if rng.random() < 0.5 else _log(rng, 80, 4096)
    if op in ("linear", "linear_bwd"):
        K, N = _log(rng, 64, 28672), _log(rng, 64, 28672)
        if rng.random() < 0.6:  # most models keep their widths multiples of 8
            K, N = K // 8 * 8, N // 8 * 8
        while 4 * T * K * N > 2.5e12:
            T //= 2
        c = dict(op=op, T=T, K=K, N=N, dt=dt, fn=rng.choice(FNS), pad=rng.choice([0, 0, 8, 3]))
        if op == "linear":
            c |= dict(bias=rng.random() < 0.5, res=rng.random() < 0.5)
        return c
    if op in ("ffn", "ffn_bwd"):
        d = _log(rng, 128, 8192)
        n = _log(rng, 2 * d, 4 * d)
        if rng.random() < 0.7:
            d, n = d // 8 * 8, n // 8 * 8
        while 12 * T * d * n > 4e12:
            T //= 2
        c = dict(op=op, T=T, d=d, n=n, dt=dt, fn=rng.choice(FNS[1:]), gated=rng.random() < 0.7,
                 bias=rng.random() < 0.5)
        if op == "ffn":
            c["save"] = rng.random() < 0.4
        return c
    d = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        d = d // 8 * 8
    return dict(op=op, T=T, d=d, xdt=rng.choice(["f32", "f32", dt]), dt=dt, pre=rng.choice(["rms", "layer"]),
                post=rng.choice(["none", "rms", "layer"]), gate=rng.choice([0, 1, _log(rng, 2, 1024)]),
                rs=rng.choice([1.0, 0.5]))


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

    def relu_bias(n):
        # the bias of a neuron that fires with probability p, p spread over its logarithm
        p = torch.exp(torch.rand(n, generator=gen, device=dev) * math.log(0.9 / 0.02) + math.log(0.02))
        return torch.special.ndtri(p).to(dt)

    s, op, T = {"case": case}, case["op"], case["T"]
    if op.startswith("linear"):
        K, N, pad = case["K"], case["N"], case["pad"]
        s["x"] = normal(T, K, pad=pad)
        s["w"] = normal(N, K, std=K ** -0.5)
        if op == "linear":
            s["b"] = normal(N, std=0.5) if case["bias"] else None
            s["r"] = normal(T, N, pad=pad) if case["res"] else None
        else:
            s["z"] = normal(T, N, pad=pad)
            s["dy"] = normal(T, N, pad=pad)
    elif op.startswith("ffn"):
        d, n, gated = case["d"], case["n"], case["gated"]
        s["x"] = normal(T, d)
        s["wg"] = normal(n, d, std=d ** -0.5) if gated else None
        s["wu"] = normal(n, d, std=d ** -0.5)
        s["wd"] = normal(d, n, std=n ** -0.5)
        relu = case["fn"] in ("relu", "sqrelu")
        first = relu_bias(n) if relu else normal(n, std=0.1)  # of the projection that the activation takes
        second = normal(n, std=0.1)
        bg, bu = (first, second) if gated else (None, first)
        s["bg"], s["bu"] = (bg, bu) if case["bias"] else (None, None)
        s["bd"] = normal(d, std=0.1) if case["bias"] else None
        if op == "ffn_bwd":
            s["dy"] = normal(T, d)
            s["g"] = normal(T, n) if gated else None
            s["u"] = normal(T, n)
            act = _f(case["fn"], (s["g"] if gated else s["u"]).float())
            s["a"] = (act * s["u"].float() if gated else act).to(dt)
    else:
        d, xdt = case["d"], DT[case["xdt"]]
        s["x"] = normal(T, d, std=2.0, t=xdt)  # (backward: the stream after the block)
        s["y"] = normal(T, d)
        for k in ("pre", "post"):
            s["w_" + k] = normal(d, std=0.2).add_(1.0) if case[k] != "none" else None
            s["b_" + k] = normal(d, std=0.2) if case[k] == "layer" else None
        groups = 1 if case["gate"] == 0 else -(-T // case["gate"])
        s["gate"] = normal(groups, d, std=0.5)
        if op == "norm_bwd":
            s["dxo"] = normal(T, d, t=xdt)
            s["dh"] = normal(T, d)
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


def _df(fn, z):
    if fn == "none":
        return torch.ones_like(z)
    if fn == "relu":
        return (z > 0).to(z.dtype)
    if fn == "sqrelu":
        return 2 * torch.clamp(z, min=0)
    if fn in ("sigmoid", "silu"):
        p = 1 / (1 + torch.exp(-z))
        return p * (1 - p) if fn == "sigmoid" else p * (1 + z * (1 - p))
    if fn == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _f(s["case"]["fn"], z)
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["x"].dtype)


def _linear_bwd(s):
    dt = s["x"].dtype
    dz = s["dy"].float() * _df(s["case"]["fn"], s["z"].float())
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt), "db": dz.sum(0).to(dt)}


def _proj(x, w, b):
    z = x @ w.float().t()
    return z if b is None else z + b.float()


def _ffn(s):
    dt, c = s["x"].dtype, s["case"]
    x = s["x"].float()
    g = _proj(x, s["wg"], s["bg"]) if c["gated"] else None
    u = _proj(x, s["wu"], s["bu"])
    a = _f(c["fn"], g) * u if c["gated"] else _f(c["fn"], u)
    y = _proj(a, s["wd"], s["bd"]).to(dt)
    if not c["save"]:
        return y
    return {"y": y, "g": None if g is None else g.to(dt), "u": u.to(dt), "a": a.to(dt)}


def _ffn_bwd(s):
    dt, c = s["x"].dtype, s["case"]
    x, dy, u, a = (s[k].float() for k in ("x", "dy", "u", "a"))
    da = dy @ s["wd"].float()
    if c["gated"]:
        g = s["g"].float()
        dg, du = da * u * _df(c["fn"], g), da * _f(c["fn"], g)
    else:
        dg, du = None, da * _df(c["fn"], u)
    dx = du @ s["wu"].float()
    if c["gated"]:
        dx = dx + dg @ s["wg"].float()
    out = {"dx": dx, "w_up": du.t() @ x, "w_down": dy.t() @ a}
    if c["gated"]:
        out["w_gate"] = dg.t() @ x
    if c["bias"]:
        out |= {"b_up": du.sum(0), "b_down": dy.sum(0)}
        if c["gated"]:
            out["b_gate"] = dg.sum(0)
    return {k: v.to(dt) for k, v in out.items()}


EPS = 1e-5


def _hat(kind, v):
    """(normalised rows, their reciprocal standard deviation)"""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r, r


def _gates(s):
    """the gate's row of each token"""
    c, g = s["case"], s["gate"].float()
    if c["gate"] == 0:
        return g
    return g[torch.arange(c["T"], device=g.device) // c["gate"]]


def _scaled(v, w, b):
    v = v if w is None else v * w.float()
    return v if b is None else v + b.float()


def _norm(s):
    c = s["case"]
    v = s["y"].float()
    if c["post"] != "none":
        v = _scaled(_hat(c["post"], v)[0], s["w_post"], s["b_post"])
    xo = c["rs"] * s["x"].float() + _gates(s) * v
    h = _scaled(_hat(c["pre"], xo)[0], s["w_pre"], s["b_pre"])
    return {"x": xo.to(s["x"].dtype), "h": h.to(s["y"].dtype)}


def _norm_grad(kind, hat, r, d):
    d = d - hat * (d * hat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - d.mean(1, keepdim=True)
    return d * r


def _norm_bwd(s):
    c, dt = s["case"], s["y"].dtype
    dh, y, gate = s["dh"].float(), s["y"].float(), _gates(s)
    hat, r = _hat(c["pre"], s["x"].float())
    D = s["dxo"].float() + _norm_grad(c["pre"], hat, r, dh * s["w_pre"].float())
    out = {"dx": (c["rs"] * D).to(s["x"].dtype), "w_pre": (dh * hat).sum(0).to(dt)}
    if c["pre"] == "layer":
        out["b_pre"] = dh.sum(0).to(dt)
    dv = gate * D
    if c["post"] == "none":
        v, dy = y, dv
    else:
        yh, ry = _hat(c["post"], y)
        v = _scaled(yh, s["w_post"], s["b_post"])
        dy = _norm_grad(c["post"], yh, ry, dv * s["w_post"].float())
        out["w_post"] = (dv * yh).sum(0).to(dt)
        if c["post"] == "layer":
            out["b_post"] = dv.sum(0).to(dt)
    out["dy"] = dy.to(dt)
    dgate = torch.zeros(s["gate"].shape, device=y.device)
    at = torch.zeros(c["T"], dtype=torch.long, device=y.device) if c["gate"] == 0 else \
        torch.arange(c["T"], device=y.device) // c["gate"]
    out["gate"] = dgate.index_add_(0, at, D * v).to(dt)
    return out


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
    if op.startswith("norm"):
        kinds = {"none": pi.PI_NORM_NONE, "rms": pi.PI_NORM_RMS, "layer": pi.PI_NORM_LAYER}
        kw = dict(pre=kinds[case["pre"]], post=kinds[case["post"]], w_pre=s["w_pre"], b_pre=s["b_pre"],
                  w_post=s["w_post"], b_post=s["b_post"], res_scale=case["rs"], gate_rows=case["gate"], eps=EPS)
        if op == "norm":
            x, h = c.norm_residual(s["x"], s["y"], s["gate"], **kw)
            return {"x": x, "h": h}
        got = c.norm_residual_bwd(s["dxo"], s["dh"], s["x"], s["y"], s["gate"], **kw)
        return {k: v for k, v in got.items() if v is not None}
    fn = getattr(pi, "PI_FN_" + case["fn"].upper())
    if op == "linear":
        return c.linear(s["x"], s["w"], s["b"], fn=fn, residual=s["r"])
    if op == "linear_bwd":
        dx, dw, db = c.linear_bwd(s["dy"], s["x"], s["w"], s["z"], fn=fn)
        return {"dx": dx, "dw": dw, "db": db}
    if op == "ffn":
        save = c.gated_ffn_save(s["x"], s["wg"], s["wu"]) if case["save"] else None
        y = c.gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], s["bg"], s["bu"], s["bd"], fn=fn, save=save)
        return y if save is None else {"y": y, "g": save[0], "u": save[1], "a": save[2]}
    got = c.gated_ffn_bwd(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], (s["g"], s["u"], s["a"]), fn=fn,
                          bias_grads=case["bias"])
    return {k: v for k, v in got.items() if v is not None}


def run(state):
    if own:
        return _own(state)
    return {"linear": _linear, "linear_bwd": _linear_bwd, "ffn": _ffn, "ffn_bwd": _ffn_bwd, "norm": _norm,
            "norm_bwd": _norm_bwd}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    op, T, e = case["op"], case["T"], 2
    if op.startswith("linear"):
        K, N = case["K"], case["N"]
        if op == "linear":
            b = T * K + N * K + T * N * (2 if case["res"] else 1) + (N if case["bias"] else 0)
            return {"bytes": e * b, "flops": 2 * T * K * N}
        z = 0 if case["fn"] == "none" else T * N
        return {"bytes": e * (T * N + z + 2 * T * K + 2 * N * K + N), "flops": 4 * T * K * N}
    if op.startswith("ffn"):
        d, n = case["d"], case["n"]
        k = 3 if case["gated"] else 2
        if op == "ffn":
            return {"bytes": e * (k * d * n + 2 * T * d + (k * T * n if case["save"] else 0)), "flops": 2 * k * T * d * n}
        return {"bytes": e * (2 * k * d * n + 3 * T * d + k * T * n), "flops": 4 * k * T * d * n}
    d, ex = case["d"], 4 if case["xdt"] == "f32" else 2
    gate = d * (1 if case["gate"] == 0 else -(-T // case["gate"]))
    if op == "norm":
        return {"bytes": T * d * (2 * ex + 2 * e) + e * gate, "flops": 10 * T * d}
    return {"bytes": T * d * (3 * ex + 3 * e) + 2 * e * gate, "flops": 30 * T * d}


# ------------------------------------------------------------------ definitions in 64 bits
def _exact_f(fn, z):
    """(f(z), f'(z)), f' by automatic differentiation of the definition."""
    z = z.detach().requires_grad_(True)
    with torch.enable_grad():
        if fn == "none":
            f = z * 1.0
        elif fn in ("relu", "sqrelu"):
            f = torch.where(z > 0, z, torch.zeros_like(z))
            f = f * f if fn == "sqrelu" else f
        elif fn == "sigmoid":
            f = torch.sigmoid(z)
        elif fn == "silu":
            f = z * torch.sigmoid(z)
        elif fn == "gelu":
            f = z * torch.special.ndtr(z)
        else:
            f = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        (df,) = torch.autograd.grad(f.sum(), z)
    return f.detach(), df


def exact(case, seed):
    s = prepare(case, seed)
    D = lambda k: None if s.get(k) is None else s[k].double()  # noqa: E731
    op = case["op"]
    if op == "linear":
        z = torch.einsum("tk,nk->tn", D("x"), D("w"))
        z = z if s["b"] is None else z + D("b")
        y = _exact_f(case["fn"], z)[0]
        return y if s["r"] is None else y + D("r")
    if op == "linear_bwd":
        dz = D("dy") * _exact_f(case["fn"], D("z"))[1]
        return {"dx": torch.einsum("tn,nk->tk", dz, D("w")), "dw": torch.einsum("tn,tk->nk", dz, D("x")),
                "db": torch.einsum("tn->n", dz)}
    if op == "ffn":
        x = D("x")
        u = torch.einsum("td,nd->tn", x, D("wu")) + (0 if s["bu"] is None else D("bu"))
        if case["gated"]:
            g = torch.einsum("td,nd->tn", x, D("wg")) + (0 if s["bg"] is None else D("bg"))
            a = _exact_f(case["fn"], g)[0] * u
        else:
            g, a = None, _exact_f(case["fn"], u)[0]
        y = torch.einsum("tn,dn->td", a, D("wd")) + (0 if s["bd"] is None else D("bd"))
        return {"y": y, "g": g, "u": u, "a": a} if case["save"] else y
    if op == "ffn_bwd":
        da = torch.einsum("td,dn->tn", D("dy"), D("wd"))
        out = {"w_down": torch.einsum("td,tn->dn", D("dy"), D("a"))}
        if case["gated"]:
            f, df = _exact_f(case["fn"], D("g"))
            dg, du = da * D("u") * df, da * f
            out["dx"] = torch.einsum("tn,nd->td", dg, D("wg")) + torch.einsum("tn,nd->td", du, D("wu"))
            out["w_gate"] = torch.einsum("tn,td->nd", dg, D("x"))
        else:
            du = da * _exact_f(case["fn"], D("u"))[1]
            out["dx"] = torch.einsum("tn,nd->td", du, D("wu"))
        out["w_up"] = torch.einsum("tn,td->nd", du, D("x"))
        if case["bias"]:
            out["b_up"], out["b_down"] = torch.einsum("tn->n", du), torch.einsum("td->d", D("dy"))
            if case["gated"]:
                out["b_gate"] = torch.einsum("tn->n", dg)
        return out

    # the norms: the definition, with gradients by automatic differentiation
    names = ("x", "y", "gate", "w_pre", "b_pre", "w_post", "b_post")
    leaf = {k: D(k) for k in names}
    if op == "norm_bwd":
        leaf = {k: None if v is None else v.requires_grad_(True) for k, v in leaf.items()}

    def normed(kind, v, w, b):
        if kind == "rms":
            out = v / ((v ** 2).mean(1, keepdim=True) + EPS).sqrt()
        else:
            out = (v - v.mean(1, keepdim=True)) / (v.var(1, keepdim=True, unbiased=False) + EPS).sqrt()
        out = out if w is None else out * w
        return out if b is None else out + b

    def branch():
        v = leaf["y"]
        if case["post"] != "none":
            v = normed(case["post"], v, leaf["w_post"], leaf["b_post"])
        rows = [0] * case["T"] if case["gate"] == 0 else [t // case["gate"] for t in range(case["T"])]
        return leaf["gate"][torch.tensor(rows, device=v.device)] * v

    if op == "norm":
        xo = case["rs"] * leaf["x"] + branch()
        return {"x": xo, "h": normed(case["pre"], xo, leaf["w_pre"], leaf["b_pre"])}
    # x is the stream after the block here: its gradient goes on to the branch and, scaled, to the stream before
    with torch.enable_grad():
        h = normed(case["pre"], leaf["x"], leaf["w_pre"], leaf["b_pre"])
        first = [k for k in ("x", "w_pre", "b_pre") if leaf[k] is not None]
        got = dict(zip(first, torch.autograd.grad(h, [leaf[k] for k in first], D("dh"))))
        Dx = got.pop("x") + D("dxo")
        second = [k for k in ("y", "gate", "w_post", "b_post") if leaf[k] is not None]
        got |= dict(zip(second, torch.autograd.grad(branch(), [leaf[k] for k in second], Dx)))
    got["dx"] = case["rs"] * Dx
    got["dy"] = got.pop("y")
    return got
