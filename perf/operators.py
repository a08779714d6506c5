"""Cases of the transformer-block operators: layer norm, matrix products with bias,
activation and residual in their epilogue, and gated feed-forward projections.

A case names an operator (``op``), a direction (``pass``: "infer" the forward pass
alone, "train" forward and backward, "force" also the backward of the input
gradient, as training on forces runs it) and its sizes.  ``run`` computes it in
plain torch operations, or through ``emulated_fp32_matrix_amd.block`` when ``own``
is set; ``exact`` gives the same values in 64 bits by automatic differentiation of
the definitions.
"""
import math

import torch

own = False

EPS = 1e-5


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # one atom's 32 neighbour tokens through a norm of the d = 256 model: latency
        {"name": "norm 32x256", "op": "norm", "pass": "infer", "rows": 32, "dim": 256},
        # the 17,280-atom system's tokens: inference and molecular dynamics
        {"name": "norm 552960x256", "op": "norm", "pass": "infer", "rows": 552960, "dim": 256},
        # the same tokens in a training step
        {"name": "norm train 552960x256", "op": "norm", "pass": "train", "rows": 552960, "dim": 256},
        # a ragged batch of the wide model trained on forces, odd width
        {"name": "norm force 12289x1023", "op": "norm", "pass": "force", "rows": 12289, "dim": 1023},
        # one token through the first feed-forward linear of the d = 256 model
        {"name": "linear 1x256x512", "op": "linear", "pass": "infer", "rows": 1, "inner": 256, "outer": 512,
         "act": "silu", "residual": False, "mode": "AUTO"},
        # second feed-forward linear and the residual sum, 17,280 atoms
        {"name": "linear 552960x512x256", "op": "linear", "pass": "infer", "rows": 552960, "inner": 512,
         "outer": 256, "act": "identity", "residual": True, "mode": "AUTO"},
        # first feed-forward linear of the d = 1024 model, 192 atoms, training
        {"name": "linear train 6144x1024x4096", "op": "linear", "pass": "train", "rows": 6144, "inner": 1024,
         "outer": 4096, "act": "gelu", "residual": False, "mode": "AUTO"},
        # odd widths and rows (a head of a model whose sizes are no multiples of a tile), six products
        {"name": "linear train 5003x387x771", "op": "linear", "pass": "train", "rows": 5003, "inner": 387,
         "outer": 771, "act": "tanh", "residual": True, "mode": "BF16X6"},
        # one atom's tokens through the gated projection of the d = 256 model
        {"name": "gated 32x256x512", "op": "gated", "pass": "infer", "rows": 32, "inner": 256, "outer": 512,
         "act": "silu", "mode": "AUTO"},
        # 17,280 atoms, inference
        {"name": "gated 552960x256x512", "op": "gated", "pass": "infer", "rows": 552960, "inner": 256,
         "outer": 512, "act": "silu", "mode": "AUTO"},
        # the d = 1024 model, 192 atoms, training with six products
        {"name": "gated train 6144x1024x2048", "op": "gated", "pass": "train", "rows": 6144, "inner": 1024,
         "outer": 2048, "act": "gelu_tanh", "mode": "BF16X6"},
        # 17,280 atoms, training
        {"name": "gated train 552960x256x512", "op": "gated", "pass": "train", "rows": 552960, "inner": 256,
         "outer": 512, "act": "silu", "mode": "AUTO"},
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 32, as models have them, else any number."""
    n = _spread(rng, lo, hi)
    return n if rng.random() < 0.3 else max(32, n // 32 * 32)


def draw(rng):
    most = max(work(c)["flops"] for c in listed()), max(work(c)["bytes"] for c in listed())
    op = rng.choice(("norm", "linear", "gated"))
    while True:
        case = {"op": op, "rows": _spread(rng, 1, 552960)}
        if op == "norm":
            case.update({"pass": rng.choice(("infer", "train", "force")), "dim": _width(rng, 64, 4096)})
        else:
            case.update({"pass": rng.choice(("infer", "train")), "inner": _width(rng, 64, 4096),
                         "outer": _width(rng, 64, 4096),
                         "act": rng.choice(("silu", "gelu", "gelu_tanh", "tanh", "relu")),
                         "mode": rng.choice(("AUTO", "AUTO", "BF16X6"))})
            if op == "linear":
                case["residual"] = rng.random() < 0.5
        w = work(case)
        if w["flops"] <= most[0] and w["bytes"] <= most[1]:
            return case


def work(case):
    r, train = case["rows"], case["pass"] != "infer"
    if case["op"] == "norm":
        d = case["dim"]
        tensors, vectors = {"infer": (2, 2), "train": (4, 4), "force": (7, 3)}[case["pass"]]
        return {"bytes": 4.0 * (tensors * r * d + vectors * d), "flops": {"infer": 8.0, "train": 24.0, "force": 60.0}[case["pass"]] * r * d}
    k, n = case["inner"], case["outer"]
    if case["op"] == "linear":
        more = r * n if case["residual"] else 0
        return {"bytes": 4.0 * ((2 if train else 1) * (r * k + k * n + n + r * n + more)),
                "flops": (6.0 if train else 2.0) * r * k * n}
    return {"bytes": 4.0 * (2 if train else 1) * (r * k + 2 * k * n + 2 * n + r * n),
            "flops": (6.0 if train else 2.0) * r * k * 2 * n}


# ---- inputs ----------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    r = case["rows"]
    s = {"case": case}
    if case["op"] == "norm":
        d = case["dim"]
        # tokens of a residual stream: a scale and an offset of their own
        s["x"] = normal(r, d) * torch.exp(0.5 * normal(r, 1)) + normal(r, 1)
        s["w"], s["b"] = 1.0 + 0.1 * normal(d), 0.1 * normal(d)
        out = d
    else:
        k, n = case["inner"], case["outer"]
        wide = 2 * n if case["op"] == "gated" else n   # gated: rows 0..n-1 gate, n..2n-1 up
        s["x"] = normal(r, k)
        s["w"], s["b"] = normal(wide, k) / math.sqrt(k), 0.1 * normal(wide)
        s["res"] = normal(r, n) if case.get("residual") else None
        out = n
    if case["pass"] != "infer":
        s["g"] = normal(r, out)                        # gradient of the output
        if case["pass"] == "force":
            s["v"] = normal(r, out)                    # gradient of the input gradient
        for name in ("x", "w", "b", "res"):
            if s.get(name) is not None:
                s[name].requires_grad_(True)
        if case["pass"] == "force":
            s["g"].requires_grad_(True)
    return s


# ---- plain forms -----------------------------------------------------------------

def _act(name, z):
    if name == "identity":
        return z
    if name == "relu":
        return torch.clamp(z, min=0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "tanh":
        return torch.tanh(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(name, z):
    if name == "identity":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "tanh":
        t = torch.tanh(z)
        return 1.0 - t * t
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _plain_norm(s):
    kind, x, w, b = s["case"]["pass"], s["x"], s["w"], s["b"]
    n = x.shape[1]

    def mean(t):
        return t.sum(dim=1, keepdim=True) / n

    c = x - mean(x)
    rstd = 1.0 / torch.sqrt(mean(c * c) + EPS)
    xhat = c * rstd
    y = xhat * w + b
    if kind == "infer":
        return y
    g = s["g"]
    a = g * w
    m_ax = mean(a * xhat)
    gx = rstd * (a - mean(a) - xhat * m_ax)
    if kind == "train":
        return y, gx, (g * xhat).sum(dim=0), g.sum(dim=0)
    v = s["v"]
    m_vx = mean(v * xhat)
    t = rstd * (v - mean(v) - xhat * m_vx)
    h = -rstd * (a * m_vx + v * m_ax)
    dx = rstd * (h - mean(h) - xhat * mean(h * xhat)) - rstd * xhat * mean(v * gx)
    return y, gx, t * w, dx, (g * t).sum(dim=0)


def _plain_linear(s):
    case, x, w, b = s["case"], s["x"], s["w"], s["b"]
    z = torch.matmul(x, w.t()) + b
    y = _act(case["act"], z)
    if s["res"] is not None:
        y = y + s["res"]
    if case["pass"] == "infer":
        return y
    dz = s["g"] if case["act"] == "identity" else s["g"] * _act_slope(case["act"], z)
    got = [y, torch.matmul(dz, w), torch.matmul(dz.t(), x), dz.sum(dim=0)]
    return got + [s["g"]] if s["res"] is not None else got


def _plain_gated(s):
    case, x, w, b = s["case"], s["x"], s["w"], s["b"]
    n = case["outer"]
    z = torch.matmul(x, w.t()) + b
    gate, up = z[:, :n], z[:, n:]
    a = _act(case["act"], gate)
    h = a * up
    if case["pass"] == "infer":
        return h
    g = s["g"]
    dz = torch.cat([g * up * _act_slope(case["act"], gate), g * a], dim=1)
    return [h, torch.matmul(dz, w), torch.matmul(dz.t(), x), dz.sum(dim=0)]


# ---- the framework's operators -----------------------------------------------------

def _own_norm(s):
    from emulated_fp32_matrix_amd import block

    y = block.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
    if s["case"]["pass"] == "infer":
        return y
    if s["case"]["pass"] == "train":
        return (y, *torch.autograd.grad(y, [s["x"], s["w"], s["b"]], s["g"]))
    (gx,) = torch.autograd.grad(y, s["x"], s["g"], create_graph=True)
    dg, dx, dw = torch.autograd.grad(gx, [s["g"], s["x"], s["w"]], s["v"])
    return y, gx, dg, dx, dw


def _own_linear(s):
    from emulated_fp32_matrix_amd import block

    case = s["case"]
    y = block.linear_act(s["x"], s["w"], s["b"], activation=case["act"], residual=s["res"], mode=case["mode"])
    if case["pass"] == "infer":
        return y
    leaves = [s["x"], s["w"], s["b"]] + ([s["res"]] if s["res"] is not None else [])
    return [y, *torch.autograd.grad(y, leaves, s["g"])]


def _own_gated(s):
    from emulated_fp32_matrix_amd import block

    case = s["case"]
    h = block.gated_linear(s["x"], s["w"], s["b"], activation=case["act"], mode=case["mode"])
    if case["pass"] == "infer":
        return h
    return [h, *torch.autograd.grad(h, [s["x"], s["w"], s["b"]], s["g"])]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "gated": _own_gated}[op](state)
    with torch.no_grad():
        return {"norm": _plain_norm, "linear": _plain_linear, "gated": _plain_gated}[op](state)


# ---- 64 bits -----------------------------------------------------------------------

def _define(case, x, w, b, res):
    """The operator's definition, differentiable, in the inputs' precision."""
    if case["op"] == "norm":
        var, mu = torch.var_mean(x, dim=-1, unbiased=False, keepdim=True)
        return (x - mu) * torch.rsqrt(var + EPS) * w + b
    z = torch.addmm(b, x, w.t())
    act = {"identity": lambda t: t, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
           "tanh": lambda t: 1.0 - 2.0 / (torch.exp(2.0 * t) + 1.0),
           "gelu": lambda t: 0.5 * t * torch.erfc(-t / math.sqrt(2.0)),
           # 1 + tanh(q) = 2 sigmoid(2 q)
           "gelu_tanh": lambda t: t * torch.sigmoid(math.sqrt(8.0 / math.pi) * (t + 0.044715 * t.pow(3)))}[case["act"]]
    if case["op"] == "gated":
        gate, up = z.chunk(2, dim=1)
        return act(gate) * up
    return act(z) if res is None else act(z) + res


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: s[k].detach().double() for k in ("x", "w", "b", "res", "g", "v") if s.get(k) is not None}
    del s
    if case["pass"] == "infer":
        with torch.no_grad():
            return _define(case, wide["x"], wide["w"], wide["b"], wide.get("res"))
    leaves = [wide[k].requires_grad_(True) for k in ("x", "w", "b", "res") if k in wide]
    y = _define(case, wide["x"], wide["w"], wide["b"], wide.get("res"))
    if case["pass"] == "train":
        got = [y.detach(), *torch.autograd.grad(y, leaves, wide["g"])]
        return tuple(got) if case["op"] == "norm" else got
    g = wide["g"].requires_grad_(True)
    (gx,) = torch.autograd.grad(y, wide["x"], g, create_graph=True)
    dg, dx, dw = torch.autograd.grad(gx, [g, wide["x"], wide["w"]], wide["v"])
    return y.detach(), gx.detach(), dg, dx, dw
