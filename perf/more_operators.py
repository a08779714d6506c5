"""Cases of the attention operators: cross attention over keys with a bias, rotary
positions, and dropout from a counter-based generator.

A case names an operator (``op``), a direction (``pass``: "infer" the forward pass
alone, "train" forward and backward, "force" also the backward of the gradients, as
training on forces runs it) and its sizes.  ``run`` computes it in plain torch
operations, or through ``emulated_fp32_matrix_amd.attention`` when ``own`` is set;
``exact`` gives the same values in 64 bits from the definitions, by automatic
differentiation where there are derivatives.
"""
import math

import numpy
import torch

own = False


# ---- the cases -----------------------------------------------------------------

def _attention(name, kind, batch, queries, keys, heads, kv_heads, dim, bias=False, ragged=False):
    case = {"op": "attention", "pass": kind, "batch": batch, "queries": queries, "keys": keys, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "bias": bias, "ragged": ragged}
    return {"name": name, **case} if name else case


def _rotary(name, kind, batch, tokens, heads, dim, part, layout, scaling, start):
    case = {"op": "rotary", "pass": kind, "batch": batch, "tokens": tokens, "heads": heads, "dim": dim, "part": part,
            "layout": layout, "scaling": scaling, "start": start}
    return {"name": name, **case} if name else case


def _dropout(name, kind, rows, dim, p, residual):
    case = {"op": "dropout", "pass": kind, "rows": rows, "dim": dim, "p": p, "residual": residual}
    return {"name": name, **case} if name else case


def listed():
    return [
        # one atom's 32 neighbour tokens, d = 256 in 8 heads: latency
        _attention("attention 1x32x32", "infer", 1, 32, 32, 8, 8, 32, bias=True),
        # the 17,280-atom system, every atom's tokens among themselves under the cutoff's
        # logarithm: molecular dynamics, training on energies, training on forces
        _attention("attention 17280x32x32", "infer", 17280, 32, 32, 8, 8, 32, bias=True),
        _attention("attention train 17280x32x32", "train", 17280, 32, 32, 8, 8, 32, bias=True),
        _attention("attention force 17280x32x32", "force", 17280, 32, 32, 8, 8, 32, bias=True),
        # one query a sequence against long encoder states of ragged lengths, shared heads: serving
        _attention("attention 8x1x8192", "infer", 8, 1, 8192, 16, 4, 64, ragged=True),
        # a decoder's queries against an encoder's states, training
        _attention("attention train 2x2048x4096", "train", 2, 2048, 4096, 16, 16, 64),
        # odd sizes and lengths, shared wide heads, trained on forces
        _attention("attention force 7x257x777", "force", 7, 257, 777, 6, 2, 80, bias=True, ragged=True),
        # one new token of each of four sequences, far from their start: latency
        _rotary("rotary 4x1", "infer", 4, 1, 16, 64, 64, "half", "parts", 1000003),
        # the large system's tokens, a quarter of the head left as it is, training
        _rotary("rotary train 17280x32", "train", 17280, 32, 8, 32, 24, "interleaved", "none", 0),
        # long sequences of wide heads
        _rotary("rotary 4x16381", "infer", 4, 16381, 16, 128, 128, "half", "base", 0),
        # one atom's tokens: latency
        _dropout("dropout 32x256", "infer", 32, 256, 0.1, True),
        # the large system's tokens with the residual stream, training
        _dropout("dropout train 552960x256", "train", 552960, 256, 0.1, True),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head(rng):
    """A head's width: mostly what models have, else any even number."""
    return rng.choice((16, 32, 48, 64, 64, 80, 96, 128)) if rng.random() < 0.8 else 2 * rng.randint(4, 64)


def draw(rng):
    most = max(work(c)["flops"] for c in listed()), max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(("attention", "attention", "rotary", "dropout"))
        if op == "attention":
            kind, dim, kv = rng.choice(("infer", "train", "force")), _head(rng), rng.choice((1, 2, 4, 8))
            heads = kv * rng.choice((1, 1, 2, 4))
            if rng.random() < 0.4:   # tokens around atoms
                n = rng.randint(4, 48)
                case = _attention(None, kind, _spread(rng, 1, 17280), n, n, heads, heads, min(dim, 64), bias=True)
            else:                    # queries against an encoder's states
                case = _attention(None, kind, _spread(rng, 1, 32), _spread(rng, 1, 2048), _spread(rng, 16, 8192), heads,
                                  kv, dim, bias=rng.random() < 0.5, ragged=rng.random() < 0.5)
        elif op == "rotary":
            dim = _head(rng)
            part = dim if rng.random() < 0.6 else 2 * rng.randint(2, dim // 2)
            case = _rotary(None, rng.choice(("infer", "train")), _spread(rng, 1, 1024), _spread(rng, 1, 16384),
                           rng.choice((1, 2, 4, 8, 16)), dim, part, rng.choice(("half", "interleaved")),
                           rng.choice(("none", "linear", "base", "parts")), rng.choice((0, 0, 1000, 1000003)))
        else:
            case = _dropout(None, rng.choice(("infer", "train")), _spread(rng, 1, 552960), _spread(rng, 16, 4096),
                            rng.choice((0.05, 0.1, 0.2, 0.5)), rng.random() < 0.5)
        w = work(case)
        if w["flops"] <= most[0] and w["bytes"] <= most[1]:
            return case


def _lengths(case):
    """Valid keys of each sequence, in some order: evenly from none to all."""
    b, n = case["batch"], case["keys"]
    return [n * i // max(b - 1, 1) for i in range(b)] if b > 1 and case["ragged"] else [n] * b


def work(case):
    if case["op"] == "attention":
        keys = sum(_lengths(case))
        pairs = float(keys) * case["queries"] * case["heads"]
        q = float(case["batch"]) * case["queries"] * case["heads"] * case["dim"]
        k = float(keys) * case["kv_heads"] * case["dim"]
        # tensors of the queries' and of the keys' shape, vectors over the keys, and products
        nq, nk, nb, products = {"infer": (2, 2, 1, 2), "train": (4, 4, 2, 7), "force": (7, 8, 4, 19)}[case["pass"]]
        return {"bytes": 4.0 * (nq * q + nk * k + (nb * keys if case["bias"] else 0)),
                "flops": 2.0 * products * pairs * case["dim"]}
    if case["op"] == "rotary":
        n = float(case["batch"]) * case["tokens"] * case["heads"] * case["dim"]
        passes = 2 if case["pass"] == "train" else 1
        return {"bytes": passes * 8.0 * n + 8.0 * case["batch"] * case["tokens"], "flops": passes * 3.0 * n}
    n = float(case["rows"]) * case["dim"]
    tensors = (3 if case["residual"] else 2) + (2 if case["pass"] == "train" else 0)
    return {"bytes": 4.0 * tensors * n, "flops": (2.0 if case["residual"] else 1.0) * n}


# ---- inputs ----------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    train = case["pass"] != "infer"
    if case["op"] == "attention":
        b, lq, lk, h, g, d = (case[n] for n in ("batch", "queries", "keys", "heads", "kv_heads", "dim"))
        s["q"], s["k"], s["v"] = normal(b, lq, h, d), normal(b, lk, g, d), normal(b, lk, g, d)
        s["bias"] = s["lengths"] = None
        if case["bias"]:
            # the logarithm of a cutoff function of the distance, nothing beyond the cutoff
            r = 1.1 * torch.rand(b, lk, generator=gen, device="cuda", dtype=torch.float32)
            s["bias"] = torch.where(r < 0.999, torch.log(0.5 + 0.5 * torch.cos(math.pi * r)), -math.inf)
        if case["ragged"]:
            order = torch.randperm(b, generator=gen, device="cuda")
            s["lengths"] = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32)[order]
        if train:
            s["g"] = normal(b, lq, h, d)                     # gradient of the output
        if case["pass"] == "force":                          # gradients of the gradients
            s["vq"], s["vk"], s["vv"] = normal(b, lq, h, d), normal(b, lk, g, d), normal(b, lk, g, d)
            s["vb"] = normal(b, lk) if case["bias"] else None
            s["g"].requires_grad_(True)
        if train:
            for name in ("q", "k", "v", "bias"):
                if s[name] is not None:
                    s[name].requires_grad_(True)
    elif case["op"] == "rotary":
        b, t, h, d = (case[n] for n in ("batch", "tokens", "heads", "dim"))
        s["x"] = normal(b, t, h, d)
        first = case["start"] + torch.randint(0, 64, (b, 1), generator=gen, device="cuda")
        s["positions"] = first + torch.arange(t, device="cuda")
        s["plan"] = _own_plan(case) if own else _plain_plan(case)
        if train:
            s["g"] = normal(b, t, h, d)
            s["x"].requires_grad_(True)
    else:
        r, d = case["rows"], case["dim"]
        s["x"] = normal(r, d)
        s["res"] = normal(r, d) if case["residual"] else None
        s["seed"] = torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=gen, device="cuda")
        if train:
            s["g"] = normal(r, d)
            s["x"].requires_grad_(True)
            if s["res"] is not None:
                s["res"].requires_grad_(True)
    return s


_FACTOR, _ORIGINAL = 8.0, 4096   # of the scaled frequencies


def _own_plan(case):
    from emulated_fp32_matrix_amd import attention

    scaled = {} if case["scaling"] == "none" else {"scaling": case["scaling"], "factor": _FACTOR}
    if case["scaling"] == "parts":
        scaled["original_length"] = _ORIGINAL
    return attention.Rotary(case["part"], layout=case["layout"], device="cuda", **scaled)


def _plain_plan(case):
    """(radians per position, magnitude): base 10,000, and its scalings for long contexts."""
    n, kind = case["part"], case["scaling"]
    base = 10000.0
    if kind == "base" and n > 2:
        base *= _FACTOR ** (n / (n - 2))
    f = torch.exp(torch.arange(0, n, 2, device="cuda", dtype=torch.float64) * (-math.log(base) / n))
    if kind == "linear":
        f = f / _FACTOR
    if kind == "parts":   # below 1 turn over the original length interpolated, above 32 kept
        w = torch.clamp((f * (_ORIGINAL / (2 * math.pi)) - 1.0) / 31.0, 0.0, 1.0)
        f = f * (w + (1.0 - w) / _FACTOR)
    return f, 0.1 * math.log(_FACTOR) + 1.0 if kind == "parts" else 1.0


# ---- plain forms -----------------------------------------------------------------

def _plain_attention(s):
    case, q, k, v, bias = s["case"], s["q"], s["k"], s["v"], s["bias"]
    b, lq, lk, h, g, d = (case[n] for n in ("batch", "queries", "keys", "heads", "kv_heads", "dim"))
    scale = 1.0 / math.sqrt(d)

    # [batch, key/value heads, queries x sharing heads or keys, dim]
    def rows(t):
        return t.reshape(b, lq, g, h // g, d).permute(0, 2, 1, 3, 4).reshape(b, g, lq * (h // g), d)

    def unrows(t):
        return t.reshape(b, g, lq, h // g, d).permute(0, 2, 1, 3, 4).reshape(b, lq, h, d)

    def cols(t):
        return t.permute(0, 2, 1, 3).contiguous()

    def uncols(t):
        return t.permute(0, 2, 1, 3).contiguous()

    alive = torch.ones(b, lk, dtype=torch.bool, device=q.device)
    if s["lengths"] is not None:
        alive = torch.arange(lk, device=q.device) < s["lengths"][:, None]
    if bias is not None:
        alive = alive & (bias > -math.inf)
    mask = alive[:, None, None, :]
    q2, k2, v2 = rows(q), cols(k), cols(v)
    z = torch.matmul(q2, k2.transpose(2, 3)) * scale
    if bias is not None:
        z = z + torch.where(alive, bias, 0.0)[:, None, None, :]
    z = torch.where(mask, z, -math.inf)
    m = z.amax(dim=3, keepdim=True)
    e = torch.exp(z - torch.where(m > -math.inf, m, 0.0))
    total = e.sum(dim=3, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    out = torch.matmul(p, v2)
    if case["pass"] == "infer":
        return unrows(out)
    do = rows(s["g"])
    dp = torch.matmul(do, v2.transpose(2, 3))
    delta = (do * out).sum(dim=3, keepdim=True)
    ds = p * (dp - delta)
    got = [unrows(out), unrows(torch.matmul(ds, k2) * scale), uncols(torch.matmul(ds.transpose(2, 3), q2) * scale),
           uncols(torch.matmul(p.transpose(2, 3), do))]
    if bias is not None:
        got.append(ds.sum(dim=2).sum(dim=1))
    if case["pass"] == "train":
        return got
    vq, vk, vv = rows(s["vq"]), cols(s["vk"]), cols(s["vv"])
    gam = (torch.matmul(vq, k2.transpose(2, 3)) + torch.matmul(q2, vk.transpose(2, 3))) * scale
    if s["vb"] is not None:
        gam = gam + s["vb"][:, None, None, :]
    mean = (p * gam).sum(dim=3, keepdim=True)
    hh = p * (gam - mean)
    t = gam * (dp - delta) - mean * dp + torch.matmul(do, vv.transpose(2, 3))
    u = p * (t - (p * t).sum(dim=3, keepdim=True))
    got += [unrows(torch.matmul(hh, v2) + torch.matmul(p, vv)),
            unrows((torch.matmul(u, k2) + torch.matmul(ds, vk)) * scale),
            uncols((torch.matmul(u.transpose(2, 3), q2) + torch.matmul(ds.transpose(2, 3), vq)) * scale),
            uncols(torch.matmul(hh.transpose(2, 3), do))]
    if bias is not None:
        got.append(u.sum(dim=2).sum(dim=1))
    return got


def _plain_rotary(s):
    case = s["case"]
    n, half = case["part"], case["part"] // 2
    f, magnitude = s["plan"]
    angle = s["positions"].double()[:, :, None, None] * f
    cos, sin = (magnitude * torch.cos(angle)).float(), (magnitude * torch.sin(angle)).float()

    def turn(x, sin):
        if case["layout"] == "half":
            a, b = x[..., :half], x[..., half:n]
        else:
            a, b = x[..., 0:n:2], x[..., 1:n:2]
        a, b = a * cos - b * sin, a * sin + b * cos
        both = torch.cat([a, b], dim=3) if case["layout"] == "half" else torch.stack([a, b], dim=4).flatten(3)
        return torch.cat([both, x[..., n:]], dim=3)

    y = turn(s["x"], sin)
    return (y, turn(s["g"], -sin)) if case["pass"] == "train" else y


def _plain_dropout(s):
    case, x = s["case"], s["x"]
    low = 0xFFFFFFFF
    n = (x.numel() + 3) // 4
    i = torch.arange(n, device=x.device)
    c = [i & low, i >> 32, s["seed"][1] & low, (s["seed"][1] >> 32) & low]
    k0, k1 = s["seed"][0] & low, (s["seed"][0] >> 32) & low
    for _ in range(10):   # Philox4x32-10
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, dim=1).reshape(-1)[:x.numel()].reshape(x.shape)
    keep = words >= int(round(case["p"] * 2 ** 32))
    scale = 1.0 / (1.0 - case["p"])
    y = torch.where(keep, x * scale, 0.0)
    if s["res"] is not None:
        y = y + s["res"]
    if case["pass"] == "infer":
        return y
    got = [y, torch.where(keep, s["g"] * scale, 0.0)]
    return got + [s["g"]] if s["res"] is not None else got


# ---- the framework's operators -----------------------------------------------------

def _own_attention(s):
    from emulated_fp32_matrix_amd import attention

    y = attention.cross_attention(s["q"], s["k"], s["v"], key_bias=s["bias"], lengths=s["lengths"])
    if s["case"]["pass"] == "infer":
        return y
    leaves = [s[n] for n in ("q", "k", "v", "bias") if s[n] is not None]
    if s["case"]["pass"] == "train":
        return [y, *torch.autograd.grad(y, leaves, s["g"])]
    first = torch.autograd.grad(y, leaves, s["g"], create_graph=True)
    second = torch.autograd.grad(first, [s["g"], *leaves],
                                 [s[n] for n in ("vq", "vk", "vv", "vb") if s[n] is not None])
    return [y, *first, *second]


def _own_rotary(s):
    y = s["plan"](s["x"], s["positions"])
    return (y, *torch.autograd.grad(y, s["x"], s["g"])) if s["case"]["pass"] == "train" else y


def _own_dropout(s):
    from emulated_fp32_matrix_amd import attention

    y = attention.dropout(s["x"], s["case"]["p"], s["seed"], residual=s["res"])
    if s["case"]["pass"] == "infer":
        return y
    return [y, *torch.autograd.grad(y, [s[n] for n in ("x", "res") if s[n] is not None], s["g"])]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "rotary": _own_rotary, "dropout": _own_dropout}[op](state)
    with torch.no_grad():
        return {"attention": _plain_attention, "rotary": _plain_rotary, "dropout": _plain_dropout}[op](state)


# ---- 64 bits -----------------------------------------------------------------------

def _exact_attention(case, s):
    names = [n for n in ("q", "k", "v", "bias") if s[n] is not None]
    kind, b, lk = case["pass"], case["batch"], case["keys"]
    beyond = torch.zeros(b, lk, dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        for i, n in enumerate(s["lengths"].tolist()):
            beyond[i, n:] = True
    share = case["heads"] // case["kv_heads"]
    # sequences at a time, by the size of their probabilities
    step = max(1, 2 ** 26 // (case["heads"] * case["queries"] * lk))
    parts = []
    for lo in range(0, b, step):
        x = {n: s[n][lo:lo + step].detach().double().requires_grad_(kind != "infer") for n in names}
        q, k, v = x["q"].transpose(1, 2), *(x[n].transpose(1, 2).repeat_interleave(share, dim=1) for n in ("k", "v"))
        z = (q @ k.transpose(2, 3).contiguous()) / math.sqrt(case["dim"])
        dead = beyond[lo:lo + step]
        if "bias" in x:
            dead = dead | torch.isneginf(x["bias"].detach())
            z = z + x["bias"].masked_fill(dead, 0.0)[:, None, None]
        z = z.masked_fill(dead[:, None, None], -1e300)
        p = torch.softmax(z, dim=-1).masked_fill(dead[:, None, None], 0.0)
        y = (p @ v).transpose(1, 2)
        if kind == "infer":
            parts.append([y.contiguous()])
            continue
        leaves, g = [x[n] for n in names], s["g"][lo:lo + step].detach().double()
        if kind == "train":
            parts.append([y.detach().contiguous(), *torch.autograd.grad(y, leaves, g)])
            continue
        g.requires_grad_(True)
        first = torch.autograd.grad(y, leaves, g, create_graph=True)
        seconds = [s[n][lo:lo + step].double() for n in ("vq", "vk", "vv", "vb")[:len(names)]]
        second = torch.autograd.grad(first, [g, *leaves], seconds)
        parts.append([y.detach().contiguous(), *(t.detach() for t in first), *second])
    got = [torch.cat(t) for t in zip(*parts)]
    return got[0] if kind == "infer" else got


def _exact_rotary(case, s):
    n, kind = case["part"], case["scaling"]
    base, magnitude, f = 10000.0, 1.0, []
    if kind == "base" and n > 2:
        base = 10000.0 * math.pow(_FACTOR, n / (n - 2))
    for i in range(n // 2):
        one = math.pow(base, -2 * i / n)
        if kind == "linear":
            one /= _FACTOR
        if kind == "parts":
            w = min(max((_ORIGINAL * one / (2 * math.pi) - 1.0) / 31.0, 0.0), 1.0)
            one = w * one + (1.0 - w) * one / _FACTOR
        f.append(one)
    if kind == "parts":
        magnitude = 1.0 + 0.1 * math.log(_FACTOR)
    angle = s["positions"].double()[..., None] * torch.tensor(f, device="cuda", dtype=torch.float64)
    unit = (magnitude * torch.polar(torch.ones_like(angle), angle))[:, :, None]

    def turn(x, unit):
        x = x.detach().double()
        y = x.clone()
        if case["layout"] == "half":
            z = torch.complex(x[..., :n // 2], x[..., n // 2:n]) * unit
            y[..., :n // 2], y[..., n // 2:n] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:n:2], x[..., 1:n:2]) * unit
            y[..., 0:n:2], y[..., 1:n:2] = z.real, z.imag
        return y

    y = turn(s["x"], unit)
    return (y, turn(s["g"], unit.conj())) if case["pass"] == "train" else y


def _exact_dropout(case, s):
    # the generator's words on the host
    seed, offset = (int(t) & (2 ** 64 - 1) for t in s["seed"].tolist())
    count, low = s["x"].numel(), numpy.uint64(0xFFFFFFFF)
    keep = numpy.empty((count + 3) // 4 * 4, dtype=bool)
    step = 1 << 20
    for lo in range(0, len(keep) // 4, step):
        i = numpy.arange(lo, min(lo + step, len(keep) // 4), dtype=numpy.uint64)
        x, y = i & low, i >> numpy.uint64(32)
        z, w = numpy.full_like(i, offset & 0xFFFFFFFF), numpy.full_like(i, offset >> 32)
        for n in range(10):
            ka = numpy.uint64(((seed & 0xFFFFFFFF) + n * 0x9E3779B9) & 0xFFFFFFFF)
            kb = numpy.uint64(((seed >> 32) + n * 0xBB67AE85) & 0xFFFFFFFF)
            left, right = x * numpy.uint64(0xD2511F53), z * numpy.uint64(0xCD9E8D57)
            x, y, z, w = (right >> numpy.uint64(32)) ^ y ^ ka, right & low, (left >> numpy.uint64(32)) ^ w ^ kb, left & low
        for j, word in enumerate((x, y, z, w)):
            keep[4 * lo + j:4 * (lo + len(i)):4] = word >= numpy.uint64(round(case["p"] * 2 ** 32))
    factor = torch.from_numpy(keep[:count]).to("cuda").reshape(s["x"].shape).double() / (1.0 - case["p"])
    y = s["x"].detach().double() * factor
    if s["res"] is not None:
        y += s["res"].detach().double()
    if case["pass"] == "infer":
        return y
    got = [y, s["g"].double() * factor]
    return got + [s["g"].double()] if s["res"] is not None else got


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "rotary": _exact_rotary, "dropout": _exact_dropout}[case["op"]](case, s)
