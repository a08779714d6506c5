"""GPU parity of cross attention (include/emu_attention.h,
emulated_fp32_matrix_amd/attention.py): outputs, gradients and the gradients'
gradients against the formulas in 64 bits, within the error that FP32
arithmetic of the same formulas may have (tests/attention_reference.py)."""
import math

import pytest
import torch

from attention_reference import Attention, close
from emulated_fp32_matrix_amd import attention
from gpu_helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def make(batch, queries, keys, heads, kv_heads, dim, bias=False, mask=False, lengths=None, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000 * queries + keys)
    x = {"q": normal(g, batch, queries, heads, dim), "k": normal(g, batch, keys, kv_heads, dim),
         "v": normal(g, batch, keys, kv_heads, dim), "bias": None, "mask": None, "lengths": None}
    if bias:
        x["bias"] = normal(g, batch, keys)
        x["bias"][torch.rand(batch, keys, generator=g, device=DEV) < 0.1] = -math.inf
    if mask:
        x["mask"] = torch.rand(batch, keys, generator=g, device=DEV) < 0.8
    if lengths is not None:
        x["lengths"] = torch.tensor(lengths, device=DEV, dtype=torch.int64)
    x["g"] = normal(g, batch, queries, heads, dim)
    x["vq"], x["vk"], x["vv"] = (normal(g, *x[n].shape) for n in "qkv")
    x["vb"] = normal(g, batch, keys)
    return x


def call(x, **over):
    a = {**x, **over}
    return attention.cross_attention(a["q"], a["k"], a["v"], key_bias=a["bias"], key_mask=a["mask"], lengths=a["lengths"],
                                     scale=a.get("scale"))


def check(x, order=2):
    """Forward, backward and its backward pass against the reference."""
    ref = Attention(x["q"], x["k"], x["v"], x["bias"], x["mask"], x["lengths"], x.get("scale"))
    worst = [close("out", call(x), ref.out())]
    if order == 0:
        return worst
    names = [n for n in ("q", "k", "v", "bias") if x[n] is not None]
    leaves = [x[n].detach().requires_grad_(True) for n in names]
    g = x["g"].detach().requires_grad_(True)
    y = call(x, **dict(zip(names, leaves)))
    close("out (recorded)", y, ref.out())
    first = ref.backward(x["g"])[:len(names)]
    for n, got, want in zip(names, torch.autograd.grad(y, leaves, x["g"], retain_graph=True), first):
        worst.append(close(f"d{n}", got, want))
    if order == 1:
        return worst
    got1 = torch.autograd.grad(y, leaves, g, create_graph=True)
    v = [x[n] for n in ("vq", "vk", "vv", "vb")[:len(names)]]
    got2 = torch.autograd.grad(got1, [g, *leaves], v)
    second = ref.backward2(x["vq"], x["vk"], x["vv"], x["vb"] if x["bias"] is not None else None)[:len(names) + 1]
    for n, got, want in zip(["g", *names], got2, second):
        worst.append(close(f"second d{n}", got, want))
    return worst


# batch, queries, keys, heads, kv_heads, dim, what masks the keys
SHAPES = [
    (1, 1, 1, 1, 1, 1, ""),
    (1, 1, 1, 1, 1, 16, "bias"),
    (2, 3, 5, 2, 1, 7, "bias"),
    (3, 16, 16, 2, 2, 16, "mask"),
    (5, 32, 32, 4, 4, 32, "bias"),
    (4, 33, 31, 2, 2, 32, "bias mask"),
    (2, 17, 48, 4, 2, 24, "lengths"),
    (2, 65, 33, 3, 3, 33, "bias"),
    (1, 130, 257, 4, 1, 64, "bias lengths"),
    (2, 100, 190, 6, 2, 80, "bias"),
    (2, 64, 70, 2, 2, 128, "mask lengths"),
    (1, 20, 300, 1, 1, 128, "bias"),
    (1, 1, 4099, 8, 2, 64, "lengths"),
    (3, 2, 1025, 4, 4, 96, "bias lengths"),
    (1, 700, 24, 2, 1, 48, "bias"),
    (1, 1500, 2, 2, 2, 128, "mask"),
    (1, 513, 515, 1, 1, 20, "bias mask lengths"),
    # at the edges of the one-launch kernels of short sequences (48 rows and keys, 32 of wide heads' second order)
    (3, 16, 16, 2, 2, 64, "bias"),
    (2, 15, 17, 3, 1, 40, "bias lengths"),
    (3, 48, 47, 2, 2, 32, "bias"),
    (2, 12, 48, 8, 2, 16, "bias mask"),
    (2, 32, 32, 2, 2, 64, "bias lengths"),
    (2, 33, 48, 2, 2, 64, "mask"),
    (2, 47, 1, 2, 1, 32, "bias"),
    (2, 1, 48, 4, 4, 50, "lengths"),
    (2, 49, 48, 1, 1, 32, "bias"),
    (2, 48, 49, 1, 1, 32, "bias"),
    (2, 48, 48, 1, 1, 65, "bias"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(t) for t in s).replace(" ", "+"))
def test_against_formulas(shape):
    batch, queries, keys, heads, kv_heads, dim, masks = shape
    lengths = [keys * (i + 1) // (batch + 1) for i in range(batch)] if "lengths" in masks else None
    x = make(batch, queries, keys, heads, kv_heads, dim, "bias" in masks, "mask" in masks, lengths)
    say("attention", shape)
    say([f"{w:.2g}" for w in check(x)])


@pytest.mark.parametrize("dim", [10, 32, 45, 64, 72, 96, 116])
def test_widths(dim):
    """Every width of the kernels, where several teams of waves stream the same side and where one does."""
    check(make(2, 230, 330, 4, 2, dim, bias=True, lengths=[290, 330]))
    check(make(3, 60, 57, 2, 2, dim, bias=True, lengths=[57, 1, 33]))


@pytest.mark.parametrize("batch,queries,keys,heads", [(40, 250, 70, 1), (3, 65, 4200, 2), (9, 30, 2100, 4), (300, 70, 60, 3)])
def test_ranges_and_runs(batch, queries, keys, heads):
    """Few and many pieces of work, one and many ranges, sequences of all lengths."""
    check(make(batch, queries, keys, heads, heads, 32, lengths=[(keys * i) // (batch - 1) for i in range(batch)]), order=2)


@pytest.mark.parametrize("queries,keys,dim", [(5, 7, 16), (32, 32, 32), (40, 300, 64), (1, 3000, 64), (200, 90, 48), (70, 200, 100)])
def test_rows_without_keys(queries, keys, dim):
    """Masked by the bias, the mask or a length of zero: zeros, and no gradients; the other sequences are not touched."""
    x = make(4, queries, keys, 2, 2, dim, bias=True, mask=True, lengths=[keys, keys, 0, keys])
    x["bias"][0] = -math.inf
    x["mask"][1] = False
    x["bias"][3, 0], x["mask"][3, 0] = 0.0, True
    check(x)
    leaves = [x[n].detach().requires_grad_(True) for n in ("q", "k", "v", "bias")]
    y = call(x, **dict(zip(("q", "k", "v", "bias"), leaves)))
    assert not y[:3].any()
    for got in torch.autograd.grad(y, leaves, x["g"]):
        assert not got[:3].any()


@pytest.mark.parametrize("queries,keys,dim", [(5, 9, 16), (32, 30, 32), (40, 300, 64), (1, 3000, 64), (300, 290, 48), (70, 200, 128)])
@pytest.mark.parametrize("trash", [math.nan, math.inf, -math.inf, 3e38])
def test_what_masked_keys_hold_is_not_used(queries, keys, dim, trash):
    x = make(3, queries, keys, 4, 2, dim, bias=True, mask=True, lengths=[keys, keys // 2, max(1, keys // 3)])
    names = ("q", "k", "v", "bias")

    def run(k, v, vk, vv):
        leaves = [x["q"].detach().requires_grad_(True), k.requires_grad_(True), v.requires_grad_(True),
                  x["bias"].detach().requires_grad_(True)]
        g = x["g"].detach().requires_grad_(True)
        y = call(x, **dict(zip(names, leaves)))
        first = torch.autograd.grad(y, leaves, g, create_graph=True)
        return [y, *first, *torch.autograd.grad(first, [g, *leaves], [x["vq"], vk, vv, x["vb"]])]

    from attention_reference import alive_keys

    dead = ~alive_keys(x["k"], x["bias"], x["mask"], x["lengths"])[:, :, None, None]
    assert bool(dead.any())
    clean = run(*(x[n].masked_fill(dead, 0.0) for n in ("k", "v", "vk", "vv")))
    dirty = run(*(x[n].masked_fill(dead, trash) for n in ("k", "v", "vk", "vv")))
    for a, b in zip(clean, dirty):
        assert bool(torch.isfinite(b).all()) and torch.equal(a, b)


@pytest.mark.parametrize("queries,keys,dim", [(5, 7, 16), (32, 32, 32), (40, 300, 64), (1, 3000, 64), (200, 90, 48)])
def test_lowest_values_as_masks(queries, keys, dim):
    """Biases of the type's lowest value: nothing beside other keys; among themselves, all alike."""
    low = torch.finfo(torch.float32).min
    x = make(2, queries, keys, 2, 2, dim, bias=True)
    x["bias"][0] = low
    x["bias"][1] = torch.where(torch.arange(keys, device=DEV) % 3 == 0, low, 0.0)
    y = call(x)
    assert float((y[0].double() - x["v"][0].double().mean(0, keepdim=True)).abs().max()) <= (keys + 8) * 2.0 ** -24 * float(
        x["v"][0].abs().mean(0).max())
    kept = torch.arange(keys, device=DEV) % 3 != 0
    want = call(x, bias=torch.where(kept, 0.0, -math.inf).expand(2, keys))
    assert float((y[1] - want[1]).abs().max()) <= 64 * 2.0 ** -24 * float(x["v"].abs().max())
    check(x)


def test_lengths_beyond_the_keys():
    x = make(4, 6, 40, 2, 2, 32, lengths=[-3, 0, 40, 2 ** 40])
    want = call(x, lengths=torch.tensor([0, 0, 40, 40], device=DEV))
    assert torch.equal(call(x), want)
    assert torch.equal(call(x, lengths=torch.tensor([-3, 0, 40, 2 ** 31 - 1], device=DEV, dtype=torch.int32)), want)


@pytest.mark.parametrize("queries,keys,dim", [(9, 20, 32), (80, 300, 64), (2, 1500, 64), (130, 130, 36), (100, 70, 33)])
def test_strides(queries, keys, dim):
    """Joint projections, head-major arrays, shared and spread-out rows: the same bits as dense arrays."""
    gen = torch.Generator(device=DEV).manual_seed(dim)
    b, h, g = 2, 4, 2
    joint = normal(gen, b, max(queries, keys), 3 * h * dim + 5)
    slices = lambda at, n, heads: joint[:, :n, at:at + heads * dim].unflatten(2, (heads, dim))
    major = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)
    spread = lambda t: torch.stack([t, t], -1)[..., 0]   # no unit stride: copied
    dense = [slices(0, queries, h).contiguous(), slices(h * dim + 1, keys, g).contiguous(), slices(2 * h * dim + 3, keys, g).contiguous()]
    bias = normal(gen, keys)
    grad = normal(gen, b, queries, h, dim)

    def run(q, k, v, bias, grad):
        leaves = [t.detach().requires_grad_(True) for t in (q, k, v, bias)]
        y = attention.cross_attention(*leaves[:3], key_bias=leaves[3])
        go = grad.detach().requires_grad_(True)
        first = torch.autograd.grad(y, leaves, go, create_graph=True)
        return [y, *first, *torch.autograd.grad(first, [go, *leaves], [leaves[0].detach(), leaves[1].detach(), leaves[2].detach(), bias.detach()])]

    want = run(*dense, bias.expand(b, keys).contiguous(), grad)
    for q, k, v, bb, gg in (
            (slices(0, queries, h), slices(h * dim + 1, keys, g), slices(2 * h * dim + 3, keys, g), bias.expand(b, keys), grad),
            (*(major(t) for t in dense), bias.expand(b, keys), major(grad)),
            (*(spread(t) for t in dense), torch.stack([bias, bias], 1)[:, 0].expand(b, keys), spread(grad))):
        for got, ref in zip(run(q, k, v, bb, gg), want):
            assert torch.equal(got, ref)
    shared = [t[:1].expand(b, *t.shape[1:]) for t in dense]
    for got, ref in zip(run(*shared, bias.expand(b, keys), grad), run(*(t.contiguous() for t in shared), bias.expand(b, keys), grad)):
        assert torch.equal(got, ref)
    one_key = dense[1][:, :1].expand(b, keys, g, dim)
    assert torch.equal(attention.cross_attention(dense[0], one_key, dense[2]),
                       attention.cross_attention(dense[0], one_key.contiguous(), dense[2]))


@pytest.mark.parametrize("queries,keys,share", [(1, 300, 4), (40, 90, 2), (200, 100, 1), (150, 100, 3)])
def test_rows_far_apart(queries, keys, share):
    """Offsets past 2^32 elements, and strides past what fast addresses hold."""
    stride = (1 << 24) + 4   # floats between tokens
    far = torch.empty(stride * (max(queries, keys) - 1) + 64 * 4, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    dense = {"q": normal(g, 1, queries, share, 32), "k": normal(g, 1, keys, 1, 32), "v": normal(g, 1, keys, 1, 32)}
    if queries <= 100:
        assert stride * (max(queries, keys) - 1) > 2 ** 30

    def apart(t, at):
        view = far[at:].as_strided(t.shape, (0, stride, 32, 1))
        view.copy_(t)
        return view

    q = dense["q"] if share > 2 else apart(dense["q"], 0)
    k, v = apart(dense["k"], 96), apart(dense["v"], 160)
    grad = normal(g, 1, queries, share, 32)

    def run(*leaves):
        leaves = [t.detach().requires_grad_(True) for t in leaves]
        y = attention.cross_attention(*leaves)
        go = grad.detach().requires_grad_(True)
        first = torch.autograd.grad(y, leaves, go, create_graph=True)
        return [y, *first, *torch.autograd.grad(first, [go, *leaves], [t.detach() for t in leaves])]

    for a, b in zip(run(q, k, v), run(*dense.values())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("batch,queries,keys,heads", [(0, 3, 4, 2), (2, 0, 4, 2), (2, 3, 0, 2), (2, 3, 4, 0), (2, 100, 0, 2), (1, 0, 500, 2)])
def test_empty(batch, queries, keys, heads):
    x = make(batch, queries, keys, heads, heads, 16, bias=True)
    leaves = [x[n].requires_grad_(True) for n in ("q", "k", "v", "bias")]
    y = call(x)
    assert y.shape == (batch, queries, heads, 16) and not y.any()
    g = x["g"].requires_grad_(True)
    first = torch.autograd.grad(y, leaves, g, create_graph=True)
    second = torch.autograd.grad(first, [g, *leaves], [torch.ones_like(t) for t in first])
    for t, like in zip([*first, *second], [*leaves, g, *leaves]):
        assert t.shape == like.shape and not t.any()


@pytest.mark.parametrize("shape", [(2, 20, 20, 4, 2, 32), (1, 3, 2000, 4, 4, 64), (2, 150, 260, 2, 1, 64), (2, 140, 90, 2, 2, 96)])
def test_same_bits_twice_and_for_fewer_wanted(shape):
    x = make(*shape, bias=True)
    names = ("q", "k", "v", "bias")

    def grads(wanted):
        leaves = {n: x[n].detach().requires_grad_(n in wanted) for n in names}
        y = call(x, **leaves)
        g = x["g"].detach().requires_grad_(True)
        first = torch.autograd.grad(y, [leaves[n] for n in wanted], g, create_graph=True)
        cot = dict(zip(names, (x["vq"], x["vk"], x["vv"], x["vb"])))
        return y, first, torch.autograd.grad(first, [g] + [leaves[n] for n in wanted], [cot[n] for n in wanted], allow_unused=True)

    y, first, second = grads(names)
    again = grads(names)
    for a, b in zip([y, *first, *second], [again[0], *again[1], *again[2]]):
        assert torch.equal(a, b)
    with torch.no_grad():
        assert torch.equal(call(x), y)
    for wanted in (("q",), ("k",), ("v",), ("bias",), ("q", "bias"), ("k", "v")):
        got = grads(wanted)
        for n, t in zip(wanted, got[1]):
            assert torch.equal(t, first[names.index(n)])


def test_second_derivatives_with_some_cotangents():
    """Cotangents that are missing count as zeros."""
    x = make(2, 70, 90, 4, 2, 40, bias=True)
    leaves = [x[n].requires_grad_(True) for n in ("q", "k", "v", "bias")]
    g = x["g"].requires_grad_(True)
    cot = [x["vq"], x["vk"], x["vv"], x["vb"]]
    first = torch.autograd.grad(call(x), leaves, g, create_graph=True)
    for keep in (0, 1, 2, 3):
        got = torch.autograd.grad(first[keep], [g, *leaves], cot[keep], retain_graph=True, allow_unused=True)
        full = torch.autograd.grad(first, [g, *leaves], [c if i == keep else torch.zeros_like(c) for i, c in enumerate(cot)],
                                   retain_graph=True)
        for a, b in zip(got, full):
            assert torch.equal(torch.zeros_like(b) if a is None else a, b)


def test_third_derivative_raises():
    x = make(1, 4, 5, 1, 1, 8)
    q = x["q"].requires_grad_(True)
    (a,) = torch.autograd.grad(call(x).square().sum(), q, create_graph=True)
    (b,) = torch.autograd.grad(a.square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="third derivative"):
        torch.autograd.grad(b.sum(), q)


def test_output_changed_in_place_raises():
    x = make(1, 4, 5, 1, 1, 8)
    y = call(x, q=x["q"].requires_grad_(True))
    y.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_refusals():
    x = make(2, 3, 5, 4, 2, 8, bias=True, mask=True, lengths=[5, 4])
    for over in (dict(q=x["q"].double()), dict(k=x["k"].half()), dict(v=x["v"].cpu()), dict(bias=x["bias"].double()),
                 dict(mask=x["mask"].int()), dict(mask=x["mask"].cpu()), dict(lengths=x["lengths"].float()), dict(lengths=x["lengths"].cpu())):
        with pytest.raises((TypeError, ValueError)):
            call(x, **over)
    for over in (dict(q=x["q"][0]), dict(k=x["k"][:, :4]), dict(k=x["k"][:1], v=x["v"][:1]), dict(q=x["q"][:, :, :3]),
                 dict(q=x["q"][..., :4]), dict(bias=x["bias"][:, :4]), dict(bias=x["bias"][0]), dict(mask=x["mask"][:1]),
                 dict(lengths=x["lengths"][:1]), dict(lengths=x["lengths"][:, None]), dict(scale=math.inf), dict(scale=1e300),
                 dict(q=x["q"].repeat(1, 1, 1, 20), k=x["k"].repeat(1, 1, 1, 20), v=x["v"].repeat(1, 1, 1, 20))):
        with pytest.raises(ValueError):
            call(x, **over)


def test_scale_and_infinite_scores():
    x = make(2, 20, 30, 2, 2, 24, bias=True)
    for scale in (0.0, -0.5, 3.0):
        x["scale"] = scale
        check(x)
    x["scale"] = None
    y = call(x, bias=torch.full_like(x["bias"], math.nan))
    assert bool(torch.isnan(y).all())
    for keys, n in ((30, 20), (300, 80)):
        x = make(2, n, keys, 2, 2, 24)
        x["q"][0, 3, 1, 2] = math.nan
        bad = torch.isnan(call(x)).all(-1)
        assert bool(bad[0, 3, 1]) and int(bad.sum()) == 1


@pytest.mark.parametrize("shape", [(3, 30, 30, 2, 2, 32), (1, 2, 700, 4, 2, 64), (2, 100, 260, 2, 2, 64)])
def test_differences(shape):
    """The gradient against differences of the operator itself, within what the outputs' own bounds leave."""
    x = make(*shape, bias=True)
    x["bias"] = x["bias"].clamp(min=-5.0)
    names = ("q", "k", "v", "bias")
    leaves = [x[n].detach().requires_grad_(True) for n in names]
    grads = torch.autograd.grad(call(x, **dict(zip(names, leaves))), leaves, x["g"])
    gen = torch.Generator(device=DEV).manual_seed(9)
    way = [normal(gen, *x[n].shape) for n in names]
    h = 2.0 ** -8
    value, bound, exact = [], 0.0, []
    for s in (1, -1):
        moved = {n: x[n] + s * h * w for n, w in zip(names, way)}
        ref = Attention(moved["q"], moved["k"], moved["v"], moved["bias"]).out()
        value.append(float((call(x, **moved).double() * x["g"].double()).sum()))
        exact.append(float((ref.v * x["g"].double()).sum()))
        bound += float((ref.e * x["g"].double().abs()).sum())
    # differences of the operator and of the formula, from the same points
    assert abs((value[0] - value[1]) - (exact[0] - exact[1])) <= 1.01 * bound
    # and the formula's differences against the gradient: the error falls with h^2
    slope = sum(float((a.double() * w.double()).sum()) for a, w in zip(grads, way))
    size = sum(float((a.double() * w.double()).abs().sum()) for a, w in zip(grads, way))
    rough = abs((exact[0] - exact[1]) / (2 * h) - slope)
    fine = []
    for s in (1, -1):
        moved = [x[n].double() + s * h / 8 * w.double() for n, w in zip(names, way)]
        fine.append(float((Attention(*moved).out().v * x["g"].double()).sum()))
    assert abs((fine[0] - fine[1]) / (h / 4) - slope) <= rough / 32 + 1e-4 * size


def test_streams():
    """Work runs on the current stream, and inputs of another stream are waited for by torch's own rules."""
    x = make(2, 100, 200, 4, 2, 64, bias=True)
    want = call(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q = x["q"] * 1.0
        got = call(x, q=q)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


@pytest.mark.parametrize("shape", [(3, 30, 30, 4, 4, 32), (1, 2, 700, 4, 2, 64), (2, 100, 260, 2, 2, 64)])
def test_captured(shape):
    """A captured force-training step, replayed with new inputs between eager work."""
    x = make(*shape, bias=True)
    names = ("q", "k", "v", "bias")
    leaves = [x[n].detach().clone().requires_grad_(True) for n in names]
    g = x["g"].detach().clone().requires_grad_(True)
    cot = [x["vq"], x["vk"], x["vv"], x["vb"]]

    def step(leaves, g):
        y = call(x, **dict(zip(names, leaves)))
        first = torch.autograd.grad(y, leaves, g, create_graph=True)
        return [y, *first, *torch.autograd.grad(first, [g, *leaves], cot)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(leaves, g)
    gen = torch.Generator(device=DEV).manual_seed(5)
    for _ in range(4):
        with torch.no_grad():
            for t in leaves + [g]:
                t.copy_(normal(gen, *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        fresh = [t.detach().clone().requires_grad_(True) for t in leaves]
        want = step(fresh, g.detach().clone().requires_grad_(True))
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_capture_with_living_results_is_refused():
    x = make(1, 4, 5, 1, 1, 8)
    q = x["q"].requires_grad_(True)
    living = call(x)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="capturing a differentiable call"):
        with torch.cuda.graph(graph):
            call(x)
    assert living.shape == q.shape


def test_outputs_end_where_they_should():
    """Through the C ABI, into arrays with guards around them, four bytes off any wider alignment."""
    import ctypes

    lib = attention._lib
    for batch, queries, keys, h, kv, dim in ((2, 3, 5, 2, 1, 7), (1, 33, 47, 2, 2, 32), (1, 2, 900, 4, 2, 64), (2, 130, 150, 2, 1, 33)):
        g = torch.Generator(device=DEV).manual_seed(queries)
        q, do = normal(g, batch, queries, h, dim), normal(g, batch, queries, h, dim)
        k, v = normal(g, batch, keys, kv, dim), normal(g, batch, keys, kv, dim)
        bias = normal(g, batch, keys)
        a = attention._Attention(batch=batch, queries=queries, keys=keys, heads=h, kv_heads=kv, dim=dim, scale=0.25,
                                 key_bias=bias.data_ptr(), key_bias_batch=keys, key_bias_key=1)
        heads = lambda t: attention._Heads(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))
        guarded = lambda n: torch.full((n + 66,), 777.0, device=DEV)
        inner = lambda t: t[33:-33]
        stream = torch.cuda.current_stream().cuda_stream
        need = ctypes.c_size_t(0)

        def space(name):
            assert getattr(lib, name)(ctypes.byref(a), ctypes.byref(need)) == 0
            t = torch.full((need.value + 512,), 85, dtype=torch.uint8, device=DEV)
            return t, t.data_ptr() + 255 & -256, need.value

        out, stats = guarded(q.numel()), guarded(2 * batch * queries * h)
        ws, at, n = space("emu_cross_attention_workspace")
        assert lib.emu_cross_attention(ctypes.byref(a), heads(q), heads(k), heads(v), inner(out).data_ptr(), inner(stats).data_ptr(),
                                       at, n, stream) == 0
        spaces = [(ws, at, n)]
        dq, dk, dv, db = guarded(q.numel()), guarded(k.numel()), guarded(k.numel()), guarded(bias.numel())
        spaces.append(space("emu_cross_attention_backward_workspace"))
        assert lib.emu_cross_attention_backward(ctypes.byref(a), heads(do), heads(q), heads(k), heads(v), inner(out).data_ptr(),
                                                inner(stats).data_ptr(), *(inner(t).data_ptr() for t in (dq, dk, dv, db)),
                                                spaces[-1][1], spaces[-1][2], stream) == 0
        second = [guarded(t.numel()) for t in (q, q, k, k, bias)]
        spaces.append(space("emu_cross_attention_backward2_workspace"))
        assert lib.emu_cross_attention_backward2(ctypes.byref(a), heads(q), heads(k), heads(v), bias.data_ptr(), keys, 1, heads(do),
                                                 heads(q), heads(k), heads(v), inner(out).data_ptr(), inner(stats).data_ptr(),
                                                 *(inner(t).data_ptr() for t in second), spaces[-1][1], spaces[-1][2], stream) == 0
        torch.cuda.synchronize()
        for t in (out, stats, dq, dk, dv, db, *second):
            assert bool((t[:33] == 777.0).all()) and bool((t[-33:] == 777.0).all())
        for t, start, n in spaces:
            off = start - t.data_ptr()
            assert bool((t[:off] == 85).all()) and bool((t[off + n:] == 85).all())
        ref = Attention(q, k, v, bias, scale=0.25)
        close("out", inner(out).view(q.shape), ref.out())
        for got, want in zip((dq, dk, dv, db), ref.backward(do)):
            close("gradient", inner(got).view(want.v.shape), want)
        for got, want in zip(second, ref.backward2(q, k, v, bias)):
            close("second", inner(got).view(want.v.shape), want)
