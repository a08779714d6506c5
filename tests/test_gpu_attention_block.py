"""The attention half of a transformer block as it is used: projections, rotary
positions, attention, dropout and the residual sum together, with their
gradients, against the same in 64 bits; dropout's seeds in modules and captured
graphs."""
import math

import pytest
import torch

from attention_reference import kept
from emulated_fp32_matrix_amd import attention, block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rotated(x, positions, rot):
    f, magnitude = attention.rotary_frequencies(rot.dim, rot.base, rot.scaling, rot.factor)
    n = rot.dim // 2
    angle = positions.double()[..., None, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    c, s = magnitude * torch.cos(angle), magnitude * torch.sin(angle)
    a, b = x[..., :n], x[..., n:2 * n]
    return torch.cat([a * c - b * s, a * s + b * c, x[..., 2 * n:]], -1)


def plain(layer, p, x, context, bias, positions, context_positions, keep=None):
    """The block in 64 bits."""
    n = x
    if layer.norm is not None:
        n = torch.nn.functional.layer_norm(x, (layer.dim,), p["norm.weight"], p.get("norm.bias"), layer.norm.eps)
    source = n if context is None else context
    lin = lambda t, name: t @ p[f"w_{name}"].t() + (p[f"b_{name}"] if f"b_{name}" in p else 0.0)
    q = lin(n, "q").unflatten(2, (layer.heads, layer.head_dim))
    k, v = lin(source, "kv").unflatten(2, (2, layer.kv_heads, layer.head_dim)).unbind(2)
    if layer.rotary is not None:
        q, k = rotated(q, positions, layer.rotary), rotated(k, context_positions, layer.rotary)
    share = layer.heads // layer.kv_heads
    q, k, v = q.transpose(1, 2), *(t.transpose(1, 2).repeat_interleave(share, 1) for t in (k, v))
    z = q @ k.transpose(2, 3).contiguous() / math.sqrt(layer.head_dim)
    if bias is not None:
        z = z + bias[:, None, None, :]
    o = lin((torch.softmax(z, -1) @ v).transpose(1, 2).flatten(2), "o")
    return x + (o if keep is None else o * keep)


@pytest.mark.parametrize("case", ["self", "context", "rotary", "shared heads, no norm"])
@pytest.mark.parametrize("tokens,keys", [(32, 32), (70, 140)])
def test_block_against_64_bits(case, tokens, keys):
    gen = torch.Generator(device=DEV).manual_seed(tokens)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    torch.manual_seed(1)
    kw = {"self": {}, "context": dict(context_dim=48), "rotary": dict(rotary=attention.Rotary(12, device=DEV)),
          "shared heads, no norm": dict(kv_heads=2, norm=False, bias=False)}[case]
    layer = attention.EmuCrossAttention(64, 4, device=DEV, mode="BF16X9", **kw)
    with torch.no_grad():
        for p in layer.parameters():
            p.add_(0.1 * rnd(*p.shape))
    x = rnd(3, tokens, 64).requires_grad_(True)
    context = None if case in ("self", "rotary") else rnd(3, keys, layer.context_dim).requires_grad_(True)
    n = tokens if context is None else keys
    bias = rnd(3, n).requires_grad_(True)
    positions = torch.arange(tokens, device=DEV) + 5000
    y = layer(x, context, key_bias=bias, positions=positions)
    leaves = [x, bias] + ([context] if context is not None else []) + list(layer.parameters())
    g = rnd(*y.shape).requires_grad_(True)
    first = torch.autograd.grad(y, leaves, g, create_graph=True)
    v = rnd(*x.shape)
    second = torch.autograd.grad(first[0], [g, x, *layer.parameters()], v, allow_unused=True)

    wide = {name: p.detach().double().requires_grad_(True) for name, p in layer.named_parameters()}
    x64, b64 = x.detach().double().requires_grad_(True), bias.detach().double().requires_grad_(True)
    c64 = None if context is None else context.detach().double().requires_grad_(True)
    y64 = plain(layer, wide, x64, c64, b64, positions, positions)
    leaves64 = [x64, b64] + ([c64] if c64 is not None else []) + list(wide.values())
    g64 = g.detach().double().requires_grad_(True)
    first64 = torch.autograd.grad(y64, leaves64, g64, create_graph=True)
    second64 = torch.autograd.grad(first64[0], [g64, x64, *wide.values()], v.double(), allow_unused=True)
    # a chain of about ten FP32 operators, each within 8 units of the largest
    # value of its results for sums of up to a few hundred terms of this size;
    # the sums over tokens of the weight gradients take their own length
    for got, want in zip([y, *first, *second], [y64, *first64, *second64]):
        if want is None:
            assert got is None or not got.any()
            continue
        size = float(want.abs().max())
        if size < 1e-12:   # (a bias that the softmax does not see)
            assert float(got.abs().max()) < 1e-3
            continue
        assert float((got.double() - want).abs().max()) <= 80 * 3 * tokens ** 0.5 * 2.0 ** -24 * size


def test_gradients_accumulate_and_training_step_runs():
    torch.manual_seed(0)
    layer = attention.EmuCrossAttention(64, 4, dropout=0.2, device=DEV)
    ffn = block.EmuGatedFFN(64, 128, device=DEV)
    x = torch.randn(4, 20, 64, device=DEV)
    for _ in range(2):
        (ffn(layer(x)) ** 2).sum().backward()
    for p in [*layer.parameters(), *ffn.parameters()]:
        assert p.grad is not None and bool(torch.isfinite(p.grad).all())


def test_dropout_in_the_block():
    torch.manual_seed(3)
    layer = attention.EmuCrossAttention(32, 2, dropout=0.25, device=DEV)
    x = torch.randn(2, 10, 32, device=DEV)
    torch.cuda.manual_seed(11)
    a = layer(x)
    torch.cuda.manual_seed(11)
    b = layer(x)
    c = layer(x)
    assert torch.equal(a, b) and not torch.equal(a, c)
    layer.eval()
    whole = layer(x)
    moved = (a - x) != 0
    assert torch.equal((a - x)[~moved], torch.zeros_like(a)[~moved]) and 0.6 < float(moved.float().mean()) < 0.9
    # kept elements are the block's own, divided by the kept share: a rounding for each of the two sums and the scale
    ratio = 4 / 3
    assert float(((a - x) - (whole - x) * ratio)[moved].abs().max()) <= 8 * 2.0 ** -24 * float(x.abs().max() + (whole - x).abs().max())


def test_dropout_captured():
    """A captured call reads its seed when it is replayed; a module's seeds come from torch's generator, which moves on."""
    seed = torch.tensor([5, 6], device=DEV)
    x = torch.randn(1000, device=DEV)
    drop = attention.EmuDropout(0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        drop(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fixed = attention.dropout(x, 0.5, seed)
        free = drop(x)
    masks = []
    for i in range(4):
        seed.copy_(torch.tensor([100 + i, i]))
        graph.replay()
        torch.cuda.synchronize()
        assert (fixed != 0).tolist() == kept(100 + i, i, range(1000), 0.5)
        assert torch.equal(fixed, attention.dropout(x, 0.5, seed))
        masks.append((free != 0).clone())
    assert all(not torch.equal(masks[0], m) for m in masks[1:])


def test_seed_changed_before_the_backward_pass_raises():
    x = torch.randn(100, device=DEV, requires_grad=True)
    seed = attention.dropout_seed(DEV)
    y = attention.dropout(x, 0.5, seed)
    seed.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_refusals():
    x = torch.randn(2, 5, 4, 16, device=DEV)
    positions, turns = torch.arange(5, device=DEV), attention.rotary_turns([1.0, 0.5], DEV)
    for args in ((x.double(), positions, turns), (x, positions.float(), turns), (x, positions, turns.int()), (x, positions.cpu(), turns),
                 (x, positions, turns.cpu())):
        with pytest.raises((TypeError, ValueError)):
            attention.rotary(*args)
    for args in ((x[0, 0], positions, turns), (x, positions[:4], turns), (x, positions.expand(3, 5), turns),
                 (x, positions, attention.rotary_turns([0.1] * 9, DEV)), (x, positions, turns[None])):
        with pytest.raises(ValueError):
            attention.rotary(*args)
    with pytest.raises(ValueError):
        attention.rotary(x, positions, turns, magnitude=math.inf)
    seed = attention.dropout_seed(DEV)
    for args, kw in (((x.half(), 0.5, seed), {}), ((x, 0.5, seed.int()), {}), ((x, 0.5, seed.cpu()), {}),
                     ((x, 0.5, seed), dict(residual=x.double()))):
        with pytest.raises((TypeError, ValueError)):
            attention.dropout(*args, **kw)
    for args, kw in (((x, 1.5, seed), {}), ((x, -0.1, seed), {}), ((x, math.nan, seed), {}), ((x, 0.5, seed[:1]), {}),
                     ((x, 0.5, seed), dict(residual=x[0]))):
        with pytest.raises(ValueError):
            attention.dropout(*args, **kw)
    layer = attention.EmuCrossAttention(64, 4, rotary=attention.Rotary(8, device=DEV), device=DEV)
    with pytest.raises(ValueError, match="positions"):
        layer(torch.zeros(1, 3, 64, device=DEV))
    with pytest.raises(NotImplementedError):
        torch.func.vmap(lambda t: attention.cross_attention(t, t, t))(torch.zeros(2, 1, 3, 2, 8, device=DEV))
