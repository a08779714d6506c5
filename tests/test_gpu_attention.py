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
