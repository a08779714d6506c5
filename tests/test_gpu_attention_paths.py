"""GPU parity of cross attention on each of its kernels' paths: every width and
number of tiles of the one-launch kernels of short sequences, of the forward
pass of few rows and of the streamed passes with and without images; maxima that
climb and fall from tile to tile and from range to range; the results of calls
that want some of the gradients; masks and lengths of other strides and types.
Outputs, gradients and the gradients' gradients against the formulas in 64 bits
(tests/attention_reference.py)."""
import ctypes
import math

import pytest
import torch

from attention_reference import alive_keys
from emulated_fp32_matrix_amd import attention
from test_gpu_attention import call, check, make, normal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("tokens", [11, 16, 27, 32, 43, 48])
@pytest.mark.parametrize("dim", [9, 16, 25, 32, 39, 48, 57, 64])
def test_short_sequences(dim, tokens):
    """One to three tiles of 16 tokens, one to four of a head, whole and cut, in every order."""
    check(make(3, tokens, tokens, 2, 2, dim, bias=True, lengths=[tokens, 1, tokens - 2]))
    check(make(2, tokens // 2, tokens, 4, 2, dim, mask=True))


@pytest.mark.parametrize("dim", [5, 16, 17, 20, 32, 35, 40, 48, 49, 50, 64, 66, 70, 80, 81, 90, 96, 97, 100, 112, 127, 128])
def test_few_rows(dim):
    """Up to 16 rows over many keys: widths that four and sixteen divide and
    that they do not, in one range and in several, keys that end inside a tile."""
    check(make(3, 3, 333, 4, 2, dim, bias=True, lengths=[333, 0, 201]))
    check(make(2, 16, 100, 2, 2, dim, mask=True, lengths=[100, 33]))
    check(make(1, 1, 1300, 8, 1, dim))


@pytest.mark.parametrize("dim", [16, 30, 32, 48, 61, 64, 80, 90, 96, 112, 127, 128])
def test_streamed(dim):
    """Teams of one and of two tiles that read the other side themselves or from
    images: 65 to 128 rows of one team, two and three teams, and four."""
    check(make(2, 100, 60, 2, 2, dim, bias=True, lengths=[60, 37]))
    check(make(1, 120, 190, 2, 2, dim, mask=True))
    check(make(2, 100, 90, 4, 2, dim, bias=True))
    check(make(1, 190, 50, 1, 1, dim, bias=True))
    check(make(1, 300, 130, 1, 1, dim, bias=True))
    check(make(1, 520, 70, 1, 1, dim, lengths=[65]))


def _slopes(keys, kind, step):
    """Biases that climb by up to 60 in all, evenly or in steps every 32 or 192 keys."""
    j = torch.arange(keys, device=DEV, dtype=torch.float32)
    if kind == "even":
        return j * (57.0 / keys)
    return step * torch.floor(j / (32 if keys <= 320 else 192 * keys / 3000))


# (Weights stay above e^-70, so that none of them is below what FP32 holds and the
# reference's bound, which is relative, applies.)
@pytest.mark.parametrize("queries,keys,dim", [(3, 300, 32), (3, 3000, 64), (70, 300, 64), (130, 300, 80), (300, 3000, 32), (20, 40, 32)])
@pytest.mark.parametrize("kind,step", [("even", 0.0), ("steps", 0.99), ("steps", 1.01), ("steps", 3.99), ("steps", 4.01)])
@pytest.mark.parametrize("falls", [False, True])
def test_maxima_that_move(queries, keys, dim, kind, step, falls):
    """Running maxima that grow by a little less and a little more than what the
    forward pass lets pass before it rescales, in every tile or range; and
    maxima that fall, whose later tiles and ranges count for almost nothing."""
    x = make(1, queries, keys, 2, 1, dim)
    x["scale"] = 0.25 / math.sqrt(dim)   # (the scores stay within about 1)
    bias = _slopes(keys, kind, step)
    x["bias"] = (bias.flip(0) if falls else bias)[None].contiguous()
    check(x)


STEPS = [0.9, 0.999, 1.0, 1.001, 1.1, 3.9, 3.999, 4.0, 4.001, 4.1]


@pytest.mark.parametrize("step", STEPS)
@pytest.mark.parametrize("queries", [70, 300])
def test_maximum_that_lags(queries, step):
    """One step after the first tile, of about what passes without a rescale: all
    of the weight lies on keys whose exponents are taken from the earlier maximum."""
    x = make(2, queries, 320, 2, 2, 64, bias=True)
    x["scale"] = 0.01
    j = torch.arange(320, device=DEV)
    x["bias"] = torch.where(j < 32, 0.0, step).expand(2, 320).contiguous()
    check(x)


@pytest.mark.parametrize("step", STEPS)
@pytest.mark.parametrize("batch,queries,dim", [(1, 3, 64), (2048, 3, 32), (1, 300, 64), (1024, 70, 64), (512, 300, 80), (128, 1000, 32)])
def test_kept_maximum_lags_by_one_at_most(batch, queries, dim, step):
    """An exponent's rounding grows with its size, so the weights' exponents are
    taken from a maximum that is at most 1 behind: scores of zero, and biases
    that are the scores then, exactly.  (Many sequences: one range of keys each.)"""
    keys = 320
    q, k = torch.zeros(1, 1, 1, dim, device=DEV).expand(batch, queries, 1, dim), torch.ones(1, 1, 1, dim, device=DEV).expand(batch, keys, 1, dim)
    bias = torch.where(torch.arange(keys, device=DEV) < 32, 0.0, step)
    a = attention._Attention(batch=batch, queries=queries, keys=keys, heads=1, kv_heads=1, dim=dim, scale=1.0,
                             key_bias=bias.data_ptr(), key_bias_batch=0, key_bias_key=1)
    heads = lambda t: attention._Heads(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))
    need = ctypes.c_size_t(0)
    assert attention._lib.emu_cross_attention_workspace(ctypes.byref(a), ctypes.byref(need)) == 0
    space = torch.empty(need.value + 256, dtype=torch.uint8, device=DEV)
    out, stats = torch.empty(batch, queries, 1, dim, device=DEV), torch.empty(batch * queries, 2, device=DEV)
    assert attention._lib.emu_cross_attention(ctypes.byref(a), heads(q), heads(k), heads(k), out.data_ptr(), stats.data_ptr(),
                                              space.data_ptr() + 255 & -256, need.value, torch.cuda.current_stream().cuda_stream) == 0
    lag = bias.max() - stats[:, 0]
    assert float(lag.min()) >= 0.0 and float(lag.max()) <= 1.0


NAMES = ("q", "k", "v", "bias")


@pytest.mark.parametrize("shape", [(2, 20, 20, 4, 2, 32), (1, 3, 2000, 4, 4, 64), (2, 150, 260, 2, 1, 64), (2, 140, 90, 2, 2, 96),
                                   (1, 60, 40, 1, 1, 64), (3, 200, 1500, 1, 1, 48)])
@pytest.mark.parametrize("wanted", [("q",), ("k",), ("v",), ("bias",), ("q", "bias"), ("k", "v"), ("q", "k"), ("v", "bias")])
def test_second_order_of_some_inputs(shape, wanted):
    """Where some inputs alone have gradients, theirs of the second order are
    those of the whole call whose other cotangents are zeros, bit for bit."""
    x = make(*shape, bias=True)
    cot = dict(zip(NAMES, (x["vq"], x["vk"], x["vv"], x["vb"])))

    def second(names, cotangents):
        leaves = {n: x[n].detach().requires_grad_(n in names) for n in NAMES}
        g = x["g"].detach().requires_grad_(True)
        first = torch.autograd.grad(call(x, **leaves), [leaves[n] for n in names], g, create_graph=True)
        got = torch.autograd.grad(first, [g] + [leaves[n] for n in names], cotangents, allow_unused=True)
        return dict(zip(("g", *names), got))

    got = second(wanted, [cot[n] for n in wanted])
    full = second(NAMES, [cot[n] if n in wanted else torch.zeros_like(cot[n]) for n in NAMES])
    for n, t in got.items():
        assert torch.equal(torch.zeros_like(full[n]) if t is None else t, full[n]), n
    assert any(bool(full[n].any()) for n in got)


@pytest.mark.parametrize("queries,keys", [(9, 20), (2, 700), (100, 300)])
def test_masks_and_lengths_as_they_come(queries, keys):
    """Masks shared by the sequences or with strides, lengths of either type with a stride."""
    x = make(3, queries, keys, 2, 2, 32, bias=True)
    gen = torch.Generator(device=DEV).manual_seed(keys)
    mask = torch.rand(keys, generator=gen, device=DEV) < 0.7
    lengths = torch.tensor([keys, keys // 2, 3], device=DEV)
    want = call(x, mask=mask.expand(3, keys).contiguous(), lengths=lengths)
    wide = torch.stack([mask, ~mask], 1).expand(3, keys, 2)[..., 0]
    for m in (mask.expand(3, keys), wide, mask[:, None].expand(keys, 3).t()):
        for n in (lengths, lengths.int(), torch.stack([lengths, -lengths], 1)[:, 0], torch.stack([lengths.int()] * 2, 1)[:, 1]):
            assert torch.equal(call(x, mask=m, lengths=n), want)


@pytest.mark.parametrize("tokens,dim", [(30, 32), (150, 64)])
def test_one_tensor_as_queries_keys_and_values(tokens, dim):
    """Its gradients are the three's sums."""
    x = make(2, tokens, tokens, 2, 2, dim, bias=True)
    one = x["q"].detach().requires_grad_(True)
    three = [x["q"].detach().clone().requires_grad_(True) for _ in range(3)]
    y = call(x, q=one, k=one, v=one)
    z = call(x, q=three[0], k=three[1], v=three[2])
    assert torch.equal(y, z)
    (got,) = torch.autograd.grad(y, one, x["g"])
    parts = torch.autograd.grad(z, three, x["g"])
    want = sum(p.double() for p in parts)
    # (two sums in FP32, in an order of autograd's own)
    assert bool(((got.double() - want).abs() <= 2.0 ** -23 * sum(p.double().abs() for p in parts)).all())


def test_alive_keys_of_the_cases_above():
    """What the cases here mean to mask is masked, and something is left."""
    x = make(3, 3, 333, 4, 2, 20, bias=True, lengths=[333, 0, 201])
    alive = alive_keys(x["k"], x["bias"], x["mask"], x["lengths"]).sum(1).tolist()
    assert alive[1] == 0 and 0 < alive[2] < alive[0] < 333
