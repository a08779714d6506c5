"""Calls of the attention operators that their documentation allows beside the
usual ones: strides that run backwards and heads that lie on each other, many
heads on one key head, a captured serving step whose lengths move on, calls on
two streams at once, gradients that are one number spread out."""
import ctypes

import pytest
import torch

from attention_reference import Attention, close
from emulated_fp32_matrix_amd import attention
from test_gpu_attention import call, check, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
lib = attention._lib


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _space(name, a):
    need = ctypes.c_size_t(0)
    assert getattr(lib, name + "_workspace")(ctypes.byref(a), ctypes.byref(need)) == 0
    t = torch.empty(need.value + 256, dtype=torch.uint8, device=DEV)
    return t, t.data_ptr() + 255 & -256, need.value


def _backwards(t):
    """A view for the C ABI of t with its sequences, tokens and heads in reverse order in memory."""
    r = t.flip(0, 1, 2).contiguous()
    last = sum((n - 1) * s for n, s in zip(r.shape[:3], r.stride()[:3]))
    return r, attention._Heads(r.data_ptr() + 4 * last, -r.stride(0), -r.stride(1), -r.stride(2))


@pytest.mark.parametrize("shape", [(2, 20, 30, 4, 2, 32), (2, 2, 300, 4, 2, 64), (2, 60, 50, 2, 2, 40), (2, 150, 200, 4, 2, 64)])
def test_strides_that_run_backwards(shape):
    batch, queries, keys, h, g, dim = shape
    x = make(*shape, bias=True)
    names = ("q", "k", "v", "g", "vq", "vk", "vv")
    kept, view = zip(*(_backwards(x[n]) for n in names))
    q, k, v, do, vq, vk, vv = view
    bias, vbias = x["bias"].flip(0, 1).contiguous(), x["vb"].flip(0, 1).contiguous()
    end = 4 * (batch * keys - 1)
    a = attention._Attention(batch=batch, queries=queries, keys=keys, heads=h, kv_heads=g, dim=dim, scale=dim ** -0.5,
                             key_bias=bias.data_ptr() + end, key_bias_batch=-keys, key_bias_key=-1)
    new = lambda t: torch.empty(t.shape, device=DEV)
    out, stats = new(x["q"]), torch.empty(batch, queries, h, 2, device=DEV)
    first, second = [new(x[n]) for n in ("q", "k", "v", "bias")], [new(x[n]) for n in ("g", "q", "k", "v", "bias")]
    w0, w1, w2 = (_space(f"emu_cross_attention{n}", a) for n in ("", "_backward", "_backward2"))
    assert lib.emu_cross_attention(ctypes.byref(a), q, k, v, out.data_ptr(), stats.data_ptr(), w0[1], w0[2], _stream()) == 0
    assert lib.emu_cross_attention_backward(ctypes.byref(a), do, q, k, v, out.data_ptr(), stats.data_ptr(),
                                            *(t.data_ptr() for t in first), w1[1], w1[2], _stream()) == 0
    assert lib.emu_cross_attention_backward2(ctypes.byref(a), vq, vk, vv, vbias.data_ptr() + end, -keys, -1, do, q, k, v,
                                             out.data_ptr(), stats.data_ptr(), *(t.data_ptr() for t in second), w2[1], w2[2],
                                             _stream()) == 0
    ref = Attention(x["q"], x["k"], x["v"], x["bias"])
    close("out", out, ref.out())
    for t, want in zip(first, ref.backward(x["g"])):
        close("gradient", t, want)
    for t, want in zip(second, ref.backward2(x["vq"], x["vk"], x["vv"], x["vb"])):
        close("second", t, want)


def test_rotary_strides_that_run_backwards():
    x = torch.randn(2, 40, 3, 32, device=DEV)
    positions = torch.randint(-99, 99, (2, 40), device=DEV)
    turns = attention.rotary_turns([0.7 ** i for i in range(12)], DEV)
    kept, view = _backwards(x)
    back = positions.flip(0, 1).contiguous()
    y = torch.empty_like(x)
    assert lib.emu_rotary(2, 40, 3, 32, view, back.data_ptr() + 8 * 79, -40, -1, turns.data_ptr(), 12, 0, 1.0, 0, y.data_ptr(),
                          _stream()) == 0
    assert torch.equal(y, attention.rotary(x, positions, turns))


@pytest.mark.parametrize("queries,keys", [(20, 30), (2, 500), (90, 200)])
def test_heads_that_lie_on_each_other(queries, keys):
    x = make(2, queries, keys, 4, 2, 32, bias=True)
    over = {n: x[n][:, :, :1].expand(x[n].shape) for n in ("q", "k", "v")}
    assert torch.equal(call(x, **over), call(x, **{n: t.contiguous() for n, t in over.items()}))


@pytest.mark.parametrize("queries,keys,heads,kv_heads", [(1, 700, 64, 1), (1, 300, 96, 2), (3, 40, 48, 1), (5, 90, 33, 1), (2, 60, 40, 2)])
def test_many_heads_on_one_key_head(queries, keys, heads, kv_heads):
    check(make(2, queries, keys, heads, kv_heads, 32, bias=True, lengths=[keys, keys // 3]))


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 64), (8, 8, 40), (40, 2, 128)])
def test_captured_serving_step_whose_lengths_move_on(heads, kv_heads, dim):
    """One new token a step against a cache of fixed size: the captured call reads the lengths of each replay."""
    x = make(3, 1, 900, heads, kv_heads, dim, lengths=[1, 1, 1])
    call(x)
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        out = call(x)
    for lengths in ([1, 500, 900], [2, 501, 0], [31, 32, 33], [900, 900, 900], [0, 0, 0]):
        x["lengths"].copy_(torch.tensor(lengths))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call(x))


def test_two_streams_at_once():
    xs = [make(2, 300, 700, 4, 2, 64, bias=True, seed=s) for s in (1, 2)]
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(8):
        for s, x, to in zip(streams, xs, got):
            with torch.cuda.stream(s):
                to.append(call(x))
    torch.cuda.synchronize()
    for to, w in zip(got, want):
        assert all(torch.equal(t, w) for t in to)


@pytest.mark.parametrize("queries,keys", [(20, 30), (2, 500), (90, 200)])
def test_gradient_that_is_one_number(queries, keys):
    x = make(2, queries, keys, 2, 2, 32, bias=True)
    names = ("q", "k", "v", "bias")

    def grads(loss):
        leaves = [x[n].detach().requires_grad_(True) for n in names]
        return torch.autograd.grad(loss(call(x, **dict(zip(names, leaves)))), leaves)

    for a, b in zip(grads(lambda y: y.sum()), grads(lambda y: (y * torch.ones_like(y)).sum())):
        assert torch.equal(a, b)
    u = torch.randn(2, 6, 2, 32, device=DEV, requires_grad=True)
    rot = attention.Rotary(32, device=DEV)
    y = attention.dropout(rot(u, torch.arange(6, device=DEV)), 0.5, torch.tensor([1, 2], device=DEV), residual=u)
    z = attention.dropout(rot(u, torch.arange(6, device=DEV)), 0.5, torch.tensor([1, 2], device=DEV), residual=u)
    (a,), (b,) = torch.autograd.grad(y.sum(), u), torch.autograd.grad((z * torch.ones_like(z)).sum(), u)
    assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(2, 20, 30, 2, 2, 32), (2, 3, 700, 4, 2, 64), (2, 90, 500, 2, 2, 64), (1, 600, 900, 1, 1, 96)])
def test_values_of_other_sizes(shape):
    """Values up to near 2^126 / keys, and small ones: powers of two in the values
    are powers of two in the results, bit for bit."""
    x = make(*shape, bias=True)
    want = call(x)
    for power in (2.0 ** -60, 2.0 ** 20, 2.0 ** 112):   # (normal numbers stay below 2^3, keys below 2^10)
        assert torch.equal(call(x, v=x["v"] * power), want * power)
