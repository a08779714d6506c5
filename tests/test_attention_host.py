"""Host-side checks of the attention operators (no GPU needed): the header
matches the binding, invalid arguments are refused before any HIP call,
workspaces are reported, the Python functions refuse what they cannot run, and
the tests' own 64-bit reference agrees with automatic differentiation and
with differences."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import emulated_fp32_matrix_amd as emu
from attention_reference import Attention, kept, philox_words
from emulated_fp32_matrix_amd import attention

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "emu_attention.h")
FAKE = 0x1000   # never dereferenced: the calls below end before any HIP call
INVALID, UNSUPPORTED = emu.STATUS_INVALID_VALUE, emu.STATUS_NOT_SUPPORTED
lib = attention._lib


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(emu_[a-z0-9_]+)\s*\(", text)))


def test_header_matches_binding_and_library():
    assert _declared() == sorted(attention.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", emu.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert not set(_declared()) - set(re.findall(r"\bT (emu_[a-z0-9_]+)$", out, flags=re.M))
    assert attention.emu_attention_version() == 100


def test_structs_match_the_header(tmp_path):
    src, exe = tmp_path / "s.c", tmp_path / "s"
    lines = []
    for name, cls in (("emu_heads_t", attention._Heads), ("emu_attention_t", attention._Attention)):
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "{HEADER}"\nint main(void) {{ {"".join(lines)} return 0; }}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in (attention._Heads, attention._Attention):
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_constants_match_header():
    text = open(HEADER).read()
    assert f"#define EMU_ATTENTION_MAX_DIM {attention.MAX_DIM}" in text
    for name, value in attention.LAYOUTS.items():
        assert re.search(rf"EMU_ROTARY_{name.upper()} = {value}\b", text)


def sizes(**over):
    a = dict(batch=2, queries=3, keys=5, heads=4, kv_heads=2, dim=8, scale=0.5)
    return attention._Attention(**{**a, **over})


def heads(data=FAKE):
    return attention._Heads(data, 1, 1, 1)


def forward(a, q=FAKE, k=FAKE, v=FAKE, out=FAKE, ws=None, bytes_=0):
    return lib.emu_cross_attention(ctypes.byref(a) if a is not None else None, heads(q), heads(k), heads(v), out, None, ws,
                                   bytes_, None)


BAD = [(dict(batch=-1), INVALID), (dict(queries=-1), INVALID), (dict(keys=-1), INVALID), (dict(heads=-4), INVALID),
       (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(dim=0), INVALID), (dict(scale=math.inf), INVALID),
       (dict(scale=math.nan), INVALID), (dict(dim=129), UNSUPPORTED), (dict(batch=2 ** 30 + 1), UNSUPPORTED),
       (dict(keys=2 ** 30 + 1), UNSUPPORTED), (dict(queries=2 ** 29), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", BAD, ids=str)
def test_bad_sizes(over, status):
    a = sizes(**over)
    n = ctypes.c_size_t(7)
    assert forward(a) == status
    for f in ("", "_backward", "_backward2"):
        assert getattr(lib, f"emu_cross_attention{f}_workspace")(ctypes.byref(a), ctypes.byref(n)) == status and n.value == 7
    z = heads()
    assert lib.emu_cross_attention_backward(ctypes.byref(a), z, z, z, z, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None) == status
    assert lib.emu_cross_attention_backward2(ctypes.byref(a), z, z, z, None, 0, 0, z, z, z, z, FAKE, FAKE, FAKE, FAKE, FAKE,
                                             FAKE, FAKE, None, 0, None) == status


def test_bad_pointers_and_workspaces():
    assert forward(None) == INVALID
    for name in ("q", "k", "v", "out"):
        assert forward(sizes(), **{name: None}) == INVALID
    a, z, none = sizes(), heads(), heads(None)
    ok = [z, z, z, z, FAKE, FAKE]
    for i in range(6):
        args = list(ok)
        args[i] = none if i < 4 else None
        assert lib.emu_cross_attention_backward(ctypes.byref(a), *args, FAKE, FAKE, FAKE, FAKE, None, 0, None) == INVALID
        assert lib.emu_cross_attention_backward2(ctypes.byref(a), z, z, z, None, 0, 0, *args, FAKE, FAKE, FAKE, FAKE, FAKE, None,
                                                 0, None) == INVALID
    # sizes that need a workspace: none, a short one, a misaligned one
    for dims in (dict(batch=1, queries=1, keys=100000, dim=64), dict(queries=300, keys=500)):
        a, n = sizes(**dims), ctypes.c_size_t(0)
        assert lib.emu_cross_attention_workspace(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value > 0
        assert forward(a) == INVALID
        assert forward(a, ws=FAKE, bytes_=n.value - 1) == INVALID
        assert forward(a, ws=FAKE + 8, bytes_=n.value) == INVALID
        for f, call in (("_backward", lambda *w: lib.emu_cross_attention_backward(
                ctypes.byref(a), *ok, FAKE, FAKE, FAKE, FAKE, *w, None)),
                        ("_backward2", lambda *w: lib.emu_cross_attention_backward2(
                            ctypes.byref(a), z, z, z, None, 0, 0, *ok, FAKE, FAKE, FAKE, FAKE, FAKE, *w, None))):
            assert getattr(lib, f"emu_cross_attention{f}_workspace")(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value > 0
            assert call(None, 0) == INVALID and call(FAKE, n.value - 1) == INVALID and call(FAKE + 4, n.value) == INVALID
    assert lib.emu_cross_attention_workspace(ctypes.byref(a), None) == INVALID


def test_nothing_to_do():
    for over in (dict(batch=0), dict(queries=0), dict(heads=0, kv_heads=0)):
        a, n = sizes(**over), ctypes.c_size_t(7)
        assert forward(a, q=None, out=None) == 0
        assert lib.emu_cross_attention_workspace(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0
    a, z, none = sizes(), heads(), heads(None)
    assert lib.emu_cross_attention_backward(ctypes.byref(a), z, z, z, z, FAKE, FAKE, None, None, None, None, None, 0, None) == 0
    assert lib.emu_cross_attention_backward2(ctypes.byref(a), none, none, none, None, 0, 0, z, z, z, z, FAKE, FAKE, None, None,
                                             None, None, None, None, 0, None) == 0


def rotary(batch=1, tokens=2, h=3, dim=8, x=FAKE, positions=FAKE, turns=FAKE, pairs=4, layout=0, magnitude=1.0, y=FAKE):
    return lib.emu_rotary(batch, tokens, h, dim, heads(x), positions, 0, 1, turns, pairs, layout, magnitude, 0, y, None)


def test_rotary_arguments():
    for over in (dict(batch=-1), dict(tokens=-1), dict(h=-1), dict(dim=-1), dict(pairs=-1), dict(pairs=5), dict(layout=2),
                 dict(layout=-1), dict(magnitude=math.nan), dict(magnitude=math.inf), dict(x=None), dict(y=None),
                 dict(positions=None), dict(turns=None)):
        assert rotary(**over) == INVALID, over
    for over in (dict(batch=2 ** 30 + 1), dict(tokens=2 ** 30 + 1), dict(dim=65537), dict(h=2 ** 28)):
        assert rotary(**over) == UNSUPPORTED, over
    for over in (dict(batch=0), dict(tokens=0), dict(h=0), dict(dim=0, pairs=0)):
        assert rotary(x=None, y=None, **over) == 0


def drop(rows=2, cols=3, x=FAKE, ldx=3, p=0.5, seed=FAKE, r=None, ldr=0, y=FAKE, ldy=3):
    return lib.emu_dropout(rows, cols, x, ldx, p, seed, r, ldr, y, ldy, None)


def test_dropout_arguments():
    for over in (dict(rows=-1), dict(cols=-1), dict(ldx=2), dict(ldy=2), dict(p=-0.1), dict(p=1.1), dict(p=math.nan), dict(x=None),
                 dict(y=None), dict(seed=None), dict(r=FAKE, ldr=2)):
        assert drop(**over) == INVALID, over
    assert drop(rows=2 ** 40, cols=2 ** 21, ldx=2 ** 21, ldy=2 ** 21) == UNSUPPORTED
    assert drop(rows=0, x=None, y=None, seed=None) == 0 and drop(cols=0, x=None, y=None, seed=None) == 0


def test_functions_refuse_host_tensors():
    x = torch.zeros(1, 2, 3, 4)
    with pytest.raises(TypeError):
        attention.cross_attention(x, x, x)
    with pytest.raises(TypeError):
        attention.rotary(x, torch.arange(2), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        attention.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="layout"):
        attention.rotary(x, torch.arange(2), torch.zeros(2, dtype=torch.int64), layout="thirds")


def test_frequencies():
    f, magnitude = attention.rotary_frequencies(8)
    assert f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15) and magnitude == 1.0
    assert attention.rotary_frequencies(8, scaling="linear", factor=4.0)[0] == pytest.approx([0.25, 0.025, 0.0025, 0.00025])
    f = attention.rotary_frequencies(8, scaling="base", factor=4.0)[0]
    assert f[0] == 1.0 and f[-1] == pytest.approx(0.001 / 4.0, rel=1e-12)   # the slowest divided by the factor
    f, magnitude = attention.rotary_frequencies(64, scaling="parts", factor=4.0, original_length=4096)
    plain = attention.rotary_frequencies(64)[0]
    turns = [4096 * x / (2 * math.pi) for x in plain]
    for x, y, t in zip(f, plain, turns):
        if t >= 32:
            assert x == pytest.approx(y, rel=1e-14)
        elif t <= 1:
            assert x == pytest.approx(y / 4.0, rel=1e-14)
        else:
            assert y / 4.0 < x < y
    assert magnitude == pytest.approx(0.1 * math.log(4.0) + 1.0)
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, scaling="cubic"), dict(dim=8, factor=0.5), dict(dim=8, base=0.5),
                dict(dim=8, base=math.inf), dict(dim=8, scaling="parts"), dict(dim=8, factor=math.nan)):
        with pytest.raises(ValueError):
            attention.rotary_frequencies(**bad)
    assert attention.rotary_turns([math.pi, -math.pi, math.pi / 2, 0.0]).tolist() == [2 ** 63 - 1, -2 ** 63, 2 ** 62, 0]
    with pytest.raises(ValueError):
        attention.rotary_turns([4.0])
    with pytest.raises(ValueError, match="layout"):
        attention.Rotary(8, layout="whole")


def test_module_arguments():
    for bad in (dict(dim=64, heads=3, kv_heads=2), dict(dim=64, heads=0), dict(dim=64, heads=2, kv_heads=0), dict(dim=65, heads=2),
                dict(dim=512, heads=2), dict(dim=64, heads=4, mode="BF16X7"), dict(dim=64, heads=4, dropout=1.5)):
        with pytest.raises(ValueError):
            attention.EmuCrossAttention(**bad)
    layer = attention.EmuCrossAttention(64, 4, kv_heads=2, context_dim=24, bias=False)
    assert {n: tuple(p.shape) for n, p in layer.named_parameters()} == {
        "norm.weight": (64,), "w_q": (64, 64), "w_kv": (64, 24), "w_o": (64, 64)}
    with pytest.raises(ValueError):
        layer(torch.zeros(2, 3, 32))
    with pytest.raises(ValueError):
        attention.EmuDropout(-0.1)
    x = torch.randn(3, 4)
    assert attention.EmuDropout(0.5).eval()(x) is x and torch.equal(attention.EmuDropout(0.0)(x, x), x + x)


# The published known answers of Philox4x32-10 (the paper's test vectors).
@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_reference(counter, key, want):
    got = philox_words(key[0] | key[1] << 32, counter[2] | counter[3] << 32, counter[0] | counter[1] << 32)
    assert tuple(got) == want
    assert kept(key[0] | key[1] << 32, counter[2] | counter[3] << 32, [0], 0.0) == [True]


# ---- the reference itself ------------------------------------------------------------

def _plain(q, k, v, bias, alive):
    share = q.shape[2] // k.shape[2]
    q, k, v = q.transpose(1, 2), *(t.transpose(1, 2).repeat_interleave(share, 1) for t in (k, v))
    z = q @ k.transpose(2, 3) / math.sqrt(q.shape[3]) + bias.masked_fill(~alive, 0.0)[:, None, None]
    p = torch.softmax(z.masked_fill(~alive[:, None, None], -1e300), -1).masked_fill(~alive[:, None, None], 0.0)
    return (p @ v).transpose(1, 2)


def test_reference_against_autograd_and_differences():
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    q, k, v, bias = rnd(2, 3, 4, 5), rnd(2, 6, 2, 5), rnd(2, 6, 2, 5), rnd(2, 6)
    bias[0, 2] = -math.inf
    alive = bias > -math.inf
    ref = Attention(q, k, v, bias)
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v, bias)]
    y = _plain(*leaves, alive)
    assert torch.allclose(ref.out().v, y, rtol=1e-12, atol=1e-12)
    g = rnd(2, 3, 4, 5).requires_grad_(True)
    first = torch.autograd.grad(y, leaves, g, create_graph=True)
    got = ref.backward(g.detach())
    for a, b in zip(got, first):
        assert torch.allclose(a.v, b, rtol=1e-10, atol=1e-12)
    cot = [rnd(*t.shape) for t in (q, k, v, bias)]
    second = torch.autograd.grad(first, [g, *leaves], cot)
    for a, b in zip(ref.backward2(*cot), second):
        assert torch.allclose(a.v, b, rtol=1e-9, atol=1e-11)
    # a gradient and a second one by differences along random directions (error: h^2, and 1e-16 / h)
    h = 1e-5
    way = [rnd(*t.shape) for t in (q, k, v, bias)]
    moved = lambda s: [t + s * h * w for t, w in zip((q, k, v, bias), way)]
    value = lambda s: float((Attention(*moved(s)).out().v * g.detach()).sum())
    slope = sum(float((a.v * w).masked_fill(~torch.isfinite(w), 0.0).sum()) for a, w in zip(got, way))
    assert (value(1) - value(-1)) / (2 * h) == pytest.approx(slope, rel=1e-7, abs=1e-7)

    def pairing(s):
        r = Attention(*moved(s))
        r.backward(g.detach())
        return sum(float((a.v * c).sum()) for a, c in zip(r.backward(g.detach()), cot))

    slope = sum(float((a.v * w).sum()) for a, w in zip(ref.backward2(*cot)[1:], way))
    assert (pairing(1) - pairing(-1)) / (2 * h) == pytest.approx(slope, rel=1e-6, abs=1e-6)
