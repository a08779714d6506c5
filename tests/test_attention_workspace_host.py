"""Workspaces of the attention calls (include/emu_attention.h): what their size
goes by, and that one asked for another call is refused.  No GPU needed: the
calls below end before any HIP call."""
import ctypes
import os

import pytest

import emulated_fp32_matrix_amd as emu
from emulated_fp32_matrix_amd import attention

lib = attention._lib
FAKE = 0x1000   # never dereferenced
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "emu_attention.h")
CALLS = ("", "_backward", "_backward2")


def struct(lengths=None, **sizes):
    return attention._Attention(scale=0.5, lengths=lengths, **sizes)


def need(call, a):
    n = ctypes.c_size_t(0)
    assert getattr(lib, f"emu_cross_attention{call}_workspace")(ctypes.byref(a), ctypes.byref(n)) == 0
    return n.value


def run(call, a, bytes_):
    z = attention._Heads(FAKE, 1, 1, 1)
    space = (FAKE, bytes_, None)
    if call == "":
        return lib.emu_cross_attention(ctypes.byref(a), z, z, z, FAKE, None, *space)
    if call == "_backward":
        return lib.emu_cross_attention_backward(ctypes.byref(a), z, z, z, z, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, *space)
    return lib.emu_cross_attention_backward2(ctypes.byref(a), z, z, z, None, 0, 0, z, z, z, z, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                             FAKE, *space)


def test_the_header_says_what_the_bytes_go_by():
    text = " ".join(open(HEADER).read().replace("*", " ").split())
    assert "ask for each call's own struct" in text and "whether lengths is NULL" in text


@pytest.mark.parametrize("call", CALLS[1:])
def test_with_and_without_lengths(call):
    sizes = dict(batch=7, queries=2000, keys=4000, heads=6, kv_heads=2, dim=80)
    plain, ragged = need(call, struct(**sizes)), need(call, struct(FAKE, **sizes))
    assert plain < ragged   # (otherwise the sizes here show nothing)
    assert run(call, struct(FAKE, **sizes), plain) == emu.STATUS_INVALID_VALUE


def test_smaller_batches_may_need_more():
    sizes = dict(queries=300, keys=4000, heads=4, kv_heads=4, dim=64)
    large, small = need("", struct(batch=18, **sizes)), need("", struct(batch=17, **sizes))
    assert large < small
    assert run("", struct(batch=17, **sizes), large) == emu.STATUS_INVALID_VALUE


@pytest.mark.parametrize("call", CALLS)
def test_nothing_else_of_the_struct_matters(call):
    """Biases, masks, their strides, the lengths' type and the scale leave the size as it is."""
    for sizes in (dict(batch=3, queries=100, keys=900, heads=4, kv_heads=2, dim=40), dict(batch=2, queries=1, keys=5000, heads=4,
                  kv_heads=4, dim=64), dict(batch=9, queries=20, keys=30, heads=2, kv_heads=2, dim=32)):
        for lengths in (None, FAKE):
            a = struct(lengths, **sizes)
            want = need(call, a)
            a.key_bias, a.key_bias_batch, a.key_bias_key, a.scale = FAKE, 7, 0, -2.0
            a.key_mask, a.key_mask_batch, a.key_mask_key = FAKE, 0, 3
            a.lengths_64 = 1 if lengths else 0
            assert need(call, a) == want
            if want:
                assert run(call, a, want - 1) == emu.STATUS_INVALID_VALUE
