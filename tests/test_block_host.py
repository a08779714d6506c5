"""Host-side checks of the transformer-block operators (no GPU needed): the
header matches the binding, invalid arguments are refused before any HIP
call, workspaces are reported, and the Python functions refuse what they
cannot run."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import emulated_fp32_matrix_amd as emu
from emulated_fp32_matrix_amd import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "emu_block.h")
FAKE = 0x1000   # never dereferenced: the calls below end before any HIP call
INVALID, UNSUPPORTED = emu.STATUS_INVALID_VALUE, emu.STATUS_NOT_SUPPORTED
lib = block._lib


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(emu_[a-z0-9_]+)\s*\(", text)))


def test_header_matches_binding_and_library():
    assert _declared() == sorted(block.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", emu.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert not set(_declared()) - set(re.findall(r"\bT (emu_[a-z0-9_]+)$", out, flags=re.M))
    assert block.emu_block_version() == 100


def test_header_compiles_as_c():
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-x", "c", HEADER], check=True)


def test_constants_match_header():
    text = open(HEADER).read()
    assert f"#define EMU_LAYER_NORM_MAX_COLS {block.LAYER_NORM_MAX_COLS}" in text
    for name, value in block.ACTIVATIONS.items():
        assert re.search(rf"EMU_ACT_{name.upper()} = {value}\b", text)


# name, valid arguments (pointers never read), then argument positions and
# values that each make the call invalid
CALLS = {
    "emu_layer_norm": ([4, 8, FAKE, 8, None, None, 1e-5, FAKE, 8, None, None, None],
                       [(0, -1), (1, 0), (2, None), (3, 7), (6, -1.0), (6, float("nan")), (7, None), (8, 7)]),
    "emu_layer_norm_backward": (
        [4, 8, FAKE, 8, FAKE, 8, None, FAKE, FAKE, FAKE, 8, None, None, None, 0, None],
        [(0, -1), (1, 0), (2, None), (3, 7), (4, None), (5, 7), (7, None), (8, None), (10, 7)]),
    "emu_layer_norm_backward2": (
        [4, 8, FAKE, 8, None, None, FAKE, 8, FAKE, 8, None, FAKE, FAKE, FAKE, 8, FAKE, 8, None, None, 0, None],
        [(0, -1), (1, 0), (3, 7), (6, None), (7, 7), (8, None), (9, 7), (11, None), (12, None), (14, 7), (16, 7)]),
    "emu_act_backward": ([4, 8, FAKE, 8, FAKE, 8, 1, FAKE, 8, None],
                         [(0, -1), (1, -1), (2, None), (3, 7), (4, None), (5, 7), (6, 6), (6, -1), (7, None), (8, 7)]),
    "emu_act_backward2": ([4, 8, FAKE, 8, FAKE, 8, FAKE, 8, 1, FAKE, 8, FAKE, 8, None],
                          [(0, -1), (2, None), (3, 7), (4, None), (6, None), (8, 6), (10, 7), (12, 7)]),
    "emu_sgemm_act": (
        [0, 4, 6, 8, FAKE, 8, FAKE, 6, None, None, 1, None, 6, None, 6, FAKE, 6, 1, None, 0, None],
        [(0, 2), (1, -1), (2, -1), (3, -1), (4, None), (5, 7), (6, None), (7, 5), (8, FAKE + 8), (10, 6), (15, None),
         (16, 5), (17, 6), (17, -1)]),
    "emu_sgemm_gated": (
        [4, 6, 8, FAKE, 8, FAKE, 8, None, None, 1, None, 12, FAKE, 6, 1, None, 0, None],
        [(0, -1), (1, -1), (2, -1), (3, None), (4, 7), (5, None), (6, 7), (7, FAKE + 8), (9, 6), (12, None), (13, 5),
         (14, 7)]),
    "emu_gated_backward": ([4, 6, FAKE, 6, FAKE, 12, 1, FAKE, 12, None],
                           [(0, -1), (1, -1), (2, None), (3, 5), (4, None), (5, 11), (6, 9), (7, None), (8, 11)]),
    "emu_gated_backward2": ([4, 6, FAKE, 12, FAKE, 6, FAKE, 12, 1, FAKE, 6, FAKE, 12, None],
                            [(0, -1), (2, None), (3, 11), (4, None), (5, 5), (6, None), (7, 11), (8, 6), (10, 5), (12, 11)]),
    "emu_wgrad": ([64, 6, 8, FAKE, 6, FAKE, 8, FAKE, 8, None, None, 0, None],
                  [(0, -1), (1, -1), (2, -1), (3, None), (4, 5), (5, None), (6, 7), (7, None), (8, 7)]),
    "emu_wgrad_act": ([64, 6, 8, FAKE, 6, FAKE, 6, 2, FAKE, 6, FAKE, 8, FAKE, 8, None, None, 0, None],
                      [(0, -1), (1, -1), (2, -1), (3, None), (4, 5), (5, None), (6, 5), (7, 6), (8, None), (9, 5),
                       (10, None), (11, 7), (12, None), (13, 7)]),
    "emu_wgrad_gated": ([64, 6, 8, FAKE, 6, FAKE, 12, 2, FAKE, 12, FAKE, 8, FAKE, 8, None, None, 0, None],
                        [(0, -1), (1, -1), (2, -1), (3, None), (4, 5), (5, None), (6, 11), (7, -1), (8, None), (9, 11),
                         (10, None), (11, 7), (12, None), (13, 7)]),
    "emu_presplit_gated": ([6, 8, FAKE, 8, 1, FAKE, None], [(0, -1), (1, -1), (2, None), (3, 7), (4, 0), (5, None), (5, FAKE + 8)]),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_invalid_arguments_refused(name):
    args, bad = CALLS[name]
    for at, value in bad:
        call = list(args)
        call[at] = value
        assert getattr(lib, name)(*call) == INVALID, (name, at, value)


def test_optional_arrays_need_a_leading_dimension():
    # Z and R are optional; when given, their leading dimension is checked
    args = list(CALLS["emu_sgemm_act"][0])
    for at in (11, 13):
        call = list(args)
        call[at], call[at + 1] = FAKE, 5
        assert lib.emu_sgemm_act(*call) == INVALID
    call = list(CALLS["emu_sgemm_gated"][0])
    call[10], call[11] = FAKE, 11
    assert lib.emu_sgemm_gated(*call) == INVALID


def test_planes_refused_in_native_mode():
    call = list(CALLS["emu_sgemm_act"][0])
    call[8], call[17] = FAKE, emu.MODES["NATIVE_F32"]
    assert lib.emu_sgemm_act(*call) == INVALID


def test_empty_calls_succeed_without_a_device():
    assert lib.emu_layer_norm(0, 8, None, 8, None, None, 1e-5, None, 8, None, None, None) == 0
    assert lib.emu_act_backward(0, 8, None, 8, None, 8, 1, None, 8, None) == 0
    assert lib.emu_act_backward(8, 0, None, 1, None, 1, 1, None, 1, None) == 0
    assert lib.emu_sgemm_act(0, 0, 6, 8, None, 8, None, 6, None, None, 1, None, 6, None, 6, None, 6, 1, None, 0, None) == 0
    assert lib.emu_sgemm_gated(4, 0, 8, None, 8, None, 8, None, None, 1, None, 1, None, 1, 1, None, 0, None) == 0
    assert lib.emu_wgrad(64, 0, 8, None, 1, FAKE, 8, None, 8, None, None, 0, None) == 0


def test_wide_layer_norm_not_supported():
    wide = block.LAYER_NORM_MAX_COLS + 1
    assert lib.emu_layer_norm(4, wide, FAKE, wide, None, None, 1e-5, FAKE, wide, None, None, None) == UNSUPPORTED
    out = ctypes.c_size_t(0)
    assert lib.emu_layer_norm_backward_workspace(4, wide, ctypes.byref(out)) == UNSUPPORTED


def test_long_inner_dimension_not_supported():
    k = 1 << 23
    assert lib.emu_sgemm_act(1, 4, 6, k, FAKE, k, FAKE, k, None, None, 1, None, 6, None, 6, FAKE, 6, 1, None, 0, None) == UNSUPPORTED
    assert lib.emu_sgemm_gated(4, 6, k, FAKE, k, FAKE, k, None, None, 1, None, 12, FAKE, 6, 1, None, 0, None) == UNSUPPORTED
    ld = 1 << 24
    assert lib.emu_wgrad(64, 6, 8, FAKE, ld, FAKE, 8, FAKE, 8, None, None, 0, None) == UNSUPPORTED
    assert lib.emu_wgrad(64, 6, 8, FAKE, 6, FAKE, ld, FAKE, 8, None, None, 0, None) == UNSUPPORTED


def _bytes(fn, *args):
    out = ctypes.c_size_t(0)
    assert fn(*args, ctypes.byref(out)) == 0
    return out.value


def test_workspace_is_checked():
    """A call that needs a workspace refuses none, a short one and a
    misaligned one."""
    need = _bytes(lib.emu_layer_norm_backward_workspace, 5000, 256)
    assert need > 0
    base = [5000, 256, FAKE, 256, FAKE, 256, None, FAKE, FAKE, FAKE, 256, FAKE, FAKE]
    for ws, size in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert lib.emu_layer_norm_backward(*base, ws, size, None) == INVALID
    need = _bytes(lib.emu_wgrad_workspace, 100000, 256, 256)
    assert need > 0
    for ws, size in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert lib.emu_wgrad(100000, 256, 256, FAKE, 256, FAKE, 256, FAKE, 256, None, ws, size, None) == INVALID


def test_workspace_queries():
    out = ctypes.c_size_t(0)
    assert lib.emu_sgemm_act_workspace(0, -1, 6, 8, None, 8, 0, 1, ctypes.byref(out)) == INVALID
    assert lib.emu_sgemm_act_workspace(0, 4, 6, 8, None, 8, 0, 1, None) == INVALID
    assert lib.emu_sgemm_act_workspace(0, 4, 6, 8, None, 7, 0, 1, ctypes.byref(out)) == INVALID
    assert lib.emu_sgemm_act_workspace(0, 4, 6, 8, None, 8, 1, 0, ctypes.byref(out)) == INVALID
    assert lib.emu_sgemm_gated_workspace(4, -6, 8, None, 8, 0, 1, ctypes.byref(out)) == INVALID
    assert lib.emu_wgrad_workspace(-1, 6, 8, ctypes.byref(out)) == INVALID
    # no rows, nothing to hold
    assert _bytes(lib.emu_sgemm_act_workspace, 1, 0, 512, 256, None, 256, 0, 1) == 0
    assert _bytes(lib.emu_wgrad_workspace, 0, 512, 256) == 0
    # the planes of op(B) at least (fewer rows take one launch without them)
    assert _bytes(lib.emu_sgemm_act_workspace, 1, 552960, 512, 256, FAKE, 256, 0, 1) >= 3 * 2 * 512 * 256
    few = ctypes.c_int(-1)
    assert lib.emu_sgemm_act_route(1, 1, 512, 256, ctypes.byref(few)) == 0 and few.value == 1
    assert lib.emu_sgemm_act_route(1, 552960, 512, 256, ctypes.byref(few)) == 0 and few.value == 0
    assert lib.emu_sgemm_act_route(1, 64, 4096, 1024, ctypes.byref(few)) == 0 and few.value == 2
    assert lib.emu_sgemm_act_route(1, 1, 512, -1, ctypes.byref(few)) == INVALID


# ---- Python functions ------------------------------------------------------------

def test_cpu_tensors_and_other_types_refused():
    x, w = torch.zeros(3, 8), torch.zeros(6, 8)
    for call in (lambda: block.layer_norm(x), lambda: block.linear_act(x, w), lambda: block.gated_linear(x, w),
                 lambda: block.layer_norm([1.0])):
        with pytest.raises(TypeError):
            call()


def test_unknown_names_refused():
    x, w = torch.zeros(3, 8), torch.zeros(6, 8)
    for call in (lambda: block.linear_act(x, w, activation="swish"), lambda: block.gated_linear(x, w, mode="FP64"),
                 lambda: block.EmuLinearAct(8, 6, activation="swish"),
                 lambda: block.EmuGatedFFN(8, 6, activation="swish")):
        with pytest.raises(ValueError):
            call()


def test_modules_hold_the_parameters_of_their_torch_counterparts():
    assert set(block.EmuLayerNorm(8).state_dict()) == set(torch.nn.LayerNorm(8).state_dict())
    assert set(block.EmuLayerNorm(8, bias=False).state_dict()) == {"weight"}
    assert not block.EmuLayerNorm(8, elementwise_affine=False).state_dict()
    assert set(block.EmuLinearAct(8, 6).state_dict()) == set(torch.nn.Linear(8, 6).state_dict())
    ffn = block.EmuGatedFFN(8, 6)
    assert {k: tuple(v.shape) for k, v in ffn.state_dict().items()} == {
        "norm.weight": (8,), "norm.bias": (8,), "w_in": (12, 8), "b_in": (12,), "out.weight": (8, 6), "out.bias": (8,)}
    assert set(block.EmuGatedFFN(8, 6, bias=False, norm=False).state_dict()) == {"w_in", "out.weight"}


def test_every_function_is_defined_once():
    names = re.findall(r"^(?:def|class) (\w+)", open(block.__file__).read(), flags=re.M)
    assert len(names) == len(set(names)) and "emu_block_version" in names
