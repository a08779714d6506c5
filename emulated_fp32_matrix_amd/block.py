"""The operators of a transformer block around :class:`EmuLinear`: layer norm,
the linear layer with its activation and residual sum in the GEMM's epilogue,
and the gated feed-forward projection, each with its backward pass, through
the C ABI of ``include/emu_block.h``.

An interatomic potential's forces are the gradient of its energy with respect
to its inputs, and training on forces differentiates that gradient again
("Unlocking Tensor Core Performance for Machine Learning Interatomic
Potentials", section "TF32x3 on Ampere GPUs").  Every function here is
therefore differentiable twice (``create_graph=True``); a third derivative
raises, and so do forward-mode derivatives, tracing (``torch.jit.trace``,
``make_fx``) and the transforms of ``torch.func`` (NotImplementedError).

    from emulated_fp32_matrix_amd import block
    n = block.layer_norm(x, weight, bias)
    y = block.linear_act(n, w, b, activation="gelu", residual=x)   # act(n w^T + b) + x
    h = block.gated_linear(n, w_in, b_in, activation="silu")       # act(gate) * up
    ffn = block.EmuGatedFFN(256, 512).cuda()                       # x + W2 (act(Wg n) * (Wu n))

Tensors are float32 on one CUDA device, any leading shape, with unit stride
along the last dimension (others are copied); work runs on the device's
current stream.  Calls allocate their outputs and workspaces with torch, so
they can be captured in a graph, which then owns them; a training step is
captured after the results of eager steps with the same parameters have been
released (a differentiable call that is captured while an input, or anything
it was made from, belongs to a living eager result is refused: the captured
backward pass would end the process; capturing the backward pass of a forward
pass that was not captured is not seen here, nor by torch's own functions).  As with
:class:`EmuLinear`, ``mode`` picks the arithmetic of the products; the weight
gradient's is FP32.

The functions and their derivatives are native (``csrc/block_torch.cpp``);
this module names them and holds the modules.  Wrong types raise TypeError,
wrong shapes and names ValueError, a failing library call :class:`EmuError` (a
RuntimeError; in a backward pass autograd passes on the RuntimeError alone).
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os

import torch

from . import _PKG, MODES, PresplitB, WeightSource, _i64, _lib, _mode, _vp
from .linear import EmuLinear

ACTIVATIONS = {"identity": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "tanh": 5}
LAYER_NORM_MAX_COLS = 16384   # EMU_LAYER_NORM_MAX_COLS

_int, _float, _size = ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_psize = ctypes.POINTER(_size)

# C functions declared in include/emu_block.h, with their argument types
_SIGNATURES = {
    "emu_block_version": [],
    "emu_layer_norm": [_i64, _i64, _vp, _i64, _vp, _vp, _float, _vp, _i64, _vp, _vp, _vp],
    "emu_layer_norm_backward_workspace": [_i64, _i64, _psize],
    "emu_layer_norm_backward": [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _size,
                                _vp],
    "emu_layer_norm_backward2": [_i64, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64,
                                 _vp, _i64, _vp, _vp, _size, _vp],
    "emu_act_backward": [_i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp],
    "emu_act_backward2": [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp],
    "emu_sgemm_act_route": [_int, _i64, _i64, _i64, ctypes.POINTER(_int)],
    "emu_sgemm_act_workspace": [_int, _i64, _i64, _i64, _vp, _i64, _int, _int, _psize],
    "emu_sgemm_act": [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _int, _vp, _i64, _vp, _i64, _vp, _i64,
                      _int, _vp, _size, _vp],
    "emu_sgemm_gated_workspace": [_i64, _i64, _i64, _vp, _i64, _int, _int, _psize],
    "emu_sgemm_gated": [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _int, _vp, _i64, _vp, _i64, _int, _vp,
                        _size, _vp],
    "emu_presplit_gated_bytes": [_i64, _i64, _int, _psize],
    "emu_presplit_gated": [_i64, _i64, _vp, _i64, _int, _vp, _vp],
    "emu_gated_backward": [_i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp],
    "emu_gated_backward2": [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp],
    "emu_wgrad_workspace": [_i64, _i64, _i64, _psize],
    "emu_wgrad": [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _size, _vp],
    "emu_wgrad_act": [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _size,
                      _vp],
    "emu_wgrad_gated_workspace": [_i64, _i64, _i64, _psize],
    "emu_wgrad_gated": [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _size,
                        _vp],
}
EXPORTS = tuple(_SIGNATURES)
for _name, _types in _SIGNATURES.items():
    getattr(_lib, _name).argtypes = _types
    getattr(_lib, _name).restype = _int


def _load_ops():
    path = os.path.join(_PKG, "_block_ops.so")
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    spec = importlib.util.spec_from_file_location("_block_ops", path)
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    return ops


_ops = _load_ops()


def emu_block_version() -> int:
    return int(_lib.emu_block_version())


def _act(activation) -> int:
    try:
        return ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, not {activation!r}") from None


def _mode_of(mode) -> int:
    m = MODES.get(mode)
    if m is None:
        if isinstance(mode, str) and mode.upper() not in MODES:
            raise ValueError(f"mode must be one of {', '.join(MODES)}, not {mode!r}")
        m = _mode(mode)
    return m


class PresplitGated:
    """A gated projection's weight split once into the BF16 planes of ``mode``
    (``presplit_gated``); ``planes`` is in the library's own layout,
    ``source`` identifies the weight."""

    def __init__(self, planes, F, K, mode, source=None):
        self.planes, self.F, self.K, self.mode, self.source = planes, int(F), int(K), mode, source


def _planes(given, kind, shape, weight, mode):
    """(planes tensor, mode of the call) of an explicit split, or (None, mode)."""
    if given is None:
        return None, mode
    if not isinstance(given, kind):
        raise TypeError(f"planes must come from {'presplit_gated' if kind is PresplitGated else 'presplit_b'}")
    if shape != tuple(weight.shape):
        raise ValueError(f"the planes are those of a weight of shape {shape}, not {tuple(weight.shape)}")
    split = _mode_of(given.mode)
    if mode != split and (mode, split) != (MODES["AUTO"], MODES["BF16X9"]):
        raise ValueError(f"the planes are split for {given.mode}")
    # (the backward pass reads the weight: both have to be the same)
    if given.source is None:
        raise ValueError("the planes do not say which weight they are those of")
    given.source.check(weight)
    return given.planes, mode


# ---- functions -------------------------------------------------------------------

def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over the last dimension (up to LAYER_NORM_MAX_COLS wide), as
    torch.nn.functional.layer_norm; differentiable twice."""
    return _ops.layer_norm(x, weight, bias, eps)


def linear_act(x, weight, bias=None, activation="identity", residual=None, mode="AUTO", planes=None):
    """act(x W^T + b) + residual, W [out, in] as in torch.nn.Linear: one GEMM
    with the bias, the activation and the residual sum in its epilogue.

    ``activation``: a key of ``ACTIVATIONS``.  ``residual``: the output's
    shape, or None.  ``planes``: ``presplit_b(weight, mode, trans_b=True)`` of
    a weight that does not change between calls (the forward product then
    skips its split); planes of another weight, and of one changed in place
    since, raise ValueError.  Differentiable twice with respect to every tensor."""
    m = _mode_of(mode)
    if planes is not None:
        planes, m = _planes(planes, PresplitB, (getattr(planes, "N", 0), getattr(planes, "K", 0)), weight, m)
    return _ops.linear_act(x, weight, bias, residual, _act(activation), m, planes)


def gated_linear(x, weight, bias=None, activation="silu", mode="AUTO", planes=None):
    """act(gate) * up with [gate | up] = x W^T + b: the first half of a gated
    feed-forward layer, both projections, the activation and the product in
    one GEMM.  W is [2 F, in]: rows 0..F-1 the gate's, F..2F-1 the up
    projection's; the bias likewise.  ``planes``: ``presplit_gated(weight,
    mode)``.  Differentiable twice."""
    m = _mode_of(mode)
    if planes is not None:
        planes, m = _planes(planes, PresplitGated, (2 * getattr(planes, "F", 0), getattr(planes, "K", 0)), weight, m)
    return _ops.gated_linear(x, weight, bias, _act(activation), m, planes)


def presplit_gated(weight, mode="BF16X9"):
    """Split a gated projection's weight [2 F, in] once, for ``gated_linear``
    calls in ``mode`` (BF16X9, also for AUTO, BF16X6, BF16X3 or BF16X1)."""
    return PresplitGated(_ops.presplit_gated(weight, _mode_of(mode)), weight.shape[0] // 2, weight.shape[1], mode,
                         WeightSource(weight))


def wgrad(dz, x, want_db=False):
    """(dz^T x, column sums of dz or None) for matrices with the same rows: the
    weight and bias gradients of a linear layer, in FP32; differentiable."""
    return _ops.wgrad(dz, x, want_db)


def act_grad(dy, z, activation):
    """dy act'(z) for matrices; differentiable once."""
    return _ops.act_grad(dy, z, _act(activation))


# ---- modules -------------------------------------------------------------------------------------

class EmuLayerNorm(torch.nn.Module):
    """torch.nn.LayerNorm over one dimension; state dicts load either way."""

    def __init__(self, dim, eps=1e-5, elementwise_affine=True, bias=True, device=None):
        super().__init__()
        self.dim, self.eps = dim, eps
        make = lambda f: torch.nn.Parameter(f(dim, device=device, dtype=torch.float32))
        self.register_parameter("weight", make(torch.ones) if elementwise_affine else None)
        self.register_parameter("bias", make(torch.zeros) if elementwise_affine and bias else None)

    def forward(self, x):
        if x.dim() < 1 or x.shape[-1] != self.dim:
            raise ValueError(f"x must end in {self.dim} features, not {tuple(x.shape)}")
        return layer_norm(x, self.weight, self.bias, self.eps)

    def extra_repr(self):
        return f"{self.dim}, eps={self.eps}, affine={self.weight is not None}, bias={self.bias is not None}"


class EmuLinearAct(EmuLinear):
    """EmuLinear with an activation and an optional residual sum in its GEMM's
    epilogue: ``layer(x, residual)`` = act(x W^T + b) + residual.  Parameters
    and modes are EmuLinear's; the weight and bias gradients run through the
    library too."""

    def __init__(self, in_features, out_features, bias=True, activation="identity", mode="AUTO", device=None):
        super().__init__(in_features, out_features, bias=bias, mode=mode, device=device)
        _act(activation)
        self.activation = activation

    @classmethod
    def from_linear(cls, linear, activation="identity", mode="AUTO"):
        m = cls(linear.in_features, linear.out_features, bias=linear.bias is not None, activation=activation,
                mode=mode, device=linear.weight.device)
        with torch.no_grad():
            m.weight.copy_(linear.weight)
            if linear.bias is not None:
                m.bias.copy_(linear.bias)
        return m

    def forward(self, x, residual=None):
        return linear_act(x, self.weight, self.bias, self.activation, residual, self.mode)

    def extra_repr(self):
        return f"{super().extra_repr()}, activation={self.activation}"


class EmuGatedFFN(torch.nn.Module):
    """A pre-norm gated feed-forward block with its residual sum:
        n = layer_norm(x);  x + W2 (act(Wg n) * (Wu n)) (+ biases)
    ``w_in`` [2 hidden, dim] holds Wg above Wu.  ``norm=False`` leaves the
    layer norm out."""

    def __init__(self, dim, hidden, activation="silu", bias=True, norm=True, eps=1e-5, mode="AUTO", device=None):
        super().__init__()
        _act(activation)
        self.dim, self.hidden, self.activation, self.mode = dim, hidden, activation, mode
        self.norm = EmuLayerNorm(dim, eps=eps, bias=bias, device=device) if norm else None
        self.w_in = torch.nn.Parameter(torch.empty(2 * hidden, dim, device=device, dtype=torch.float32))
        self.register_parameter("b_in", torch.nn.Parameter(
            torch.zeros(2 * hidden, device=device, dtype=torch.float32)) if bias else None)
        self.out = EmuLinearAct(hidden, dim, bias=bias, mode=mode, device=device)
        torch.nn.init.kaiming_uniform_(self.w_in, a=math.sqrt(5))

    def forward(self, x):
        n = x if self.norm is None else self.norm(x)
        h = gated_linear(n, self.w_in, self.b_in, self.activation, self.mode)
        return self.out(h, residual=x)

    def extra_repr(self):
        return f"dim={self.dim}, hidden={self.hidden}, activation={self.activation}, mode={self.mode}"
