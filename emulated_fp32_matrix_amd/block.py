"""The operators of a transformer block around :class:`EmuLinear`: layer norm,
the linear layer with its activation and residual sum in the GEMM's epilogue,
and the gated feed-forward projection, each with its backward pass, through
the C ABI of ``include/emu_block.h``.

An interatomic potential's forces are the gradient of its energy with respect
to its inputs, and training on forces differentiates that gradient again
("Unlocking Tensor Core Performance for Machine Learning Interatomic
Potentials", section "TF32x3 on Ampere GPUs").  Every function here is
therefore differentiable twice (``create_graph=True``); a third derivative is
refused by torch.

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
released (a capture that finds them alive is refused).  As with
:class:`EmuLinear`, ``mode`` picks the arithmetic of the products; the weight
gradient's is FP32.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import (MODES, OP_N, OP_T, STATUS_SUCCESS, EmuError, _check_matrix, _i64, _ld, _lib, _mode, _vp,
               emu_presplit_b, emu_presplit_b_bytes, select_mode)
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


def emu_block_version() -> int:
    return int(_lib.emu_block_version())


# ---- marshalling ---------------------------------------------------------------

def _act(activation) -> int:
    try:
        return ACTIVATIONS[activation]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, not {activation!r}") from None


def _mode_of(mode) -> int:
    if isinstance(mode, str) and mode.upper() not in MODES:
        raise ValueError(f"mode must be one of {', '.join(MODES)}, not {mode!r}")
    return _mode(mode)


def _check(t, name, device=None):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError(f"{name} must be a float32 CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, not {t.device}")


def _vector(t, name, n, device):
    """The data of an optional vector of length n."""
    if t is None:
        return None
    _check(t, name, device)
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be a vector of length {n}")
    return t if t.is_contiguous() else t.contiguous()


def _rows(t, width):
    """t as a matrix with unit stride along its last dimension: a view where
    the leading dimensions allow one."""
    t = t.detach()
    if t.dim() != 2:
        # (an empty tensor cannot infer its row count)
        t = t.reshape(-1, width) if t.numel() else t.reshape(math.prod(t.shape[:-1]), width)
    if t.shape[0] > 1 and t.stride(0) < width or width > 1 and t.stride(1) != 1:
        t = t.contiguous()
    return t


def _empty(rows, cols, like):
    return torch.empty((rows, cols), dtype=torch.float32, device=like.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


class _on:
    """Enters the device of a tensor if another one is current; gives the
    device's current stream."""

    __slots__ = ("guard", "stream")

    def __init__(self, device):
        self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)
        self.stream = torch.cuda.current_stream(device).cuda_stream or None

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


def _done(status, where):
    if status != STATUS_SUCCESS:
        raise EmuError(int(status), where)


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _asked_bytes(fn, *args):
    out = _size(0)
    _done(fn(*args, ctypes.byref(out)), fn.__name__)
    return out.value


def _wants_grad(*tensors):
    if not torch.is_grad_enabled():
        return False
    for t in tensors:
        if t is not None and t.requires_grad:
            return True
    return False


# ---- products -------------------------------------------------------------------

def _product(a, w, trans_b, bias, act, residual, z, mode, planes=None):
    """act(a @ op(w) + bias) + residual for matrices; z receives the
    pre-activation when given."""
    M, K = a.shape
    N = w.shape[0] if trans_b else w.shape[1]
    c = _empty(M, N, a)
    op = OP_T if trans_b else OP_N
    with _on(a.device) as stream:
        pa, lda = _ptr(a), _ld(a)
        ws = _workspace(_asked_bytes(_lib.emu_sgemm_act_workspace, op, M, N, K, pa, lda, 0 if planes is None else 1,
                                     mode), a.device)
        _done(_lib.emu_sgemm_act(op, M, N, K, pa, lda, _ptr(w), _ld(w), _ptr(planes), _ptr(bias), act, _ptr(z),
                                 N, _ptr(residual), 0 if residual is None else _ld(residual), _ptr(c), max(N, 1),
                                 mode, _ptr(ws), 0 if ws is None else ws.numel(), stream), "emu_sgemm_act")
    return c


def _gated(a, w, bias, act, z, mode, planes=None):
    M, K = a.shape
    F = w.shape[0] // 2
    c = _empty(M, F, a)
    with _on(a.device) as stream:
        pa, lda = _ptr(a), _ld(a)
        ws = _workspace(_asked_bytes(_lib.emu_sgemm_gated_workspace, M, F, K, pa, lda, 0 if planes is None else 1,
                                     mode), a.device)
        _done(_lib.emu_sgemm_gated(M, F, K, pa, lda, _ptr(w), _ld(w), _ptr(planes), _ptr(bias), act, _ptr(z),
                                   2 * F, _ptr(c), max(F, 1), mode, _ptr(ws), 0 if ws is None else ws.numel(), stream),
              "emu_sgemm_gated")
    return c


def wgrad(dz, x, want_db=False):
    """(dz^T x, column sums of dz or None) for matrices with the same rows:
    the weight and bias gradients of a linear layer, in FP32."""
    _check_matrix(dz, "dz")
    _check_matrix(x, "x")
    _check(x, "x", dz.device)
    if dz.shape[0] != x.shape[0]:
        raise ValueError(f"row counts differ: {dz.shape[0]} vs {x.shape[0]}")
    return _wgrad(dz, x, want_db)


def _wgrad(dz, x, want_db):
    rows, M = dz.shape
    N = x.shape[1]
    dw = _empty(M, N, dz)
    db = torch.empty(M, dtype=torch.float32, device=dz.device) if want_db else None
    with _on(dz.device) as stream:
        ws = _workspace(_asked_bytes(_lib.emu_wgrad_workspace, rows, M, N), dz.device)
        _done(_lib.emu_wgrad(rows, M, N, _ptr(dz), _ld(dz), _ptr(x), _ld(x), _ptr(dw), max(N, 1), _ptr(db), _ptr(ws),
                             0 if ws is None else ws.numel(), stream), "emu_wgrad")
    return dw, db


def _wgrad_from(dy, z, act, x, want_db, gated):
    """(dz, dz^T x, column sums of dz or None), dz the activation's (gated:
    the gated product's) backward pass."""
    rows, M = dy.shape
    N, wide = x.shape[1], z.shape[1]
    dz, dw = _empty(rows, wide, dy), _empty(wide, N, dy)
    db = torch.empty(wide, dtype=torch.float32, device=dy.device) if want_db else None
    asked, run = (_lib.emu_wgrad_gated_workspace, _lib.emu_wgrad_gated) if gated \
        else (_lib.emu_wgrad_workspace, _lib.emu_wgrad_act)
    with _on(dy.device) as stream:
        ws = _workspace(_asked_bytes(asked, rows, M, N), dy.device)
        _done(run(rows, M, N, _ptr(dy), _ld(dy), _ptr(z), _ld(z), act, _ptr(dz), max(wide, 1), _ptr(x), _ld(x),
                  _ptr(dw), max(N, 1), _ptr(db), _ptr(ws), 0 if ws is None else ws.numel(), stream), run.__name__)
    return dz, dw, db


def _fuse_act(x):
    """Whether the activation's backward pass runs inside the weight gradient:
    every 128 columns of x repeat it, which pays for up to two such tiles."""
    return x.shape[-1] <= 256


class _GatedPlanes:
    """Planes of a gated projection's weight, rebuilt when it changes."""

    def __init__(self):
        self.key = None
        self.planes = None

    def get(self, w, mode):
        key = (w.data_ptr(), tuple(w.shape), w._version, mode, w.device)
        if key != self.key:
            F, K = w.shape[0] // 2, w.shape[1]
            nbytes = _asked_bytes(_lib.emu_presplit_gated_bytes, F, K, mode)
            planes = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=w.device)
            with _on(w.device) as stream:
                _done(_lib.emu_presplit_gated(F, K, _ptr(w), _ld(w), mode, _ptr(planes), stream),
                      "emu_presplit_gated")
            self.planes, self.key = planes, key
        return self.planes


class _Planes:
    """Planes of op(B) of a weight, rebuilt when it changes."""

    def __init__(self, trans_b):
        self.trans_b = trans_b
        self.key = None
        self.planes = None

    def get(self, w, mode):
        key = (w.data_ptr(), tuple(w.shape), w._version, mode, w.device)
        if key != self.key:
            K, N = (w.shape[1], w.shape[0]) if self.trans_b else w.shape
            st, nbytes = emu_presplit_b_bytes(N, K, mode)
            _done(st, "emu_presplit_b_bytes")
            planes = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=w.device)
            with _on(w.device) as stream:
                _done(emu_presplit_b(OP_T if self.trans_b else OP_N, N, K, w.data_ptr(), _ld(w), mode,
                                     planes.data_ptr(), stream), "emu_presplit_b")
            self.planes, self.key = planes, key
        return self.planes


def _planes_for(cache, w, M, N, K, mode):
    """The cached planes of w where the call would split it, else None."""
    if cache is None or mode == MODES["NATIVE_F32"] or not (M and N and K):
        return None
    if mode == MODES["AUTO"]:
        few = _int(0)
        _done(_lib.emu_sgemm_act_route(OP_T, M, N, K, ctypes.byref(few)), "emu_sgemm_act_route")
        if few.value or select_mode(M, N, K) != "BF16X9":
            return None
        return cache.get(w, MODES["BF16X9"])
    return cache.get(w, mode)


# ---- differentiable pieces ---------------------------------------------------------

class _Refuse(torch.autograd.Function):
    """out, connected to the tensors it was made from by a derivative that
    raises: a gradient taken through it never goes missing silently."""

    @staticmethod
    def forward(ctx, out, *sources):
        return out.view_as(out)

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("the block operators are differentiable twice: a third derivative is not implemented")


def _claim_leaves(ctx, device):
    """Refuses a call captured in a graph whose leaves still belong to an
    eager call.  A leaf's gradient node keeps the stream of the first call
    that used the leaf, as long as any result of it lives; a captured backward
    pass would make that stream wait for the captured one, and ending such a
    capture ends the process."""
    stream = torch.cuda.current_stream(device).cuda_stream
    for node, _ in ctx.next_functions:
        if node is None or type(node).__name__ != "AccumulateGrad":
            continue
        if node.metadata.setdefault("emu_block_stream", stream) != stream and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("capturing a differentiable call whose parameters or inputs still belong to the results "
                               "of an earlier call on another stream: release those results first, or make the "
                               "earlier call on the capturing stream")


def _last_derivative(backward):
    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        with torch.no_grad():
            outs = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return outs
        sources = [t for t in (*grads, *ctx.saved_tensors) if t is not None and t.requires_grad]
        if not sources:
            return outs
        return tuple(_Refuse.apply(o, *sources) if isinstance(o, torch.Tensor) else o for o in outs)

    return wrapped


class _Product(torch.autograd.Function):
    """a @ op(w) in `mode`, op(w) = w^T (trans_w) or w; the input-gradient
    product of the layers below, differentiable again."""

    @staticmethod
    def forward(ctx, a, w, trans_w, mode, caches):
        ctx.save_for_backward(a, w)
        ctx.trans_w, ctx.mode, ctx.caches = trans_w, mode, caches
        a2, w2 = _rows(a, a.shape[-1]), _rows(w, w.shape[-1])
        N = w.shape[0] if trans_w else w.shape[1]
        planes = None
        if caches is not None and w2.data_ptr() == w.data_ptr():
            planes = _planes_for(caches[0 if trans_w else 1], w2, a2.shape[0], N, a2.shape[1], mode)
        return _product(a2, w2, trans_w, None, 0, None, None, mode, planes)

    @staticmethod
    def backward(ctx, g):
        a, w = ctx.saved_tensors
        ga = gw = None
        if ctx.needs_input_grad[0]:
            ga = _Product.apply(g, w, not ctx.trans_w, ctx.mode, ctx.caches)
        if ctx.needs_input_grad[1]:
            gw = _WeightGrad.apply(g, a, False, ctx.mode)[0] if ctx.trans_w \
                else _WeightGrad.apply(a, g, False, ctx.mode)[0]
        return ga, gw, None, None, None


class _WeightGrad(torch.autograd.Function):
    """(dz^T x, column sums of dz) for matrices, differentiable again: with P
    and q the gradients of the two, dz gets x P^T + q and x gets dz P."""

    @staticmethod
    def forward(ctx, dz, x, want_db, mode):
        ctx.save_for_backward(dz, x)
        ctx.mode = mode
        ctx.set_materialize_grads(False)
        return _wgrad(_rows(dz, dz.shape[1]), _rows(x, x.shape[1]), want_db)

    @staticmethod
    def backward(ctx, P, q):
        dz, x = ctx.saved_tensors
        gdz = gx = None
        if ctx.needs_input_grad[0]:
            if P is not None:
                gdz = _Product.apply(x, P, True, ctx.mode, None)
            if q is not None:
                gdz = q.expand(dz.shape[0], -1) if gdz is None else gdz + q
        if ctx.needs_input_grad[1] and P is not None:
            gx = _Product.apply(dz, P, False, ctx.mode, None)
        return gdz, gx, None, None


class _ActBackward(torch.autograd.Function):
    """dz = dy act'(z) for matrices."""

    @staticmethod
    def forward(ctx, dy, z, act):
        ctx.save_for_backward(dy, z)
        ctx.act = act
        d, zz = _rows(dy, dy.shape[1]), _rows(z, z.shape[1])
        rows, cols = zz.shape
        out = _empty(rows, cols, zz)
        with _on(zz.device) as stream:
            _done(_lib.emu_act_backward(rows, cols, _ptr(d), _ld(d), _ptr(zz), _ld(zz), act, _ptr(out), max(cols, 1),
                                        stream), "emu_act_backward")
        return out

    @staticmethod
    @_last_derivative
    def backward(ctx, v):
        dy, z = ctx.saved_tensors
        v, d, zz = _rows(v, v.shape[1]), _rows(dy, dy.shape[1]), _rows(z, z.shape[1])
        rows, cols = zz.shape
        gdy = _empty(rows, cols, zz) if ctx.needs_input_grad[0] else None
        gz = _empty(rows, cols, zz) if ctx.needs_input_grad[1] else None
        with _on(zz.device) as stream:
            _done(_lib.emu_act_backward2(rows, cols, _ptr(v), _ld(v), _ptr(d), _ld(d), _ptr(zz), _ld(zz), ctx.act,
                                         _ptr(gdy), max(cols, 1), _ptr(gz), max(cols, 1), stream),
                  "emu_act_backward2")
        return gdy, gz, None


class _GatedBackward(torch.autograd.Function):
    """dZ = [dh u act'(g) | dh act(g)] for Z = [g | u]."""

    @staticmethod
    def forward(ctx, dh, z, act):
        ctx.save_for_backward(dh, z)
        ctx.act = act
        d, zz = _rows(dh, dh.shape[1]), _rows(z, z.shape[1])
        rows, F = d.shape
        out = _empty(rows, 2 * F, zz)
        with _on(zz.device) as stream:
            _done(_lib.emu_gated_backward(rows, F, _ptr(d), _ld(d), _ptr(zz), _ld(zz), act, _ptr(out),
                                          max(2 * F, 1), stream), "emu_gated_backward")
        return out

    @staticmethod
    @_last_derivative
    def backward(ctx, v):
        dh, z = ctx.saved_tensors
        v, d, zz = _rows(v, v.shape[1]), _rows(dh, dh.shape[1]), _rows(z, z.shape[1])
        rows, F = d.shape
        gdh = _empty(rows, F, zz) if ctx.needs_input_grad[0] else None
        gz = _empty(rows, 2 * F, zz) if ctx.needs_input_grad[1] else None
        with _on(zz.device) as stream:
            _done(_lib.emu_gated_backward2(rows, F, _ptr(v), _ld(v), _ptr(d), _ld(d), _ptr(zz), _ld(zz), ctx.act,
                                           _ptr(gdh), max(F, 1), _ptr(gz), max(2 * F, 1), stream),
                  "emu_gated_backward2")
        return gdh, gz, None


def _first_order_grads(ctx, gy, z, x, weight, gated):
    """(dx, dW, db) where dW is asked for and nothing is differentiated again:
    the activation's backward pass runs inside the weight gradient's."""
    K = weight.shape[1]
    g2 = _rows(gy, gy.shape[-1])
    dz, gw, gb = _wgrad_from(g2, z, ctx.act, _rows(x, K), ctx.has_bias and ctx.needs_input_grad[2], gated)
    gx = None
    if ctx.needs_input_grad[0]:
        gx = _Product.apply(dz, weight, False, ctx.mode, ctx.caches).reshape(ctx.x_shape)
    return gx, gw, gb


def _layer_grads(ctx, dz, x, weight, has_bias):
    """(dx, dW, db) of z = x W^T + b from dz, each where asked for."""
    gx = gw = gb = None
    if ctx.needs_input_grad[0]:
        gx = _Product.apply(dz, weight, False, ctx.mode, ctx.caches).reshape(ctx.x_shape)
    want_b = has_bias and ctx.needs_input_grad[2]
    if ctx.needs_input_grad[1] or want_b:
        x2 = x if x.dim() == 2 else x.reshape(dz.shape[0], weight.shape[1])
        gw, gb = _WeightGrad.apply(dz, x2, want_b, ctx.mode)
        if not ctx.needs_input_grad[1]:
            gw = None
    return gx, gw, gb


# ---- linear layer with activation and residual ----------------------------------------

class _LinearAct(torch.autograd.Function):
    """y = act(x W^T + b) + residual; the pre-activation z is an output of its
    own, so that the backward pass, which reads it, can be differentiated."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, act, mode, caches):
        _claim_leaves(ctx, x.device)
        ctx.set_materialize_grads(False)
        ctx.act, ctx.mode, ctx.caches = act, mode, caches
        ctx.x_shape = x.shape
        ctx.has_bias = bias is not None
        N, K = weight.shape
        x2, w2 = _rows(x, K), _rows(weight, K)
        res = None if residual is None else _rows(residual, N)
        planes = _planes_for(caches[0], w2, x2.shape[0], N, K, mode) if caches is not None else None
        z = _empty(x2.shape[0], N, x2) if act != 0 else None
        y = _product(x2, w2, True, bias, act, res, z, mode, planes).view(x.shape[:-1] + (N,))
        ctx.save_for_backward(x, weight, z)
        return y, z

    @staticmethod
    def backward(ctx, gy, gz):
        x, weight, z = ctx.saved_tensors
        N = weight.shape[0]
        if gz is None and z is not None and ctx.needs_input_grad[1] and not torch.is_grad_enabled() and _fuse_act(x):
            gx, gw, gb = _first_order_grads(ctx, gy, z, x, weight, False)
            return gx, gw, gb, gy if ctx.needs_input_grad[3] else None, None, None, None
        dz = None
        if gy is not None:
            g2 = gy.reshape(math.prod(ctx.x_shape[:-1]), N)
            dz = g2 if z is None else _ActBackward.apply(g2, z, ctx.act)
        if gz is not None:
            dz = gz if dz is None else dz + gz
        if dz is None:
            return None, None, None, None, None, None, None
        gx, gw, gb = _layer_grads(ctx, dz, x, weight, ctx.has_bias)
        return gx, gw, gb, gy if ctx.needs_input_grad[3] else None, None, None, None


def _check_layer(x, weight, bias, out):
    _check(x, "x")
    _check(weight, "weight", x.device)
    if weight.dim() != 2:
        raise ValueError("weight must be 2-D")
    if x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x must end in {weight.shape[1]} features, not {tuple(x.shape)}")
    if bias is not None and (bias.dim() != 1 or bias.shape[0] != out):
        raise ValueError(f"bias must be a vector of length {out}")


def linear_act(x, weight, bias=None, activation="identity", residual=None, mode="AUTO", _caches=None):
    """act(x W^T + b) + residual, W [out, in] as in torch.nn.Linear: one GEMM
    with the bias, the activation and the residual sum in its epilogue.

    ``activation``: a key of ``ACTIVATIONS``.  ``residual``: the output's
    shape, or None.  Differentiable twice with respect to every tensor."""
    act, m = _act(activation), _mode_of(mode)
    _check_layer(x, weight, bias, weight.shape[0])
    N, K = weight.shape
    bias = _vector(bias, "bias", N, x.device)
    if residual is not None:
        _check(residual, "residual", x.device)
        if residual.shape != x.shape[:-1] + (N,):
            raise ValueError(f"residual must have shape {tuple(x.shape[:-1] + (N,))}")
    if _wants_grad(x, weight, bias, residual):
        return _LinearAct.apply(x, weight, bias, residual, act, m, _caches)[0]
    x2, w2 = _rows(x, K), _rows(weight, K)
    res = None if residual is None else _rows(residual, N)
    planes = _planes_for(_caches[0], w2, x2.shape[0], N, K, m) if _caches is not None else None
    y = _product(x2, w2, True, bias, act, res, None, m, planes)
    return y if x.dim() == 2 else y.view(x.shape[:-1] + (N,))


# ---- gated feed-forward projection -------------------------------------------------------

class _GatedLinear(torch.autograd.Function):
    """h = act(g) u, [g | u] = Z = x W^T + b; Z is an output of its own (see
    _LinearAct)."""

    @staticmethod
    def forward(ctx, x, weight, bias, act, mode, caches):
        _claim_leaves(ctx, x.device)
        ctx.set_materialize_grads(False)
        ctx.act, ctx.mode, ctx.caches = act, mode, None if caches is None else (None, caches[1])
        ctx.x_shape = x.shape
        ctx.has_bias = bias is not None
        wide, K = weight.shape
        x2, w2 = _rows(x, K), _rows(weight, K)
        planes = _planes_for(caches[0], w2, x2.shape[0], wide, K, mode) if caches is not None else None
        z = _empty(x2.shape[0], wide, x2)
        h = _gated(x2, w2, bias, act, z, mode, planes).view(x.shape[:-1] + (wide // 2,))
        ctx.save_for_backward(x, weight, z)
        return h, z

    @staticmethod
    def backward(ctx, gh, gz):
        x, weight, z = ctx.saved_tensors
        if gz is None and ctx.needs_input_grad[1] and not torch.is_grad_enabled() and _fuse_act(x):
            return (*_first_order_grads(ctx, gh, z, x, weight, True), None, None, None)
        dz = None
        if gh is not None:
            dz = _GatedBackward.apply(gh.reshape(z.shape[0], z.shape[1] // 2), z, ctx.act)
        if gz is not None:
            dz = gz if dz is None else dz + gz
        if dz is None:
            return None, None, None, None, None, None
        gx, gw, gb = _layer_grads(ctx, dz, x, weight, ctx.has_bias)
        return gx, gw, gb, None, None, None


def gated_linear(x, weight, bias=None, activation="silu", mode="AUTO", _caches=None):
    """act(gate) * up with [gate | up] = x W^T + b: the first half of a gated
    feed-forward layer, both projections, the activation and the product in
    one GEMM.  W is [2 F, in]: rows 0..F-1 the gate's, F..2F-1 the up
    projection's; the bias likewise.  Differentiable twice."""
    act, m = _act(activation), _mode_of(mode)
    _check_layer(x, weight, bias, weight.shape[0])
    wide, K = weight.shape
    if wide % 2:
        raise ValueError("weight must hold as many gate rows as up rows")
    bias = _vector(bias, "bias", wide, x.device)
    if _wants_grad(x, weight, bias):
        return _GatedLinear.apply(x, weight, bias, act, m, _caches)[0]
    x2, w2 = _rows(x, K), _rows(weight, K)
    planes = _planes_for(_caches[0], w2, x2.shape[0], wide, K, m) if _caches is not None else None
    h = _gated(x2, w2, bias, act, None, m, planes)
    return h if x.dim() == 2 else h.view(x.shape[:-1] + (wide // 2,))


# ---- layer norm ------------------------------------------------------------------------------

def _norm_forward(x2, weight, bias, eps, keep):
    rows, cols = x2.shape
    y = _empty(rows, cols, x2)
    stats = torch.empty((2, rows), dtype=torch.float32, device=x2.device) if keep else None
    with _on(x2.device) as stream:
        p = _ptr(stats)
        _done(_lib.emu_layer_norm(rows, cols, _ptr(x2), _ld(x2), _ptr(weight), _ptr(bias), eps, _ptr(y), cols, p,
                                  None if p is None else p + 4 * rows, stream), "emu_layer_norm")
    return y, stats


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        _claim_leaves(ctx, x.device)
        cols = x.shape[-1]
        y, stats = _norm_forward(_rows(x, cols), weight, bias, eps, True)
        ctx.save_for_backward(x, weight, stats)
        ctx.has_bias = bias is not None
        return y.view(x.shape)

    @staticmethod
    def backward(ctx, gy):
        x, weight, stats = ctx.saved_tensors
        want = (ctx.needs_input_grad[0], ctx.needs_input_grad[1], ctx.has_bias and ctx.needs_input_grad[2])
        gx, gw, gb = _LayerNormBackward.apply(gy, x, weight, stats, want)
        return gx, gw, gb, None


class _LayerNormBackward(torch.autograd.Function):
    """(dx, dweight, dbias); its gradient with respect to x is the whole one,
    through the mean and the deviation too."""

    @staticmethod
    def forward(ctx, gy, x, weight, stats, want):
        ctx.save_for_backward(gy, x, weight, stats)
        ctx.set_materialize_grads(False)
        cols = x.shape[-1]
        g2, x2 = _rows(gy, cols), _rows(x, cols)
        rows = x2.shape[0]
        dx = _empty(rows, cols, x2) if want[0] else None
        sums = torch.empty((2, cols), dtype=torch.float32, device=x2.device) if want[1] or want[2] else None
        dw = sums[0] if want[1] else None
        db = sums[1] if want[2] else None
        with _on(x2.device) as stream:
            ws = None
            if sums is not None:
                ws = _workspace(_asked_bytes(_lib.emu_layer_norm_backward_workspace, rows, cols), x2.device)
            p = _ptr(stats)
            _done(_lib.emu_layer_norm_backward(rows, cols, _ptr(g2), _ld(g2), _ptr(x2), _ld(x2), _ptr(weight), p,
                                               p + 4 * rows, _ptr(dx), cols, _ptr(dw), _ptr(db), _ptr(ws),
                                               0 if ws is None else ws.numel(), stream), "emu_layer_norm_backward")
        return None if dx is None else dx.view(x.shape), dw, db

    @staticmethod
    @_last_derivative
    def backward(ctx, v, p, q):
        gy, x, weight, stats = ctx.saved_tensors
        cols = x.shape[-1]
        g2, x2 = _rows(gy, cols), _rows(x, cols)
        rows = x2.shape[0]
        v2 = None if v is None else _rows(v, cols)
        p, q = (None if t is None else t.contiguous() for t in (p, q))
        gdy = _empty(rows, cols, x2) if ctx.needs_input_grad[0] else None
        gx = _empty(rows, cols, x2) if ctx.needs_input_grad[1] else None
        gw = torch.empty(cols, dtype=torch.float32, device=x2.device) \
            if weight is not None and ctx.needs_input_grad[2] else None
        with _on(x2.device) as stream:
            ws = None
            if gw is not None:
                ws = _workspace(_asked_bytes(_lib.emu_layer_norm_backward_workspace, rows, cols), x2.device)
            st = _ptr(stats)
            _done(_lib.emu_layer_norm_backward2(rows, cols, _ptr(v2), 0 if v2 is None else _ld(v2), _ptr(p), _ptr(q),
                                                _ptr(g2), _ld(g2), _ptr(x2), _ld(x2), _ptr(weight), st,
                                                st + 4 * rows, _ptr(gdy), cols, _ptr(gx), cols, _ptr(gw), _ptr(ws),
                                                0 if ws is None else ws.numel(), stream), "emu_layer_norm_backward2")
        return (None if gdy is None else gdy.view(x.shape), None if gx is None else gx.view(x.shape), gw, None, None)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over the last dimension (up to LAYER_NORM_MAX_COLS wide), as
    torch.nn.functional.layer_norm; differentiable twice."""
    _check(x, "x")
    if x.dim() < 1 or not 1 <= x.shape[-1] <= LAYER_NORM_MAX_COLS:
        raise ValueError(f"layer_norm takes 1 to {LAYER_NORM_MAX_COLS} features, not {tuple(x.shape)}")
    cols = x.shape[-1]
    weight = _vector(weight, "weight", cols, x.device)
    bias = _vector(bias, "bias", cols, x.device)
    if _wants_grad(x, weight, bias):
        return _LayerNorm.apply(x, weight, bias, float(eps))
    y = _norm_forward(_rows(x, cols), weight, bias, float(eps), False)[0]
    return y if x.dim() == 2 else y.view(x.shape)


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
        if x.shape[-1] != self.dim:
            raise ValueError(f"x must end in {self.dim} features, not {tuple(x.shape)}")
        return layer_norm(x, self.weight, self.bias, self.eps)

    def extra_repr(self):
        return f"{self.dim}, eps={self.eps}, affine={self.weight is not None}, bias={self.bias is not None}"


class EmuLinearAct(EmuLinear):
    """EmuLinear with an activation and an optional residual sum in its GEMM's
    epilogue: ``layer(x, residual)`` = act(x W^T + b) + residual.  Parameters,
    modes and ``cache_weights`` are EmuLinear's; the weight and bias gradients
    run through the library too."""

    def __init__(self, in_features, out_features, bias=True, activation="identity", mode="AUTO", device=None,
                 cache_weights=False):
        super().__init__(in_features, out_features, bias=bias, mode=mode, device=device, cache_weights=False)
        _act(activation)
        self.activation = activation
        self._caches = (_Planes(True), _Planes(False)) if cache_weights else None

    @classmethod
    def from_linear(cls, linear, activation="identity", mode="AUTO", cache_weights=False):
        m = cls(linear.in_features, linear.out_features, bias=linear.bias is not None, activation=activation,
                mode=mode, device=linear.weight.device, cache_weights=cache_weights)
        with torch.no_grad():
            m.weight.copy_(linear.weight)
            if linear.bias is not None:
                m.bias.copy_(linear.bias)
        return m

    def forward(self, x, residual=None):
        return linear_act(x, self.weight, self.bias, self.activation, residual, self.mode, self._caches)

    def extra_repr(self):
        return f"{super().extra_repr()}, activation={self.activation}"


class EmuGatedFFN(torch.nn.Module):
    """A pre-norm gated feed-forward block with its residual sum:
        n = layer_norm(x);  x + W2 (act(Wg n) * (Wu n)) (+ biases)
    ``w_in`` [2 hidden, dim] holds Wg above Wu.  ``norm=False`` leaves the
    layer norm out."""

    def __init__(self, dim, hidden, activation="silu", bias=True, norm=True, eps=1e-5, mode="AUTO", device=None,
                 cache_weights=False):
        super().__init__()
        _act(activation)
        self.dim, self.hidden, self.activation, self.mode = dim, hidden, activation, mode
        self.norm = EmuLayerNorm(dim, eps=eps, bias=bias, device=device) if norm else None
        self.w_in = torch.nn.Parameter(torch.empty(2 * hidden, dim, device=device, dtype=torch.float32))
        self.register_parameter("b_in", torch.nn.Parameter(
            torch.zeros(2 * hidden, device=device, dtype=torch.float32)) if bias else None)
        self.out = EmuLinearAct(hidden, dim, bias=bias, mode=mode, device=device, cache_weights=cache_weights)
        self._caches = (_GatedPlanes(), _Planes(False)) if cache_weights else None
        torch.nn.init.kaiming_uniform_(self.w_in, a=math.sqrt(5))

    def forward(self, x):
        n = x if self.norm is None else self.norm(x)
        h = gated_linear(n, self.w_in, self.b_in, self.activation, self.mode, self._caches)
        return self.out(h, residual=x)

    def extra_repr(self):
        return f"dim={self.dim}, hidden={self.hidden}, activation={self.activation}, mode={self.mode}"
