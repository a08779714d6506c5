"""The operators of a transformer block's attention half, beside the linears,
norms and feed-forward projections of :mod:`.block`: attention of queries over
keys of another length, rotary positions, and dropout with the residual sum,
through the C ABI of ``include/emu_attention.h``.

An interatomic potential lets the tokens of an atom's neighbours attend to each
other under a bias, the logarithm of the cutoff function; its forces are the
gradient of the energy, and training on forces differentiates that gradient
once more ("Unlocking Tensor Core Performance for Machine Learning Interatomic
Potentials", section "TF32x3 on Ampere GPUs").  :func:`cross_attention` is
therefore differentiable twice, with respect to the bias too; the other two
are linear and have every derivative.

    from emulated_fp32_matrix_amd import attention
    o = attention.cross_attention(q, k, v, key_bias=log_cutoff)   # [batch, tokens, heads, dim]
    rot = attention.Rotary(64, device="cuda")
    q = rot(q, positions)
    y = attention.dropout(h, 0.1, attention.dropout_seed("cuda"), residual=x)
    layer = attention.EmuCrossAttention(256, 8, dropout=0.1).cuda()
    y = layer(x, context, key_bias=log_cutoff)

Tensors, streams, capturing in graphs and errors are as in :mod:`.block`.
``cross_attention`` keeps its output for its backward pass: changing it in
place before that raises, as with torch's own functions.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _i64, _lib, _vp
from .block import EmuLayerNorm, _mode_of, _ops, _psize, linear_act

MAX_DIM = 128   # EMU_ATTENTION_MAX_DIM
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = ("linear", "base", "parts")

_int, _float, _double, _size = ctypes.c_int, ctypes.c_float, ctypes.c_double, ctypes.c_size_t


class _Heads(ctypes.Structure):   # emu_heads_t
    _fields_ = [("data", _vp), ("batch", _i64), ("token", _i64), ("head", _i64)]


class _Attention(ctypes.Structure):   # emu_attention_t
    _fields_ = [("batch", _i64), ("queries", _i64), ("keys", _i64), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("scale", _float), ("key_bias", _vp),
                ("key_bias_batch", _i64), ("key_bias_key", _i64), ("key_mask", _vp), ("key_mask_batch", _i64),
                ("key_mask_key", _i64), ("lengths", _vp), ("lengths_64", ctypes.c_int32)]


_pattn = ctypes.POINTER(_Attention)

# C functions declared in include/emu_attention.h, with their argument types
_SIGNATURES = {
    "emu_attention_version": [],
    "emu_cross_attention_workspace": [_pattn, _psize],
    "emu_cross_attention": [_pattn, _Heads, _Heads, _Heads, _vp, _vp, _vp, _size, _vp],
    "emu_cross_attention_backward_workspace": [_pattn, _psize],
    "emu_cross_attention_backward": [_pattn, _Heads, _Heads, _Heads, _Heads, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _size,
                                     _vp],
    "emu_cross_attention_backward2_workspace": [_pattn, _psize],
    "emu_cross_attention_backward2": [_pattn, _Heads, _Heads, _Heads, _vp, _i64, _i64, _Heads, _Heads, _Heads, _Heads,
                                      _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _size, _vp],
    "emu_rotary": [_i64, _i64, _i64, _i64, _Heads, _vp, _i64, _i64, _vp, _i64, _int, _float, _int, _vp, _vp],
    "emu_dropout": [_i64, _i64, _vp, _i64, _double, _vp, _vp, _i64, _vp, _i64, _vp],
}
EXPORTS = tuple(_SIGNATURES)
for _name, _types in _SIGNATURES.items():
    getattr(_lib, _name).argtypes = _types
    getattr(_lib, _name).restype = _int


def emu_attention_version() -> int:
    return int(_lib.emu_attention_version())


# ---- functions -------------------------------------------------------------------

def cross_attention(q, k, v, key_bias=None, key_mask=None, lengths=None, scale=None):
    """softmax(scale q k^T + key_bias) v for each sequence and head.

    ``q`` [batch, queries, heads, dim]; ``k``, ``v`` [batch, keys, kv_heads,
    dim], heads a multiple of kv_heads: query head h reads key head h // (heads
    / kv_heads).  Any strides with unit stride along dim (others are copied), so
    slices of a joint projection and transposed [batch, heads, tokens, dim]
    arrays are read in place.  Self attention is the case of q, k and v from
    one source.  ``scale``: 1 / sqrt(dim) by default.

    Keys take part that are among the first ``lengths[b]`` (int32 or int64,
    [batch], on the device), whose ``key_mask`` (bool [batch, keys]) is True
    and whose ``key_bias`` (float32 [batch, keys], differentiable) is not
    -inf; the others' keys and values are not used, whatever they hold.  A row
    without keys gives zeros.  Returns [batch, queries, heads, dim].
    Differentiable twice with respect to q, k, v and key_bias."""
    return _ops.cross_attention(q, k, v, key_bias, key_mask, lengths, scale)


def rotary(x, positions, turns, layout="half", magnitude=1.0):
    """Rotate pairs of each head of ``x`` [..., tokens, heads, dim] by angles
    that grow with the token's position; :class:`Rotary` keeps ``turns`` and
    the rest.

    ``positions``: int32 or int64, [tokens] or x's shape up to its tokens.
    ``turns``: int64 [pairs] (:func:`rotary_turns`): frequencies as 2^-64 turns
    per position.  ``layout``: pairs are elements (i, i + pairs) ("half") or (2
    i, 2 i + 1) ("interleaved") of the first 2 pairs; the rest is copied."""
    return _ops.rotary(x, positions, turns, _layout(layout), magnitude)


def dropout(x, p, seed, residual=None):
    """x / (1 - p) where kept, 0 where dropped (with probability p), plus
    ``residual``; also where x is not finite.

    ``seed``: int64 [2] on x's device (:func:`dropout_seed`), a generator's key
    and stream: the mask is a function of it and of the element's number, made
    again in the backward pass and never stored.  A captured call reads the
    seed when it is replayed."""
    return _ops.dropout(x, p, seed, residual)


def dropout_seed(device, generator=None):
    """A seed for :func:`dropout` from torch's generator (which a captured
    graph advances with every replay)."""
    return torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), device=device, generator=generator)


def _layout(layout) -> int:
    try:
        return LAYOUTS[layout]
    except (KeyError, TypeError):
        raise ValueError(f"layout must be one of {', '.join(LAYOUTS)}, not {layout!r}") from None


def rotary_frequencies(dim, base=10000.0, scaling=None, factor=1.0, original_length=None):
    """(radians per position of each of dim / 2 pairs, magnitude) for
    ``rotary``: base^(-2 i / dim), scaled for contexts ``factor`` times as long
    as those trained on:
      "linear": divided by factor (positions interpolated);
      "base": base multiplied by factor^(dim / (dim - 2)), which divides the
        slowest frequency by factor and keeps the fastest;
      "parts": frequencies of more than 32 turns over ``original_length`` kept,
        of less than 1 divided by factor, linearly between; magnitude 0.1
        ln(factor) + 1."""
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and positive, not {dim}")
    if scaling is not None and scaling not in SCALINGS:
        raise ValueError(f"scaling must be None or one of {', '.join(SCALINGS)}, not {scaling!r}")
    if not base >= 1.0 or not factor >= 1.0 or math.isinf(base) or math.isinf(factor):
        raise ValueError("base and factor must be finite and at least 1")
    if scaling == "parts" and not (original_length and original_length > 0):
        raise ValueError("scaling 'parts' needs the original_length")
    if scaling == "base" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = [base ** (-2 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "parts":
        kept = [min(max((original_length * x / (2 * math.pi) - 1.0) / 31.0, 0.0), 1.0) for x in f]
        f = [x * (w + (1.0 - w) / factor) for x, w in zip(f, kept)]
    return f, 0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0


def rotary_turns(frequencies, device=None):
    """Radians per position (at most pi in size) as ``rotary`` takes them: an
    int64 tensor of 2^-64 turns per position."""
    turns = [float(f) / (2 * math.pi) for f in frequencies]
    if not all(abs(t) <= 0.5 for t in turns):
        raise ValueError("frequencies must be at most half a turn per position")
    fixed = [min(max(int(math.ldexp(t, 64)), -2 ** 63), 2 ** 63 - 1) for t in turns]
    return torch.tensor(fixed, dtype=torch.int64, device=device)


# ---- modules -------------------------------------------------------------------------------------

class Rotary(torch.nn.Module):
    """Rotary positions of the first ``dim`` elements of a head:
    ``rot(x, positions)``; frequencies as :func:`rotary_frequencies`."""

    def __init__(self, dim, base=10000.0, layout="half", scaling=None, factor=1.0, original_length=None, device=None):
        super().__init__()
        _layout(layout)
        f, self.magnitude = rotary_frequencies(dim, base, scaling, factor, original_length)
        self.dim, self.base, self.layout, self.scaling, self.factor = dim, base, layout, scaling, factor
        self.register_buffer("turns", rotary_turns(f, device), persistent=False)

    def forward(self, x, positions):
        return rotary(x, positions, self.turns, self.layout, self.magnitude)

    def extra_repr(self):
        more = f", scaling={self.scaling}, factor={self.factor}" if self.scaling else ""
        return f"{self.dim}, base={self.base}, layout={self.layout}{more}"


class EmuDropout(torch.nn.Module):
    """Dropout with an optional residual sum, ``drop(x, residual)``; a new mask
    each call, from torch's generator.  Without training it is x (+ residual)."""

    def __init__(self, p=0.1):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must be between 0 and 1, not {p}")
        self.p = p

    def forward(self, x, residual=None):
        if not self.training or self.p == 0.0:
            return x if residual is None else x + residual
        return dropout(x, self.p, dropout_seed(x.device), residual)

    def extra_repr(self):
        return f"p={self.p}"


class EmuCrossAttention(torch.nn.Module):
    """A pre-norm attention block with its residual sum:
        n = layer_norm(x);  x + dropout(W_o attention(W_q n, W_kv context))
    ``layer(x)`` attends to n itself, ``layer(x, context)`` to a context of
    ``context_dim`` features and another length.  ``w_kv`` [2 kv_heads dim,
    context_dim] holds the keys' rows above the values'.  ``rotary``: a
    :class:`Rotary` applied to queries and keys, whose positions the call
    gives (``positions`` [tokens] or [batch, tokens]; ``context_positions``)."""

    def __init__(self, dim, heads, kv_heads=None, head_dim=None, context_dim=None, rotary=None, dropout=0.0, bias=True,
                 norm=True, eps=1e-5, mode="AUTO", device=None):
        super().__init__()
        kv_heads = heads if kv_heads is None else kv_heads
        if heads < 1 or kv_heads < 1 or heads % kv_heads:
            raise ValueError(f"heads must be a multiple of kv_heads, not {heads} and {kv_heads}")
        if head_dim is None:
            if dim % heads:
                raise ValueError(f"{dim} features do not divide into {heads} heads: give head_dim")
            head_dim = dim // heads
        if not 1 <= head_dim <= MAX_DIM:
            raise ValueError(f"heads must be 1 to {MAX_DIM} wide, not {head_dim}")
        _mode_of(mode)
        self.dim, self.heads, self.kv_heads, self.head_dim, self.mode = dim, heads, kv_heads, head_dim, mode
        self.context_dim = dim if context_dim is None else context_dim
        self.norm = EmuLayerNorm(dim, eps=eps, bias=bias, device=device) if norm else None
        self.rotary = rotary
        self.drop = EmuDropout(dropout)
        for name, rows, cols in (("q", heads * head_dim, dim), ("kv", 2 * kv_heads * head_dim, self.context_dim),
                                 ("o", dim, heads * head_dim)):
            w = torch.nn.Parameter(torch.empty(rows, cols, device=device, dtype=torch.float32))
            torch.nn.init.kaiming_uniform_(w, a=math.sqrt(5))
            self.register_parameter(f"w_{name}", w)
            self.register_parameter(f"b_{name}", torch.nn.Parameter(
                torch.zeros(rows, device=device, dtype=torch.float32)) if bias else None)

    def forward(self, x, context=None, key_bias=None, key_mask=None, lengths=None, positions=None,
                context_positions=None):
        if x.dim() != 3 or x.shape[-1] != self.dim:
            raise ValueError(f"x must be [batch, tokens, {self.dim}], not {tuple(x.shape)}")
        n = x if self.norm is None else self.norm(x)
        source = n if context is None else context
        if source.dim() != 3 or source.shape[0] != x.shape[0] or source.shape[-1] != self.context_dim:
            raise ValueError(f"the context must be [{x.shape[0]}, tokens, {self.context_dim}], not {tuple(source.shape)}")
        q = linear_act(n, self.w_q, self.b_q, mode=self.mode).unflatten(2, (self.heads, self.head_dim))
        kv = linear_act(source, self.w_kv, self.b_kv, mode=self.mode).unflatten(2, (2, self.kv_heads, self.head_dim))
        k, v = kv[:, :, 0], kv[:, :, 1]
        if self.rotary is not None:
            if positions is None or (context is not None and context_positions is None):
                raise ValueError("the block's rotary positions need positions and, with a context, context_positions")
            q, k = self.rotary(q, positions), self.rotary(k, positions if context is None else context_positions)
        o = cross_attention(q, k, v, key_bias, key_mask, lengths).flatten(2)
        if self.drop.training and self.drop.p > 0.0:   # (its own mode: it may be sampled in a block that does not train)
            return self.drop(linear_act(o, self.w_o, self.b_o, mode=self.mode), x)
        return linear_act(o, self.w_o, self.b_o, residual=x, mode=self.mode)

    def extra_repr(self):
        return (f"dim={self.dim}, heads={self.heads}, kv_heads={self.kv_heads}, head_dim={self.head_dim}, "
                f"context_dim={self.context_dim}, mode={self.mode}")
