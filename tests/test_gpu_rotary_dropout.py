"""GPU parity of rotary positions and dropout (include/emu_attention.h) against
their definitions: rotations in 64 bits, the generator's words in Python
integers."""
import math

import pytest
import torch

from attention_reference import U, kept
from emulated_fp32_matrix_amd import attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rotate(x, positions, frequencies, layout, magnitude, inverse=False):
    """x [batch, tokens, heads, dim] in 64 bits; positions [batch, tokens]."""
    n = len(frequencies)
    angle = positions.double()[:, :, None, None] * torch.tensor(frequencies, dtype=torch.float64, device=x.device)
    c, s = magnitude * torch.cos(angle), magnitude * torch.sin(-angle if inverse else angle)
    y = x.double().clone()
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    size = torch.zeros_like(y)   # of what the products round
    size[..., first] = size[..., second] = magnitude * (a.abs() + b.abs())
    return y, size


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("batch,tokens,heads,dim,part,start,scaling", [
    (1, 1, 1, 2, 2, 0, None), (2, 5, 3, 7, 6, 11, None), (1, 33, 8, 32, 32, 0, "linear"), (3, 17, 4, 64, 24, 5000, "base"),
    (2, 40, 2, 128, 128, 1000003, "parts"), (4, 1, 16, 64, 64, -70001, None), (1, 2000, 5, 50, 50, 2 ** 40, None),
    (2, 3, 2, 33, 10, 3, "parts"), (700, 9, 12, 96, 64, 100, None),
    (2, 3, 2, 2600, 2500, 7, None), (1, 2, 1, 1030, 1030, 7, "base"), (2, 300, 1, 6, 4, 0, None), (3, 11, 70, 8, 8, 1, None)])
def test_rotary(layout, batch, tokens, heads, dim, part, start, scaling):
    g = torch.Generator(device=DEV).manual_seed(dim)
    x = torch.randn(batch, tokens, heads, dim, generator=g, device=DEV).requires_grad_(True)
    positions = start + torch.randint(0, 50, (batch, 1), generator=g, device=DEV) + torch.arange(tokens, device=DEV)
    rot = attention.Rotary(part, layout=layout, scaling=scaling, factor=4.0 if scaling else 1.0, original_length=2048,
                           device=DEV)
    frequencies, magnitude = attention.rotary_frequencies(part, scaling=scaling, factor=4.0 if scaling else 1.0,
                                                          original_length=2048)
    y = rot(x, positions)
    want, size = rotate(x.detach(), positions, frequencies, layout, magnitude)
    # cosine and sine to 2^-23, times the magnitude and the element, a sum: 4.5
    # roundings of u; the reference's own angle is off by 2^-53 of itself
    far = 2.0 ** -52 * float(positions.abs().max())
    bound = (5 * U + far) * size + 1e-40
    assert bool(((y.double() - want).abs() <= bound).all())
    v = torch.randn(y.shape, generator=g, device=DEV).requires_grad_(True)
    (gx,) = torch.autograd.grad(y, x, v, create_graph=True)
    want, size = rotate(v.detach(), positions, frequencies, layout, magnitude, inverse=True)
    assert bool(((gx.double() - want).abs() <= (5 * U + far) * size + 1e-40).all())
    w = torch.randn(y.shape, generator=g, device=DEV)
    (gv,) = torch.autograd.grad(gx, v, w)
    want, size = rotate(w, positions, frequencies, layout, magnitude)
    assert bool(((gv.double() - want).abs() <= (5 * U + far) * size + 1e-40).all())


def test_far_positions_are_exact_turns():
    """Positions a whole number of turns apart rotate alike: 2^-64 turns are counted exactly."""
    turns = torch.tensor([2 ** 62, 2 ** 40, -2 ** 63], device=DEV)   # a quarter, 2^-24 and half a turn a position
    x = torch.randn(1, 4, 2, 6, device=DEV)
    near = torch.tensor([0, 1, 2, 3], device=DEV)
    for far in (2 ** 24, -2 ** 24, 2 ** 50, 3 * 2 ** 60):
        assert torch.equal(attention.rotary(x, near, turns), attention.rotary(x, near + far, turns))
    y = attention.rotary(x, near, turns)
    assert torch.equal(y[0, 1, :, 0], -x[0, 1, :, 3]) and torch.equal(y[0, 1, :, 3], x[0, 1, :, 0])
    assert torch.equal(y[0, 2, :, 0], -x[0, 2, :, 0])


def test_rotary_strides_and_types():
    g = torch.Generator(device=DEV).manual_seed(1)
    wide = torch.randn(2, 9, 3, 4, 40, generator=g, device=DEV)
    rot = attention.Rotary(16, device=DEV)
    positions = torch.arange(9, device=DEV)
    for x in (wide[:, :, 1], wide[:, :, 2, :, 3:35], wide[:, :, 0].transpose(1, 2).contiguous().transpose(1, 2),
              wide[:, :, 0].transpose(2, 3).contiguous().transpose(2, 3), wide[:1, :, 0].expand(2, 9, 4, 40)):
        want = rot(x.contiguous(), positions)
        assert torch.equal(rot(x, positions), want)
        assert torch.equal(rot(x, positions.int()), want)
        assert torch.equal(rot(x, positions.expand(2, 9)), want)
        assert torch.equal(rot(x[1], positions), want[1])
    five = wide[:, :, :, :, :20].permute(0, 2, 1, 3, 4)   # [2, 3, 9, 4, 20]
    assert torch.equal(rot(five, positions), torch.stack([rot(five[:, i], positions) for i in range(3)], 1))
    assert rot(wide[:, :0, 0], positions[:0]).shape == (2, 0, 4, 40)


SEED = (0x123456789ABCDEF0, -5)


def seed_tensor(key=SEED[0], offset=SEED[1]):
    return torch.tensor([key, offset], device=DEV)


@pytest.mark.parametrize("shape,p", [((1,), 0.5), ((3, 5), 0.1), ((7, 4), 0.9), ((2, 3, 6), 0.25), ((33, 1), 0.5), ((257, 31), 0.1)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout_mask(shape, p, residual):
    x = torch.randn(shape, device=DEV, requires_grad=True)
    r = torch.randn(shape, device=DEV, requires_grad=True) if residual else None
    y = attention.dropout(x, p, seed_tensor(), residual=r)
    keep = torch.tensor(kept(*SEED, range(x.numel()), p), device=DEV).reshape(shape)
    scale = torch.tensor(1.0 / (1.0 - p), device=DEV, dtype=torch.float32)
    want = torch.where(keep, x.detach() * scale, torch.zeros((), device=DEV))
    if residual:
        want = want + r.detach()
    assert torch.equal(y, want)
    g = torch.randn(shape, device=DEV, requires_grad=True)
    grads = torch.autograd.grad(y, [x] + ([r] if residual else []), g, create_graph=True)
    assert torch.equal(grads[0], torch.where(keep, g * scale, torch.zeros((), device=DEV)))
    if residual:
        assert torch.equal(grads[1], g)
    w = torch.randn(shape, device=DEV)
    (gg,) = torch.autograd.grad(grads[0], g, w)
    assert torch.equal(gg, torch.where(keep, w * scale, torch.zeros((), device=DEV)))


@pytest.mark.parametrize("rows,cols,stride", [(9, 8, 12), (9, 7, 7), (9, 7, 11), (5, 1, 3), (1, 13, 20), (40, 33, 40)])
def test_dropout_rows_apart(rows, cols, stride):
    """The mask goes by the element's number, whatever the strides."""
    x = torch.randn(rows, stride, device=DEV)[:, :cols]
    r = torch.randn(rows, stride + 3, device=DEV)[:, 2:cols + 2]
    want = attention.dropout(x.contiguous(), 0.3, seed_tensor(), residual=r.contiguous())
    assert torch.equal(attention.dropout(x, 0.3, seed_tensor(), residual=r), want)
    assert torch.equal(attention.dropout(x, 0.3, seed_tensor()), attention.dropout(x.contiguous(), 0.3, seed_tensor()))


def test_dropout_ends():
    x = torch.tensor([1.0, math.inf, math.nan, -2.0, 0.0, 3.0], device=DEV)
    assert torch.equal(attention.dropout(x, 0.0, seed_tensor())[3:], x[3:])
    assert torch.equal(attention.dropout(x, 1.0, seed_tensor()), torch.zeros_like(x))
    assert attention.dropout(x[:0], 0.5, seed_tensor()).shape == (0,)
    assert attention.dropout(x[0], 0.0, seed_tensor()).shape == ()


def test_dropout_counts_past_32_bits():
    """Elements past 2^34, whose blocks of four are past 2^32 (69 GB in, as much out)."""
    n = (1 << 34) + 64
    x = torch.ones(n, device=DEV)
    y = attention.dropout(x, 0.5, seed_tensor())
    del x
    for at in (0, (1 << 32) - 32, (1 << 34) - 32, (1 << 34)):
        assert (y[at:at + 64] != 0).tolist() == kept(*SEED, range(at, at + 64), 0.5)


def test_kept_share():
    x = torch.ones(1000, 1000, device=DEV)
    for p in (0.1, 0.5, 0.9):
        share = float((attention.dropout(x, p, attention.dropout_seed(DEV)) != 0).double().mean())
        assert abs(share - (1 - p)) < 6 * math.sqrt(p * (1 - p) / 1e6)   # six standard deviations
