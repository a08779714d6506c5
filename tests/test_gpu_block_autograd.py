"""The block operators inside autograd: outputs changed in place, frozen
parameters, inputs that are views, force training of the linear layer."""
import pytest
import torch

import block_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu
U = ref.U


def _block():
    from emulated_fp32_matrix_amd import block

    return block


def _randn(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to("cuda:0")


def _calls():
    """name -> (function of the leaves, leaves), for 2-D and 3-D inputs."""
    block = _block()
    out = {}
    for shape in ((6, 16), (2, 3, 16)):
        x, w, b = _randn(1, *shape), _randn(2, 8, 16, scale=0.25), _randn(3, 8)
        r, nw, nb = _randn(4, *shape[:-1], 8), _randn(5, 16), _randn(6, 16)
        dims = f"{len(shape)}-D"
        out[f"layer_norm {dims}"] = (block.layer_norm, (x, nw, nb))
        out[f"layer_norm plain {dims}"] = (block.layer_norm, (x,))
        out[f"linear_act {dims}"] = (lambda x, w, b, r: block.linear_act(x, w, b, "silu", r), (x, w, b, r))
        out[f"linear_act identity {dims}"] = (lambda x, w: block.linear_act(x, w), (x, w))
        out[f"gated_linear {dims}"] = (lambda x, w, b: block.gated_linear(x, w, b), (x, w, b))
    dz, z, x = _randn(7, 6, 8), _randn(8, 6, 8), _randn(9, 6, 16)
    out["wgrad"] = (lambda dz, x: block.wgrad(dz, x, True)[0], (dz, x))
    out["wgrad db"] = (lambda dz, x: block.wgrad(dz, x, True)[1], (dz, x))
    out["act_grad"] = (lambda dz, z: block.act_grad(dz, z, "tanh"), (dz, z))
    return out


@pytest.mark.parametrize("name", sorted(["wgrad", "wgrad db", "act_grad"] + [
    f"{f} {d}" for f in ("layer_norm", "layer_norm plain", "linear_act", "linear_act identity", "gated_linear")
    for d in ("2-D", "3-D")]))
def test_outputs_may_be_changed_in_place(name):
    """y.mul_, then backward: the gradients of 2 y + 1, as with torch's own
    operators; the input gradients of create_graph and the second derivatives
    likewise."""
    f, inputs = _calls()[name]
    leaves = [t.clone().requires_grad_(True) for t in inputs]
    want_y = f(*leaves)
    cot = _randn(11, *want_y.shape)
    used = [t for t, g in zip(leaves, torch.autograd.grad(want_y, leaves, cot, allow_unused=True)) if g is not None]
    want = torch.autograd.grad(f(*leaves), used, 2.0 * cot)
    y = f(*leaves)
    y.mul_(2.0).add_(1.0)
    assert torch.equal(y, 2.0 * want_y + 1.0)
    for got, one in zip(torch.autograd.grad(y, used, cot), want):
        assert torch.equal(got, one)
    if name == "act_grad":   # (differentiable once)
        return
    # the first derivatives, in place, then a second time
    first = torch.autograd.grad(f(*leaves), used, cot, create_graph=True)
    plain = [g for g in first if g.requires_grad]
    if not plain:
        return
    cots = [_randn(12 + i, *g.shape) for i, g in enumerate(plain)]
    want2 = torch.autograd.grad(plain, used, [-2.0 * c for c in cots], allow_unused=True, create_graph=True)
    again = [g for g in torch.autograd.grad(f(*leaves), used, cot, create_graph=True) if g.requires_grad]
    for g in again:
        g.neg_().mul_(2.0)
    got2 = torch.autograd.grad(again, used, cots, allow_unused=True, create_graph=True)
    for got, one in zip(got2, want2):
        assert (got is None) == (one is None)
        if got is not None:
            # (negation and doubling are exact, sums of several paths may be ordered otherwise)
            assert float((got - one).detach().abs().max()) <= 8 * U * float(one.detach().abs().max())
            got.neg_()   # the last derivatives too


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("create_graph", [False, True])
def test_bias_alone(gated, create_graph):
    """The weight frozen, the bias trained: its gradient without the weight's
    product, which would need an array of the weight's size."""
    block = _block()
    rows, K, N = 700, 2048, 4096
    x, w, b = _randn(1, rows, K), _randn(2, N, K, scale=K**-0.5), _randn(3, N).requires_grad_(True)
    f = (lambda: block.gated_linear(x, w, b)) if gated else (lambda: block.linear_act(x, w, b, "silu"))
    y = f()
    g = _randn(4, *y.shape)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    (db,) = torch.autograd.grad(y, b, g, create_graph=create_graph)
    used = torch.cuda.max_memory_allocated() - before
    z, zb = ref.product(x.double(), w.double(), b, "AUTO")
    F = N // 2
    if gated:
        d1, _, s1, _ = ref.slopes("silu", z[:, :F])
        dz = torch.cat([g * z[:, F:] * d1, g * ref.act("silu", z[:, :F])], dim=1)
        size = torch.cat([g.abs() * (z[:, F:].abs() + zb[:, F:]) * (24 * U * s1 + 1.2 * zb[:, :F]) + g.abs() * zb[:, F:] * d1.abs(),
                          g.abs() * (ref.act_bound("silu", z[:, :F]) + 1.2 * zb[:, :F])], dim=1) + 2 * U * dz.abs()
    else:
        d1, _, s1, _ = ref.slopes("silu", z)
        dz = g * d1
        size = g.abs() * (24 * U * s1 + 1.2 * zb) + U * dz.abs()
    assert ref.worst(db.detach(), dz.sum(0), (rows + 10) * U * dz.abs().sum(0) + 1.01 * size.sum(0) + 1e-30) <= 1.0
    say(f"bias alone, gated {gated}, create_graph {create_graph}: {used} bytes")
    # dz (rows x N) and, of the sums, at most 128 partial rows
    assert used <= 4 * (rows * N + 130 * N) + (1 << 16)


@pytest.mark.parametrize("bias_trained,weight_trained", [(True, False), (False, True), (True, True), (False, False)])
def test_frozen_parameters(bias_trained, weight_trained):
    """Only what is trained gets a gradient, and the one that it gets with
    everything trained (the bias' to the order of its sum)."""
    block = _block()
    x, w, b, r = _randn(1, 300, 64), _randn(2, 80, 64, scale=0.125), _randn(3, 80), _randn(4, 300, 80)
    g = _randn(5, 300, 80)
    every = [t.clone().requires_grad_(True) for t in (x, w, b, r)]
    full = torch.autograd.grad(block.linear_act(*every[:3], "gelu", every[3]), every, g)
    some = [t.clone().requires_grad_(on) for t, on in zip((x, w, b, r), (True, weight_trained, bias_trained, False))]
    y = block.linear_act(*some[:3], "gelu", some[3])
    leaves = [t for t in some if t.requires_grad]
    for create in (False, True):
        for t, got in zip(leaves, torch.autograd.grad(y, leaves, g, create_graph=create, retain_graph=True)):
            at = next(i for i, s in enumerate(some) if s is t)
            assert float((got - full[at]).abs().max()) <= 64 * U * float(full[at].abs().max()) + (300 * U * float(g.abs().sum(0).max()) if at == 2 else 0)


def test_rows_far_apart():
    """A slice whose rows lie further apart than the weight gradient's kernel
    reaches: as input, as output gradient, and in wgrad."""
    block = _block()
    far = torch.zeros(5, 17_000_000, device="cuda:0")
    far[:, :112] = _randn(1, 5, 112)
    x, g = far[:, :64], far[:, 64:112]
    for K in (64, 8):
        w, b = _randn(2, 48, K, scale=0.125).requires_grad_(True), _randn(3, 48).requires_grad_(True)
        got = torch.autograd.grad(block.linear_act(x[:, :K], w, b, "silu"), (w, b), g)
        want = torch.autograd.grad(block.linear_act(x[:, :K].contiguous(), w, b, "silu"), (w, b), g.contiguous())
        assert all(torch.equal(u, v) for u, v in zip(got, want))
        y = block.linear_act(x[:, :K], w, b)
        assert torch.equal(torch.autograd.grad(y, w, g)[0], block.wgrad(g.contiguous(), x[:, :K].contiguous())[0])
    assert all(torch.equal(u, v) for u, v in zip(block.wgrad(g, x, True), block.wgrad(g.contiguous(), x.contiguous(), True)))
    wg = _randn(4, 96, 64, scale=0.125).requires_grad_(True)
    got = torch.autograd.grad(block.gated_linear(x, wg), wg, g)[0]
    assert torch.equal(got, torch.autograd.grad(block.gated_linear(x.contiguous(), wg), wg, g.contiguous())[0])
    far_x = far[:, 100:100 + 300]   # wider than the fused pass takes
    w = _randn(5, 48, 300, scale=0.05).requires_grad_(True)
    got = torch.autograd.grad(block.linear_act(far_x, w, None, "gelu"), w, g)[0]
    assert torch.equal(got, torch.autograd.grad(block.linear_act(far_x.contiguous(), w, None, "gelu"), w, g.contiguous())[0])


def test_rows_of_one_stride_are_not_copied():
    """A slice of the last dimension of a 3-D tensor has rows a fixed distance
    apart: read where they are."""
    block = _block()
    wide = _randn(1, 40, 50, 600)
    x = wide[:, :, 44:556]
    want = block.layer_norm(x.contiguous())
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    y = block.layer_norm(x)
    assert torch.cuda.max_memory_allocated() - before <= 4 * y.numel() + 512
    assert torch.equal(y, want)
    w = _randn(2, 48, 512, scale=0.05)
    for view in (wide[:, :, 44:556], wide[::2, :, 44:556], wide[:, ::2, 44:556], wide[:, :1, 44:556], wide[:1, :, 44:556],
                 wide.transpose(0, 1)[:, :, 44:556], wide[:1].expand(3, 50, 600)[:, :, 44:556], wide[:, 0, 44:556], wide[0, 0, 44:556],
                 wide[:0, :, 44:556], wide[:, :, None, 44:556]):
        flat = view.contiguous()
        assert torch.equal(block.layer_norm(view), block.layer_norm(flat))
        assert torch.equal(block.linear_act(view, w, None, "silu", mode="BF16X9"), block.linear_act(flat, w, None, "silu", mode="BF16X9"))


@pytest.mark.parametrize("mode", ["AUTO", "BF16X9", "NATIVE_F32"])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("shape", [(150, 64), (3, 50, 64)])
def test_force_training_of_the_linear_layer(mode, name, shape):
    """Energy and force loss through one linear layer with its activation and
    residual, against torch float64.  A second-order gradient passes about ten
    FP32 operations, each with a relative error near 1e-7 in the norm: 1e-5
    leaves a factor of ten."""
    block = _block()
    x, w, b = _randn(1, *shape), _randn(2, 48, 64, scale=0.125), _randn(3, 48)
    r, c = _randn(4, *shape[:-1], 48), _randn(5, *shape[:-1], 48)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b, r)]
    wide = [t.double().requires_grad_(True) for t in (x, w, b, r)]

    def loss_of(f, ts):
        y = f(*ts)
        energy = (torch.tanh(y) * c.to(y.dtype)).sum()
        force = torch.autograd.grad(energy, [ts[0], ts[3]], create_graph=True)
        return y, *force, energy + (force[0] ** 2).sum() + (force[1] ** 3).sum()

    got = loss_of(lambda x, w, b, r: block.linear_act(x, w, b, name, r, mode=mode), leaves)
    want = loss_of(lambda x, w, b, r: ref.act(name, x @ w.t() + b) + r, wide)
    pairs = list(zip(("y", "force", "residual's force"), got, want))
    pairs += list(zip(("x", "w", "b", "r"), torch.autograd.grad(got[3], leaves), torch.autograd.grad(want[3], wide)))
    for what, a, e in pairs:
        assert a.shape == e.shape
        rel = float((a.detach().double() - e.detach()).norm() / e.detach().norm())
        say(f"linear {mode} {name} {len(shape)}-D {what}: {rel:.2e}")
        assert rel <= 1e-5, (what, rel)


@pytest.mark.parametrize("gated", [False, True])
def test_force_training_of_the_bias_alone(gated):
    """With the weight frozen the bias' second-order gradient is the one that
    it has with everything trained, to the order of its sums."""
    block = _block()
    x, w, b = _randn(1, 300, 64), _randn(2, 96, 64, scale=0.125), _randn(3, 96)

    def grads(weight_trained):
        xs, ws, bs = x.clone().requires_grad_(True), w.clone().requires_grad_(weight_trained), b.clone().requires_grad_(True)
        y = block.gated_linear(xs, ws, bs) if gated else block.linear_act(xs, ws, bs, "gelu")
        fx, fb = torch.autograd.grad((y * y).sum(), (xs, bs), create_graph=True)
        return torch.autograd.grad((fx ** 2).sum() + (fb ** 2).sum(), (bs, xs))

    for got, want in zip(grads(False), grads(True)):
        # sums of 300 rows, each rounding below 2^-24 of the terms' sum
        assert float((got - want).norm()) <= 600 * U * float(want.norm())
