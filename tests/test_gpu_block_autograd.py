"""The block operators inside autograd: outputs changed in place."""
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
