"""Captured calls whose inputs lead out of the capture: refused in the forward
pass (the captured backward pass would end the process), at every function and
through views.  Nothing here captures a backward pass of a refused call."""
import pytest
import torch

from emulated_fp32_matrix_amd import block

pytestmark = pytest.mark.gpu


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to("cuda:0")


def _capture(f):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


CALLS = {
    "wgrad": lambda x, w, z: block.wgrad(x, z)[0],
    "act_grad": lambda x, w, z: block.act_grad(x, x, "silu"),
    "a transposed weight": lambda x, w, z: block.linear_act(z, w.t()),
    "a reshaped input": lambda x, w, z: block.layer_norm(x.view(8, 5, 16)),
    "a slice of a weight": lambda x, w, z: block.gated_linear(z, w[2:8]),
    "a bias made from a leaf": lambda x, w, z: block.linear_act(z, w.detach(), 2.0 * w[0]),
    "a residual of a leaf": lambda x, w, z: block.linear_act(z.detach(), w.detach(), None, "silu", x + 1.0),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_living_results_are_refused(name):
    f = CALLS[name]
    x, w = _randn(1, 40, 16).requires_grad_(True), _randn(2, 16, 16).requires_grad_(True)
    z = _randn(3, 40, 16)
    kept = f(x, w, z)
    with pytest.raises(RuntimeError, match="earlier call on another stream"):
        _capture(lambda: f(x, w, z))
    torch.cuda.synchronize()
    want = kept.detach().clone()
    del kept
    g, out = _capture(lambda: f(x, w, z).detach())
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_an_input_made_outside_is_refused():
    """h was made before the capture: a backward pass that reaches it leaves
    the capture.  Detached, or made inside, it may be captured."""
    x = _randn(1, 40, 16).requires_grad_(True)
    h = 2.0 * x
    with pytest.raises(RuntimeError, match="detach"):
        _capture(lambda: block.layer_norm(h))
    torch.cuda.synchronize()
    want = block.layer_norm(h.detach())
    cot = _randn(2, 40, 16)
    g, out = _capture(lambda: block.layer_norm(h.detach()))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del h

    def step():
        y = block.layer_norm(2.0 * x)
        return [y.detach(), *torch.autograd.grad(y, x, cot)]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g, out = _capture(step)
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_streams_of_one_capture_are_one():
    """A branch on a second stream that the capture forked and joined."""
    x, w = _randn(1, 40, 16).requires_grad_(True), _randn(2, 16).requires_grad_(True)
    side = torch.cuda.Stream()

    def forward():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            h = block.layer_norm(x, w)
        here.wait_stream(side)
        return block.layer_norm(h, w).detach()

    want = forward().clone()
    torch.cuda.synchronize()
    g, out = _capture(forward)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_without_gradients_nothing_is_refused():
    x, w, z = _randn(1, 40, 16).requires_grad_(True), _randn(2, 16, 16).requires_grad_(True), _randn(3, 40, 16)
    h = 2.0 * x
    kept = [f(x, w, z) for f in CALLS.values()]
    with torch.no_grad():
        want = block.layer_norm(h)
        g, out = _capture(lambda: block.layer_norm(h))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(kept) == len(CALLS)
