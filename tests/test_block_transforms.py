"""The block operators under what does not run torch's backward graph:
forward-mode derivatives, tracers and function transforms.  Their kernels are
no torch operators, so a tangent would go missing and a recorded program would
return memory that nothing writes; every such call is refused, before anything
else is looked at (so most of it shows on the CPU)."""
import pytest
import torch
import torch.autograd.forward_ad as fw
from torch.fx.experimental.proxy_tensor import make_fx

from emulated_fp32_matrix_amd import block


def _case(device):
    g = torch.Generator().manual_seed(1)
    t = {k: torch.randn(*s, generator=g).to(device) for k, s in
         {"x": (5, 8), "w": (6, 8), "b": (6,), "r": (5, 6), "nw": (8,), "nb": (8,), "dz": (5, 6)}.items()}
    calls = {
        "layer_norm": (lambda t: block.layer_norm(t["x"], t["nw"], t["nb"]), ("x", "nw", "nb")),
        "linear_act": (lambda t: block.linear_act(t["x"], t["w"], t["b"], "silu", t["r"]), ("x", "w", "b", "r")),
        "gated_linear": (lambda t: block.gated_linear(t["x"], t["w"], t["b"]), ("x", "w", "b")),
        "wgrad": (lambda t: block.wgrad(t["dz"], t["x"])[0], ("dz", "x")),
        "act_grad": (lambda t: block.act_grad(t["dz"], t["r"], "tanh"), ("dz", "r")),
    }
    return t, calls


DEVICES = ["cpu", pytest.param("cuda:0", marks=pytest.mark.gpu)]


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("recorded", [False, True])
def test_forward_mode_is_refused_at_every_input(device, recorded):
    t, calls = _case(device)
    if recorded:
        t = {k: v.requires_grad_(True) for k, v in t.items()}
    for name, (f, inputs) in calls.items():
        for at in inputs:
            with fw.dual_level():
                dual = dict(t)
                dual[at] = fw.make_dual(t[at].detach().clone(), torch.ones_like(t[at]))
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    f(dual)
                with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                    f(dual)


@pytest.mark.parametrize("device", DEVICES)
def test_tracers_are_refused(device):
    t, calls = _case(device)
    for name, (f, inputs) in calls.items():
        x = t[inputs[0]]
        g = lambda v: f({**t, inputs[0]: v})
        with pytest.raises(NotImplementedError, match="traced"):
            torch.jit.trace(g, (x,), check_trace=False)
        for mode in ("real", "fake"):
            with pytest.raises(NotImplementedError, match="traced"):
                make_fx(g, tracing_mode=mode, _allow_non_fake_inputs=True)(x)
        with pytest.raises(NotImplementedError):
            torch.func.functionalize(g)(x)


@pytest.mark.parametrize("device", DEVICES)
def test_function_transforms_are_refused(device):
    t, calls = _case(device)
    for name, (f, inputs) in calls.items():
        x = t[inputs[0]]
        g = lambda v: f({**t, inputs[0]: v})
        with pytest.raises(NotImplementedError):
            torch.func.jvp(g, (x,), (torch.ones_like(x),))
        with pytest.raises(NotImplementedError):
            torch.func.grad(lambda v: g(v).sum())(x)
        with pytest.raises(NotImplementedError):
            torch.func.vmap(g)(torch.stack([x, x]))


def test_tensors_with_their_own_dispatch_are_refused():
    from torch._subclasses.fake_tensor import FakeTensorMode

    t, calls = _case("cpu")
    with FakeTensorMode() as mode:
        fake = mode.from_tensor(t["x"])
        with pytest.raises(NotImplementedError):
            block.layer_norm(fake)
    with pytest.raises(NotImplementedError, match="plain tensors"):
        block.layer_norm(fake)


def test_other_modes_and_parameters_are_not_refused():
    """What sees no kernel and needs none passes the check (these tensors are
    then refused for their device): parameters, a mode that counts operators."""
    from torch.utils.flop_counter import FlopCounterMode

    x = torch.nn.Parameter(torch.zeros(3, 8))
    with pytest.raises(TypeError):
        block.layer_norm(x)
    with FlopCounterMode(display=False), pytest.raises(TypeError):
        block.layer_norm(x)


@pytest.mark.gpu
def test_a_gradient_with_a_tangent_is_refused():
    """Forward over reverse: the backward pass of an ordinary call, given a
    gradient that carries a tangent."""
    t, calls = _case("cuda:0")
    for name in ("layer_norm", "linear_act", "gated_linear"):
        f, inputs = calls[name]
        leaves = {k: t[k].clone().requires_grad_(True) for k in inputs}
        y = f({**t, **leaves})
        with fw.dual_level():
            g = fw.make_dual(torch.ones_like(y), torch.ones_like(y))
            with pytest.raises(NotImplementedError, match="forward-mode"):
                torch.autograd.grad(y, list(leaves.values()), g)
