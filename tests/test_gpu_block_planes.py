"""Weights split beforehand are held to the weight that a call passes with
them: its storage, layout and version."""
import pytest
import torch

import emulated_fp32_matrix_amd as emu
from emulated_fp32_matrix_amd import block

pytestmark = pytest.mark.gpu


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to("cuda:0")


def test_planes_of_the_other_orientation_are_refused():
    """A square weight: planes of x W are not those of x W^T."""
    x, w = _randn(1, 40, 64), _randn(2, 64, 64)
    with pytest.raises(ValueError, match="planes"):
        block.linear_act(x, w, planes=emu.presplit_b(w))
    want = block.linear_act(x, w, mode="BF16X9")
    assert torch.equal(block.linear_act(x, w, mode="BF16X9", planes=emu.presplit_b(w, trans_b=True)), want)
    # the same matrix, given as op(B) = B: the planes of x W^T
    wt = w.t().contiguous()
    assert torch.equal(block.linear_act(x, wt.t(), mode="BF16X9", planes=emu.presplit_b(wt)), want)


def test_planes_of_a_weight_that_changed_are_refused():
    x, w = _randn(1, 40, 64), torch.nn.Parameter(_randn(2, 96, 64))
    pb, pg = emu.presplit_b(w, trans_b=True), block.presplit_gated(w)
    with torch.no_grad():
        block.linear_act(x, w, planes=pb)
        block.gated_linear(x, w, planes=pg)
        w.add_(1.0)
        for call in (lambda: block.linear_act(x, w, planes=pb), lambda: block.gated_linear(x, w, planes=pg)):
            with pytest.raises(ValueError, match="changed"):
                call()


def test_planes_of_another_weight_are_refused():
    x, w, other = _randn(1, 40, 64), _randn(2, 96, 64), _randn(3, 96, 64)
    both = _randn(4, 192, 64)
    pb, pg, first = emu.presplit_b(w, trans_b=True), block.presplit_gated(w), emu.presplit_b(both[:96], trans_b=True)
    for call in (lambda: block.linear_act(x, other, planes=pb), lambda: block.gated_linear(x, other, planes=pg),
                 lambda: block.linear_act(x, both[96:], planes=first)):
        with pytest.raises(ValueError, match="another weight"):
            call()
    block.linear_act(x, both[:96], planes=first)
    # a weight that took the freed one's place in memory is another one
    at = w.data_ptr()
    del w
    w = _randn(5, 96, 64)
    assert w.data_ptr() == at
    with pytest.raises(ValueError, match="another weight"):
        block.linear_act(x, w, planes=pb)


def test_planes_fit_every_view_of_their_weight():
    """A parameter, its detached view and a slice that is the whole of it are
    the same weight; planes do not keep the weight's memory."""
    x, w = _randn(1, 40, 64), torch.nn.Parameter(_randn(2, 96, 64))
    want = block.linear_act(x, w.detach(), mode="BF16X9")
    pb = emu.presplit_b(w.detach(), trans_b=True)
    for view in (w, w.detach(), w[:], w.view(96, 64)):
        assert torch.equal(block.linear_act(x, view, mode="BF16X9", planes=pb), want)
    with torch.inference_mode():   # (no version counter there)
        v = _randn(2, 96, 64)
        pv = emu.presplit_b(v, trans_b=True)
        assert torch.equal(block.linear_act(x, v, mode="BF16X9", planes=pv), want)
    before = torch.cuda.memory_allocated()
    big = torch.zeros(4096, 1024, device="cuda:0")
    p = emu.presplit_b(big, trans_b=True)
    held = p.planes.numel()
    del big
    assert torch.cuda.memory_allocated() - before <= held + 512


def test_sgemm_presplit_needs_no_weight():
    """Planes alone are enough where the call passes no weight."""
    x, w = _randn(1, 40, 64), _randn(2, 96, 64)
    want = emu.sgemm(x, w, mode="BF16X9", trans_b=True)
    pb = emu.presplit_b(w, trans_b=True)
    w.zero_()
    del w
    assert torch.equal(emu.sgemm_presplit(x, pb, ksplit=1), want)
