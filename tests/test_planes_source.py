"""How planes know their weight (no GPU needed: it is a matter of storages and
version counters)."""
import copy
import pickle

import pytest
import torch

import emulated_fp32_matrix_amd as emu
from emulated_fp32_matrix_amd import block


def test_the_same_matrix_passes_and_others_do_not():
    w = torch.nn.Parameter(torch.randn(6, 6))
    source = emu.WeightSource(w.detach())
    for same in (w, w.detach(), w[:], w.view(6, 6), w.t().t()):
        source.check(same)
    for other in (w.t(), w.detach().clone(), torch.randn(6, 6), w[:5], torch.randn(7, 6)[1:]):
        with pytest.raises(ValueError, match="another"):
            source.check(other)
    with torch.no_grad():
        w.mul_(2.0)
    with pytest.raises(ValueError, match="changed"):
        source.check(w)
    emu.WeightSource(w).check(w)


def test_a_freed_weight_is_never_taken_for_another():
    for _ in range(50):
        w = torch.randn(64, 64)
        source = emu.WeightSource(w)
        del w
        with pytest.raises(ValueError, match="another"):
            source.check(torch.randn(64, 64))


def test_inference_tensors():
    with torch.inference_mode():
        w = torch.randn(4, 4)
        emu.WeightSource(w).check(w)


def test_copies_and_pickles_of_planes():
    """A copy shares the reference to the storage (which is counted), a pickle
    has none and is refused where a weight is passed."""
    w = torch.randn(8, 4)
    pb = emu.PresplitB(torch.zeros(16, dtype=torch.uint8), 8, 4, "BF16X9", emu.WeightSource(w))
    for _ in range(3):
        for other in (copy.copy(pb), copy.deepcopy(pb)):
            other.source.check(w)
    assert pickle.loads(pickle.dumps(pb)).source is None
    with pytest.raises(ValueError, match="which weight"):
        block.linear_act(torch.zeros(2, 4), w, planes=pickle.loads(pickle.dumps(pb)))
    del pb, other
    copy.deepcopy(w)
