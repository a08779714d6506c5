"""The attention block's module with its operators replaced by plain torch (no
GPU needed): which of its parts run, in which modes."""
import pytest
import torch

from emulated_fp32_matrix_amd import attention


@pytest.fixture
def plain(monkeypatch):
    """The module's operators in plain torch; dropout's calls are recorded."""
    calls = []

    def linear_act(x, w, b=None, residual=None, mode="AUTO"):
        y = torch.nn.functional.linear(x, w, b)
        return y if residual is None else y + residual

    def cross_attention(q, k, v, key_bias=None, key_mask=None, lengths=None, scale=None):
        p = torch.softmax(torch.einsum("bqhd,bkhd->bhqk", q, k) / q.shape[-1] ** 0.5, -1)
        return torch.einsum("bhqk,bkhd->bqhd", p, v)

    def dropout(x, p, seed, residual=None):
        calls.append((p, residual is not None))
        return 2.0 * x if residual is None else 2.0 * x + residual   # (told from the undropped sum)

    monkeypatch.setattr(attention, "linear_act", linear_act)
    monkeypatch.setattr(attention, "cross_attention", cross_attention)
    monkeypatch.setattr(attention, "dropout", dropout)
    monkeypatch.setattr(attention, "dropout_seed", lambda device, generator=None: torch.zeros(2, dtype=torch.int64))
    return calls


@pytest.mark.parametrize("block_trains", [True, False])
@pytest.mark.parametrize("drop_trains", [True, False])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_dropout_goes_by_its_own_mode(plain, block_trains, drop_trains, p):
    """The dropout module's mode decides, as it does for the module alone: with
    layer.eval() and layer.drop.train() dropout is sampled."""
    torch.manual_seed(0)
    layer = attention.EmuCrossAttention(16, 2, dropout=p, norm=False)
    layer.train(block_trains)
    layer.drop.train(drop_trains)
    x = torch.randn(2, 3, 16)
    y = layer(x)
    dropped = drop_trains and p > 0.0
    assert plain == ([(p, True)] if dropped else [])
    layer.drop.eval()
    inner = layer(x) - x
    assert torch.allclose(y, x + (2.0 if dropped else 1.0) * inner, atol=1e-6)
