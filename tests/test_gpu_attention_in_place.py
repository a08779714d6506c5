"""Outputs in the place of inputs, where include/emu_attention.h allows them:
rotary positions and dropout through the C ABI; and the block's dropout where
the block itself does not train."""
import pytest
import torch

from emulated_fp32_matrix_amd import attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("batch,tokens,heads,dim,part", [(1, 1, 1, 2, 2), (2, 5, 3, 7, 6), (3, 40, 4, 64, 24), (2, 300, 8, 32, 32),
                                                         (700, 9, 2, 96, 66), (1, 3, 2, 2600, 2500), (2, 9, 70, 50, 0)])
@pytest.mark.parametrize("inverse", [0, 1])
def test_rotary(layout, batch, tokens, heads, dim, part, inverse):
    gen = torch.Generator(device=DEV).manual_seed(dim)
    x = torch.randn(batch, tokens, heads, dim, generator=gen, device=DEV)
    positions = torch.randint(-9999, 9999, (batch, tokens), generator=gen, device=DEV)
    turns = attention.rotary_turns([0.9 ** i for i in range(part // 2)], DEV)

    def run(at, y):
        view = attention._Heads(at.data_ptr(), at.stride(0), at.stride(1), at.stride(2))
        assert attention._lib.emu_rotary(batch, tokens, heads, dim, view, positions.data_ptr(), tokens, 1, turns.data_ptr(), part // 2,
                                         attention.LAYOUTS[layout], 1.25, inverse, y.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream) == 0
        return y

    want = run(x, torch.empty_like(x))
    if not inverse:
        assert torch.equal(want, attention.rotary(x, positions, turns, layout, 1.25))
    here = x.clone()
    assert torch.equal(run(here, here), want)


@pytest.mark.parametrize("rows,cols,ld", [(1, 13, 13), (9, 8, 8), (9, 8, 12), (9, 7, 7), (9, 7, 11), (40, 33, 40), (300, 256, 256)])
@pytest.mark.parametrize("place", ["x", "x, with a residual", "residual"])
def test_dropout(rows, cols, ld, place):
    gen = torch.Generator(device=DEV).manual_seed(cols)
    x, r = (torch.randn(rows, ld, generator=gen, device=DEV) for _ in range(2))
    seed = torch.tensor([77, -3], device=DEV)
    residual = None if place == "x" else r

    def run(x, r, y):
        assert attention._lib.emu_dropout(rows, cols, x.data_ptr(), ld, 0.3, seed.data_ptr(), None if r is None else r.data_ptr(), ld,
                                          y.data_ptr(), ld, torch.cuda.current_stream().cuda_stream) == 0
        return y

    want = run(x, residual, torch.full_like(x, 5.0))
    assert torch.equal(want[:, :cols], attention.dropout(x[:, :cols], 0.3, seed, None if residual is None else r[:, :cols]))
    assert bool((want[:, cols:] == 5.0).all())
    kept = x.clone() if place != "residual" else r.clone()
    got = run(kept, residual, kept) if place != "residual" else run(x, kept, kept)
    assert torch.equal(got[:, :cols], want[:, :cols])
    assert torch.equal(got[:, cols:], (x if place != "residual" else r)[:, cols:])


@pytest.mark.parametrize("tokens", [10, 70])
def test_dropout_sampled_in_a_block_that_does_not_train(tokens):
    torch.manual_seed(3)
    layer = attention.EmuCrossAttention(32, 2, dropout=0.25, device=DEV).eval()
    x = torch.randn(2, tokens, 32, device=DEV)
    whole = layer(x).detach()
    assert torch.equal(whole, layer(x))
    layer.drop.train()
    a, b = layer(x).detach(), layer(x).detach()
    assert not torch.equal(a, b)
    moved = (a - x) != 0
    assert 0.6 < float(moved.float().mean()) < 0.9
    # kept elements are the block's own over the kept share: roundings of two sums and the scale
    assert float(((a - x) - (whole - x) * (4 / 3))[moved].abs().max()) <= 8 * 2.0 ** -24 * float(x.abs().max() + (whole - x).abs().max())
    layer.train()
    layer.drop.eval()
    assert torch.equal(layer(x), whole)   # (neither drops: one call and the same)
