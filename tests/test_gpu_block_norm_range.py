"""Layer norm of rows far from zero: the mean is good to its own rounding, and
columns past a row's end never enter a result."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
U = ref.U


def _block():
    from emulated_fp32_matrix_amd import block

    return block


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to("cuda:0")


@pytest.mark.parametrize("cols", [3, 63, 200, 256, 700, 1000, 2500, 5000, 16000])
def test_constant_rows(cols):
    """x - mean(x) is zero in a constant row, whatever its value: y is the
    bias, the deviations are zero and dx is the gradient less its mean."""
    block = _block()
    eps = 1e-5
    values = torch.tensor([0.1, -3.3, 1000003.0, -16777213.0, 1.2345679e12, -9.8765434e25, 3.3333333e-20], device="cuda:0")
    x = values[:, None].expand(len(values), cols).contiguous()
    w, b = _randn(1, cols), _randn(2, cols)
    stats = torch.empty(2, len(values), device="cuda:0")
    y = torch.empty_like(x)
    assert block._lib.emu_layer_norm(len(values), cols, x.data_ptr(), cols, w.data_ptr(), b.data_ptr(), eps, y.data_ptr(), cols,
                                     stats[0].data_ptr(), stats[1].data_ptr(), torch.cuda.current_stream().cuda_stream or None) == 0
    assert torch.equal(stats[0], values)
    assert torch.equal(y, b.expand_as(x))
    xg, wg = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    dy = _randn(3, len(values), cols)
    dx, dw = torch.autograd.grad(block.layer_norm(xg, wg, b, eps), (xg, wg), dy)
    assert bool((dw == 0).all())
    a = dy.double() * w.double()
    want = (a - a.mean(-1, keepdim=True)) * eps**-0.5
    # the sums and products of ref.norm_backward with xhat = 0
    bound = 192 * U * eps**-0.5 * (a.abs() + a.abs().mean(-1, keepdim=True))
    assert float(((dx.double() - want).abs() / bound).max()) <= 1.0


def test_mean_to_its_own_rounding():
    """A large offset under a small spread: the mean kept for the backward pass
    is the exact one to a unit in its last place."""
    block = _block()
    for cols in (100, 256, 1023, 4097):
        x = 4096.0 + _randn(cols, 64, cols)
        stats = torch.empty(2, 64, device="cuda:0")
        y = torch.empty_like(x)
        assert block._lib.emu_layer_norm(64, cols, x.data_ptr(), cols, None, None, 1e-5, y.data_ptr(), cols, stats[0].data_ptr(),
                                         stats[1].data_ptr(), torch.cuda.current_stream().cuda_stream or None) == 0
        mu = x.double().mean(-1)
        # half a unit of the sum's rounding, and the sum of the centred row:
        # 64 additions of terms near 1, 2^-18 of the offset's unit (2^-11)
        assert float((stats[0].double() - mu).abs().max()) <= 0.51 * 2.0**-11


@pytest.mark.parametrize("cols", [50, 100, 200])
def test_columns_past_the_end_stay_out(cols):
    """Where mean times reciprocal deviation overflows, the columns that a
    lane holds past the row's end must not turn the row's sums into NaN."""
    block = _block()
    x = torch.full((3, cols), 2.0**120, device="cuda:0")
    x[1] = _randn(1, cols)
    xg = x.clone().requires_grad_(True)
    w = _randn(2, cols).requires_grad_(True)
    dy = _randn(3, 3, cols)
    dx, dw = torch.autograd.grad(block.layer_norm(xg, w, None), (xg, w), dy)
    a = dy.double() * w.detach().double()
    want = (a - a.mean(-1, keepdim=True)) * 1e-5**-0.5
    bound = 192 * U * 1e-5**-0.5 * (a.abs() + a.abs().mean(-1, keepdim=True))
    for r in (0, 2):
        assert bool(torch.isfinite(dx[r]).all())
        assert float(((dx[r].double() - want[r]).abs() / bound[r]).max()) <= 1.0
    value, bnd = ref.norm_backward(x[1:2], w.detach(), dy[1:2], 1e-5)[0]
    assert ref.worst(dx[1:2], value, bnd) <= 1.0
    value, bnd = ref.norm_backward(x[1:2], w.detach(), dy[1:2], 1e-5)[1]
    assert ref.worst(dw, value, bnd) <= 1.0   # (xhat is zero in the other rows)


def test_means_that_are_not_finite():
    """An infinity, a NaN or a sum past FP32's range: the mean that the FP32
    formula gives is kept, and the row's y is NaN; its neighbours are as alone."""
    block = _block()
    inf = float("inf")
    for cols in (100, 256, 3000):
        x = _randn(cols, 6, cols)
        x[1] = 3e38
        x[2] = -3e38
        x[3, 7] = inf
        x[4, 9] = float("nan")
        stats = torch.empty(2, 6, device="cuda:0")
        y = torch.empty_like(x)
        assert block._lib.emu_layer_norm(6, cols, x.data_ptr(), cols, None, None, 1e-5, y.data_ptr(), cols, stats[0].data_ptr(),
                                         stats[1].data_ptr(), torch.cuda.current_stream().cuda_stream or None) == 0
        mean = stats[0].tolist()
        assert mean[1] == inf and mean[2] == -inf and mean[3] == inf and mean[4] != mean[4]
        assert bool(torch.isnan(y[1:5]).all())
        for r in (0, 5):
            assert torch.equal(y[r], block.layer_norm(x[r:r + 1])[0])
