"""Products of very many columns: the routes of one launch end where a launch's
threads would pass 2^32."""
import ctypes

import pytest
import torch

import emulated_fp32_matrix_amd as emu
from emulated_fp32_matrix_amd import block

LIMIT = 1 << 26


def test_one_launch_routes_end_before_a_launch_does():
    route = ctypes.c_int(-1)
    lib = block._lib
    for N in (LIMIT + 1, 1 << 27, (1 << 30) - 5, 1 << 30):
        for M, K in ((1, 4), (1, 64), (17, 4), (1, 1)):
            assert lib.emu_sgemm_act_route(1, M, N, K, ctypes.byref(route)) == 0 and route.value == 0, (M, N, K)
    for N in (1000, 4096):
        assert lib.emu_sgemm_act_route(1, 1, N, 4, ctypes.byref(route)) == 0 and route.value != 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [LIMIT - 3, LIMIT + 5, 2 * LIMIT + 3])
@pytest.mark.parametrize("mode", ["AUTO", "BF16X1", "NATIVE_F32"])
def test_very_wide_products(N, mode):
    """Whole numbers: exact in every mode."""
    w = torch.randint(-8, 9, (N, 4), device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(1)).float()
    b = (torch.arange(N, device="cuda:0") % 7).float()
    x = torch.tensor([[1.0, -2.0, 3.0, 5.0]], device="cuda:0")
    z = w[:, 0] - 2.0 * w[:, 1] + 3.0 * w[:, 2] + 5.0 * w[:, 3] + b
    assert torch.equal(block.linear_act(x, w, b, "relu", mode=mode)[0], torch.relu(z))
    F = N // 2
    got = block.gated_linear(x, w[:2 * F], b[:2 * F], "relu", mode=mode)[0]
    assert torch.equal(got, torch.relu(z[:F]) * z[F:2 * F])


@pytest.mark.gpu
def test_very_wide_without_inputs():
    """K = 0: the bias, its activation and the residual."""
    N = LIMIT + 6
    b = (torch.arange(N, device="cuda:0") % 9).float() - 4.0
    r = (torch.arange(N, device="cuda:0") % 5).float()[None]
    x, w = torch.zeros(1, 0, device="cuda:0"), torch.zeros(N, 0, device="cuda:0")
    assert torch.equal(block.linear_act(x, w, b, "relu", r)[0], torch.relu(b) + r[0])
    assert torch.equal(block.gated_linear(x, w, b, "relu")[0], torch.relu(b[:N // 2]) * b[N // 2:])
    assert bool((block.linear_act(x, w) == 0).all())
