"""The weight gradient with whole numbers: every sum is exact in FP32 (below
2^24), so a row left out, counted twice or put in the wrong place shows, at any
number of rows.  Plain, and with the activation's or the gated product's
backward pass inside, in both widths of the kernel's tile."""
import ctypes
import random

import pytest
import torch

import block_reference as ref
import wgrad_plan
from gpu_helpers import say

# rows, M, N: widths off the tiles' edges, last slabs partly filled
WIDE = [(1234, 777, 1300), (700, 2050, 1030), (2000, 1300, 390), (60, 2050, 2100)]
NARROW = [(20000, 36, 64), (4099, 130, 259), (1000, 256, 256), (33, 129, 127), (100001, 40, 130), (300, 1030, 1028)]
GATED_WIDE = [(1234, 389, 1300), (700, 1026, 1030), (60, 1026, 2100)]
GATED_NARROW = [(20000, 18, 64), (4099, 65, 259), (33, 64, 127)]


def _block():
    from emulated_fp32_matrix_amd import block

    return block


def _whole(seed, most, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).float()


def test_plan_of_the_shapes_below():
    """The model of the plan agrees with the library's workspaces, and the
    shapes below reach the tiles that they are named for."""
    lib, need = _block()._lib, ctypes.c_size_t(0)
    rng = random.Random(5)
    seen = set()
    for _ in range(3000):
        rows, M, N = (int(2 ** rng.uniform(0, t)) for t in (17, 12, 12))
        for gated, query in ((False, lib.emu_wgrad_workspace), (True, lib.emu_wgrad_gated_workspace)):
            assert query(rows, M, N, ctypes.byref(need)) == 0
            assert need.value == wgrad_plan.workspace(rows, M, N, gated), (rows, M, N, gated)
            wn, segs = wgrad_plan.plan(rows, M, N, gated)
            seen.add((wn, segs > 1))
    assert seen == {(2, False), (2, True), (4, False), (4, True)}
    for shapes, gated, wn in ((WIDE, False, 4), (NARROW, False, 2), (GATED_WIDE, True, 4), (GATED_NARROW, True, 2)):
        plans = [wgrad_plan.plan(*s, gated) for s in shapes]
        assert all(p[0] == wn for p in plans) and any(p[1] > 1 for p in plans) and any(p[1] == 1 for p in plans), plans


def test_the_comparison_sees_a_lost_row_and_rounded_operands():
    """On the CPU, with the mistake in the reference: one row less, or operands
    rounded to 8 bits, changes the whole-number result."""
    for rows, M, N in ((20000, 36, 64), (4099, 130, 259)):
        dz, x = _whole(1, 400, rows, M), _whole(2, 1, rows, N)
        want = dz.double().t() @ x.double()
        assert float(want.abs().max()) < 2**24
        for row in (0, rows // 2, rows - 1):
            keep = torch.arange(rows) != row
            assert not torch.equal(dz[keep].double().t() @ x[keep].double(), want)
        assert not torch.equal(dz.bfloat16().double().t() @ x.double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,M,N", WIDE + NARROW)
def test_wgrad_is_exact_on_whole_numbers(rows, M, N):
    block = _block()
    small = min(400, (2**24 - 1) // rows)
    for mz, mx in ((small, 1), (1, small)):
        dz, x = _whole(1, mz, rows, M).cuda(), _whole(2, mx, rows, N).cuda()
        say(f"wgrad {rows}x{M}x{N}, plan {wgrad_plan.plan(rows, M, N)}, up to {mz} and {mx}")
        dw, db = block.wgrad(dz, x, want_db=True)
        assert torch.equal(dw.double(), dz.double().t().contiguous() @ x.double())
        assert torch.equal(db.double(), dz.double().sum(0))


def _fused(rows, M, N, dy, z, act, x, gated):
    """emu_wgrad_act / emu_wgrad_gated with leading dimensions wider than the
    rows; what lies between the rows of dZ and dW stays."""
    block = _block()
    lib, need, wide = block._lib, ctypes.c_size_t(0), 2 * M if gated else M
    query = lib.emu_wgrad_gated_workspace if gated else lib.emu_wgrad_workspace
    call = lib.emu_wgrad_gated if gated else lib.emu_wgrad_act
    assert query(rows, M, N, ctypes.byref(need)) == 0
    ws = torch.empty(max(need.value, 1), dtype=torch.uint8, device="cuda:0")
    dz = torch.full((rows, wide + 3), 7.0, device="cuda:0")
    dw = torch.full((wide, N + 5), 7.0, device="cuda:0")
    db = torch.empty(wide, device="cuda:0")
    assert call(rows, M, N, dy.data_ptr(), dy.stride(0), z.data_ptr(), z.stride(0), act, dz.data_ptr(), wide + 3, x.data_ptr(),
                x.stride(0), dw.data_ptr(), N + 5, db.data_ptr(), ws.data_ptr(), need.value,
                torch.cuda.current_stream().cuda_stream or None) == 0
    assert bool((dz[:, wide:] == 7.0).all()) and bool((dw[:, N:] == 7.0).all())
    return dz[:, :wide], dw[:, :N], db


def _flat(name, seed, *shape):
    """Pre-activations where act is 0 or whole and act' 0 or 1 (both but for
    tails below 2^-60): +-50, for tanh 0 and 50."""
    up = torch.randint(0, 2, shape, generator=torch.Generator().manual_seed(seed)).float()
    return 50.0 * up if name == "tanh" else 100.0 * up - 50.0


TAIL = 2.0**-30   # of the exact value: rows times tails below 2^-60


@pytest.mark.gpu
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("rows,M,N", WIDE + NARROW[:4])
def test_wgrad_act_is_exact_on_whole_numbers(rows, M, N, name):
    block = _block()
    dy, x = _whole(1, 2, rows, M + 1).cuda()[:, :M], _whole(2, 2, rows, N + 2).cuda()[:, :N]
    z = _flat(name, 3, rows, M).cuda()
    slope = torch.ones_like(z) if name == "identity" else (z == 0 if name == "tanh" else z > 0).float()
    want = (dy * slope).double()
    say(f"wgrad_act {name} {rows}x{M}x{N}, plan {wgrad_plan.plan(rows, M, N)}")
    dz, dw, db = _fused(rows, M, N, dy, z, block.ACTIVATIONS[name], x, False)
    for got, exact in ((dz, want), (dw, want.t().contiguous() @ x.double()), (db, want.sum(0))):
        assert float((got.double() - exact).abs().max()) <= TAIL
    assert torch.equal(dz, block.act_grad(dy.contiguous(), z, name))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("rows,F,N", GATED_WIDE + GATED_NARROW)
def test_wgrad_gated_is_exact_on_whole_numbers(rows, F, N, name):
    block = _block()
    dh, x = _whole(1, 1, rows, F + 1).cuda()[:, :F], _whole(2, 1, rows, N + 2).cuda()[:, :N]
    g, u = _flat(name, 3, rows, F).cuda(), _whole(4, 2, rows, F).cuda()
    slope = torch.ones_like(g) if name == "identity" else (g == 0 if name == "tanh" else g > 0).float()
    value = g if name == "identity" else (g > 0).float() * (1.0 if name == "tanh" else 50.0)
    want = torch.cat([dh * u * slope, dh * value], dim=1).double()
    say(f"wgrad_gated {name} {rows}x{F}x{N}, plan {wgrad_plan.plan(rows, F, N, True)}")
    dz, dw, db = _fused(rows, F, N, dh, torch.cat([g, u], dim=1), block.ACTIVATIONS[name], x, True)
    for got, exact in ((dz, want), (dw, want.t().contiguous() @ x.double()), (db, want.sum(0))):
        assert float((got.double() - exact).abs().max()) <= TAIL


@pytest.mark.gpu
@pytest.mark.parametrize("name", ref.ACTS)
def test_fused_backward_passes_at_ordinary_values(name):
    """dZ of the fused passes, in the wide tiles, is the element-wise passes'
    bit for bit, and dW the plain product's of that dZ where both run the same
    plan."""
    block = _block()
    for rows, M, N in WIDE[:2]:
        g = torch.Generator().manual_seed(rows)
        dy, z, x = (torch.randn(rows, n, generator=g).cuda() for n in (M, M, N))
        dz, dw, db = _fused(rows, M, N, dy, 3.0 * z, block.ACTIVATIONS[name], x, False)
        assert torch.equal(dz, block.act_grad(dy, 3.0 * z, name))
        dw2, db2 = block.wgrad(dz.contiguous(), x, want_db=True)
        assert torch.equal(dw, dw2) and torch.equal(db, db2)
    for rows, F, N in GATED_WIDE[:2]:
        g = torch.Generator().manual_seed(rows)
        dh, z, x = (torch.randn(rows, n, generator=g).cuda() for n in (F, 2 * F, N))
        dz, dw, db = _fused(rows, F, N, dh, 3.0 * z, block.ACTIVATIONS[name], x, True)
        want = torch.empty(rows, 2 * F, device="cuda:0")
        assert block._lib.emu_gated_backward(rows, F, dh.data_ptr(), F, (3.0 * z).data_ptr(), 2 * F, block.ACTIVATIONS[name],
                                             want.data_ptr(), 2 * F, torch.cuda.current_stream().cuda_stream or None) == 0
        assert torch.equal(dz, want)
