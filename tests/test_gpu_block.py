"""GPU parity of the transformer-block operators (include/emu_block.h and
emulated_fp32_matrix_amd.block) against 64-bit plain forms, element by element
within bounds that count roundings (tests/block_reference.py)."""
import ctypes

import pytest
import torch

import block_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu
U = ref.U
MODES = ("AUTO", "BF16X9", "BF16X6", "NATIVE_F32", "BF16X3")


def _block():
    from emulated_fp32_matrix_amd import block

    return block


def _randn(seed, *shape, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to("cuda:0")


def _within(label, got, want):
    value, bound = want
    w = ref.worst(got, value, bound)
    say(f"{label}: {w:.3f} of the bound")
    assert w <= 1.0, f"{label}: {w:.3f} of the bound"


# ---- layer norm --------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 2), (33, 63), (5, 64), (17, 127), (300, 256), (40, 257), (33, 512), (9, 513), (130, 1023),
               (7, 2048), (6, 3000), (5, 4096), (4, 8191), (3, 16384), (20000, 65)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("affine", ["both", "weight", "none"])
def test_layer_norm_and_its_derivatives(rows, cols, affine):
    block = _block()
    eps = 1e-5
    x = (_randn(rows + cols, rows, cols, scale=2.0) + _randn(1, rows, 1)).requires_grad_(True)
    w = _randn(2, cols, scale=0.2, shift=1.0).requires_grad_(True) if affine != "none" else None
    b = _randn(3, cols).requires_grad_(True) if affine == "both" else None
    dy = _randn(4, rows, cols).requires_grad_(True)
    v = _randn(5, rows, cols)
    say(f"layer norm {rows}x{cols} {affine}")
    y = block.layer_norm(x, w, b, eps)
    _within("y", y.detach(), ref.norm(x, w, b, eps))
    with torch.no_grad():
        assert torch.equal(block.layer_norm(x, w, b, eps), y)
    leaves = [t for t in (x, w, b) if t is not None]
    grads = torch.autograd.grad(y, leaves, dy, create_graph=True)
    want = ref.norm_backward(x, w, dy, eps)
    for name, got, one in zip(("dx", "dweight", "dbias"), grads, want):
        _within(name, got.detach(), one)
    # second order: v on dx, p on dweight, q on dbias
    p = _randn(6, cols) if w is not None else None
    q = _randn(7, cols) if b is not None else None
    inner = [t for t in (dy, x, w) if t is not None]
    got2 = torch.autograd.grad(grads, inner, [t for t in (v, p, q) if t is not None], retain_graph=True)
    want2 = ref.norm_backward2(x, w, dy, v, p, q, eps)
    for name, got, one in zip(("gdy", "gx", "gweight"), got2, want2):
        _within(name, got, one)
    if w is not None:   # only the weight's gradient is differentiated
        got2 = torch.autograd.grad(grads[1], inner, p, allow_unused=True)
        want2 = ref.norm_backward2(x, w, dy, None, p, None, eps)
        for name, got, one in zip(("gdy of dweight", "gx of dweight", "gw of dweight"), got2, want2):
            _within(name, got, one)


def test_layer_norm_matches_differences():
    """Central differences of the 64-bit form at a few entries, for the HIP
    gradient of sum(g * y)."""
    block = _block()
    x = _randn(1, 5, 40).requires_grad_(True)
    w, b, g = _randn(2, 40), _randn(3, 40), _randn(4, 5, 40)
    (dx,) = torch.autograd.grad(block.layer_norm(x, w, b), x, g)
    h = 1e-4
    for r, c in ((0, 0), (2, 17), (4, 39)):
        e = torch.zeros(5, 40, dtype=torch.float64, device="cuda:0")
        e[r, c] = h
        f = lambda t: float((ref.norm(t, w, b, 1e-5)[0] * g.double()).sum())
        d = (f(x.double() + e) - f(x.double() - e)) / (2 * h)
        # central differences are off by h^2 / 6 times a third derivative of
        # order 10, and by 64-bit roundings of a sum of 200 terms over 2 h
        assert abs(float(dx[r, c]) - d) <= 1e-6 * max(1.0, abs(d))


def test_layer_norm_strides_shapes_and_empty_rows():
    block = _block()
    wide = _randn(1, 50, 300)
    w, b = _randn(2, 200), _randn(3, 200)
    x = wide[:, 40:240]                                  # row stride 300, 16-byte aligned start
    _within("column slice", block.layer_norm(x, w, b), ref.norm(x, w, b, 1e-5))
    x = wide[::3, 1:201]                                 # row stride 900, unaligned start
    _within("row and column slice", block.layer_norm(x, w, b), ref.norm(x, w, b, 1e-5))
    x = _randn(4, 200, 30).t()                           # columns strided: copied
    _within("transposed", block.layer_norm(x, w, b), ref.norm(x, w, b, 1e-5))
    x = _randn(5, 2, 3, 200)
    y = block.layer_norm(x, w, b)
    assert y.shape == x.shape
    _within("4-D", y.reshape(6, 200), ref.norm(x.reshape(6, 200), w, b, 1e-5))
    x = _randn(6, 1, 200).expand(7, 200)
    _within("expanded", block.layer_norm(x, w, b), ref.norm(x, w, b, 1e-5))
    x = torch.zeros(0, 200, device="cuda:0", requires_grad=True)
    wg = w.clone().requires_grad_(True)
    y = block.layer_norm(x, wg, b)
    assert y.shape == (0, 200)
    gx, gw = torch.autograd.grad(y, (x, wg), torch.zeros_like(y))
    assert gx.shape == (0, 200) and bool((gw == 0).all())


def test_layer_norm_special_rows():
    """A constant row gives the bias; rows with an infinity or a NaN stay NaN
    without touching their neighbours."""
    block = _block()
    for cols in (64, 200, 3000):
        x = _randn(cols, 6, cols)
        x[1] = 3.25
        x[3, 5] = float("inf")
        x[4, 7] = float("nan")
        w, b = _randn(1, cols), _randn(2, cols)
        y = block.layer_norm(x, w, b)
        assert torch.equal(y[1], b)
        assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4]).all())
        for r in (0, 2, 5):
            assert torch.equal(y[r], block.layer_norm(x[r:r + 1], w, b)[0])


def test_layer_norm_offset_row_means():
    """Rows whose mean is far larger than their deviation: the squared
    deviations are summed, not moments subtracted."""
    block = _block()
    x = _randn(1, 64, 256, scale=1.0, shift=4096.0)
    _within("offset", block.layer_norm(x), ref.norm(x, None, None, 1e-5))


def test_layer_norm_in_place_and_untouched_surroundings():
    """Raw calls: y over x, dx over dy, leading dimensions wider than the row;
    what lies between the rows stays as it was."""
    block = _block()
    lib, s = block._lib, torch.cuda.current_stream().cuda_stream or None
    for rows, cols, ld in ((37, 61, 70), (20, 256, 260), (5, 2500, 2501)):
        buf = _randn(rows, rows, ld)
        x = buf.clone()
        stats = torch.empty(2, rows, device="cuda:0")
        want = ref.norm(buf[:, :cols], None, None, 1e-5)
        assert lib.emu_layer_norm(rows, cols, x.data_ptr(), ld, None, None, 1e-5, x.data_ptr(), ld, stats[0].data_ptr(),
                                  stats[1].data_ptr(), s) == 0
        _within(f"in place {rows}x{cols}", x[:, :cols], want)
        assert torch.equal(x[:, cols:], buf[:, cols:])
        g = _randn(7, rows, ld)
        dx = g.clone()
        assert lib.emu_layer_norm_backward(rows, cols, dx.data_ptr(), ld, buf.data_ptr(), ld, None, stats[0].data_ptr(),
                                           stats[1].data_ptr(), dx.data_ptr(), ld, None, None, None, 0, s) == 0
        _within(f"dx in place {rows}x{cols}", dx[:, :cols], ref.norm_backward(buf[:, :cols], None, g[:, :cols], 1e-5)[0])
        assert torch.equal(dx[:, cols:], g[:, cols:])


# ---- activations ------------------------------------------------------------------------

def _points():
    z = torch.cat([torch.linspace(-12, 12, 4801), torch.linspace(-100, 100, 401), torch.tensor(
        [0.0, -0.0, 1e-30, -1e-30, 1e-6, -1e-6, 1e4, -1e4, 1e20, -1e20, 3e38, -3e38])])
    return z.to("cuda:0")


@pytest.mark.parametrize("name", ref.ACTS)
def test_activation_values_and_slopes(name):
    """act through a product with the identity (exact in BF16X9), its slopes
    through the element-wise passes."""
    block = _block()
    z = _points()
    n = z.numel()
    one = torch.eye(1, device="cuda:0")
    zz = z.reshape(n, 1)
    small = zz[zz.abs() <= 1e4].reshape(-1, 1)
    for mode in ("BF16X9", "AUTO"):
        y = block.linear_act(small, one, None, activation=name, mode=mode)
        z64 = small.double()
        _within(f"{name} {mode}", y, (ref.act(name, z64), ref.act_bound(name, z64) + 2.0**-140))
    d1, d2, s1, s2 = ref.slopes(name, zz.double())
    dy, v = _randn(1, n, 1), _randn(2, n, 1)
    tiny = 2.0**-110   # where exponentials and reciprocals fall below 2^-126
    got = block.act_grad(dy, zz, name)
    _within(f"{name}'", got, (dy.double() * d1, dy.double().abs() * (24 * U * s1.nan_to_num(0, 0, 0) + tiny)))
    dyg, zg = dy.clone().requires_grad_(True), small.clone().requires_grad_(True)
    m = small.shape[0]
    out = block.act_grad(dyg[:m], zg, name)
    gdy, gz = torch.autograd.grad(out, (dyg, zg), v[:m])
    d1, d2, s1, s2 = ref.slopes(name, small.double())
    _within(f"{name}' again", gdy[:m], (v[:m].double() * d1, v[:m].double().abs() * (24 * U * s1 + tiny)))
    scale = (v[:m] * dy[:m]).double()
    _within(f"{name}''", gz, (scale * d2, scale.abs() * (48 * U * s2 + tiny)))


@pytest.mark.parametrize("name", ref.ACTS)
def test_activation_keeps_nan(name):
    block = _block()
    z = torch.tensor([[float("nan"), 1.0, float("nan"), -1.0]], device="cuda:0")
    dy = torch.ones_like(z)
    y = block.linear_act(torch.tensor([[float("nan")]], device="cuda:0"), torch.ones(3, 1, device="cuda:0"),
                         activation=name)
    assert bool(torch.isnan(y).all())
    if name not in ("identity", "relu"):
        d = block.act_grad(dy, z, name)
        assert torch.isnan(d).tolist() == [[True, False, True, False]]


# ---- linear layer with activation and residual ---------------------------------------------

LINEAR_SHAPES = [(1, 1, 1), (1, 512, 256), (16, 40, 64), (17, 33, 31), (33, 768, 100), (64, 130, 257), (65, 128, 64),
                 (129, 127, 36), (200, 771, 387), (300, 256, 96), (257, 516, 32)]


def _linear_case(M, N, K, residual, seed=0):
    x = _randn(seed + 1, M, K)
    w = _randn(seed + 2, N, K, scale=K**-0.5)
    b = _randn(seed + 3, N)
    r = _randn(seed + 4, M, N) if residual else None
    return x, w, b, r


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
@pytest.mark.parametrize("mode", MODES)
def test_linear_act_forward(M, N, K, mode):
    block = _block()
    for i, name in enumerate(ref.ACTS):
        x, w, b, r = _linear_case(M, N, K, i % 2 == 0, seed=i)
        bias = b if i != 2 else None
        say(f"linear {M}x{N}x{K} {mode} {name}")
        y = block.linear_act(x, w, bias, activation=name, residual=r, mode=mode)
        z, zb = ref.product(x.double(), w.double(), bias, mode)
        want = ref.act(name, z)
        bound = ref.act_bound(name, z) + 1.2 * zb
        if r is not None:
            want = want + r.double()
            bound = bound + U * want.abs()
        _within("y", y, (want, bound * 1.01 + 1e-30))


@pytest.mark.parametrize("M,N,K", [(1, 512, 256), (33, 70, 64), (129, 127, 36), (200, 771, 387), (1000, 256, 128)])
@pytest.mark.parametrize("mode,name", [("AUTO", "silu"), ("BF16X9", "gelu"), ("BF16X6", "tanh"), ("NATIVE_F32", "gelu_tanh"),
                                       ("AUTO", "identity"), ("AUTO", "relu")])
def test_linear_act_gradients(M, N, K, mode, name):
    block = _block()
    x, w, b, r = _linear_case(M, N, K, True)
    if name == "relu":   # keep z away from the kink
        x, w, b = x.abs(), w.abs() * torch.sign(_randn(9, N, 1)), b * 0
    leaves = [t.requires_grad_(True) for t in (x, w, b, r)]
    g = _randn(5, M, N)
    say(f"linear gradients {M}x{N}x{K} {mode} {name}")
    y = block.linear_act(x, w, b, activation=name, residual=r, mode=mode)
    dx, dw, db, dr = torch.autograd.grad(y, leaves, g)
    x64, w64, g64 = x.detach().double(), w.detach().double(), g.double()
    z, zb = ref.product(x64, w64, b, mode)
    d1, d2, s1, s2 = ref.slopes(name, z)
    dz = g64 * d1
    curve = 0.0 if name in ("identity", "relu") else 1.2   # |act''| <= 1.2
    dzb = g64.abs() * (24 * U * s1 + curve * zb) + U * dz.abs()
    if name == "identity":
        dzb = 0 * dzb
    delta = ref.DELTA[mode]
    _within("dx", dx, (dz @ w64, ((2 * N + 10) * U + delta) * (dz.abs() @ w64.abs()) + 1.01 * (dzb @ w64.abs()) + 1e-30))
    _within("dW", dw, (dz.t() @ x64, (2 * M + 10) * U * (dz.abs().t() @ x64.abs()) + 1.01 * (dzb.t() @ x64.abs()) + 1e-30))
    _within("db", db, (dz.sum(0), (M + 10) * U * dz.abs().sum(0) + 1.01 * dzb.sum(0) + 1e-30))
    assert torch.equal(dr, g)


def test_linear_act_matches_sgemm_in_the_explicit_modes():
    """The product is emu_sgemm's bit for bit (bias and residual added after
    it, one rounding each), and z, kept for the backward pass, changes no
    output."""
    import emulated_fp32_matrix_amd as emu

    block = _block()
    for M, N, K in ((300, 260, 100), (130, 128, 64), (70, 36, 387)):
        x, w, b, r = _linear_case(M, N, K, True)
        for mode in ("BF16X9", "BF16X6", "BF16X3", "BF16X1", "NATIVE_F32"):
            t = emu.sgemm(x, w, mode=mode, trans_b=True)
            want = (t + b) + r
            got = block.linear_act(x, w, b, residual=r, mode=mode)
            assert torch.equal(got, want), (M, N, K, mode)
            y = block.linear_act(x, w, b, activation="silu", mode=mode)
            x2 = x.clone().requires_grad_(True)
            assert torch.equal(block.linear_act(x2, w, b, activation="silu", mode=mode), y)


def _raw_linear(x, w, trans_b, bias, act, mode, z=None):
    """emu_sgemm_act with op(B) = w or w^T and wider leading dimensions than
    the rows; what lies between the rows of C and Z stays."""
    import emulated_fp32_matrix_amd as emu

    block = _block()
    lib, (M, K) = block._lib, x.shape
    N = w.shape[0] if trans_b else w.shape[1]
    c = torch.full((M, N + 3), 7.0, device="cuda:0")
    zz = torch.full((M, N + 5), 7.0, device="cuda:0")
    need = ctypes.c_size_t(0)
    args = (int(trans_b), M, N, K, x.data_ptr(), x.stride(0))
    assert lib.emu_sgemm_act_workspace(*args, 0, emu.MODES[mode], ctypes.byref(need)) == 0
    ws = torch.empty(max(need.value, 1), dtype=torch.uint8, device="cuda:0")
    assert lib.emu_sgemm_act(*args, w.data_ptr(), w.stride(0), None, bias.data_ptr(), act, zz.data_ptr(), N + 5, None, N,
                             c.data_ptr(), N + 3, emu.MODES[mode], ws.data_ptr(), need.value,
                             torch.cuda.current_stream().cuda_stream) == 0
    assert bool((c[:, N:] == 7.0).all()) and bool((zz[:, N:] == 7.0).all())
    return c[:, :N], zz[:, :N]


@pytest.mark.parametrize("mode", ["AUTO", "BF16X9", "BF16X6", "NATIVE_F32"])
def test_sgemm_act_both_layouts_of_b(mode):
    """B stored K x N and N x K give the same bits; Z is the product plus the
    bias, C its activation."""
    block = _block()
    for M, N, K in ((1, 70, 33), (40, 64, 128), (300, 260, 100), (150, 131, 387)):
        x, w, b, _ = _linear_case(M, N, K, False)
        c1, z1 = _raw_linear(x, w, True, b, 2, mode)
        c2, z2 = _raw_linear(x, w.t().contiguous(), False, b, 2, mode)
        assert torch.equal(c1, c2) and torch.equal(z1, z2), (M, N, K)
        assert torch.equal(z1, block.linear_act(x, w, b, mode=mode))
        assert torch.equal(c1, block.linear_act(x, w, b, activation="silu", mode=mode))


@pytest.mark.parametrize("mode", ["AUTO", "BF16X9", "BF16X6"])
def test_planes_bitwise(mode):
    """Weights split once beforehand: the results of the calls that split."""
    import emulated_fp32_matrix_amd as emu

    block = _block()
    split = "BF16X9" if mode == "AUTO" else mode
    for M in (30000,) if mode == "AUTO" else (100, 300, 6144):   # (AUTO takes the FP32 kernel for fewer rows)
        x, w, b, r = _linear_case(M, 200, 96, True)
        pb = emu.presplit_b(w, mode=split, trans_b=True)
        pg = block.presplit_gated(w, split)
        assert torch.equal(block.linear_act(x, w, b, "gelu", r, mode=mode, planes=pb),
                           block.linear_act(x, w, b, "gelu", r, mode=mode)), M
        assert torch.equal(block.gated_linear(x, w, b, mode=mode, planes=pg), block.gated_linear(x, w, b, mode=mode)), M
    x1 = x[:3]   # few rows: AUTO without planes runs FP32, with them the emulation
    got = block.linear_act(x1, w, b, mode=mode, planes=pb)
    z, zb = ref.product(x1.double(), w.double(), b, mode)
    _within("few rows with planes", got, (z, zb))
    with pytest.raises(ValueError):
        block.linear_act(x, w, b, mode="BF16X3", planes=pb)
    with pytest.raises(ValueError):
        block.linear_act(x, w[:100], None, mode=mode, planes=pb)
    with pytest.raises(TypeError):
        block.gated_linear(x, w, b, mode=mode, planes=pb)


# one row, rows and columns past a tile's end, k past a chunk's, widths below
# four, tiles of 32 x 32 and of 64 x 64, fewer and more of them than CUs
FEW = [(1, 4, 4), (1, 3, 7), (5, 2, 3), (33, 5, 6), (31, 37, 129), (65, 96, 64), (64, 64, 127), (130, 70, 387),
       (257, 513, 34), (1000, 640, 130), (700, 500, 261), (2000, 260, 72),
       (4109, 300, 66), (1100, 1102, 131)]


@pytest.mark.parametrize("mode", ["BF16X9", "BF16X6", "BF16X3", "BF16X1"])
def test_few_rows_in_the_explicit_modes(mode):
    """One launch for few rows gives emu_sgemm's product bit for bit: both
    layouts of B, planes, z, the residual and the gated product; inf and NaN
    stay in their rows and columns."""
    import emulated_fp32_matrix_amd as emu

    block = _block()
    for M, N, K in FEW:
        x, w, b, r = _linear_case(M, N, K, True)
        t = emu.sgemm(x, w, mode=mode, trans_b=True)
        pb = emu.presplit_b(w, mode=mode, trans_b=True)
        say(f"{M}x{N}x{K} {mode}")
        assert torch.equal(block.linear_act(x, w, b, residual=r, mode=mode), (t + b) + r), (M, N, K)
        assert torch.equal(block.linear_act(x, w, b, residual=r, mode=mode, planes=pb), (t + b) + r), (M, N, K)
        for trans_b, op in ((True, w), (False, w.t().contiguous())):
            c, z = _raw_linear(x, op, trans_b, b, 0, mode)
            assert torch.equal(c, t + b) and torch.equal(z, t + b), (M, N, K, trans_b)
        F = N // 2
        wg, bg = w[:2 * F].contiguous(), b[:2 * F].contiguous()
        zz = (t + b)[:, :2 * F]
        want = torch.relu(zz[:, :F]) * zz[:, F:]
        assert torch.equal(block.gated_linear(x, wg, bg, "relu", mode=mode), want), (M, N, K)
        pg = block.presplit_gated(wg, mode)
        assert torch.equal(block.gated_linear(x, wg, bg, "relu", mode=mode, planes=pg), want), (M, N, K)
        xg = x.clone().requires_grad_(True)
        assert torch.equal(block.gated_linear(xg, wg, bg, "relu", mode=mode), want), (M, N, K)
    x, w, b, r = _linear_case(70, 70, 130, True)
    x[3, 5], x[40, 129], w[9, 0] = float("inf"), float("nan"), float("-inf")
    t = emu.sgemm(x, w, mode=mode, trans_b=True)
    c, z = _raw_linear(x, w, True, b, 0, mode)
    cn, _ = _raw_linear(x, w.t().contiguous(), False, b, 0, mode)
    bad = ~torch.isfinite(t)
    assert int(bad.sum()) == 2 * 70 + 68 and torch.equal(bad, ~torch.isfinite(c)) and torch.equal(bad, ~torch.isfinite(cn))
    assert torch.equal(c[~bad], (t + b)[~bad]) and torch.equal(cn[~bad], c[~bad])
    assert torch.equal(torch.isnan(t), torch.isnan(c)) and torch.equal(torch.isnan(c), torch.isnan(cn))


@pytest.mark.parametrize("M,N,K", [(40, 4096, 600), (129, 771, 387), (1000, 640, 260), (70, 64, 2050)])
def test_few_rows_in_auto(M, N, K):
    """AUTO's one launch against the 64-bit form, and with nine products (route
    2) BF16X9's bits; the gated product of the same weight."""
    block = _block()
    few = ctypes.c_int(-1)
    assert block._lib.emu_sgemm_act_route(1, M, N, K, ctypes.byref(few)) == 0
    say(f"{M}x{N}x{K}: route {few.value}")
    assert few.value != 0
    x, w, b, r = _linear_case(M, N, K, True)
    y = block.linear_act(x, w, b, "identity", r)
    if few.value == 2:
        assert torch.equal(y, block.linear_act(x, w, b, "identity", r, mode="BF16X9"))
    z, zb = ref.product(x.double(), w.double(), b, "AUTO")
    want = z + r.double()
    _within("sum", y, (want, 1.01 * (zb + U * want.abs())))
    F = N // 2
    wg, bg = w[:2 * F].contiguous(), b[:2 * F].contiguous()
    z, zb = ref.product(x.double(), wg.double(), bg, "AUTO")
    a, u, ab, ub = torch.relu(z[:, :F]), z[:, F:], zb[:, :F], zb[:, F:]
    _within("gated", block.gated_linear(x, wg, bg, "relu"), (a * u, 1.01 * (ab * (u.abs() + ub) + a * ub) + U * (a * u).abs() + 1e-30))


# (M, N, K): every tile split, the last round split, 64- and 128-row tiles, none
@pytest.mark.parametrize("M,N,K", [(6144, 1024, 1024), (768, 512, 4096), (700, 640, 2048), (3300, 1200, 1024), (2000, 640, 2048), (20000, 260, 160)])
def test_auto_plans(M, N, K):
    """The K split plans of AUTO with the fused epilogues: bit for bit
    emu_sgemm's product where the epilogue adds one rounding, and the gated
    projection against the linear one with its rows reordered."""
    import emulated_fp32_matrix_amd as emu

    block = _block()
    few = ctypes.c_int(-1)
    assert block._lib.emu_sgemm_act_route(1, M, N, K, ctypes.byref(few)) == 0
    say(f"{M}x{N}x{K}: plan {emu.select_plan(M, N, K)}, few rows {few.value}")
    assert few.value == 0 and emu.select_mode(M, N, K) == "BF16X9"
    x, w, b, r = _linear_case(M, N, K, True)
    t = emu.sgemm(x, w, mode="AUTO", trans_b=True)
    assert torch.equal(block.linear_act(x, w, b, residual=r), (t + b) + r)
    z, zb = ref.product(x.double(), w.double(), b, "AUTO")
    y = block.linear_act(x, w, b, "gelu", r)
    want = ref.act("gelu", z) + r.double()
    _within("gelu", y, (want, 1.01 * (ref.act_bound("gelu", z) + 1.2 * zb + U * want.abs())))
    # [g | u] = t + b: the gated product of the same weight, bit for bit where
    # the plan splits whole rows of tiles (its tiles hold other columns)
    F = N // 2
    zz = t + b
    h = block.gated_linear(x, w, b, "relu")
    if emu.select_plan(M, N, K)[2] % -(-N // 128) == 0:
        assert torch.equal(h, torch.relu(zz[:, :F]) * zz[:, F:])
    a, u, ab, ub = torch.relu(z[:, :F]), z[:, F:], zb[:, :F], zb[:, F:]
    _within("gated", h, (a * u, 1.01 * (ab * (u.abs() + ub) + a * ub) + U * (a * u).abs() + 1e-30))
    xg = x.clone().requires_grad_(True)
    h2 = block.gated_linear(xg, w, b, "relu")   # keeps Z
    assert torch.equal(h2, h)


def test_linear_act_strides_batches_and_empty():
    block = _block()
    x = _randn(1, 2, 3, 5, 64)
    w, b = _randn(2, 40, 64, scale=0.125), _randn(3, 40)
    res = _randn(4, 2, 3, 5, 40)
    y = block.linear_act(x, w, b, activation="gelu", residual=res)
    assert y.shape == (2, 3, 5, 40)
    assert torch.equal(y.reshape(30, 40), block.linear_act(x.reshape(30, 64), w, b, "gelu", res.reshape(30, 40)))
    wide = _randn(5, 300, 100)
    for xs in (wide[:, 4:68], wide[::2, 3:67], wide[:64].t()[4:68].t()):
        _y = block.linear_act(xs, w, b, "silu", mode="BF16X9")
        assert torch.equal(_y, block.linear_act(xs.contiguous(), w, b, "silu", mode="BF16X9"))
    ws = _randn(6, 40, 200)[:, 10:74]
    assert torch.equal(block.linear_act(wide[:, :64].contiguous(), ws, b), block.linear_act(wide[:, :64].contiguous(), ws.contiguous(), b))
    empty = torch.zeros(0, 64, device="cuda:0", requires_grad=True)
    wg = w.clone().requires_grad_(True)
    y = block.linear_act(empty, wg, b, "silu")
    assert y.shape == (0, 40)
    gx, gw = torch.autograd.grad(y, (empty, wg), torch.zeros_like(y))
    assert gx.shape == (0, 64) and bool((gw == 0).all())
    # no input features: the bias alone
    y = block.linear_act(torch.zeros(100, 0, device="cuda:0"), torch.zeros(40, 0, device="cuda:0"), b, "relu")
    assert torch.equal(y, torch.relu(b).expand(100, 40))


@pytest.mark.parametrize("mode", ["AUTO", "BF16X9"])
def test_linear_act_isolates_rows(mode):
    """A row with a NaN or an infinity leaves the others as they are."""
    block = _block()
    for M in (40, 200):
        x, w, b, r = _linear_case(M, 96, 64, True)
        want = block.linear_act(x, w, b, "silu", r, mode=mode)
        x2 = x.clone()
        x2[7, 3] = float("nan")
        x2[11, 5] = float("inf")
        got = block.linear_act(x2, w, b, "silu", r, mode=mode)
        keep = torch.ones(M, dtype=torch.bool, device="cuda:0")
        keep[7] = keep[11] = False
        assert torch.equal(got[keep], want[keep])
        assert bool(torch.isnan(got[7]).all()) and not bool(torch.isfinite(got[11]).any())


# ---- gated projection ---------------------------------------------------------------------------

GATED_SHAPES = [(1, 1, 1), (1, 512, 256), (16, 20, 64), (33, 31, 33), (64, 65, 100), (65, 64, 64), (129, 130, 36),
                (200, 387, 259), (300, 512, 96), (700, 48, 128)]


def _gated_reference(x, w, b, name, mode):
    z, zb = ref.product(x.double(), w.double(), b, mode)
    F = w.shape[0] // 2
    return z[:, :F], z[:, F:], zb[:, :F], zb[:, F:]


@pytest.mark.parametrize("M,F,K", GATED_SHAPES)
@pytest.mark.parametrize("mode", MODES)
def test_gated_forward(M, F, K, mode):
    block = _block()
    for i, name in enumerate(("silu", "gelu", "gelu_tanh", "tanh")):
        x, w, b, _ = _linear_case(M, 2 * F, K, False, seed=i)
        bias = b if i != 1 else None
        say(f"gated {M}x{F}x{K} {mode} {name}")
        h = block.gated_linear(x, w, bias, activation=name, mode=mode)
        g, u, gb, ub = _gated_reference(x, w, bias, name, mode)
        a = ref.act(name, g)
        ab = ref.act_bound(name, g) + 1.2 * gb
        _within("h", h, (a * u, 1.01 * (ab * (u.abs() + ub) + a.abs() * ub) + U * (a * u).abs() + 1e-30))


@pytest.mark.parametrize("M,F,K", [(1, 512, 256), (33, 31, 33), (129, 130, 36), (200, 387, 259), (700, 128, 128)])
@pytest.mark.parametrize("mode,name", [("AUTO", "silu"), ("BF16X6", "gelu_tanh"), ("NATIVE_F32", "gelu"), ("BF16X9", "tanh")])
def test_gated_gradients(M, F, K, mode, name):
    block = _block()
    x, w, b, _ = _linear_case(M, 2 * F, K, False)
    leaves = [t.requires_grad_(True) for t in (x, w, b)]
    dh = _randn(5, M, F)
    say(f"gated gradients {M}x{F}x{K} {mode} {name}")
    h = block.gated_linear(x, w, b, activation=name, mode=mode)
    dx, dw, db = torch.autograd.grad(h, leaves, dh)
    x64, w64, d64 = x.detach().double(), w.detach().double(), dh.double()
    g, u, gb, ub = _gated_reference(x.detach(), w.detach(), b, name, mode)
    a = ref.act(name, g)
    d1, _, s1, _ = ref.slopes(name, g)
    dz = torch.cat([d64 * u * d1, d64 * a], dim=1)
    dgb = d64.abs() * ((u.abs() + ub) * (24 * U * s1 + 1.2 * gb) + ub * d1.abs()) + 2 * U * dz[:, :F].abs()
    dub = d64.abs() * (ref.act_bound(name, g) + 1.2 * gb) + U * dz[:, F:].abs()
    dzb = torch.cat([dgb, dub], dim=1)
    delta = ref.DELTA[mode]
    _within("dx", dx, (dz @ w64, ((4 * F + 10) * U + delta) * (dz.abs() @ w64.abs()) + 1.01 * (dzb @ w64.abs()) + 1e-30))
    _within("dW", dw, (dz.t() @ x64, (2 * M + 10) * U * (dz.abs().t() @ x64.abs()) + 1.01 * (dzb.t() @ x64.abs()) + 1e-30))
    _within("db", db, (dz.sum(0), (M + 10) * U * dz.abs().sum(0) + 1.01 * dzb.sum(0) + 1e-30))


def test_gated_strides_batches_and_empty():
    block = _block()
    w, b = _randn(2, 80, 64, scale=0.125), _randn(3, 80)
    x = _randn(1, 4, 25, 64)
    h = block.gated_linear(x, w, b)
    assert h.shape == (4, 25, 40) and torch.equal(h.reshape(100, 40), block.gated_linear(x.reshape(100, 64), w, b))
    wide = _randn(5, 300, 100)
    for xs in (wide[:, 4:68], wide[::2, 3:67]):
        assert torch.equal(block.gated_linear(xs, w, b, mode="BF16X9"), block.gated_linear(xs.contiguous(), w, b, mode="BF16X9"))
    empty = torch.zeros(0, 64, device="cuda:0", requires_grad=True)
    wg = w.clone().requires_grad_(True)
    h = block.gated_linear(empty, wg, b)
    gx, gw = torch.autograd.grad(h, (empty, wg), torch.zeros_like(h))
    assert h.shape == (0, 40) and gx.shape == (0, 64) and bool((gw == 0).all())
    assert block.gated_linear(x, torch.zeros(0, 64, device="cuda:0")).shape == (4, 25, 0)


# ---- weight gradient ---------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,M,N", [(1, 1, 1), (31, 5, 7), (32, 128, 128), (33, 129, 127), (1000, 256, 256), (4099, 130, 259),
                                      (20000, 36, 64), (64, 700, 390), (300, 1030, 1028)])
def test_wgrad(rows, M, N):
    block = _block()
    dz, x = _randn(1, rows, M), _randn(2, rows, N)
    dw, db = block.wgrad(dz, x, want_db=True)
    d64, x64 = dz.double(), x.double()
    say(f"wgrad {rows}x{M}x{N}")
    _within("dW", dw, (d64.t() @ x64, (2 * rows + 10) * U * (d64.abs().t() @ x64.abs())))
    _within("db", db, (d64.sum(0), (rows / 16 + 80) * U * d64.abs().sum(0)))
    again, none = block.wgrad(dz, x)
    assert none is None and torch.equal(again, dw)
    wide = _randn(3, rows, M + N + 3)
    dzs, xs = wide[:, 1:1 + M], wide[:, 2 + M:2 + M + N]
    dws, dbs = block.wgrad(dzs, xs, want_db=True)
    assert torch.equal(dws, block.wgrad(dzs.contiguous(), xs.contiguous())[0])


def test_wgrad_refusals_and_empty():
    block = _block()
    dz, x = _randn(1, 10, 8), _randn(2, 11, 4)
    with pytest.raises(ValueError):
        block.wgrad(dz, x)
    with pytest.raises(ValueError):
        block.wgrad(dz[0], x)
    assert torch.equal(block.wgrad(dz.t(), x[:8])[0], block.wgrad(dz.t().contiguous(), x[:8])[0])   # strided: copied
    dw, db = block.wgrad(dz[:0], x[:0], want_db=True)
    assert dw.shape == (8, 4) and bool((dw == 0).all()) and bool((db == 0).all())
    dw, db = block.wgrad(dz, x[:10, :0], want_db=True)
    assert dw.shape == (8, 0)
    _within("db alone", db, (dz.double().sum(0), 90 * U * dz.double().abs().sum(0)))


# ---- the operators together ------------------------------------------------------------------------------

def _ffn64(ffn, x):
    p = {k: v.detach().double().requires_grad_(True) for k, v in ffn.named_parameters()}
    x64 = x.detach().double().requires_grad_(True)

    def run(t):
        n = torch.nn.functional.layer_norm(t, (t.shape[-1],), p["norm.weight"], p["norm.bias"], 1e-5)
        g, u = (n @ p["w_in"].t() + p["b_in"]).chunk(2, dim=-1)
        return t + (ref.act(ffn.activation, g) * u) @ p["out.weight"].t() + p["out.bias"]

    return run, p, x64


@pytest.mark.parametrize("mode,activation,rows", [("AUTO", "silu", 40), ("AUTO", "gelu", 400), ("BF16X6", "gelu_tanh", 400),
                                                  ("NATIVE_F32", "tanh", 130)])
def test_feed_forward_block_energy_and_force_loss(mode, activation, rows):
    """LayerNorm, gated projection and output layer with its residual as one
    block: y, the forces -dE/dx and the gradients of an energy + force loss
    against torch float64.  The relative errors of FP32 products of a few
    hundred terms are near 1e-7 each; a second-order gradient passes about
    twenty such operations one after the other: 1e-5 leaves a factor of five."""
    block = _block()
    torch.manual_seed(3)
    ffn = block.EmuGatedFFN(64, 96, activation=activation, mode=mode, device="cuda:0")
    with torch.no_grad():
        ffn.norm.weight.add_(0.1 * torch.randn_like(ffn.norm.weight))
        ffn.norm.bias.add_(0.1 * torch.randn_like(ffn.norm.bias))
        ffn.b_in.add_(0.1 * torch.randn_like(ffn.b_in))
    x = _randn(1, rows, 64).requires_grad_(True)
    c = _randn(2, rows, 64)

    def loss_of(fn, xx, cc):
        y = fn(xx)
        energy = (y * torch.tanh(y) * cc).sum()
        (force,) = torch.autograd.grad(energy, xx, create_graph=True)
        return y, force, energy / rows + (force**2).sum()

    y, f, loss = loss_of(ffn, x, c)
    params = dict(ffn.named_parameters())
    got = torch.autograd.grad(loss, list(params.values()) + [x])
    run, p64, x64 = _ffn64(ffn, x)
    y64, f64, loss64 = loss_of(run, x64, c.double())
    want = torch.autograd.grad(loss64, [p64[k] for k in params] + [x64])
    rel = lambda a, b: float((a.detach().double() - b.detach()).norm() / b.detach().norm())
    for name, a, b in [("y", y, y64), ("force", f, f64)] + list(zip(list(params) + ["x"], got, want)):
        e = rel(a, b)
        say(f"block {mode} {activation} {rows} rows {name}: {e:.2e}")
        assert e <= 1e-5, (name, e)


def test_third_derivative_is_refused():
    block = _block()
    x = _randn(1, 8, 16).requires_grad_(True)
    y = block.layer_norm(x).pow(2).sum()
    (g,) = torch.autograd.grad(y, x, create_graph=True)
    (h,) = torch.autograd.grad(g.pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(h.sum(), x)


def test_streams_and_interleaved_calls():
    """Calls issued at once on several streams, interleaved, give the results
    of the calls alone."""
    block = _block()
    cases = []
    for i, rows in enumerate((40, 500, 3000, 129)):
        x, w, b, r = _linear_case(rows, 128, 64, True, seed=10 * i)
        wg, bg = _randn(50 + i, 192, 64, scale=0.125), _randn(60 + i, 192)
        cases.append((x, w, b, r, wg, bg))

    def run(c):
        x, w, b, r, wg, bg = c
        n = block.layer_norm(x)
        return (block.linear_act(n, w, b, "silu", r, mode="BF16X9"), block.gated_linear(n, wg, bg), block.wgrad(r, n, True)[0])

    alone = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    for _ in range(3):
        for i, (s, c) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                outs[i].append(run(c))
    torch.cuda.synchronize()
    for one, many in zip(alone, outs):
        for got in many:
            assert all(torch.equal(a, b) for a, b in zip(one, got))


def test_host_threads_at_once():
    """Training steps from four host threads, each on its own stream: the
    gradients of the steps alone."""
    import threading

    block = _block()
    torch.manual_seed(5)
    ffns = [block.EmuGatedFFN(64, 96, device="cuda:0") for _ in range(4)]
    xs = [_randn(i, 150 + 400 * i, 64) for i in range(4)]

    def step(i):
        x = xs[i].clone().requires_grad_(True)
        y = ffns[i](x)
        return [t.detach() for t in (y, *torch.autograd.grad((y * y).sum(), [x, *ffns[i].parameters()]))]

    alone = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    got[i] = step(i)
            s.synchronize()
        except Exception as e:   # noqa: BLE001 (reported by the main thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for a, b in zip(alone, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_views_that_stand_for_a_negative():
    """The imaginary part of a conjugate is stored with the other sign."""
    block = _block()

    def negative(t):
        v = torch.complex(torch.zeros_like(t), t).conj().imag
        assert v.is_neg()
        return v

    x, w, b, r = _linear_case(40, 36, 64, True)
    for f in (lambda x, w, b, r: block.linear_act(x, w, b, "silu", r), lambda x, w, b, r: block.gated_linear(x, w, b),
              lambda x, w, b, r: block.layer_norm(r, b, b), lambda x, w, b, r: block.wgrad(r, x)[0]):
        assert torch.equal(f(negative(x), negative(w), negative(b), negative(r)), f(-x, -w, -b, -r))
    x1, x2 = x.clone().requires_grad_(True), x.clone().requires_grad_(True)
    block.layer_norm(x1).backward(negative(x))
    block.layer_norm(x2).backward(-x)
    assert torch.equal(x1.grad, x2.grad)


def test_one_tensor_in_several_places():
    """x as input and residual, one weight in two layers: their gradients add
    up."""
    block = _block()
    x, w = _randn(1, 200, 64).requires_grad_(True), _randn(2, 64, 64, scale=0.125).requires_grad_(True)
    g = _randn(3, 200, 64)
    y = block.linear_act(block.linear_act(x, w, None, "silu", x), w, None, "tanh", x)
    dx, dw = torch.autograd.grad(y, (x, w), g)
    x64, w64 = x.detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
    f = lambda t, name: ref.act(name, t @ w64.t()) + x64
    wx, ww = torch.autograd.grad(f(f(x64, "silu"), "tanh"), (x64, w64), g.double())
    # two layers of products of 64 terms: each relative error near 1e-7
    for got, want in ((dx, wx), (dw, ww)):
        assert float((got.double() - want).norm() / want.norm()) <= 2e-6


def test_graphs_replay_and_share_nothing():
    """Two captured graphs (inference, and a training step's forward and
    backward) replayed in turn, on two streams, with eager work between: each
    replay equals the eager result."""
    block = _block()
    torch.manual_seed(1)
    ffn = block.EmuGatedFFN(64, 128, device="cuda:0")
    x1, x2 = _randn(1, 700, 64), _randn(2, 900, 64).requires_grad_(True)
    g2 = _randn(3, 900, 64)
    params = list(ffn.parameters())

    def infer():
        with torch.no_grad():
            return [ffn(x1)]

    def train():
        y = ffn(x2)
        return [y, *torch.autograd.grad(y, params + [x2], g2)]

    # (no result keeps an eager autograd graph of the parameters alive)
    eager = [[t.detach().clone() for t in f()] for f in (infer, train)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in (infer, train):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(4):
        for out in outs:
            for t in out:
                t.detach().zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        block.gated_linear(_randn(turn, 2000, 64), _randn(9, 256, 64))   # eager work beside them
        torch.cuda.synchronize()
        for want, got in zip(eager, outs):
            for k, (a, b) in enumerate(zip(want, got)):
                assert torch.equal(a, b), (turn, k)


def test_capture_with_a_living_eager_graph_is_refused():
    """The parameters' gradient nodes of a living eager result belong to the
    eager stream; a captured backward pass through them would end the process,
    so the captured forward is refused before it."""
    block = _block()
    layer = block.EmuGatedFFN(32, 32, device="cuda:0")
    x = _randn(1, 100, 32)
    calls = [lambda: layer(x), lambda: layer.norm(x), lambda: layer.out(x), lambda: block.gated_linear(x, layer.w_in)]
    kept = [f() for f in calls]
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="earlier call on another stream"):
            with torch.cuda.graph(g):
                f()
    torch.cuda.synchronize()
    want = [t.detach().clone() for t in kept]
    del kept
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [f().detach() for f in calls]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_shape_and_device_refusals():
    block = _block()
    x, w, b = _randn(1, 4, 8), _randn(2, 6, 8), _randn(3, 6)
    cpu = torch.zeros(6)
    bad = [lambda: block.linear_act(x, w[:, :7], b), lambda: block.linear_act(x, w, b[:5]),
           lambda: block.linear_act(x, w, b, residual=_randn(4, 4, 5)), lambda: block.linear_act(x, w[0], b),
           lambda: block.gated_linear(x, w[:5], None), lambda: block.layer_norm(x, b),
           lambda: block.layer_norm(_randn(1, 2, block.LAYER_NORM_MAX_COLS + 1)),
           lambda: block.EmuLayerNorm(9, device="cuda:0")(x)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: block.linear_act(x, w, cpu), lambda: block.linear_act(x.double(), w.double()),
                 lambda: block.layer_norm(x.half()), lambda: block.linear_act(x, w.cpu())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        block.layer_norm(x, eps=-1.0)


def test_large_offsets():
    """More than 2^31 elements: rows past that offset are read and written
    where they belong (4.3 GiB arrays, a row of 4096 wide)."""
    block = _block()
    cols, rows = 4096, (1 << 31) // 4096 + 300
    x = torch.empty(rows, cols, device="cuda:0")
    x[:] = 1.0
    tail = _randn(1, 300, cols)
    x[-300:] = tail
    y = block.layer_norm(x)
    _within("last rows", y[-300:], ref.norm(tail, None, None, 1e-5))
    assert bool((y[: 1000] == 0).all())
    del y
    w = _randn(2, 8, cols, scale=cols**-0.5)
    x[:-300] = 0.0
    z = block.linear_act(x, w, None, "silu", mode="BF16X9")
    assert torch.equal(z[-300:], block.linear_act(tail, w, None, "silu", mode="BF16X9"))
    dz = torch.zeros(rows, 8, device="cuda:0")
    dz[-300:] = _randn(3, 300, 8)
    dw, db = block.wgrad(dz, x, True)
    want = dz[-300:].double().t() @ tail.double()
    _within("dW", dw, (want, 610 * U * (dz[-300:].double().abs().t() @ tail.double().abs())))
