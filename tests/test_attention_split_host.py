"""The three pieces that the attention kernels split their operands into, and
the six of nine products that they keep (csrc/emu_attn_split.h): what is left
out, against what include/emu_attention.h says of it.  No GPU needed."""
import os
import re

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def pieces(x):
    """hi, mid, lo of FP32 values, each in 64 bits."""
    r = lambda t: t.to(torch.bfloat16).to(torch.float32)   # to nearest even
    hi = r(x)
    mid = r(x - hi)
    lo = (x - hi) - mid
    assert torch.equal(r(lo), lo)
    return [t.double() for t in (hi, mid, lo)]


def stated():
    """The header's bound of what the six products leave out of one."""
    text = " ".join(open(os.path.join(ROOT, "include", "emu_attention.h")).read().replace("*", " ").split())
    n, = re.findall(r"leave out (?:at most|less than) 2\^-(\d+) of a product", text)
    return 2.0 ** -int(n)


def left_out(a, b):
    (ah, am, al), (bh, bm, bl) = pieces(a), pieces(b)
    kept = al * bh + ah * bl + am * bm + am * bh + ah * bm + ah * bh
    exact = a.double() * b.double()
    # (64 bits hold the terms and their sums here: 48 bits and a few more)
    return ((exact - kept) / exact).abs()


def test_the_pair_that_loses_most():
    """mid near 2^-8 and lo near 2^-17 of a value just above a power of two:
    the two products mid lo that are left out come near 2^-24."""
    a = torch.tensor([1 + 2.0 ** -8 - 2.0 ** -17 - 2.0 ** -23], dtype=torch.float32)
    lost = float(left_out(a, a)[0])
    assert 1.9 * 2.0 ** -25 < lost < 2.0 ** -24
    assert lost <= stated()


def test_every_mantissa_stays_below_the_stated_bound():
    """What is left out of a b is at most (m_a l_b + l_a m_b + l_a l_b) |a b|,
    m and l the pieces' shares: by their largest over all mantissas, and for the
    squares as they are."""
    bits = torch.arange(1 << 23, dtype=torch.int32) + 0x3F800000   # 1 .. 2; other binades scale
    x = bits.view(torch.float32)
    hi, mid, lo = pieces(x)
    assert torch.equal(hi + mid + lo, x.double())
    m, l = float((mid / x.double()).abs().max()), float((lo / x.double()).abs().max())
    assert 2 * m * l + l * l <= stated()
    assert float(left_out(x, x).max()) <= 2 * m * l + l * l
