"""Angles of far positions at frequencies of any size below 2^26, on the GPU,
against position * frequency reduced in 90 decimal digits."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

from _paged import U, assert_close
from _rope import T, TINY

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _two_pi():
    """By Machin's formula."""
    def arctan_of_one_over(n):
        term, total, k = Decimal(1) / n, Decimal(1) / n, 1
        while abs(term) > Decimal(10) ** -88:
            term /= -n * n
            k += 2
            total += term / k
        return total
    return 8 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239))


def _angles(positions, freq):
    """[positions, frequencies] in 64 bits, within half a turn of 0."""
    getcontext().prec = 90
    turn = _two_pi()
    out = []
    for f in freq.tolist():
        f = Decimal(f)
        out.append([float((p * f).remainder_near(turn)) for p in positions.tolist()])
    return torch.tensor(out, dtype=torch.float64).T


@pytest.mark.parametrize("first", [0, 10 ** 6, 2 ** 31 - 700, -2 ** 31])
@pytest.mark.parametrize("freq", [
    [2.0 ** 26 - 4, 2.0 ** 25 + 2, 1.3 * 2 ** 25, -1.9 * 2 ** 24, 3.1e7, 2.0 ** 23 + 1, 1.5e6, 33333.3],
    [1.0, 0.7, -0.33, 1e-3, 2.5, 200.1, 1e-9, 255.9]])
def test_angles(ra, first, freq):
    """Rows of (1, 0): a cosine and a sine themselves, where they are close to 0
    too.  A function is off by 2^-21 (tests/_rope.py), and rounded once to the type."""
    S, dtype = 700, torch.float16
    freq = torch.tensor(freq)
    pos = (torch.arange(S, dtype=torch.int64) + first).to(torch.int32)
    x = torch.zeros((1, 1, S, 64), dtype=dtype)
    x[..., :8] = 1.0
    got, _ = ra.qk_norm_rope_fwd(x.cuda(), x[:, :0].cuda(), pos.cuda(), freq.cuda())
    angle = _angles(pos, freq)
    want = torch.zeros((S, 64), dtype=torch.float64)
    want[:, :8], want[:, 8:16] = angle.cos(), angle.sin()
    assert_close(got[0, 0], want, U[dtype] * want.abs() + TINY[dtype] + 2.0 ** -21 + 3 * T, "turned rows")
    near = (want[:, :16].abs() < 0.02) & (want[:, :16] != 0)
    assert first == 0 or near.any()      # what rounding to the type hides least
    assert math.isfinite(float(got.float().sum()))
