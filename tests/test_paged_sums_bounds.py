"""The bounds of tests/_paged_sums.py see the mistakes that they are for: planted
here in the 64-bit reference, on the CPU."""
import pytest
import torch

from _paged import make
from _paged_sums import balance, misses, reference, spread


@pytest.mark.parametrize("dtype,rho", [(torch.bfloat16, 2.0 ** -16), (torch.bfloat16, 2.0 ** -8),
                                       (torch.float16, 2.0 ** -11)])
@pytest.mark.parametrize("mistake", [None, "a share lost", "a step lost", "a share twice", "two shares exchanged",
                                     "a factor missed"])
def test_a_wrong_part_is_seen(dtype, rho, mistake):
    """A share is what one of 19 blocks has of a head's context, a step 128 keys."""
    n = 38911
    x = make([n], [2], 2, 1, 64, 64, dtype, seed=1)
    spread(x, 64, 2)
    share = slice(6 * 2048, 7 * 2048)

    def planted(p, i):
        p = p.clone()
        if mistake == "a share lost":
            p[:, share] = 0
        elif mistake == "a step lost":
            p[:, 2560:2688] = 0
        elif mistake == "a share twice":
            p[:, share] *= 2
        elif mistake == "two shares exchanged":
            p[:, share], p[:, 20480:22528] = p[:, 20480:22528].clone(), p[:, share].clone()
        elif mistake == "a factor missed":
            p[:, share] *= 1.25
        return p

    got = reference(x, planted=planted)["o"].to(dtype)
    worst, mean = misses(got, reference(x), dtype, rho, 16)
    if mistake is None:
        assert worst <= 1 and mean <= 1
    else:
        assert mean > 4


@pytest.mark.parametrize("n", [2, 7, 40])
def test_weights_rounded_once_are_seen(n):
    """bf16 weights without what rounding leaves, against weights in two parts."""
    x = make([n] * 6, [1] * 6, 8, 8, 64, 16, torch.bfloat16, seed=n)
    balance(x)
    ref = reference(x)

    def once(p, i):
        w = p / p.max()
        return w.to(torch.bfloat16).double() * p.max()

    def twice(p, i):
        w = (p / p.max()).float()
        upper = (w.view(torch.int32) & -65536).view(torch.float32)
        return (upper.double() + (w - upper).to(torch.bfloat16).double()) * p.max().double()

    for planted, holds in ((once, False), (twice, True)):
        got = reference(x, planted=planted)["o"].to(torch.bfloat16)
        worst, mean = misses(got, ref, torch.bfloat16, 2.0 ** -16, 1)
        assert (worst <= 1 and mean <= 1) if holds else (worst > 2 and mean > 4), (worst, mean)
