"""rope_inv_freq's mixture between divided and kept frequencies, number by
number."""
import math

import pytest
import torch

import long_context_exact_ring_gb300 as ra


@pytest.mark.parametrize("rot,base,length,factor,fast,slow", [
    (64, 1e4, 4096, 40.0, 32.0, 1.0), (128, 1e6, 32768, 4.0, 32.0, 1.0), (128, 5e5, 8192, 8.0, 4.0, 1.0)])
def test_parts_mix_linearly_in_the_turns(rot, base, length, factor, fast, slow):
    f, amplitude = ra.rope_inv_freq(rot, base, scaling="parts", factor=factor, original_length=length, beta_fast=fast,
                                    beta_slow=slow, device="cpu")
    assert amplitude == 0.1 * math.log(factor) + 1.0
    between = 0
    for i in range(rot // 2):
        x = base ** (-2 * i / rot)
        turns = length * x / (2 * math.pi)
        kept = (turns - slow) / (fast - slow)
        if kept >= 1:
            want = x
        elif kept <= 0:
            want = x / factor
        else:
            want = kept * x + (1 - kept) * x / factor
            between += 1
        assert abs(float(f[i]) - want) <= 2.0 ** -23 * want
    assert between >= 4


def test_parts_of_one_pair_by_hand():
    """Two pairs, 1 and 1/100: over 40 pi * 100 positions the second turns 20 times,
    halfway between 10 and 30."""
    f, _ = ra.rope_inv_freq(4, 1e4, scaling="parts", factor=5.0, original_length=round(4000 * math.pi), beta_fast=30.0,
                            beta_slow=10.0, device="cpu")
    assert f[0] == 1.0 and abs(float(f[1]) / (0.01 * (0.5 + 0.5 / 5)) - 1) < 1e-4
    assert f.dtype == torch.float32
