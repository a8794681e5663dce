"""The bounds of tests/_rope_sums.py see the mistakes that they are for: planted
here in the 64-bit reference, on the CPU."""
import pytest
import torch

from _rope_sums import SHAPES, case, weight_grad_and_tol


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_wrong_sum_is_seen(shape, interleaved):
    x = case(shape, torch.bfloat16)
    for name in "qk":
        dw, tol, terms = weight_grad_and_tol(x["d" + name], x[name], x["w" + name], x["pos"][:, None], x["freq"], 1e-5,
                                             interleaved, 1.0)

        def worst(got):
            return float(((got - dw).abs() / tol).max())
        assert worst(dw.float().double()) < 1
        assert worst(dw - terms[-1, -1, -1]) > 2, "a row lost"
        assert worst(dw - terms[-1, :, -1].sum(0)) > 2, "a token lost"
        tokens = terms.sum(1)
        assert worst(tokens.to(torch.bfloat16).double().sum((0, 1))) > 2, "tokens' sums in 16 bits"
