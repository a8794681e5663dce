"""The weights' gradients of the norm and rotation within bounds that show a lost
row, a lost token and a sum kept in 16 bits (tests/_rope_sums.py;
tests/test_rope_sums_bounds.py plants them); several batch rows with several
tokens to a warp among the shapes."""
import pytest
import torch

from _paged import assert_close
from _rope import backward_and_tol, forward_and_tol
from _rope_sums import SHAPES, case, weight_grad_and_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,interleaved", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("norm", ["qk", "q", "k"])
def test_rows_and_weights(ra, shape, dtype, interleaved, norm):
    x = case(shape, dtype)
    w = {n: x["w" + n] if n in norm else None for n in "qk"}
    how = dict(eps=1e-5, interleaved=interleaved, **{n + "_weight": None if t is None else t.cuda() for n, t in w.items()})
    rows, grads = [x[n].cuda() for n in "qk"], [x["d" + n].cuda() for n in "qk"]
    at = (x["pos"].cuda(), x["freq"].cuda())
    y = ra.qk_norm_rope_fwd(*rows, *at, **how)
    got = ra.qk_norm_rope_bwd(*grads, *rows, *at, **how)
    for i, n in enumerate("qk"):
        args = (x["pos"][:, None], x["freq"], 1e-5, interleaved, 1.0)
        assert_close(y[i], *forward_and_tol(x[n], w[n], *args), n)
        dx, _, tol, _ = backward_and_tol(x["d" + n], x[n], w[n], *args)
        assert_close(got[i], dx, tol, "d" + n)
        if w[n] is not None:
            dw, tol, _ = weight_grad_and_tol(x["d" + n], x[n], w[n], *args)
            assert_close(got[2 + i], dw, tol, "weight of " + n)


@pytest.mark.parametrize("shape", SHAPES[1:4])
def test_rows_are_not_read_without_weights(ra, shape):
    """The gradients themselves may stand for them."""
    x = case(shape, torch.bfloat16)
    q, k, dq, dk = [x[n].cuda() for n in ("q", "k", "dq", "dk")]
    at = (x["pos"].cuda(), x["freq"].cuda())
    want = ra.qk_norm_rope_bwd(dq, dk, q, k, *at)
    got = ra.qk_norm_rope_bwd(dq, dk, dq, dk, *at)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[2] is None and got[3] is None
    got = ra.qk_norm_rope_bwd(dq, dk, dq, dk, *at, dq_in=dq, dk_in=dk)
    assert got[0] is dq and torch.equal(dq, want[0]) and torch.equal(dk, want[1])
