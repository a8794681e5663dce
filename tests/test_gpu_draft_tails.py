"""Draws of draft_verify from rows whose weights are small: residuals behind a
token that holds nearly all of a row, rows far below 1 in sum, single weights down
to the smallest numbers.

A weight of the definition is w = max(target - draft, 0), or the target's own, in
64 bits.  The kernel holds it in whole units, cut, where the sum of V weights has
at least 2^36 of them or the unit is 2^-149, the step of fp32 itself; a
difference may be rounded to fp32 first.  So, with W the exact sum, no partial
sum is off by more than e W, e = V 2^-36 + 2^-24, nor is W itself, and for the
token x drawn with v
    w_x > 0,   w_0 + .. + w_(x-1) <= (v + 2 e) W,   w_0 + .. + w_x > (v - 2 e) W.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BELOW = 1 - 2.0 ** -24


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _row(seed, vocab, token, top, mass, peak=3.0):
    """fp32 probabilities: `top` at the token, `mass` over the others, a softmax of
    normal logits."""
    g = torch.Generator().manual_seed(seed)
    w = torch.softmax(torch.randn(vocab, generator=g, dtype=torch.float64) * peak, 0)
    w[token] = 0
    w *= mass / w.sum()
    w[token] = top
    return w.float()


def _draws(ra, target, draft, token, n, seed, u=BELOW):
    """The tokens that n requests draw, each with one drafted token, from the same
    row; and their random numbers, one in each n-th of [0, 1)."""
    v = (torch.arange(n) + torch.rand(n, generator=torch.Generator().manual_seed(seed))) / n
    rows = target.cuda().repeat(2 * n, 1)
    other = None if draft is None else draft.cuda().repeat(2 * n, 1)
    ids = [7 % target.shape[0], token] * n
    got = ra.draft_verify(rows, other, _i32(ids), _i32(list(range(0, 2 * n + 1, 2))), torch.full((2 * n,), u).cuda(),
                          v.float().cuda())
    assert got[0].tolist() == [0] * n and got[2].tolist() == [1] * n       # none stands
    return got[1].tolist(), v.float().double()


def _check(tokens, v, w):
    """w: the definition's weights in 64 bits."""
    total, cum = w.sum(), torch.cumsum(w, 0)
    e = len(w) * 2.0 ** -36 + 2.0 ** -24
    x = torch.tensor(tokens)
    assert (w[x] > 0).all(), "a token without a weight"
    assert (cum[x] - w[x] <= (v + 2 * e) * total).all() and (cum[x] > (v - 2 * e) * total).all()


MASSES = [(1 - 2.0 ** -4, 2.0 ** -4), (1 - 2.0 ** -9, 2.0 ** -9), (1 - 2.0 ** -22, 2.0 ** -22),
          (1 - 2.0 ** -24, 2.0 ** -24), (0.5, 2.0 ** -40), (0.5, 2.0 ** -62), (0.5, 2.0 ** -101), (0.5, 2.0 ** -130)]


@pytest.mark.parametrize("vocab,n", [(5, 200), (4097, 100), (131071, 40), (262144, 16)])
@pytest.mark.parametrize("top,mass", MASSES)
@pytest.mark.parametrize("outright", [False, True])
def test_behind_a_token_that_holds_nearly_all(ra, vocab, n, top, mass, outright):
    token = vocab // 3
    target = _row(vocab, vocab, token, top, mass)
    draft = None
    if not outright:       # more of the drafted token, less of the others
        draft = target * 0.25
        draft[token] = min(1.0, 1.5 * top)
    w = target.double()
    if outright:
        w[token] = 0
    else:
        w = (w - draft.double()).clamp(min=0)
    assert w[token] == 0 and w.sum() > 0
    tokens, v = _draws(ra, target, draft, token, n, 1)
    assert token not in tokens
    _check(tokens, v, w)


@pytest.mark.parametrize("weight", [2.0 ** -43, 2.0 ** -44, 2.0 ** -45, 2.0 ** -90, 2.0 ** -126, 2.0 ** -149])
@pytest.mark.parametrize("outright", [False, True])
def test_one_small_residual_is_drawn(ra, weight, outright):
    """Nothing else is left: it is drawn, and the token that was refused is not."""
    for vocab, at in ((9, 8), (70001, 41234)):
        target = torch.zeros(vocab)
        target[3], target[at] = 0.5, weight
        draft = None
        if not outright:
            draft = torch.zeros(vocab)
            draft[3] = 1.0
        tokens, _ = _draws(ra, target, draft, 3, 5, 2)
        assert tokens == [at] * 5


def test_a_residual_of_neighbouring_numbers(ra):
    """target - draft is one step of fp32, at a value far above the weights' unit and
    at one far below."""
    for value in (0.25, 2.0 ** -30, 2.0 ** -60, 2.0 ** -126):
        target = torch.tensor([0.5, value, value, 0.0, value])
        draft = target.clone()
        draft[0] = 1.0
        target[2] = torch.nextafter(target[2], torch.tensor(1.0))
        target[4] = torch.nextafter(target[4], torch.tensor(1.0))
        tokens, v = _draws(ra, target, draft, 0, 40, 3)
        assert set(tokens) == {2, 4}
        _check(tokens, v, (target.double() - draft.double()).clamp(min=0))


def test_without_a_residual_the_row_itself(ra):
    """The drafted token alone has a weight, or the draft says what the target does."""
    target = torch.zeros(300)
    target[11] = 2.0 ** -50
    for draft in (None, target.clone()):
        got = ra.draft_verify(target.cuda().repeat(2, 1), None if draft is None else draft.cuda().repeat(2, 1),
                              _i32([0, 11]), _i32([0, 2]), torch.ones(2).cuda(), torch.tensor([0.5]).cuda())
        assert [t.tolist() for t in got] == [[0], [11], [1]]


@pytest.mark.parametrize("mass", [1.0, 2.0 ** -9, 2.0 ** -50, 2.0 ** -120, 2.0 ** -140])
def test_rows_of_any_sum(ra, mass):
    """Nothing drafted: from the row itself, which need not sum to 1."""
    vocab, n = 50001, 30
    row = _row(3, vocab, 5, 0.0, mass)
    v = (torch.arange(n) + 0.5) / n
    got = ra.draft_verify(row.cuda().repeat(n, 1), None, _i32([0] * n), _i32(list(range(n + 1))), torch.zeros(n).cuda(),
                          v.cuda())
    _check(got[1].tolist(), v.double(), row.double())


def test_the_draw_does_not_depend_on_the_batch(ra):
    """Blocks share a row differently in a large batch and alone."""
    vocab, n = 30011, 1500
    token = 77
    target = _row(9, vocab, token, 1 - 2.0 ** -20, 2.0 ** -20)
    many, _ = _draws(ra, target, None, token, n, 4)
    v = (torch.arange(n) + torch.rand(n, generator=torch.Generator().manual_seed(4))) / n
    for i in (0, 1, 700, n - 1):
        got = ra.draft_verify(target.cuda().repeat(2, 1), None, _i32([7, token]), _i32([0, 2]),
                              torch.full((2,), BELOW).cuda(), v[i:i + 1].float().cuda())
        assert got[1].tolist() == [many[i]]
