"""Pages outside the pool in a step of the serving loop: what each of the three
calls does with them, and which of them says so."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("bad", ["in the table", "on the free list"])
def test_a_step_over_a_bad_page_is_reported_by_its_attention(ra, new, bad):
    """The plan gives tokens on a bad page no slot, the append leaves them out,
    and the attention of the same step, which reads the page, reports it.  The
    other request is as it would be alone."""
    ps, H, d, num = 16, 2, 64, 8
    lens, table = _i32([40, 24]), _i32([[0, 1, 2, -1, -1], [3, 4, -1, -1, -1]])
    free, counts = _i32([7, 6, 5] + [-1] * 5), _i32([3, 0])
    if bad == "in the table":
        table[0, 2] = num                 # holds tokens 32 .. 47
    else:
        lens[0] = 48                      # the next token takes a page
        free[2] = -9                      # the first to go
    pools = [torch.zeros(num, ps, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    news = [new, 1]
    rows = torch.ones(sum(news), 1, d, dtype=torch.bfloat16, device="cuda")
    new_lens, cu, slots, left = ra.paged_kv_plan(lens, _i32(news), table, free, counts, ps, sum(news))
    inside = 48 - int(lens[0]) if bad == "in the table" else 16      # of the new tokens, how many the page takes
    assert slots[:min(inside, new)].tolist() == [-1] * min(inside, new)
    assert slots[-1].item() == 4 * ps + 24 % ps and int(left[1]) == 0
    ra.paged_kv_append(rows, rows, *pools, slots)
    stored = new + 1 - min(inside, new)
    for p in pools:
        assert float(p.float().sum()) == stored * d
    assert ra.check_status() == ra.RA_OK          # no slot is none to report
    q = torch.ones(sum(news), H, d, dtype=torch.bfloat16, device="cuda")
    o, lse = ra.paged_attn_fwd(q, *pools, table, new_lens, cu, True)
    assert ra.check_status() == ra.RA_ERR_BAD_PAGE
    # request 1: 24 keys of zeros and one of ones
    e = torch.exp(torch.tensor(d / d ** 0.5, dtype=torch.float64))
    want = e / (24 + e)
    # half a step of O and of the weights, 2^-8 each
    assert float((o[-1].double() - want.cuda()).abs().max()) <= 2 * 2.0 ** -8 * float(want)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
