"""Drafts in a serving loop: tokens are added, attended and partly taken back,
and no page is lost or held twice."""
import random

import pytest
import torch

from _paged import assert_close, attn_ref, pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _take_back(s, kept):
    """As the documentation has it: pages behind the new lengths go on the stack."""
    column = torch.arange(s["table"].shape[1], device="cuda")
    have, keep = ((x[:, None] + s["ps"] - 1) // s["ps"] for x in (s["lens"], kept))
    back = ((column >= keep) & (column < have)).flatten()
    num = s["free"].numel()
    at = torch.where(back, s["counts"][0] + back.cumsum(0) - 1, num)
    s["free"].copy_(torch.cat([s["free"], s["free"][:1]]).index_copy_(0, at, s["table"].flatten())[:num])
    s["counts"][0] += back.sum()
    s["lens"].copy_(kept)


def _held(s):
    """Pages of the requests and of the stack, as lists."""
    lens, table, count = s["lens"].tolist(), s["table"].tolist(), int(s["counts"][0])
    held = [p for a, row in zip(lens, table) for p in row[:pages(a, s["ps"])]]
    return held + s["free"][:count].tolist()


@pytest.mark.parametrize("captured", [False, True])
def test_drafts_are_taken_back(ra, captured):
    n, width, ps, H, H_kv, d, num = 4, 9, 8, 4, 2, 64, 40
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(ps=ps, table=torch.full((n, width), -1, **i32), free=torch.arange(num, **i32),
             counts=torch.tensor([num, 0], **i32), lens=torch.zeros(n, **i32))
    pools = [torch.full((num, ps, H_kv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rng, g = random.Random(5), torch.Generator().manual_seed(5)
    kept, new = torch.zeros(n, **i32), torch.full((n,), 6, **i32)
    T = 6 * n
    q, k, v = (torch.zeros(T, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, H_kv, H_kv))

    def step():
        _take_back(s, kept)
        lens, cu, slots, _ = ra.paged_kv_plan(s["lens"], new, s["table"], s["free"], s["counts"], ps, T,
                                              seq_lens_out=s["lens"], counts_out=s["counts"])
        ra.paged_kv_append(k, v, *pools, slots)
        return ra.paged_attn_fwd(q, *pools, s["table"], lens, cu, True, max_q=6)

    graph = None
    truth, draft = [[] for _ in range(n)], None       # the rows of K that each request has accepted; the last draft's
    for turn in range(40):
        if draft is not None:
            for i in range(n):
                stay = rng.randint(0, 6)
                truth[i] += draft[6 * i:6 * i + stay]
                if len(truth[i]) > width * ps - 12:
                    truth[i] = truth[i][:rng.randint(0, 20)]       # a request that goes back a long way
        kept.copy_(torch.tensor([len(x) for x in truth], dtype=torch.int32))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        draft = list(k.cpu())
        if captured and graph is None and turn == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                o, lse = step()
        if graph is not None:
            graph.replay()
        else:
            o, lse = step()
        assert sorted(_held(s)) == list(range(num)), f"turn {turn}"
        lens = [len(x) + 6 for x in truth]
        assert s["lens"].tolist() == lens
        if turn % 13 == 12:
            x = dict(q=q.cpu(), k_cache=pools[0].cpu(), v_cache=pools[1].cpu(), table=s["table"].cpu(), lens=lens,
                     news=[6] * n, cu=[6 * i for i in range(n + 1)])
            for i in range(n):
                c = torch.arange(lens[i])
                want = torch.stack(truth[i] + draft[6 * i:6 * i + 6])
                assert torch.equal(x["k_cache"][x["table"][i].long()[c // ps], c % ps], want)
            o_ref, lse_ref, tol_o, tol_lse = attn_ref(x, True)
            assert_close(o, o_ref, tol_o, "O")
            assert_close(lse, lse_ref, tol_lse, "LSE")
    assert ra.check_status() == ra.RA_OK
