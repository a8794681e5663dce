"""Pages that a window hides for good, given back before their request ends:
their table entries name no page, and paged_kv_plan and paged_kv_trim pass over
them when they give a request's pages back."""
import random

import pytest
import torch

from _paged import assert_close, pages, plan_ref
from _window import window_ref

pytestmark = pytest.mark.gpu

NONE = [-1, -2 ** 31, 2 ** 31 - 1]      # and num_pages


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _state(rng, n, width, page_size, spare, share):
    """Lengths, tables with entries of no page (about `share` of them), the stack."""
    lens = [rng.randint(0, width * page_size) for _ in range(n)]
    used = [pages(a, page_size) for a in lens]
    ids = list(range(sum(used) + spare + 3))
    rng.shuffle(ids)
    table, at, back = [], 0, []
    for u in used:
        row = ids[at:at + u]
        at += u
        for x in range(u):
            if rng.random() < share:
                back.append(row[x])
                row[x] = rng.choice(NONE + [len(ids)])
        table.append(row + [-9] * (width - u))
    free = back + ids[at:at + spare]
    return lens, table, free + [-1] * (len(ids) - len(free)), [len(free), 31]


SHAPES = [(1, 1, 8, 0), (1, 5000, 8, 3), (3, 4, 16, 5), (8, 700, 16, 9), (33, 5, 48, 40), (500, 40, 16, 900),
          (1025, 3, 64, 700), (8192, 2, 8, 3000)]


@pytest.mark.parametrize("n,width,page_size,spare", SHAPES)
@pytest.mark.parametrize("share", [0.01, 0.5, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(ra, n, width, page_size, spare, share, in_place):
    rng = random.Random(n + width)
    lens, table, free, counts = _state(rng, n, width, page_size, spare, share)
    num = len(free)
    new = [rng.choice([-1, -1, 0, 1, rng.randint(1, 3 * page_size)]) for _ in range(n)]
    tokens = sum(max(q, 0) for q in new) + 2
    # the reference: what is given back first, then the plan of the others
    top, stack = counts[0], list(free)
    for a, q, row in zip(lens, new, table):
        if q < 0:
            for p in row[:pages(a, page_size)]:
                if 0 <= p < num:
                    stack[top] = p
                    top += 1
    left = [0 if q < 0 else a for a, q in zip(lens, new)]
    want = plan_ref(left, new, table, stack, [top, 0], page_size, tokens)
    # (its slots on an entry of no page are -1)
    slots = list(want[2])
    for i, q in enumerate(new):
        for t in range(max(q, 0)):
            if slots[want[1][i] + t] != -1:
                p = want[4][i][(lens[i] + t) // page_size]
                if not 0 <= p < num:
                    slots[want[1][i] + t] = -1
    top = want[3][0]      # above it the stack holds nothing
    t, f, s, c = _i32(table), _i32(free), _i32(lens), _i32(counts)
    for _ in range(1 if in_place else 2):                    # a repeat changes nothing
        got = ra.paged_kv_plan(s, _i32(new), t, f, c, page_size, tokens, seq_lens_out=s if in_place else None,
                               counts_out=c if in_place else None)
        assert [x.tolist() for x in got] + [t.tolist()] == [want[0], want[1], slots, want[3], want[4]]
        assert f.tolist()[:top] == want[5][:top]


@pytest.mark.parametrize("n,width,page_size,spare", SHAPES)
@pytest.mark.parametrize("share", [0.01, 0.5, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_trim(ra, n, width, page_size, spare, share, in_place):
    rng = random.Random(n + width + 1)
    lens, table, free, counts = _state(rng, n, width, page_size, spare, share)
    num = len(free)
    drop = [rng.choice([0, -4, 1, rng.randint(0, a), a, 2 ** 31 - 1]) for a in lens]
    out, stack, top = [], list(free), counts[0]
    for a, x, row in zip(lens, drop, table):
        x = min(max(x, 0), a)
        out.append(a - x)
        for p in row[pages(a - x, page_size):pages(a, page_size)]:
            if 0 <= p < num:
                stack[top] = p
                top += 1
    t, f, s, c = _i32(table), _i32(free), _i32(lens), _i32(counts)
    for _ in range(1 if in_place else 2):                    # a repeat changes nothing
        got = ra.paged_kv_trim(s, _i32(drop), t, f, c, page_size, seq_lens_out=s if in_place else None,
                               counts_out=c if in_place else None)
        assert [x.tolist() for x in got] + [f.tolist()[:top]] == [out, [top, counts[1]], stack[:top]]
    assert t.tolist() == table


def test_a_stack_that_is_too_full_stays_inside(ra):
    """Counts that make no sense beside entries of no page: nothing outside the
    buffers is written."""
    ps, num = 16, 12
    guard = torch.full((3 * 64,), 55, dtype=torch.int32, device="cuda")
    table = [[1, -1, 3, 4, 5, 99]] * 5
    for have in (-3, 5, 11, 2 ** 31 - 1):
        for call in ("plan", "trim"):
            free = guard[64:64 + num]
            state = (_i32([96] * 5), _i32([-1, 1, -1, -1, 0] if call == "plan" else [96, 0, 40, 7, 96]), _i32(table), free,
                     _i32([have, 0]), ps)
            out = ra.paged_kv_plan(*state, 3)[3] if call == "plan" else ra.paged_kv_trim(*state)[1]
            assert 0 <= int(out[0]) <= num
            assert (guard[:64] == 55).all() and (guard[64 + num:] == 55).all()
            guard[64:64 + num] = 55


@pytest.mark.parametrize("captured", [False, True])
def test_a_window_that_gives_its_pages_back(ra, captured):
    """A serving loop over contexts longer than the pool: pages behind the window
    go on the stack as they are hidden, requests end and are shortened in between.
    No page is lost or held twice, and attention is right throughout."""
    n, width, ps, H, H_kv, d, num, window, sinks, m = 4, 40, 8, 4, 2, 64, 48, 37, 5, 6
    lens, table = _i32([0] * n), torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    free, counts = torch.arange(num, dtype=torch.int32, device="cuda"), _i32([num, 0])
    new, drop = _i32([m] * n), _i32([0] * n)
    pools = [torch.full((num, ps, H_kv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rng, g = random.Random(8), torch.Generator().manual_seed(8)
    q, k, v = (torch.zeros(m * n, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, H_kv, H_kv))

    def step():
        ra.paged_kv_trim(lens, drop, table, free, counts, ps, seq_lens_out=lens, counts_out=counts)
        _, cu, slots, _ = ra.paged_kv_plan(lens, new, table, free, counts, ps, m * n, seq_lens_out=lens,
                                           counts_out=counts)
        ra.paged_kv_append(k, v, *pools, slots)
        return ra.paged_attn_window_fwd(q, *pools, table, lens, cu, window, sinks, max_q=m)

    graph = None
    truth = [([], []) for _ in range(n)]      # rows of K and V, by request
    for turn in range(90):
        news, drops = [m] * n, [0] * n
        for i in range(n):
            a = len(truth[i][0])
            if a > width * ps - 2 * m or rng.random() < 0.03:
                news[i] = -1
            elif a >= 3:
                drops[i] = rng.choice([0, 0, 1, 3])
        new.copy_(torch.tensor(news))
        drop.copy_(torch.tensor(drops))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        if captured and graph is None and turn == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                o, lse = step()
        if graph is not None:
            graph.replay()
        else:
            o, lse = step()
        at, cu = 0, [0]
        for i in range(n):
            kept = len(truth[i][0]) - drops[i]
            for rows, fresh in zip(truth[i], (k, v)):
                del rows[kept:]
                if news[i] < 0:
                    rows.clear()
                else:
                    rows += list(fresh[at:at + m].cpu())
            at += max(news[i], 0)
            cu.append(at)
        have = [len(t[0]) for t in truth]
        assert lens.tolist() == have and counts.tolist()[1] == 0
        rows, count = table.tolist(), counts.tolist()[0]
        held = [p for a, row in zip(have, rows) for p in row[:pages(a, ps)] if p != -1]
        assert sorted(held + free.tolist()[:count]) == list(range(num)), f"turn {turn}"
        if turn % 11 == 10:
            ref = dict(q=q.cpu(), k_cache=torch.zeros(n * width, ps, H_kv, d, dtype=torch.bfloat16),
                       table=torch.arange(n * width).view(n, width), lens=have,
                       news=[max(x, 0) for x in news], cu=cu)
            ref["v_cache"] = ref["k_cache"].clone()
            for i in range(n):
                for pool, t in zip((ref["k_cache"], ref["v_cache"]), truth[i]):
                    if t:
                        pool[i * width:(i + 1) * width].view(-1, H_kv, d)[:len(t)] = torch.stack(t)
            o_ref, lse_ref, tol_o, tol_lse = window_ref(ref, window, sinks)
            assert_close(o[:cu[-1]], o_ref[:cu[-1]], tol_o[:cu[-1]], "O")
            assert_close(lse[:, :cu[-1]], lse_ref[:, :cu[-1]], tol_lse[:, :cu[-1]], "LSE")
        # what no token will see again, three taken back at most, goes on the stack
        for i, a in enumerate(have):
            for x in range(pages(sinks, ps), max(0, a - 3 - window + 1) // ps):
                if rows[i][x] != -1:
                    free[count] = rows[i][x]
                    table[i, x] = -1
                    rows[i][x] = -1
                    count += 1
        counts[0] = count
    assert ra.check_status() == ra.RA_OK
