"""The paged key/value cache on the GPU, against plain references in whole
numbers and 64 bits (tests/_paged.py, where the tolerances are derived)."""
import random

import pytest
import torch

import workloads
from _paged import assert_close, attn_ref, attn_ref_causal, make, pages, plan_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# Bookkeeping
# ---------------------------------------------------------------------------
def _random_state(rng, n, width, page_size, spare, chunk):
    lens = [rng.randint(0, width * page_size) for _ in range(n)]
    used = [pages(a, page_size) for a in lens]
    ids = list(range(sum(used) + spare + 3))
    rng.shuffle(ids)
    table, at = [], 0
    for u in used:
        table.append(ids[at:at + u] + [-9] * (width - u))
        at += u
    free = ids[at:at + spare] + [-1] * (len(ids) - spare)
    new = [rng.choice([-1, 0, 1, 1, 1, rng.randint(1, chunk)]) for _ in range(n)]
    return lens, new, table, free, [spare, 123]


@pytest.mark.parametrize("n,width,page_size,spare,chunk,slack", [
    (1, 1, 8, 1, 4, 0), (3, 4, 16, 0, 9, 2), (8, 8, 16, 9, 40, 5), (33, 5, 48, 40, 100, 0), (500, 40, 16, 900, 300, 7),
    (1025, 3, 64, 700, 90, 1), (8192, 2, 8, 3000, 10, 0)])
@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(ra, n, width, page_size, spare, chunk, slack, seed, in_place):
    rng = random.Random(1000 * n + seed)
    lens, new, table, free, counts = _random_state(rng, n, width, page_size, spare, chunk)
    tokens = sum(max(q, 0) for q in new) + (slack if seed == 0 else -min(slack, 3))
    tokens = max(tokens, 0)
    want = plan_ref(lens, new, table, free, counts, page_size, tokens)
    wide = _i32([row + [77] * 3 for row in table])          # rows wider than the table
    t, f, s, c = wide[:, :width], _i32(free), _i32(lens), _i32(counts)
    for _ in range(1 if in_place else 2):                    # a repeat changes nothing
        got = ra.paged_kv_plan(s, _i32(new), t, f, c, page_size, tokens, seq_lens_out=s if in_place else None,
                               counts_out=c if in_place else None)
        assert [x.tolist() for x in got] + [t.tolist(), f.tolist()] == list(want)
    assert (wide[:, width:] == 77).all()
    assert ra.check_status() == ra.RA_OK


def test_plan_over_odd_lengths_stays_inside(ra):
    """Lengths and counts that make no sense: nothing outside the buffers is
    touched, and what comes out is in range."""
    width, ps, num, tokens = 4, 16, 12, 30
    lens = [-5, 10 ** 6, 3, 64, 2 ** 31 - 1, -2 ** 31]
    new = [4, 4, 2 ** 31 - 1, -1, -2 ** 31, 7]
    guard = torch.full((3 * 64,), 55, dtype=torch.int32, device="cuda")
    for have in (-3, 5, 2 ** 31 - 1):
        table, free = _i32([[1, 2, 99, -4]] * 6), _i32(list(range(num)))
        slots = guard[64:64 + tokens]
        out = ra.paged_kv_plan(_i32(lens), _i32(new), table, free, _i32([have, 0]), ps, tokens, slots=slots)
        assert ((out[0] >= 0) & (out[0] <= width * ps)).all()
        assert ((slots >= -1) & (slots < num * ps)).all()
        assert 0 <= int(out[3][0]) <= num
        assert (guard[:64] == 55).all() and (guard[64 + tokens:] == 55).all()
        guard[64:64 + tokens] = 55


@pytest.mark.parametrize("tokens", [0, 5])
def test_plan_without_requests(ra, tokens):
    """A loop that has run dry: the pages stay free, no slot is given."""
    free = _i32([4, 2, 0, 1, 3])
    for in_place in (False, True):
        counts, cu = _i32([3, 9]), _i32([77])
        out = ra.paged_kv_plan(_i32([]), _i32([]), torch.empty(0, 4, dtype=torch.int32, device="cuda"), free, counts, 16,
                               tokens, cu_q=cu, counts_out=counts if in_place else None)
        assert [x.tolist() for x in out] == [[], [0], [-1] * tokens, [3, 0]]
    assert free.tolist() == [4, 2, 0, 1, 3]


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,d,ps", [(1, 1, 64, 8), (5, 2, 128, 16), (77, 5, 64, 48), (1000, 8, 128, 16)])
@pytest.mark.parametrize("layout", ["thd", "htd", "padded"])
def test_append(ra, dtype, T, H, d, ps, layout):
    g = torch.Generator("cuda").manual_seed(T)
    num = pages(T, ps) + 3
    kv = torch.randn((T, 2, H, d), generator=g, device="cuda").to(dtype)
    shape = {"thd": (num, ps, H, d), "htd": (num, H, ps, d), "padded": (num, ps, H + 1, d + 8)}[layout]
    store = [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2)]

    def view(x):
        return x if layout == "thd" else x.transpose(1, 2) if layout == "htd" else x[:, :, :H, :d]

    slots = torch.randperm(num * ps, generator=g, device="cuda")[:T].to(torch.int32)
    slots[::7] = -1
    want = [x.clone() for x in store]
    for i, w in enumerate(want):
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                view(w)[s // ps, s % ps] = kv[t, i]
    k, v = kv[:, 0], kv[:, 1].transpose(0, 1).contiguous().transpose(0, 1)
    ra.paged_kv_append(k, v, view(store[0]), view(store[1]), slots)
    assert torch.equal(store[0], want[0]) and torch.equal(store[1], want[1])
    assert ra.check_status() == ra.RA_OK


def test_append_slot_outside_the_pool(ra):
    """Bad slots are left out and reported; the others are stored."""
    pool = [torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    ra.paged_kv_append(k, k, *pool, _i32([3, 16, -2, -1]))
    assert ra.check_status() == ra.RA_ERR_BAD_PAGE
    assert ra.check_status() == ra.RA_OK
    for x in pool:
        assert float(x.sum()) == 64 and float(x[0, 3].sum()) == 64


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def _run(ra, x, causal, **kw):
    args = [x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q")]
    if x["k_cache"].stride(1) < x["k_cache"].stride(2):      # .cuda() keeps strides of dense tensors
        assert args[1].stride() == x["k_cache"].stride()
    return ra.paged_attn_fwd(*args, causal, **kw)


def _check(ra, x, causal, scale=None, **kw):
    o, lse = _run(ra, x, causal, scale=scale, **kw)
    assert ra.check_status() == ra.RA_OK
    o_ref, lse_ref, tol_o, tol_lse = attn_ref(x, causal, scale)
    rows = x["cu"][-1]
    assert_close(o[:rows], o_ref[:rows], tol_o[:rows], "O")
    assert_close(lse[:, :rows], lse_ref[:, :rows], tol_lse[:, :rows], "LSE")
    return o, lse


BATCHES = {
    "one_key": ([1], [1]),
    "one_token": ([131], [1]),
    "decode": ([1, 7, 8, 9, 16, 128, 129, 300], [1] * 8),
    "short_and_empty": ([0, 3, 0, 5, 40], [0, 1, 2, 9, 0]),      # rows without keys, requests without rows
    "verify": ([50, 17, 260], [3, 5, 4]),
    "prompt": ([37, 150], [37, 150]),
    "chunks": ([300, 514, 90], [45, 130, 1]),
    "tiles": ([128, 256, 384, 127], [128, 1, 129, 64]),
}


@pytest.mark.parametrize("batch", sorted(BATCHES))
@pytest.mark.parametrize("H,H_kv", [(4, 4), (8, 2), (7, 1), (32, 2)])
@pytest.mark.parametrize("d,dtype,page_size,layout", [
    (128, torch.bfloat16, 16, "thd"), (64, torch.float16, 8, "htd"), (128, torch.float16, 48, "htd"),
    (64, torch.bfloat16, 256, "thd")])
def test_attn(ra, batch, H, H_kv, d, dtype, page_size, layout):
    lens, news = BATCHES[batch]
    x = make(lens, news, H, H_kv, d, page_size, dtype, layout=layout, seed=len(batch))
    _check(ra, x, causal=True)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("batch", ["decode", "short_and_empty", "chunks"])
def test_attn_not_causal(ra, batch, dtype, d):
    lens, news = BATCHES[batch]
    _check(ra, make(lens, news, 8, 4, d, 24, dtype, seed=3), causal=False, scale=0.3)


@pytest.mark.parametrize("max_q", [1, 64, 10 ** 6, 2 ** 32 + 1])
def test_attn_does_not_depend_on_the_hint(ra, max_q):
    lens, news = BATCHES["chunks"]
    x = make(lens, news, 8, 2, 128, 16, torch.bfloat16, seed=9)
    _check(ra, x, True, max_q=max_q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attn_large_scores(ra, dtype):
    """Scores in the hundreds: the running maximum moves all the time."""
    x = make([700, 333], [1, 70], 8, 2, 64, 16, dtype, seed=5, peak=60.0)
    _check(ra, x, True)


def test_attn_many_small_weights_fp16(ra):
    """One key stands 25 binary orders above 4000 others, whose weights, with
    the first key's at 1, would all round to 0 in fp16."""
    x = make([4001], [1], 1, 1, 64, 16, torch.float16, seed=6)
    x["q"].zero_()
    x["q"][0, 0, 0] = 1.0
    keys = x["k_cache"]
    keys[torch.isfinite(keys)] = 0.0
    page = x["table"][0, 0]
    keys[page, 0, 0, 0] = 25 * 0.6931
    x["v_cache"][torch.isfinite(x["v_cache"])] = 64.0
    x["v_cache"][page, 0] = 0.0
    _check(ra, x, True, scale=1.0)


@pytest.mark.parametrize("news", [[1, 3], [40, 130]])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attn_values_a_row_does_not_see(ra, news, what, where):
    """A later token's K or V of any value leaves the earlier rows alone, and
    reaches the rows that see it."""
    lens = [60, 290]
    x = make(lens, news, 4, 2, 128, 16, torch.bfloat16, seed=8)
    for i in range(2):
        key = lens[i] - (news[i] + 1) // 2                 # one of the new tokens
        cache = x[where + "_cache"]
        cache[x["table"][i, key // 16], key % 16, 1] = float(what)
    o, lse = _run(ra, x, True)
    o_ref, lse_ref, tol_o, tol_lse = attn_ref(x, True)
    clean = torch.isfinite(lse_ref.T) & torch.isfinite(o_ref).all(-1)
    assert not clean.all() and clean.any()
    got = o.cpu().double()
    assert ((got - o_ref).abs() <= tol_o)[clean].all()
    assert ((lse.cpu().double() - lse_ref).abs().T <= tol_lse.T)[clean].all()
    if where == "v":
        assert torch.equal(torch.isfinite(got), torch.isfinite(o_ref))


def test_attn_nan_query_stays_in_its_row(ra):
    x = make([33, 400], [1, 150], 4, 2, 128, 16, torch.bfloat16, seed=8)
    x["q"][5, 2, 7] = float("nan")
    o, lse = _run(ra, x, True)
    bad = torch.isnan(o).any(-1).cpu()
    assert bad[5, 2] and int(bad.sum()) == 1
    assert torch.isnan(lse[2, 5]) and int(torch.isnan(lse).sum()) == 1


@pytest.mark.parametrize("batch", ["decode", "chunks"])
def test_attn_strided_and_padded(ra, batch):
    """q and O inside wider storage, rows behind the last request untouched."""
    lens, news = BATCHES[batch]
    x = make(lens, news, 8, 2, 128, 16, torch.bfloat16, seed=2, rows_behind=9)
    T = x["q"].shape[0]
    wide = torch.randn((T, 3, 8, 128)).to(torch.bfloat16)
    wide[:, 1] = x["q"]
    o = torch.full((8, T, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, T), 6.0, device="cuda")
    y = dict(x)
    args = [x[n].cuda() for n in ("k_cache", "v_cache", "table", "seq_lens", "cu_q")]
    ra.paged_attn_fwd(wide.cuda()[:, 1], *args, True, o=o.transpose(0, 1)[:, :, :128], lse=lse)
    o_ref, lse_ref, tol_o, tol_lse = attn_ref(y, True)
    rows = x["cu"][-1]
    got = o.transpose(0, 1)
    assert_close(got[:rows, :, :128], o_ref[:rows], tol_o[:rows], "O")
    assert_close(lse[:, :rows], lse_ref[:, :rows], tol_lse[:, :rows], "LSE")
    assert (got[rows:] == 5).all() and (got[:, :, 128:] == 5).all() and (lse[:, rows:] == 6).all()


@pytest.mark.parametrize("news", [[1, 1], [1, 70]])
def test_attn_page_outside_the_pool(ra, news):
    """A bad page's keys read as zero rows, and the status says so."""
    x = make([80, 100], news, 4, 2, 64, 16, torch.bfloat16, seed=4)
    bad = dict(x, table=x["table"].clone())
    num = x["k_cache"].shape[0]
    for i, value in ((0, num), (1, -1)):
        p = int(x["table"][i, 2])
        x["k_cache"][p], x["v_cache"][p] = 0, 0
        bad["table"][i, 2] = value
    o, lse = _run(ra, bad, True)
    assert ra.check_status() == ra.RA_ERR_BAD_PAGE
    o_ref, lse_ref, tol_o, tol_lse = attn_ref(x, True)
    assert_close(o, o_ref, tol_o, "O")
    assert_close(lse, lse_ref, tol_lse, "LSE")


def test_attn_lengths_beyond_the_buffers(ra):
    """cu_q and seq_lens past q's rows and the table: cut, not followed."""
    x = make([64, 64], [2, 2], 4, 2, 64, 16, torch.bfloat16, seed=4)
    x["table"] = x["table"][:, :4].contiguous()
    x["seq_lens"] = torch.tensor([10 ** 6, -4], dtype=torch.int32)
    x["cu_q"] = torch.tensor([0, 2, 999], dtype=torch.int32)
    o, lse = _run(ra, x, True)
    assert ra.check_status() == ra.RA_OK
    y = dict(x, lens=[64, 0])
    o_ref, lse_ref, tol_o, tol_lse = attn_ref(y, True)
    assert_close(o, o_ref, tol_o, "O")
    assert_close(lse, lse_ref, tol_lse, "LSE")


def test_attn_offsets_past_32_bits(ra):
    """Pages more than 2^32 elements into the pool."""
    ps, H, d = 64, 8, 128
    num = (1 << 32) // (ps * H * d) + 40
    x = make([150, 70], [1, 66], 16, H, d, ps, torch.bfloat16, seed=1)
    pools = [torch.empty((num, ps, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = x["k_cache"].shape[0]
    for big, name in zip(pools, ("k_cache", "v_cache")):
        big[num - small:] = x[name].cuda()
    table = x["table"].cuda() + (num - small)
    o, lse = ra.paged_attn_fwd(x["q"].cuda(), *pools, table, x["seq_lens"].cuda(), x["cu_q"].cuda(), True)
    o_ref, lse_ref, tol_o, tol_lse = attn_ref(x, True)
    assert_close(o, o_ref, tol_o, "O")
    assert_close(lse, lse_ref, tol_lse, "LSE")
    # and appended there
    rows = torch.ones(3, H, d, dtype=torch.bfloat16, device="cuda")
    slots = _i32([num * ps - 1, num * ps - 2, 0])
    ra.paged_kv_append(rows, rows, *pools, slots)
    for big in pools:
        assert (big[num - 1, ps - 2:] == 1).all() and (big[0, 0] == 1).all()


def test_attn_other_stream_and_shared_workspace_of_two_graphs(ra):
    lens, news = BATCHES["chunks"]
    x = make(lens, news, 8, 2, 128, 16, torch.bfloat16, seed=11)
    want = _run(ra, x, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _run(ra, x, True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # one workspace, full of other bits, behind two graphs replayed in turn
    T, H, d = x["q"].shape
    ws = torch.full((ra.paged_attn_workspace_size(3, T, H, 2, d),), 255, dtype=torch.uint8, device="cuda")
    args = [x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q")]
    graphs, outs = [], []
    for causal in (True, False):
        o, lse = torch.zeros_like(args[0]), torch.zeros(H, T, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ra.paged_attn_fwd(*args, causal, o=o, lse=lse, workspace=ws)
        graphs.append(g)
        outs.append((o, lse))
    for _ in range(3):
        for g in graphs:
            g.replay()
    assert torch.equal(outs[0][0], want[0]) and torch.equal(outs[0][1], want[1])
    other = _run(ra, x, False)
    assert torch.equal(outs[1][0], other[0]) and torch.equal(outs[1][1], other[1])


@pytest.mark.parametrize("H,H_kv", [(128, 1), (100, 1), (43, 1), (17, 1), (16, 1), (34, 2)])
@pytest.mark.parametrize("news", [[1, 1, 0], [2, 3, 5]])
def test_attn_large_groups(ra, H, H_kv, news):
    """Groups that fill a tile of 128 rows, or leave some of it over."""
    _check(ra, make([150, 64, 9], news, H, H_kv, 64, 8, torch.bfloat16, seed=H), True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("news", [[1], [3, 1, 1], [40, 1, 9]])
def test_attn_many_short_requests(ra, d, news):
    """More requests than threads, each with a few keys; some without rows."""
    rng = random.Random(d)
    n = 700
    lens = [rng.choice([0, 1, 7, 8, 33, 64, 100]) for _ in range(n)]
    q = [min(rng.choice(news + [0]), max(a, 1)) for a in lens]
    _check(ra, make(lens, q, 2, 1, d, 8, torch.bfloat16, seed=n), True)


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("d,page_size", [(64, 512), (128, 136)])
def test_attn_one_context_over_all_blocks(ra, new, d, page_size):
    """A context cut into as many parts as there are blocks, its last key
    tiles short."""
    for length in (152 * 128 + 1, 152 * 256 - 1):
        x = make([length], [new], 2, 1, d, page_size, torch.float16, seed=new)
        _check(ra, x, True)


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("odd", [None, "inf", "nan"])
def test_attn_whole_tiles_between_cut_ones(ra, d, dtype, odd):
    """Prompts of several key tiles, many tiles to a block: those between a
    share's first and last begin in the middle of their keys.  A value of V that
    only the later rows see reaches those alone."""
    lens = [520, 300, 401, 640, 129, 575] * 4
    x = make(lens, [a - 7 * (i % 3) for i, a in enumerate(lens)], 16, 8, d, 16, dtype, seed=d)
    for i, a in enumerate(lens if odd else []):
        key = a * 2 // 3 - i
        x["v_cache"][x["table"][i, key // 16], key % 16, i % 8, i] = float(odd)
    o, lse = _run(ra, x, True)
    assert ra.check_status() == ra.RA_OK
    o_ref, lse_ref, tol_o, tol_lse = attn_ref_causal(x)
    assert bool(torch.isfinite(o_ref).all()) == (odd is None)
    assert_close(o, o_ref, tol_o, "O")
    assert_close(lse, lse_ref, tol_lse, "LSE")


def test_attn_different_strides_for_keys_and_values(ra):
    """K by tokens, V by heads, both inside wider storage; a wider table."""
    x = make([90, 300], [1, 60], 8, 2, 64, 16, torch.bfloat16, seed=7)
    num = x["k_cache"].shape[0]
    k = torch.full((num, 16, 3, 72), float("nan"), dtype=torch.bfloat16)
    v = torch.full((num + 2, 2, 24, 64), float("nan"), dtype=torch.bfloat16)
    k[:, :, 1:, :64] = x["k_cache"]
    v[:num, :, :16] = x["v_cache"].transpose(1, 2)
    table = torch.full((2, x["table"].shape[1] + 5), 3, dtype=torch.int32)
    table[:, :-5] = x["table"]
    o, lse = ra.paged_attn_fwd(x["q"].cuda(), k.cuda()[:, :, 1:, :64], v.cuda()[:num, :, :16].transpose(1, 2),
                               table.cuda()[:, :-5], x["seq_lens"].cuda(), x["cu_q"].cuda(), True)
    o_ref, lse_ref, tol_o, tol_lse = attn_ref(x, True)
    assert_close(o, o_ref, tol_o, "O")
    assert_close(lse, lse_ref, tol_lse, "LSE")


def test_attn_two_calls_at_once(ra):
    """Two streams, each with a workspace of its own, over one pool."""
    x = make([5000, 2000, 77], [1, 140, 30], 8, 2, 128, 16, torch.bfloat16, seed=12)
    args = [x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q")]
    want = ra.paged_attn_fwd(*args, True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in streams:
            got.append(ra.paged_attn_fwd(*args, True, stream=s))
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_attn_results_do_not_change_from_call_to_call(ra):
    x = make([5000, 2000, 77] * 3, [1, 140, 30] * 3, 8, 2, 64, 16, torch.float16, seed=13)
    want = _run(ra, x, True)
    for _ in range(5):
        got = _run(ra, x, True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attn_part_contexts_merge_to_the_whole(ra):
    """Attention over two halves of a context, merged as ring steps are."""
    x = make([512], [1], 4, 2, 128, 16, torch.bfloat16, seed=15)
    whole_o, whole_lse = _check(ra, x, False)
    parts = []
    for a in (0, 16):
        y = dict(x, table=x["table"][:, a:a + 16].contiguous(), seq_lens=torch.tensor([256], dtype=torch.int32))
        o, lse = _run(ra, y, False)
        parts.append((o.float()[None].transpose(1, 2).contiguous(), lse[None].contiguous()))
    (oa, la), (ob, lb) = parts
    o, lse = ra.attn_merge_partials(oa, la, ob, lb)
    # each part's O and the whole's are rounded: u max |O| each, the parts'
    # weights summing to 1, and the weights' own rounding u max |v|
    u = 2.0 ** -8
    bound = 2 * u * max(float(x.abs().max()) for x in (oa, ob)) + 2 * u * 5
    assert float((o[0].transpose(0, 1) - whole_o.float()).abs().max()) <= bound
    assert float((lse[0] - whole_lse).abs().max()) <= 1e-4


def test_attn_tiny_wait_limit_reports_or_completes(ra):
    """Waits that run out end the kernels and are reported; the next call is
    right again."""
    x = make([4000, 900], [300, 1], 8, 2, 128, 16, torch.bfloat16, seed=16)
    want = _run(ra, x, True)
    assert ra.check_status() == ra.RA_OK
    try:
        ra.set_wait_limit_ns(1)
        for _ in range(3):
            _run(ra, x, True)
            assert ra.check_status() in (ra.RA_OK, ra.RA_ERR_DEVICE_TIMEOUT)
    finally:
        ra.set_wait_limit_ns(0)
    got = _run(ra, x, True)
    assert ra.check_status() == ra.RA_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


FIRST_CALL = """
import torch
import long_context_exact_ring_gb300 as ra
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
args = [i([0, 0]), i([3, 2]), i([[-1] * 4] * 2), i(list(range(8))), i([8, 0])]
out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in (2, 3, 5, 2)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ra.paged_kv_plan(*args, 8, 5, seq_lens_out=out[0], cu_q=out[1], slots=out[2], counts_out=out[3])
g.replay()
torch.cuda.synchronize()
assert [x.tolist() for x in out] == [[3, 2], [0, 3, 5], [56, 57, 58, 48, 49], [6, 0]], out
"""


def test_first_call_inside_a_capture(ra):
    """A process whose first call of the library is captured."""
    import subprocess
    import sys
    subprocess.run([sys.executable, "-c", FIRST_CALL], check=True, timeout=300)


def test_profile_names_the_kernels(ra):
    x = make([300, 200], [60, 1], 4, 2, 64, 16, torch.bfloat16, seed=17)
    ra.profile_reset()
    ra.profile_enable(True)
    try:
        _run(ra, x, True)
    finally:
        ra.profile_enable(False)
    counts = {k: v[0] for k, v in ra.profile_read().items()}
    ra.profile_reset()
    assert [counts["paged_" + k] for k in ("rows_kernel", "tiles_kernel", "join_kernel", "plan_kernel")] == [1, 1, 1, 0]


def test_refusals_on_the_gpu(ra):
    """Arguments that do not belong together, refused before a launch."""
    x = make([33], [2], 4, 2, 64, 16, torch.bfloat16, seed=18)
    a = {n: x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q")}

    def call(**kw):
        b = dict(a, **kw)
        extra = {k: b.pop(k) for k in list(b) if k not in a}
        return ra.paged_attn_fwd(b["q"], b["k_cache"], b["v_cache"], b["table"], b["seq_lens"], b["cu_q"], True, **extra)

    for wrong, kind in (
            (dict(q=a["q"].float()), TypeError), (dict(k_cache=a["k_cache"].half()), TypeError),
            (dict(v_cache=a["v_cache"][:-1]), ValueError), (dict(seq_lens=a["seq_lens"].long()), TypeError),
            (dict(cu_q=a["cu_q"][:1]), ValueError), (dict(table=a["table"].cpu()), ValueError),
            (dict(q=a["q"][:, :3]), ValueError), (dict(o=torch.empty_like(a["q"])[:1]), ValueError),
            (dict(lse=torch.empty(2, 4, device="cuda")), ValueError), (dict(scale=-1.0), ra.RingAttnError),
            (dict(q=a["q"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
            (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), ra.RingAttnError)):
        with pytest.raises(kind):
            call(**wrong)
    k = a["q"][:, :2]
    with pytest.raises(ValueError):
        ra.paged_kv_append(k, k[:1], a["k_cache"], a["v_cache"], _i32([0, 1]))
    with pytest.raises(ra.RingAttnError):
        ra.paged_kv_append(k, k, a["k_cache"][:, :12], a["v_cache"][:, :12], _i32([0, 1]))
    with pytest.raises(ValueError):
        ra.paged_kv_plan(_i32([0]), _i32([1, 1]), a["table"], _i32([0]), _i32([1, 0]), 16, 1)
    assert ra.check_status() == ra.RA_OK


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def _server(n, width, ps, H_kv, d, num, dtype):
    pools = [torch.full((num, ps, H_kv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    return dict(pools=pools, table=torch.full((n, width), -1, dtype=torch.int32, device="cuda"), ps=ps,
                free=torch.arange(num, dtype=torch.int32, device="cuda"), counts=_i32([num, 0]), lens=_i32([0] * n))


def _step(ra, srv, new, q, k, v, causal=True, **kw):
    lens, cu, slots, _ = ra.paged_kv_plan(srv["lens"], new, srv["table"], srv["free"], srv["counts"], srv["ps"],
                                          q.shape[0], seq_lens_out=srv["lens"], counts_out=srv["counts"])
    ra.paged_kv_append(k, v, *srv["pools"], slots)
    return ra.paged_attn_fwd(q, *srv["pools"], srv["table"], lens, cu, causal, **kw)


@pytest.mark.parametrize("H,H_kv,d", [(8, 2, 128), (4, 4, 64)])
def test_prompts_in_chunks_equal_whole_sequences(ra, H, H_kv, d):
    """Two prompts fed chunk by chunk and then token by token give what
    ring_attn_fwd gives for the whole sequences."""
    S = 384
    g = torch.Generator().manual_seed(0)
    q = torch.randn((2, H, S, d), generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn((2, H_kv, S, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    want_o, want_lse = ra.ring_attn_fwd(q, k, v, 1, True)
    srv = _server(2, 24, 16, H_kv, d, 50, torch.bfloat16)
    got_o, got_lse = torch.zeros_like(want_o), torch.zeros_like(want_lse)
    at = [0, 0]
    steps = [(100, 7), (28, 121), (200, 200), (53, 0), (1, 1), (1, 1), (1, 2), (0, 52)]
    for new in steps:
        part = [torch.cat([x[i, :, at[i]:at[i] + new[i]].transpose(0, 1) for i in range(2)]) for x in (q, k, v)]
        o, lse = _step(ra, srv, _i32(new), *part)
        row = 0
        for i in range(2):
            got_o[i, :, at[i]:at[i] + new[i]] = o[row:row + new[i]].transpose(0, 1)
            got_lse[i, :, at[i]:at[i] + new[i]] = lse[:, row:row + new[i]]
            row += new[i]
            at[i] += new[i]
    assert at == [S, S] and ra.check_status() == ra.RA_OK
    assert srv["lens"].tolist() == [S, S] and srv["counts"].tolist() == [2, 0]
    # Either result is within u (|O| + A) of the exact one, A <= max |v|
    # weighted, and rounded once more; 4 u max |v| covers both.
    assert float((got_o.double() - want_o.double()).abs().max()) <= 4 * 2.0 ** -8 * float(v.abs().max())
    assert float((got_lse - want_lse).abs().max()) <= 1e-3
    # ending both gives every page back
    ra.paged_kv_plan(srv["lens"], _i32([-1, -1]), srv["table"], srv["free"], srv["counts"], 16, 0,
                     seq_lens_out=srv["lens"], counts_out=srv["counts"])
    assert srv["counts"].tolist() == [50, 0] and sorted(srv["free"].tolist()) == list(range(50))


def test_captured_decode_step_replays_as_contexts_grow(ra):
    """A whole step captured once: lengths, pages and results move on with
    every replay."""
    n, H, H_kv, d, ps = 3, 8, 2, 128, 16
    srv = _server(n, 8, ps, H_kv, d, 20, torch.bfloat16)
    g = torch.Generator().manual_seed(3)
    rows = [[torch.randn((n, h, d), generator=g).to(torch.bfloat16).cuda() for h in (H, H_kv, H_kv)]
            for _ in range(40)]
    q, k, v = (torch.empty_like(x) for x in rows[0])
    new = _i32([1] * n)
    for x, y in zip((q, k, v), rows[0]):
        x.copy_(y)
    _step(ra, srv, new, q, k, v, max_q=1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = _step(ra, srv, new, q, k, v, max_q=1)
    for step in range(1, 40):
        for x, y in zip((q, k, v), rows[step]):
            x.copy_(y)
        graph.replay()
        if step in (1, 15, 16, 39):
            length = step + 1
            x = dict(q=q.cpu(), k_cache=srv["pools"][0].cpu(), v_cache=srv["pools"][1].cpu(),
                     table=srv["table"].cpu(), lens=[length] * n, news=[1] * n, cu=list(range(n + 1)))
            assert srv["lens"].tolist() == [length] * n
            o_ref, lse_ref, tol_o, tol_lse = attn_ref(x, True)
            assert_close(o, o_ref, tol_o, "O")
            assert_close(lse, lse_ref, tol_lse, "LSE")
            keys = torch.stack([y[1] for y in rows[:length]], 1).cpu()
            for i in range(n):
                c = torch.arange(length)
                assert torch.equal(x["k_cache"][x["table"][i].long()[c // ps], c % ps], keys[i])


def test_decode_over_the_long_shape(ra):
    """The last token of the 128K grouped-query shape, against 64 bits."""
    w = workloads.FWDBWD_GQA_128K
    g = torch.Generator("cuda").manual_seed(5)
    ps, num = 64, w.S // 64
    pools = [torch.randn((num, ps, w.H_kv, w.d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    table = torch.randperm(num, generator=g, device="cuda").to(torch.int32)[None]
    for new in (1, 5):
        q = torch.randn((new, w.H, w.d), generator=g, device="cuda").to(torch.bfloat16)
        o, lse = ra.paged_attn_fwd(q, *pools, table, _i32([w.S]), _i32([0, new]), True, max_q=new)
        assert ra.check_status() == ra.RA_OK
        k, v = (p[table[0].long()].flatten(0, 1) for p in pools)
        for h in (0, 13, 31):
            s = (q[:, h].double() @ k[:, h // 4].double().T) * w.scale
            for t in range(new):
                s[t, w.S - new + t + 1:] = float("-inf")
            want = torch.logsumexp(s, 1)
            p, vh = torch.exp(s - want[:, None]), v[:, h // 4].double()
            ref = p @ vh
            # E of tests/_paged.py is below 2^-12 here, n 2^-23 is 2^-6 u
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -6) * (p @ vh.abs())
            assert float((lse[h].double() - want).abs().max()) <= 1e-3
            assert bool(((o[:, h].double() - ref).abs() <= tol).all())
