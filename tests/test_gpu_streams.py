"""Calls on a stream of their own (stream=): what they allocate is not memory
that work queued on the current stream still uses, and what they return may be
used on the current stream and dropped there."""
import pytest
import torch

from _paged import make

pytestmark = pytest.mark.gpu

SLEEP = 100_000_000     # clock ticks, about 50 ms


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _free_memory_with_queued_writes(sizes):
    """Blocks of these sizes, free to the current stream, which has yet to
    write them."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(SLEEP)
    for b in blocks:
        b.fill_(0x7f)


def _check(call, sizes):
    """call(stream) -> tensors; the same results whatever the current stream is at."""
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _free_memory_with_queued_writes(sizes)
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # read late on the current stream, dropped, and the call repeated
    torch.cuda._sleep(SLEEP)
    kept = [t.clone() for t in got]
    del got
    for _ in range(2):
        for t in call(side):
            with torch.cuda.stream(side):
                t.zero_()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


@pytest.mark.parametrize("news", [[1, 1, 1], [1, 130, 30]])
def test_paged_attn_on_its_own_stream(ra, news):
    x = make([5000, 2000, 77], news, 8, 2, 128, 16, torch.bfloat16, seed=12)
    args = [x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q")]
    T, H, d = args[0].shape
    _check(lambda s: ra.paged_attn_fwd(*args, True, stream=s),
           [2 * T * H * d, 4 * T * H, ra.paged_attn_workspace_size(3, T, H, 2, d)])


def test_paged_plan_on_its_own_stream(ra):
    i32 = dict(dtype=torch.int32, device="cuda")
    n, tokens = 300, 5000
    lens, new = torch.arange(n, **i32), torch.full((n,), 16, **i32)
    table = torch.arange(n * 40, **i32).reshape(n, 40)
    free, counts = torch.arange(n * 40, n * 42, **i32), torch.tensor([n * 2, 0], **i32)
    _check(lambda s: ra.paged_kv_plan(lens, new, table, free, counts, 16, tokens, stream=s),
           [4 * n, 4 * (n + 1), 4 * tokens, 8])


@pytest.mark.parametrize("handle", [0, 1, 2, "of a stream"])
def test_paged_calls_on_a_stream_given_by_its_handle(ra, handle):
    """The calls run on the stream that the handle names (0 to 2: the default
    ones), behind what is queued there."""
    x = make([700, 90], [1, 30], 8, 2, 128, 16, torch.bfloat16, seed=3)
    q, k, v, table, lens, cu = (x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q"))
    want = ra.paged_attn_fwd(q, k, v, table, lens, cu, True)
    stream = torch.cuda.Stream() if handle == "of a stream" else torch.cuda.default_stream()
    late, rows, pools = torch.zeros_like(q), k[:2, 0], [torch.zeros_like(k) for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(SLEEP)
        late.copy_(q)
        for p in pools:
            p.fill_(1.0)
    handle = stream.cuda_stream if handle == "of a stream" else handle
    with torch.cuda.stream(torch.cuda.Stream()):
        got = ra.paged_attn_fwd(late, k, v, table, lens, cu, True, stream=handle)
        ra.paged_kv_append(rows, rows, *pools, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for p in pools:
        assert torch.equal(p[0, :2].nan_to_num(7.0), rows.nan_to_num(7.0)) and (p[1:] == 1).all()


def _ring_inputs(dtype=torch.bfloat16):
    g = torch.Generator("cuda").manual_seed(4)
    return [torch.randn((1, 4, 512, 64), generator=g, device="cuda").to(dtype) for _ in range(4)]


@pytest.mark.parametrize("name", ["ring_attn_fwd", "ring_attn_fwd_f32", "ring_attn_fwd_emulated",
                                  "ring_attn_fwd_ulysses_emulated"])
def test_ring_forward_on_its_own_stream(ra, name):
    q, k, v, _ = _ring_inputs(torch.float32 if name == "ring_attn_fwd_f32" else torch.bfloat16)
    work = {"ring_attn_fwd": 1, "ring_attn_fwd_f32": ra.fwd_f32_workspace_size(1, 4, 4, 512, 64),
            "ring_attn_fwd_emulated": ra.emulated_workspace_size(1, 4, 512, 64),
            "ring_attn_fwd_ulysses_emulated": ra.ulysses_workspace_size(1, 4, 4, 512, 64)}[name]
    _check(lambda s: getattr(ra, name)(q, k, v, 2, True, stream=s), [q.numel() * q.element_size(), 4 * 4 * 512, work])


def test_ring_backward_and_merge_on_their_own_stream(ra):
    q, k, v, do = _ring_inputs()
    o, lse = ra.ring_attn_fwd(q, k, v, 2, True)
    # dQ is summed in no fixed order: dK and dV are compared bit by bit
    _check(lambda s: ra.ring_attn_bwd(q, k, v, o, lse, do, 2, True, stream=s)[1:],
           [2 * q.numel()] * 3 + [ra.bwd_workspace_size(1, 4, 512, 64)])
    a, b, lse_b = o.float(), do.float(), lse + 1
    _check(lambda s: ra.attn_merge_partials(a, lse, b, lse_b, stream=s), [4 * q.numel(), 4 * 4 * 512])


@pytest.mark.parametrize("fork", [False, True])
def test_captured_on_a_stream_that_is_named(ra, fork):
    """stream= inside a capture: the capture's own stream, or one that forks off
    it and joins it again."""
    x = make([700, 90, 3000], [1, 30, 1], 8, 2, 128, 16, torch.bfloat16, seed=3)
    args = [x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q")]
    want = ra.paged_attn_fwd(*args, True)
    q, k, v, _ = _ring_inputs()
    want_ring = ra.ring_attn_fwd(q, k, v, 2, True)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        stream = side if fork else main
        side.wait_stream(main)
        got = ra.paged_attn_fwd(*args, True, stream=stream)
        ring = ra.ring_attn_fwd(q, k, v, 2, True, stream=stream)
        main.wait_stream(side)
    for _ in range(2):
        for t in (*got, *ring):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *ring), (*want, *want_ring)))
