"""Infinities in V of a paged cache: a row that sees one gets it, with its sign,
whichever kernel serves the row; infinities of both signs in one column give
NaN.  The weights of these batches are far from underflow in every type."""
import pytest
import torch

from _paged import assert_close, attn_ref, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _put(x, request, key, head, col, value):
    ps = x["v_cache"].shape[1]
    x["v_cache"][x["table"][request, key // ps], key % ps, head, col] = value


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_q", [1, 10 ** 6])      # paged_rows_kernel for all; both kernels
@pytest.mark.parametrize("lens,news,H,H_kv", [
    ([1, 1], [1, 1], 2, 1),             # one key, of weight 1
    ([2, 3, 17], [1, 1, 1], 4, 2),      # less than a step of keys
    ([400, 256], [1, 1], 4, 2),         # units whose keys every row sees
    ([60, 290], [3, 7], 4, 2),          # units that end inside the new tokens
    ([60, 290], [40, 130], 4, 2),       # rows for tiles of 128
])
def test_infinity_in_v(ra, dtype, d, max_q, lens, news, H, H_kv):
    x = make(lens, news, H, H_kv, d, 16, dtype, seed=len(lens) + d, peak=0.5)
    inf = float("inf")
    for i, length in enumerate(lens):
        first = length // 3                                  # every row sees it, unless the request is all new
        late = length - (news[i] + 1) // 2                   # only the later of several new tokens do
        _put(x, i, first, 0, 3, inf)
        _put(x, i, first, H_kv - 1, 8, -inf)
        _put(x, i, late, 0, 20, -inf)
        _put(x, i, late, H_kv - 1, d - 1, inf)
        if first != late:
            _put(x, i, first, 0, 41, inf)
            _put(x, i, late, 0, 41, -inf)
    args = [x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q")]
    o, lse = ra.paged_attn_fwd(*args, True, max_q=max_q)
    assert ra.check_status() == ra.RA_OK
    o_ref, lse_ref, tol_o, tol_lse = attn_ref(x, True)
    assert torch.isinf(o_ref).any()
    assert_close(o, o_ref, tol_o, "O")
    assert_close(lse, lse_ref, tol_lse, "LSE")
