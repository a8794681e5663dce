"""paged_attn_fwd's sums over contexts cut into many parts, and its weights,
within bounds that show a lost, doubled or misplaced part and a weight rounded
once (tests/_paged_sums.py; tests/test_paged_sums_bounds.py plants them)."""
import pytest
import torch

from _paged import U, assert_close, make
from _paged_sums import balance, misses, reference, spread

pytestmark = pytest.mark.gpu

BLOCKS = 152


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    return m


def _check(ra, x, rho, units, **kw):
    args = [x[n].cuda() for n in ("q", "k_cache", "v_cache", "table", "seq_lens", "cu_q")]
    o, lse = ra.paged_attn_fwd(*args, True, **kw)
    assert ra.check_status() == ra.RA_OK
    ref = reference(x, "cuda")
    worst, mean = misses(o, ref, x["q"].dtype, rho, units)
    assert worst <= 1 and mean <= 1, (worst, mean)
    n = max(x["lens"])
    assert_close(lse, ref["lse"], ref["e"][..., 0].T + n * 2.0 ** -24 + 2.0 ** -23 * ref["lse"].abs(), "LSE")


def _rho(dtype, rows_kernel):
    return 2.0 ** -16 if rows_kernel and dtype == torch.bfloat16 else U[dtype]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,news,H,H_kv,d,ps", [
    ([38911], [1], 2, 1, 64, 64),            # one head over all blocks
    ([38911], [2], 8, 1, 128, 128),          # a full tile of 16 rows
    ([65613], [1], 8, 2, 128, 16),
    ([20000, 9001, 70, 31000], [1, 3, 1, 2], 8, 2, 64, 48),
])
def test_few_new_tokens(ra, dtype, lens, news, H, H_kv, d, ps):
    x = make(lens, news, H, H_kv, d, ps, dtype, seed=sum(lens))
    spread(x, 64, 3)
    unit = 128 if d == 128 else 256
    total = sum(-(-a // unit) + 2 for a in lens) * H_kv
    _check(ra, x, _rho(dtype, True), total // BLOCKS + 1, max_q=1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,news,H,H_kv,d,ps", [
    ([38911], [70], 2, 1, 64, 64),
    ([38911], [300], 1, 1, 128, 136),
    ([65613], [40], 8, 2, 128, 16),
    ([9000, 2501, 700], [300, 40, 700], 4, 2, 64, 48),
])
def test_many_new_tokens(ra, dtype, lens, news, H, H_kv, d, ps):
    x = make(lens, news, H, H_kv, d, ps, dtype, seed=sum(lens))
    spread(x, 64, 4)
    step = 2 * (128 // (H // H_kv))
    total = sum((-(-a // 128) + 3) * -(-q // step) for a, q in zip(lens, news)) * H_kv
    _check(ra, x, _rho(dtype, False), max(5, total // BLOCKS + 1), max_q=max(news))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [2, 7, 40, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_few_new_tokens(ra, dtype, n, d):
    """O close to 0: what rounding a weight leaves out would show."""
    x = make([n] * 6, [1] * 6, 8, 8, d, 16, dtype, seed=n)
    balance(x)
    _check(ra, x, _rho(dtype, True), 3, max_q=1)
