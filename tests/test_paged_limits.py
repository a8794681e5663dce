"""Sizes of the paged calls at the edge of what their 32-bit indexes hold,
refused or accepted on the host; nothing is launched here."""
import pytest

FAKE = 1 << 20    # aligned and not null; never dereferenced


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    m.load_library()
    return m


@pytest.mark.parametrize("tokens", [(1 << 30) + 1, 2 ** 31 - 16384, 2 ** 31 - 1])
def test_plan_refuses_more_slots_than_its_indexes_hold(ra, tokens):
    """Threads step through the slots 2^14 at a time in 32 bits."""
    rc = ra.load_library().paged_kv_plan(FAKE, FAKE, 4, FAKE, 8, 8, FAKE, 32, FAKE, 16, tokens, FAKE, FAKE, FAKE, FAKE,
                                         None)
    assert rc == ra.RA_ERR_UNSUPPORTED
