"""The paged key/value cache calls without a GPU: argument checks before
anything is launched, and the index arithmetic that device data decides."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_exact_ring_gb300", "csrc")
FAKE = 1 << 20    # aligned and not null; never dereferenced


@pytest.fixture(scope="module")
def ra():
    import long_context_exact_ring_gb300 as m
    from long_context_exact_ring_gb300 import build
    build.build()
    m.load_library()
    return m


def _plan(ra, n=4, stride=8, max_pages=8, num_pages=32, page_size=16, tokens=4, table=FAKE, lens=FAKE, slots=FAKE):
    return ra.load_library().paged_kv_plan(lens, FAKE, n, table, stride, max_pages, FAKE, num_pages, FAKE, page_size,
                                           tokens, FAKE, FAKE, slots, FAKE, None)


@pytest.mark.parametrize("change,code", [
    (dict(n=-1), -1), (dict(tokens=-1), -1), (dict(max_pages=0), -1), (dict(stride=7), -1), (dict(num_pages=0), -1),
    (dict(page_size=0), -1), (dict(page_size=20), -2), (dict(n=8193), -2), (dict(num_pages=1 << 27), -2),
    (dict(max_pages=1 << 27, stride=1 << 27), -2), (dict(n=8192, max_pages=1 << 18, stride=1 << 18), -2),
    (dict(table=0), -1), (dict(table=FAKE + 2), -1), (dict(lens=FAKE + 1), -1), (dict(slots=0), -1),
])
def test_plan_refuses(ra, change, code):
    assert _plan(ra, **change) == code


def _strides(*x):
    return (ctypes.c_longlong * len(x))(*x)


def _append(ra, k=FAKE, ks=None, cache=FAKE, cs=None, slots=FAKE, tokens=4, H=2, d=128, pages=8, ps=16):
    return ra.load_library().paged_kv_append(k, ks, FAKE, None, cache, cs, FAKE, None, slots, tokens, H, d, pages, ps,
                                             None)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), -1), (dict(H=0), -1), (dict(d=96), -2), (dict(ps=12), -2), (dict(pages=0), -1),
    (dict(pages=1 << 27), -2), (dict(k=0), -1), (dict(k=FAKE + 8), -1), (dict(cache=0), -1), (dict(slots=0), -1),
    (dict(slots=FAKE + 2), -1), (dict(ks=_strides(4, 128)), -1), (dict(ks=_strides(256, -128)), -1),
    (dict(cs=_strides(1 << 35, 256, 128)), -1), (dict(cs=_strides(4096, 0, 128)), -1),
])
def test_append_refuses(ra, change, code):
    assert _append(ra, **change) == code


def test_empty_append_touches_nothing(ra):
    assert _append(ra, tokens=0, k=0, cache=0, slots=0) == 0


def _attn(ra, q=FAKE, qs=None, kc=FAKE, cs=None, table=FAKE, stride=8, o=FAKE, lse=FAKE, dtype=0, n=2, tokens=4, H=8,
          Hkv=2, d=128, pages=32, ps=16, max_pages=8, max_q=4, causal=1, scale=0.1, ws=FAKE, ws_bytes=None):
    lib = ra.load_library()
    if ws_bytes is None:
        ws_bytes = lib.paged_attn_workspace_size(n, tokens, H, Hkv, d)
    return lib.paged_attn_fwd(q, qs, kc, cs, FAKE, None, table, stride, FAKE, FAKE, o, None, lse, dtype, n, tokens, H,
                              Hkv, d, pages, ps, max_pages, max_q, causal, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(n=-1), -1), (dict(tokens=-1), -1), (dict(H=0), -1), (dict(H=9), -1), (dict(Hkv=0), -1), (dict(d=96), -2),
    (dict(d=256), -2), (dict(ps=17), -2), (dict(pages=0), -1), (dict(max_pages=0), -1), (dict(stride=7), -1),
    (dict(max_pages=1 << 27, stride=1 << 27), -2), (dict(max_q=-1), -1), (dict(causal=2), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(dtype=2), -1),
    (dict(H=258, Hkv=2), -2), (dict(tokens=1 << 30), -2), (dict(pages=1 << 27), -2), (dict(q=0), -1),
    (dict(q=FAKE + 8), -1), (dict(kc=FAKE + 4), -1), (dict(o=0), -1), (dict(lse=FAKE + 2), -1), (dict(table=0), -1),
    (dict(ws=0), -1), (dict(ws=FAKE + 16), -1), (dict(ws_bytes=0), -1), (dict(qs=_strides(1024, 12)), -1),
    (dict(cs=_strides(1 << 35, 256, 128)), -1),
])
def test_attn_refuses(ra, change, code):
    assert _attn(ra, **change) == code


def test_empty_attn_touches_nothing(ra):
    assert _attn(ra, n=0, q=0, kc=0, table=0, o=0, lse=0, ws=0) == 0
    assert _attn(ra, tokens=0, q=0, kc=0, table=0, o=0, lse=0, ws=0) == 0


def test_workspace_does_not_depend_on_lengths(ra):
    size = ra.paged_attn_workspace_size
    assert size(0, 4, 8, 2, 128) == size(2, 0, 8, 2, 128) == size(2, 4, 8, 3, 128) == size(2, 4, 8, 2, 96) == 0
    assert size(2, 4, 8, 2, 128) > 0


def test_bad_page_status_has_a_name(ra):
    assert ra.status_string(ra.RA_ERR_BAD_PAGE) == "RA_ERR_BAD_PAGE"


def test_binding_refuses_host_tensors(ra):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    pool = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ra.paged_kv_plan(i(2), i(2), i(2, 4), i(8), i(2), 16, 2)
    with pytest.raises(ValueError):
        ra.paged_kv_append(x[:, :2], x[:, :2], pool, pool, i(2))
    with pytest.raises(ValueError):
        ra.paged_attn_fwd(x, pool, pool, i(2, 4), i(2), i(3), True)
    with pytest.raises(TypeError):
        ra.paged_attn_fwd(None, pool, pool, i(2, 4), i(2), i(3), True)


INDEX_PROGRAM = r"""
#include "paged_index.h"
#include <climits>
#include <cstdio>
#include <initializer_list>
using namespace ra::paged;
int main()
{
    const int odd[] = {INT_MIN, -5, -1, 0, 1, 7, 8, 40, 41, 1000, INT_MAX};
    for (int tokens : {0, 1, 40})
        for (int width : {1, 5, 1 << 20})
            for (int ps : {8, 48, 256})
                for (int a : odd) for (int b : odd) for (int len : odd) {
                    const Request r = cut_request(a, b, len, tokens, width, ps);
                    if (r.first < 0 || r.q < 0 || r.first + r.q > tokens || r.len < 0 ||
                        r.len > (long long)width * ps) { std::printf("cut %d %d %d\n", a, b, len); return 1; }
                    if (a >= 0 && b >= a && b <= tokens && (r.first != a || r.q != b - a)) return 2;
                    if (len >= 0 && len <= (long long)width * ps && r.len != len) return 3;
                    if (r.len > 0 && page_index(r.len - 1, ps, -1) >= width) return 4;
                }
    for (int s = 3; s < 12; ++s)
        for (int key = 0; key < 100000; key += 7)
            if (page_index(key, 1 << s, s) != page_index(key, 1 << s, -1)) return 5;
    for (int page : odd)
        if (page_ok(page, 41) != (page >= 0 && page < 41)) return 6;
    // shares of the work: sums of a request's tiles against the tiles one by one
    for (int q : {1, 31, 32, 33, 64, 100, 509, 1500})
        for (int len : {0, 1, 5, 63, 64, 65, 128, 500, 509, 512, 4096, 131072})
            for (int causal : {0, 1}) for (int step : {1, 2, 36, 64, 256}) for (int unit : {16, 128}) {
                const TileWork w{q, len, causal, step, unit, unit == 16 ? 0 : 3};
                long long sum = 0;
                for (int t = 0; t < w.tiles(); ++t) {
                    if (w.before(t) != sum) { std::printf("sum %d %d %d %d\n", q, len, step, t); return 8; }
                    if (w.tile_of(sum, 0, w.tiles()) != t || w.tile_of(sum + w.units(t) + w.extra - 1, t, w.tiles()) != t) return 9;
                    int seen = causal ? len - q + ((t + 1) * step < q ? (t + 1) * step : q) : len;
                    if (seen < 0) seen = 0;
                    if (w.units(t) < 1 || w.units(t) * unit < seen || (w.units(t) > 1 && (w.units(t) - 1) * unit >= seen))
                        return 10;
                    sum += w.units(t) + w.extra;
                }
                if (w.before(w.tiles()) != sum) return 11;
            }
    for (long long total : {0ll, 1ll, 151ll, 152ll, 153ll, 99999ll, (1ll << 32) + 5, (1ll << 58) + 12345})
        for (int blocks : {1, 2, 152, 256, 65535}) {
            long long at = 0;
            for (int b = 0; b < blocks; ++b) {
                const Share s = share_of(total, blocks, b);
                if (s.start != at || s.count < total / blocks || s.count > total / blocks + 1) return 13;
                at += s.count;
            }
            if (at != total) return 14;
        }
    for (long long size : {1ll, 7ll, 1ll << 40})
        for (int count : {1, 2, 8, 1000})
            for (int x : {0, 1, 6, 7, 500, 999})
                if (x < count && (quotient_below(x * size, size, count) != x ||
                                  quotient_below(x * size + size - 1, size, count) != x)) return 15;
    if (cut_units(0, 3) != 0 || cut_units(3, 3) != 0 || cut_units(4, 3) != 1 || cut_units(7, 0) != 7) return 16;
    {   // the largest that the calls accept
        const TileWork w{1 << 30, 1 << 30, 1, 1, 16, 3};
        if (w.before(w.tiles()) <= 0 || w.tile_of(w.before(w.tiles()) - 1, 0, w.tiles()) != w.tiles() - 1) return 12;
    }
    // rows past 2^32 elements, and a row behind the last page never named
    const PoolLayout l{8ll * 16 * 128, 128, 16 * 128};
    if (row_offset(l, 1 << 20, 15, 7) != (1ll << 20) * l.sp + 15 * 128 + 7ll * 16 * 128) return 7;
    return 0;
}
"""


def test_index_arithmetic_stays_in_range(tmp_path):
    cxx = shutil.which("g++") or pytest.skip("no g++")
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(INDEX_PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


@pytest.mark.parametrize("seed", range(4))
def test_plan_reference_keeps_every_page_once(seed):
    """The tests' own reference: no page is lost or given twice."""
    import random

    from _paged import pages, plan_ref
    rng = random.Random(seed)
    ps, n, width, num = 8, 5, 6, 24
    lens, table, free, count = [0] * n, [[-1] * width for _ in range(n)], list(range(num)), [num, 0]
    for _ in range(40):
        new = [rng.choice([-1, 0, 1, 1, 5, 20]) for _ in range(n)]
        lens, cu, slots, count, table, free = plan_ref(lens, new, table, free, count, ps, 60)
        held = [p for a, row in zip(lens, table) for p in row[:pages(a, ps)]]
        assert sorted(held + free[:count[0]]) == list(range(num))
        got = [s for s in slots if s >= 0]
        assert len(set(got)) == len(got)
