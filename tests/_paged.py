"""Plain references of the paged key/value cache calls, in whole numbers and
64 bits, and the inputs the tests share.

Tolerances of paged_attn_fwd, from the roundings it makes.  u is half a step
of the type (2^-8 bf16, 2^-11 fp16).  A score is a d-term fp32 sum: off by at
most d 2^-24 B, B = scale sum_i |q_i k_i|; its scaling and the subtraction of
the reference each add 2^-24 of a value no larger than 4 max |s| + 32, and
the exponential 2^-22: together E.  A weight is off by E and, rounded for the
product with V, by u; sums over n keys add n 2^-24.  With A = sum_c p_c |v_c|
    |O - O_ref| <= u |O_ref| + (u + 2 E + n 2^-23) A
    |LSE - LSE_ref| <= E + n 2^-24 + 2^-23 |LSE_ref|.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def pages(tokens, page_size):
    return -(-tokens // page_size)


def make(lens, news, H, H_kv, d, page_size, dtype, *, layout="thd", seed=0, peak=1.0, rows_behind=0):
    """CPU tensors of a batch: pools that hold NaN wherever no key was
    written, table entries of no page behind each context."""
    g = torch.Generator().manual_seed(seed)
    used = [pages(a, page_size) for a in lens]
    num_pages = sum(used) + 2
    ids = torch.randperm(num_pages, generator=g).to(torch.int32)
    n, width = len(lens), max(used + [1]) + 1
    table = torch.full((n, width), -7, dtype=torch.int32)
    at = 0
    for i, x in enumerate(used):
        table[i, :x] = ids[at:at + x]
        at += x
    pools = []
    for _ in range(2):
        c = torch.full((num_pages, page_size, H_kv, d), float("nan"), dtype=dtype)
        for i, a in enumerate(lens):
            for p in range(used[i]):
                m = min(page_size, a - p * page_size)
                c[table[i, p], :m] = torch.randn((m, H_kv, d), generator=g).to(dtype)
        if layout == "htd":
            c = c.transpose(1, 2).contiguous().transpose(1, 2)
        pools.append(c)
    T = sum(news) + rows_behind
    q = (torch.randn((T, H, d), generator=g) * peak).to(dtype)
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    return dict(q=q, k_cache=pools[0], v_cache=pools[1], table=table, lens=list(lens), news=list(news), cu=cu,
                seq_lens=torch.tensor(lens, dtype=torch.int32), cu_q=torch.tensor(cu, dtype=torch.int32))


def attn_ref(x, causal, scale=None):
    """(O, LSE, tolerance of O, tolerance of LSE) in 64 bits; rows of no
    request are NaN in all four."""
    q, ps = x["q"], x["k_cache"].shape[1]
    T, H, d = q.shape
    H_kv = x["k_cache"].shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    u = U[q.dtype]
    o = torch.full((T, H, d), float("nan"), dtype=torch.float64)
    lse = torch.full((H, T), float("nan"), dtype=torch.float64)
    tol_o, tol_lse = torch.zeros_like(o), torch.zeros_like(lse)
    for i, length in enumerate(x["lens"]):
        c = torch.arange(length)
        page = x["table"][i].long()[c // ps] if length else c
        k = x["k_cache"][page, c % ps].double()
        v = x["v_cache"][page, c % ps].double()
        for t in range(x["news"][i]):
            row = x["cu"][i] + t
            m = max(0, length - x["news"][i] + t + 1) if causal else length
            for h in range(H):
                j = h // (H // H_kv)
                if m == 0:
                    o[row, h], lse[h, row] = 0.0, float("-inf")
                    continue
                qr = q[row, h].double()
                s = scale * (k[:m, j] @ qr)
                b = scale * (k[:m, j].abs() @ qr.abs()).max()
                big = s.max()
                w = torch.exp(s - big)
                total = w.sum()
                p = w / total
                o[row, h] = p @ v[:m, j]
                lse[h, row] = big + total.log()
                e = d * 2.0 ** -24 * b + 2.0 ** -23 * (4 * s.abs().max() + 32) + 2.0 ** -22
                tol_o[row, h] = u * o[row, h].abs() + (u + 2 * e + m * 2.0 ** -23) * (p @ v[:m, j].abs())
                tol_lse[h, row] = e + m * 2.0 ** -24 + 2.0 ** -23 * lse[h, row].abs()
    return o, lse, tol_o, tol_lse


def attn_ref_causal(x):
    """attn_ref(x, True) for longer batches: a matrix product for each request
    and head.  V may hold infinities and NaN."""
    q, ps = x["q"], x["k_cache"].shape[1]
    T, H, d = q.shape
    H_kv = x["k_cache"].shape[2]
    scale, u = 1.0 / math.sqrt(d), U[q.dtype]
    o = torch.full((T, H, d), float("nan"), dtype=torch.float64)
    lse = torch.full((H, T), float("nan"), dtype=torch.float64)
    tol_o, tol_lse = torch.zeros_like(o), torch.zeros_like(lse)
    for i, length in enumerate(x["lens"]):
        c = torch.arange(length)
        page = x["table"][i].long()[c // ps]
        k = x["k_cache"][page, c % ps].double()
        v = x["v_cache"][page, c % ps].double()
        rows = slice(x["cu"][i], x["cu"][i] + x["news"][i])
        m = length - x["news"][i] + torch.arange(x["news"][i]) + 1       # keys that a row sees
        seen = c[None, :] < m[:, None]
        for h in range(H):
            j = h // (H // H_kv)
            qr = q[rows, h].double()
            s = scale * (qr @ k[:, j].T)
            b = (scale * (qr.abs() @ k[:, j].abs().T)).where(seen, 0.0).amax(1)
            most = s.abs().where(seen, 0.0).amax(1)
            s = s.where(seen, float("-inf"))
            lse[h, rows] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            finite = torch.where(torch.isfinite(v[:, j]), v[:, j], 0.0)
            out = p @ finite
            e = d * 2.0 ** -24 * b + 2.0 ** -23 * (4 * most + 32) + 2.0 ** -22
            tol_o[rows, h] = u * out.abs() + (u + 2 * e + m * 2.0 ** -23)[:, None] * (p @ finite.abs())
            tol_lse[h, rows] = e + m * 2.0 ** -24 + 2.0 ** -23 * lse[h, rows].abs()
            for key, col in (~torch.isfinite(v[:, j])).nonzero().tolist():
                out[:, col] += torch.where(seen[:, key], p[:, key] * v[key, j, col], 0.0)
            o[rows, h] = out
    return o, lse, tol_o, tol_lse


def assert_close(got, want, tol, what):
    got = got.detach().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(torch.where(inf, got, 0.0), torch.where(inf, want, 0.0)), f"{what}: infinities"
    err = torch.where(torch.isfinite(want), (got - want).abs() - tol, -1.0)
    worst = float(err.max()) if err.numel() else -1.0
    assert worst <= 0, f"{what}: {worst:.3e} beyond the tolerance"


def plan_ref(seq_lens, new_lens, table, free, counts, page_size, tokens):
    """One request after the other.  Lists in, lists out:
    (seq_lens, cu_q, slots, counts, table, free)."""
    table, stack, top = [list(r) for r in table], list(free), counts[0]
    width = len(table[0]) if table else 0
    for i, q in enumerate(new_lens):
        if q < 0:
            for p in table[i][:pages(seq_lens[i], page_size)]:
                stack[top] = p
                top += 1
    out, cu, slots, refused, empty = [], [0], [-1] * tokens, 0, False
    for i, (a, q) in enumerate(zip(seq_lens, new_lens)):
        cu.append(cu[-1] + max(q, 0))
        if q < 0:
            out.append(0)
            continue
        have, want = pages(a, page_size), pages(a + q, page_size)
        ok = want <= width and cu[-1] <= tokens
        if ok and want > have and (empty or want - have > top):
            ok, empty = False, True
        if not ok:
            refused += 1
            out.append(a)
            continue
        for p in range(have, want):
            top -= 1
            table[i][p] = stack[top]
        for t in range(q):
            slots[cu[i] + t] = table[i][(a + t) // page_size] * page_size + (a + t) % page_size
        out.append(a + q)
    return out, cu, slots, [top, refused], table, stack
