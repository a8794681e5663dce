"""References and bounds for the sums of paged_attn_fwd over long contexts, and
for its weights, in 64 bits.

V is constant over ranges of keys and differs from range to range (spread), so
that a part of a context that is lost, counted twice or weighted by another
part's factor moves O by far more than the bounds.

Bounds, counting the roundings as they are made.  E is the error of a weight
before it is rounded (tests/_paged.py); rho what rounding it leaves: 2^-16 where
bf16 weights are multiplied in two parts (paged_rows_kernel), else half a step
u.  A block adds `units` pieces of keys one behind the other, at most 10
additions, rescalings and exponentials each, then 8 warps and at most 160 parts
are added: with 2^-22 for each (a tensor core cuts where it aligns),
sigma = (10 units + 168) 2^-22.  A = sum_c p_c |v_c|.
    every entry:   |O - O_ref| <= u |O_ref| + (rho + 2 E + sigma) A
    on average:    the rounding of one weight is independent of another's, so
                   the mean square over all entries stays below
                   4 mean(u^2 O_ref^2 + rho^2 sum_c p_c^2 v_c^2)
                   plus 2 mean(((2 E + sigma) A)^2)
where the factor 4 is room for what the mean of some thousand entries, not
quite independent, may be off by."""
import math

import torch

from _paged import U


def spread(x, size, seed):
    """V of a batch of tests/_paged.py: one value for each range of `size` keys,
    column and head, of magnitude 0.5 to 1 and any sign."""
    g = torch.Generator().manual_seed(seed)
    v, ps = x["v_cache"], x["v_cache"].shape[1]
    for i, length in enumerate(x["lens"]):
        c = torch.arange(length)
        values = torch.rand((length // size + 1, *v.shape[2:]), generator=g) * 0.5 + 0.5
        values *= (torch.rand(values.shape, generator=g) < 0.5) * 2.0 - 1.0
        v[x["table"][i].long()[c // ps], c % ps] = values[c // size].to(v.dtype)


def reference(x, device="cpu", scale=None, planted=None):
    """Causal attention in 64 bits, as a dict: o, lse, a (sum p |v|), s2 (sum p^2
    v^2), e (E).  planted(p, i) -> p changes the weights [rows, keys] of request i
    before they meet V: a mistake for a test of the bounds."""
    q, ps = x["q"], x["k_cache"].shape[1]
    T, H, d = q.shape
    group = H // x["k_cache"].shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = {n: torch.zeros((T, H, d), dtype=torch.float64) for n in ("o", "a", "s2")}
    out["e"] = torch.zeros((T, H, 1), dtype=torch.float64)
    out["lse"] = torch.zeros((H, T), dtype=torch.float64)
    for i, length in enumerate(x["lens"]):
        c = torch.arange(length)
        page = x["table"][i].long()[c // ps]
        rows = slice(x["cu"][i], x["cu"][i] + x["news"][i])
        seen = (c[None, :] < (length - x["news"][i] + torch.arange(x["news"][i]) + 1)[:, None]).to(device)
        for h in range(H):
            if h % group == 0:
                k = x["k_cache"][page, c % ps, h // group].to(device).double()
                v = x["v_cache"][page, c % ps, h // group].to(device).double()
            qr = q[rows, h].to(device).double()
            s = scale * (qr @ k.T)
            b = (scale * (qr.abs() @ k.abs().T)).where(seen, 0.0).amax(1)
            most = s.abs().where(seen, 0.0).amax(1)
            s = s.where(seen, float("-inf"))
            p = torch.softmax(s, 1)
            out["lse"][h, rows] = torch.logsumexp(s, 1).cpu()
            out["a"][rows, h] = (p @ v.abs()).cpu()
            out["s2"][rows, h] = (p ** 2 @ v ** 2).cpu()
            out["e"][rows, h, 0] = (d * 2.0 ** -24 * b + 2.0 ** -23 * (4 * most + 32) + 2.0 ** -22).cpu()
            out["o"][rows, h] = ((p if planted is None else planted(p, i)) @ v).cpu()
    return out


def misses(got, ref, dtype, rho, units):
    """By how much O misses the bound of its entries (the worst entry over its
    bound) and that of the mean square: (x, y), both at most 1 where it holds."""
    u = U[dtype]
    sigma = (10 * units + 168) * 2.0 ** -22
    err = (got.detach().cpu().double() - ref["o"]).abs()
    rest = (2 * ref["e"] + sigma) * ref["a"]
    worst = (err / (u * ref["o"].abs() + rho * ref["a"] + rest)).max()
    mean = 4 * (u ** 2 * ref["o"] ** 2 + rho ** 2 * ref["s2"]).mean() + 2 * (rest ** 2).mean()
    return float(worst), float((err ** 2).mean() / mean)


def balance(x):
    """Sets V's first key of every request so that O is close to 0 (one query
    head to a key/value head, one new token): rounding O then hides nothing of
    the weights' errors."""
    ps = x["v_cache"].shape[1]
    for i, length in enumerate(x["lens"]):
        c = torch.arange(length)
        page, row = x["table"][i].long()[c // ps], x["cu"][i]
        for h in range(x["q"].shape[1]):
            s = (x["k_cache"][page, c % ps, h].double() @ x["q"][row, h].double()) / math.sqrt(x["q"].shape[2])
            p = torch.softmax(s, 0)
            v = x["v_cache"][page, c % ps, h].double()
            first = v[0] - (p @ v) / p[0]
            x["v_cache"][page[0], 0, h] = first.to(x["v_cache"].dtype)
