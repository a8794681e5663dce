"""The paged key/value cache operators, case by case: what a serving program
calls between a prompt's first chunk and its last token.

    plan     paged_kv_plan: pages, slots and lengths of the next step
    append   paged_kv_append: the new tokens' K and V rows into the pool
    attn     paged_attn_fwd: the new tokens' attention over their contexts

Each case runs either through this package (``own`` true) or in its plain
form: elementary torch operations, 32-bit arithmetic, rounded once at the end.
"""
import math
import random

import torch

own = False

if own:   # the plain forms need nothing of the package
    import long_context_exact_ring_gb300  # noqa: F401

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _pages(tokens, page_size):
    return -(-tokens // page_size)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _plan(name, n, ctx, chunk, page_size, mode):
    """n requests with up to ctx cached tokens; mode decode adds one token to
    each, chunk gives a quarter of them up to `chunk` new tokens, churn also
    ends a fifth of them and leaves the pool short of a few pages."""
    return {"name": name, "op": "plan", "n": n, "ctx": ctx, "chunk": chunk, "page_size": page_size,
            "mode": mode, "lens_seed": n}


def _append(name, tokens, pad, kv_heads, d, page_size, dtype, layout):
    """`tokens` rows into a pool of twice as many, `pad` unused rows behind
    them; layout thd is [pages, page_size, heads, d], htd keeps each head's
    page together."""
    return {"name": name, "op": "append", "tokens": tokens, "pad": pad, "kv_heads": kv_heads, "d": d,
            "page_size": page_size, "dtype": dtype, "layout": layout, "lens_seed": tokens}


def _attn(name, n, ctx, new, heads, kv_heads, d, page_size, dtype="bf16", layout="thd", spread="equal",
          causal=True, peak=1.0):
    """n requests of `ctx` cached tokens, the new ones among them.  spread:
    equal gives every request ctx tokens and `new` new ones; ragged spreads
    the contexts over (0, ctx] and the new tokens over [1, new]; mixed gives
    one request in eight a chunk of `new` tokens and the rest one token."""
    return {"name": name, "op": "attn", "n": n, "ctx": ctx, "new": new, "heads": heads,
            "kv_heads": kv_heads, "d": d, "page_size": page_size, "dtype": dtype, "layout": layout,
            "spread": spread, "causal": causal, "peak": peak, "lens_seed": n + ctx + new}


def listed():
    return [
        # the bookkeeping of one decode step of a small server: latency only
        _plan("plan_decode_n8", 8, 4096, 1, 16, "decode"),
        # a large server's step: prompt chunks among decodes, finished
        # requests handing their pages on, a pool that runs out
        _plan("plan_churn_n500", 500, 131072, 4096, 16, "churn"),
        # one decode step's K and V rows
        _append("append_decode_t64", 64, 0, 8, 128, 16, "bf16", "thd"),
        # a prompt's chunk of all 32 heads, the batch padded to a round size
        _append("append_chunk_t16001", 16001, 383, 32, 128, 64, "bf16", "htd"),
        # one user, a short conversation, one token: the latency of a token
        _attn("decode_n1_ctx777", 1, 777, 1, 32, 8, 128, 16),
        # a busy server's decode step: 64 ragged contexts, 32 heads over 8
        _attn("decode_n64_ragged16k", 64, 16384, 1, 32, 8, 128, 16, spread="ragged"),
        # one token of the 128K, 32-head multi-head shape: all of its cache is read
        _attn("decode_n1_ctx128k_mha", 1, 131072, 1, 32, 32, 128, 64, layout="htd"),
        # a draft of up to 6 tokens checked at once, 7 heads to a key/value head
        _attn("verify_n24_new6_fp16", 24, 8191, 6, 28, 4, 128, 32, dtype="fp16", spread="ragged"),
        # a prompt's chunk in the middle of a long context
        _attn("chunk_509_ctx32k", 1, 32768, 509, 32, 8, 128, 16, peak=3.0),
        # the largest: the last 2048 tokens of a 128K prompt
        _attn("chunk_2048_ctx128k", 1, 131072, 2048, 32, 8, 128, 64),
        # a step of decodes and prompt chunks together, head dimension 64
        _attn("mixed_n40_d64_fp16", 40, 12000, 1024, 16, 2, 64, 48, dtype="fp16", spread="mixed"),
        # short prompts from their first token on, multi-head
        _attn("prompts_n9_new1500", 9, 1500, 1500, 16, 16, 128, 128, layout="htd", spread="ragged"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    top = {}
    for c in listed():
        for key, value in work(c).items():
            top[c["op"], key] = max(value, top.get((c["op"], key), 0))
    kind = rng.choice(["plan", "append", "attn", "attn", "attn", "attn"])
    while True:
        page_size = rng.choice([8, 16, 16, 32, 48, 64, 128, 256])
        layout = rng.choice(["thd", "htd"])
        dtype = rng.choice(["bf16", "fp16"])
        if kind == "plan":
            case = _plan("", _log(rng, 1, 500), _log(rng, 64, 131072), _log(rng, 1, 4096), max(page_size, 16),
                         rng.choice(["decode", "chunk", "churn"]))
        elif kind == "append":
            case = _append("", _log(rng, 1, 16001), rng.choice([0, 0, rng.randint(1, 300)]),
                           rng.choice([1, 2, 4, 5, 8, 16, 32]), rng.choice([64, 128]), page_size, dtype, layout)
        else:
            heads, kv_heads = rng.choice([(32, 8), (32, 32), (16, 2), (16, 16), (28, 4), (8, 1), (20, 4), (64, 8),
                                          (5, 5), (12, 1)])
            spread = rng.choice(["equal", "ragged", "ragged", "mixed"])
            new = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, 2048), _log(rng, 17, 2048)])
            ctx = _log(rng, 1, 131072)
            case = _attn("", _log(rng, 1, 128), ctx, min(new, ctx), heads, kv_heads, rng.choice([64, 128]),
                         page_size, dtype, layout, spread, rng.random() < 0.85, rng.choice([1.0, 1.0, 3.0]))
        case["lens_seed"] = rng.randrange(1 << 30)
        del case["name"]
        w = work(case)
        if all(w[key] <= top[kind, key] for key in w):
            return case


def _attn_lens(case):
    """Per request: tokens in the cache (the new ones included), new tokens."""
    rng = random.Random(case["lens_seed"])
    kv, new = [], []
    for i in range(case["n"]):
        if case["spread"] == "equal":
            length, q = case["ctx"], case["new"]
        else:
            length = rng.randint(1, case["ctx"])
            if case["spread"] == "mixed":
                q = case["new"] if i % 8 == 0 else 1
            else:
                q = rng.randint(1, case["new"])
        kv.append(length)
        new.append(min(q, length))
    return kv, new


def _plan_lens(case):
    """Per request: cached tokens, new tokens (-1: finished)."""
    rng = random.Random(case["lens_seed"])
    kv, new = [], []
    for i in range(case["n"]):
        kv.append(rng.randint(0, case["ctx"] - 1))
        q = 1
        if case["mode"] != "decode" and i % 4 == 0:
            q = rng.randint(1, case["chunk"])
        if case["mode"] == "churn" and rng.random() < 0.2:
            q = -1
        new.append(min(q, case["ctx"] - kv[-1]))
    return kv, new


def work(case):
    if case["op"] == "plan":
        ps = case["page_size"]
        kv, new = _plan_lens(case)
        tokens = sum(max(q, 0) for q in new)
        moved = sum(_pages(a, ps) if q < 0 else _pages(a + q, ps) - _pages(a, ps) for a, q in zip(kv, new))
        return {"bytes": 4 * (4 * case["n"] + 2 * moved + tokens), "flops": tokens}
    if case["op"] == "append":
        row = case["kv_heads"] * case["d"] * 2
        return {"bytes": 4 * row * case["tokens"] + 4 * (case["tokens"] + case["pad"]), "flops": 0}
    kv, new = _attn_lens(case)
    d, heads, kv_heads = case["d"], case["heads"], case["kv_heads"]
    pairs = sum(q * a - (q * (q - 1) // 2 if case["causal"] else 0) for a, q in zip(kv, new))
    rows = sum(new) * heads
    nbytes = (2 * sum(kv) * kv_heads * d * 2 + rows * (2 * d * 2 + 4)
              + 4 * sum(_pages(a, case["page_size"]) for a in kv) + 8 * case["n"])
    return {"bytes": nbytes, "flops": 4 * d * heads * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _pool(num_pages, page_size, kv_heads, d, dtype, layout, g):
    """One of the two pools, as a [pages, page_size, heads, d] view."""
    if layout == "htd":
        return torch.randn((num_pages, kv_heads, page_size, d), generator=g, device="cuda",
                           dtype=dtype).transpose(1, 2)
    return torch.randn((num_pages, page_size, kv_heads, d), generator=g, device="cuda", dtype=dtype)


def _int(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    ps = case["page_size"]
    if case["op"] == "plan":
        kv, new = _plan_lens(case)
        used = [_pages(a, ps) for a in kv]
        max_pages = _pages(case["ctx"], ps) + 1
        need = sum(_pages(a + q, ps) - u for a, q, u in zip(kv, new, used) if q > 0)
        released = sum(u for q, u in zip(new, used) if q < 0)
        # churn: about one needed page in twenty is missing, so the last
        # requests have to wait
        spare = need + 10 if case["mode"] != "churn" else max(0, need - need // 20 - 1 - released)
        num_pages = sum(used) + spare
        ids = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["n"], max_pages), -1, dtype=torch.int32, device="cuda")
        used_d = _int(used).long()
        where = torch.arange(max_pages, device="cuda")[None, :] < used_d[:, None]
        table[where] = ids[:sum(used)]
        free = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
        free[:spare] = ids[sum(used):]
        tokens = max(1, sum(max(q, 0) for q in new) + case["lens_seed"] % 8)
        return {"case": case, "seq_lens": _int(kv), "new_lens": _int(new), "table": table, "free": free,
                "counts": _int([spare, 0]), "tokens": tokens,
                "seq_lens_out": torch.empty(case["n"], dtype=torch.int32, device="cuda"),
                "cu_q": torch.empty(case["n"] + 1, dtype=torch.int32, device="cuda"),
                "slots": torch.empty(tokens, dtype=torch.int32, device="cuda"),
                "counts_out": torch.empty(2, dtype=torch.int32, device="cuda")}
    dtype, d, kv_heads = _TYPES[case["dtype"]], case["d"], case["kv_heads"]
    if case["op"] == "append":
        total = case["tokens"] + case["pad"]
        num_pages = _pages(2 * case["tokens"] + 1, ps)
        slots = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        # runs of neighbouring slots, as pages give them, in any order of pages
        pages = torch.randperm(num_pages, generator=g, device="cuda")
        order = (pages[:, None] * ps + torch.arange(ps, device="cuda")).flatten()
        slots[:case["tokens"]] = order[:case["tokens"]].to(torch.int32)
        # K and V come as parts of one projection's rows
        kv = torch.randn((total, 2, kv_heads, d), generator=g, device="cuda", dtype=dtype)
        return {"case": case, "k": kv[:, 0], "v": kv[:, 1], "slots": slots, "tokens": case["tokens"],
                "k_cache": _pool(num_pages, ps, kv_heads, d, dtype, case["layout"], g),
                "v_cache": _pool(num_pages, ps, kv_heads, d, dtype, case["layout"], g)}
    kv, new = _attn_lens(case)
    used = [_pages(a, ps) for a in kv]
    num_pages = sum(used) + 3
    ids = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["n"], max(used) + 2), -1, dtype=torch.int32, device="cuda")
    where = torch.arange(table.shape[1], device="cuda")[None, :] < _int(used).long()[:, None]
    table[where] = ids[:sum(used)]
    caches = [_pool(num_pages, ps, kv_heads, d, dtype, case["layout"], g) for _ in range(2)]
    # what lies behind a context in its last page was never written: any bits
    last = table.long().gather(1, (_int(used).long() - 1)[:, None])
    behind = torch.arange(ps, device="cuda")[None, :] >= (_int(kv).long() - ps * (_int(used).long() - 1))[:, None]
    request, offset = behind.nonzero(as_tuple=True)
    for c in caches:
        c[last[request, 0], offset] = float("nan")
    q = torch.randn((sum(new), case["heads"], d), generator=g, device="cuda", dtype=dtype) * case["peak"]
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    return {"case": case, "q": q, "k_cache": caches[0], "v_cache": caches[1], "table": table,
            "seq_lens": _int(kv), "cu_q": _int(cu), "kv": kv, "new": new, "max_q": max(new)}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "attn": _own_attn}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[op](state)


def _own_plan(s):
    import long_context_exact_ring_gb300 as ra
    ra.paged_kv_plan(s["seq_lens"], s["new_lens"], s["table"], s["free"], s["counts"], s["case"]["page_size"],
                     s["tokens"], seq_lens_out=s["seq_lens_out"], cu_q=s["cu_q"], slots=s["slots"],
                     counts_out=s["counts_out"])
    return {"seq_lens": s["seq_lens_out"], "cu_q": s["cu_q"], "slots": s["slots"], "counts": s["counts_out"],
            "table": s["table"], "free": s["free"]}


def _own_append(s):
    import long_context_exact_ring_gb300 as ra
    ra.paged_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attn(s):
    import long_context_exact_ring_gb300 as ra
    o, lse = ra.paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["cu_q"],
                               s["case"]["causal"], max_q=s["max_q"])
    return {"o": o, "lse": lse}


def _plain_plan(s):
    ps, tokens = s["case"]["page_size"], s["tokens"]
    table, free = s["table"], s["free"]
    n, max_pages = table.shape
    length, new, have = s["seq_lens"].long(), s["new_lens"].long(), s["counts"][0].long()
    ended = new < 0
    new = new.clamp(min=0)
    pages = (length + ps - 1) // ps
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    column = torch.arange(max_pages, device="cuda")[None, :]
    # finished requests push their pages
    back = torch.where(ended, pages, 0)
    target = have + (back.cumsum(0) - back)[:, None] + column
    target = torch.where(column < back[:, None], target, free.numel())
    stack = torch.cat([free, free.new_zeros(1)])
    stack[target.flatten()] = table.flatten()
    free.copy_(stack[:-1])
    have = have + back.sum()
    # the others pop theirs, in order, while the stack lasts
    after = (length + new + ps - 1) // ps
    fits = ~ended & (after <= max_pages) & (cu[1:] <= tokens)
    need = torch.where(fits, after - pages, 0)
    upto = need.cumsum(0)
    granted = fits & ((need == 0) | (upto <= have))
    take = have - 1 - ((upto - need)[:, None] + column - pages[:, None])
    popped = (column >= pages[:, None]) & (column < after[:, None]) & granted[:, None]
    table.copy_(torch.where(popped, stack[take.clamp(0, free.numel() - 1)], table))
    # one slot for every new token
    t = torch.arange(tokens, device="cuda")
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=n - 1)
    pos = length[r] + t - cu[r]
    page = table[r, (pos // ps).clamp(0, max_pages - 1)]
    s["slots"].copy_(torch.where((t < cu[-1]) & granted[r], page * ps + pos % ps, -1))
    s["seq_lens_out"].copy_(torch.where(ended, 0, torch.where(granted, length + new, length)))
    s["cu_q"].copy_(cu)
    s["counts_out"].copy_(torch.stack([have - torch.where(granted, need, 0).sum(), (~granted & ~ended).sum()]))
    return {"seq_lens": s["seq_lens_out"], "cu_q": s["cu_q"], "slots": s["slots"], "counts": s["counts_out"],
            "table": table, "free": free}


def _plain_append(s):
    ps, t = s["case"]["page_size"], s["tokens"]
    slots = s["slots"][:t].long()
    for rows, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        cache[slots // ps, slots % ps] = rows[:t]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    case = s["case"]
    q, heads, kv_heads, d = s["q"], case["heads"], case["kv_heads"], case["d"]
    group, scale = heads // kv_heads, 1.0 / math.sqrt(d)
    o = torch.empty_like(q)
    lse = torch.empty((heads, q.shape[0]), dtype=torch.float32, device="cuda")
    first = 0
    for i, (length, new) in enumerate(zip(s["kv"], s["new"])):
        pages = s["table"][i, :_pages(length, case["page_size"])].long()
        keys = s["k_cache"][pages].flatten(0, 1)[:length].float().permute(1, 2, 0)       # [kv, d, len]
        values = s["v_cache"][pages].flatten(0, 1)[:length].float().transpose(0, 1)      # [kv, len, d]
        block = max(1, (1 << 29) // (length * group))     # rows at a time, to bound the scores
        hblock = max(1, (1 << 29) // (length * group * min(new, block)))
        for a in range(0, new, block):
            b = min(new, a + block)
            hidden = None
            if case["causal"] and new > 1:
                pos = torch.arange(length - new + a, length - new + b, device="cuda")
                hidden = torch.arange(length, device="cuda")[None, :] > pos[:, None]     # [rows, len]
            for h in range(0, kv_heads, hblock):
                e = min(kv_heads, h + hblock)
                x = q[first + a:first + b, h * group:e * group].float() * scale
                x = x.unflatten(1, (e - h, group)).permute(1, 2, 0, 3)                   # [kv, group, rows, d]
                score = (x.flatten(1, 2) @ keys[h:e]).unflatten(1, (group, b - a))
                if hidden is not None:
                    score.masked_fill_(hidden, float("-inf"))
                m = score.amax(-1, keepdim=True)
                p = score.sub_(m).exp_()
                total = p.sum(-1, keepdim=True)
                out = (p.flatten(1, 2) @ values[h:e]).unflatten(1, (group, b - a)) / total
                o[first + a:first + b, h * group:e * group] = out.permute(2, 0, 1, 3).flatten(1, 2).to(q.dtype)
                lse[h * group:e * group, first + a:first + b] = (m + total.log()).squeeze(-1).flatten(0, 1)
        first += new
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------------------
# From the definitions, in whole numbers or 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "append":
        ps = case["page_size"]
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                s["k_cache"][slot // ps, slot % ps] = s["k"][t]
                s["v_cache"][slot // ps, slot % ps] = s["v"][t]
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if work(case)["flops"] > 6e12:
        return None
    return _exact_attn(s)


def _exact_plan(s):
    """One request after the other, one page after the other."""
    ps, width = s["case"]["page_size"], s["table"].shape[1]
    lens, new = s["seq_lens"].tolist(), s["new_lens"].tolist()
    rows, stack, top = s["table"].tolist(), s["free"].tolist(), s["counts"].tolist()[0]
    for i, q in enumerate(new):
        if q < 0:
            for page in rows[i][:_pages(lens[i], ps)]:
                stack[top] = page
                top += 1
    slots, cu, out, refused, short = [-1] * s["tokens"], [0], [], 0, False
    for i, (a, q) in enumerate(zip(lens, new)):
        cu.append(cu[-1] + max(q, 0))
        if q < 0:
            out.append(0)
            continue
        have, want = _pages(a, ps), _pages(a + q, ps)
        ok = want <= width and cu[-1] <= s["tokens"]
        if ok and want > have and (short or want - have > top):
            ok, short = False, True      # pages go out in order: nobody overtakes
        if not ok:
            refused += 1
            out.append(a)
            continue
        for p in range(have, want):
            top -= 1
            rows[i][p] = stack[top]
        for t in range(q):
            slots[cu[i] + t] = rows[i][(a + t) // ps] * ps + (a + t) % ps
        out.append(a + q)
    return {"seq_lens": _int(out), "cu_q": _int(cu), "slots": _int(slots), "counts": _int([top, refused]),
            "table": _int(rows), "free": _int(stack)}


def _exact_attn(s):
    case = s["case"]
    q, d, ps = s["q"], case["d"], case["page_size"]
    group = case["heads"] // case["kv_heads"]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full((case["heads"], q.shape[0]), float("-inf"), dtype=torch.float64, device="cuda")
    cu = s["cu_q"].tolist()
    for i, length in enumerate(s["kv"]):
        c = torch.arange(length, device="cuda")
        page, offset = s["table"][i].long()[c // ps], c % ps
        for kvh in range(case["kv_heads"]):
            k = s["k_cache"][page, offset, kvh].double()
            v = s["v_cache"][page, offset, kvh].double()
            for h in range(kvh * group, kvh * group + group):
                step = max(1, (1 << 27) // length)
                for a in range(cu[i], cu[i + 1], step):
                    b = min(cu[i + 1], a + step)
                    score = (q[a:b, h].double() @ k.T) / math.sqrt(d)
                    if case["causal"]:
                        pos = torch.arange(a, b, device="cuda") - cu[i + 1] + length
                        score = torch.where(c[None, :] <= pos[:, None], score, float("-inf"))
                    lse[h, a:b] = torch.logsumexp(score, 1)
                    o[a:b, h] = torch.exp(score - lse[h, a:b, None]) @ v
    return {"o": o, "lse": lse}
