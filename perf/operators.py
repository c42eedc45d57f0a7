"""Cases of the paged key-value cache and masked attention operators, for timing and checking.

Each case is one call as a serving program makes it, on synthetic inputs:

  append   new K/V rows of several sequences written into their pages
  decode   one new token per sequence attends over its paged cache
  evict    the cache cut back to a budget by accumulated attention weight
  masked   attention of many queries under document / prefix / causal bounds, with capped
           scores and a distance bias

`run` computes a case with elementary torch operations where `own` is false and with the
library's calls where it is true; `exact` computes it in 64 bits.  Sizes (lengths, documents)
follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

# heads / kv heads 24 / 8: the width of the 640x368 configuration with three query heads to a
# key head; 924 / 1200: its unit's tokens and the slice appended per unit; 57,600: its cache.
_LISTED = [
    # one decode step of 16 sessions, the smallest write
    dict(name="append 16 x 1", op="append", dtype="bf16", n_seq=16, kv_heads=8, dim=128, rows_lo=1,
         rows_hi=1, cached=2048, page=64, sizes=1),
    # a unit's slice for each of 8 sessions, all heads kept, pages of an odd size
    dict(name="append 8 x 1200", op="append", dtype="bf16", n_seq=8, kv_heads=24, dim=128,
         rows_lo=1100, rows_hi=1200, cached=4000, page=100, sizes=2),
    # two short sessions: latency
    dict(name="decode 2 x 300", op="decode", dtype="bf16", n_seq=2, heads=24, kv_heads=8, dim=128,
         len_lo=230, len_hi=300, page=16, cap=0.0, bias=False, weights=False, moved=False, sizes=3),
    # a serving batch of ragged sessions, weights kept for eviction, capped scores
    dict(name="decode 16 x 12k weights", op="decode", dtype="bf16", n_seq=16, heads=24, kv_heads=8,
         dim=128, len_lo=500, len_hi=12000, page=64, cap=30.0, bias=False, weights=True, moved=False,
         sizes=4),
    # one session over the whole 57,600-token cache, a key head per query head, distance bias
    dict(name="decode 1 x 57600", op="decode", dtype="bf16", n_seq=1, heads=24, kv_heads=24, dim=128,
         len_lo=57600, len_hi=57600, page=1200, cap=0.0, bias=True, weights=False, moved=False, sizes=5),
    # fp32, evicted caches (positions no longer in slot order), bias, weights
    dict(name="decode fp32 8 x 4k", op="decode", dtype="fp32", n_seq=8, heads=8, kv_heads=2, dim=64,
         len_lo=900, len_hi=4000, page=24, cap=0.0, bias=True, weights=True, moved=True, sizes=6),
    # four sessions cut from about 1.2 units to one
    dict(name="evict 4 x 1200 to 924", op="evict", dtype="bf16", n_seq=4, kv_heads=8, dim=128,
         len_lo=950, len_hi=1200, keep=924, first=4, recent=128, page=16, sizes=7),
    # a batch of long sessions cut back to 30,000 tokens
    dict(name="evict 16 x 36k to 30k", op="evict", dtype="bf16", n_seq=16, kv_heads=8, dim=128,
         len_lo=30500, len_hi=36000, keep=30000, first=4, recent=2048, page=64, sizes=8),
    # a short turn over a cached context
    dict(name="masked 48 over 2148", op="masked", dtype="bf16", n_q=48, n_kv=2148, heads=24, kv_heads=8,
         dim=128, docs=1, causal=True, prefix=False, cap=30.0, bias=False, tail=0, sizes=9),
    # a packed prefill of ragged documents, capped scores, padding behind the last one
    dict(name="masked 8192 packed cap", op="masked", dtype="bf16", n_q=8192, n_kv=8192, heads=24,
         kv_heads=8, dim=128, docs=9, causal=True, prefix=False, cap=50.0, bias=False, tail=57, sizes=10),
    # prompts seen whole (prefix) before causal answers, distance bias, a key head per query head
    dict(name="masked 8000 prefix bias", op="masked", dtype="bf16", n_q=8000, n_kv=8000, heads=24,
         kv_heads=24, dim=128, docs=2, causal=True, prefix=True, cap=0.0, bias=True, tail=0, sizes=11),
    # the fp32 mode, everything on
    dict(name="masked fp32 1000", op="masked", dtype="fp32", n_q=1000, n_kv=1400, heads=4, kv_heads=2,
         dim=64, docs=5, causal=True, prefix=True, cap=20.0, bias=True, tail=11, sizes=12),
]
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "evict", "masked", "masked"])
    dtype = "bf16" if rng.random() < 0.75 else "fp32"
    kv = rng.choice([1, 2, 3, 4, 8, 12])
    dim = 128 if dtype == "bf16" else rng.choice([32, 64, 96, 128])
    c = dict(op=op, dtype=dtype, kv_heads=kv, dim=dim, sizes=rng.randrange(1 << 20))
    if op == "append":
        hi = _log(rng, 1, 1200)
        c.update(n_seq=_log(rng, 1, 16), rows_lo=max(1, hi // 2), rows_hi=hi, cached=_log(rng, 1, 5000),
                 page=rng.choice([1, 7, 16, 64, 100, 256]))
    elif op == "decode":
        n_seq = _log(rng, 1, 16)
        hi = min(_log(rng, 1, 16000 if dtype == "bf16" else 4000), 1300000 // (n_seq * kv))
        c.update(n_seq=n_seq, heads=kv * rng.choice([1, 2, 3, 4, 8, 12, 16]),
                 len_lo=max(1, hi // 5), len_hi=hi, page=rng.choice([1, 5, 16, 48, 64, 100, 256]),
                 cap=rng.choice([0.0, 20.0, 50.0]), bias=rng.random() < 0.4, weights=rng.random() < 0.5,
                 moved=rng.random() < 0.3)
    elif op == "evict":
        n_seq = _log(rng, 1, 16)
        hi = min(_log(rng, 40, 30000), 4000000 // (n_seq * kv))
        keep = max(8, int(hi * rng.uniform(0.4, 0.97)))
        c.update(n_seq=n_seq, len_lo=max(1, hi // 3), len_hi=hi, keep=keep, first=rng.choice([0, 4]),
                 recent=rng.randrange(0, keep // 2 + 1), page=rng.choice([1, 7, 16, 64, 100]))
    else:
        n = _log(rng, 1, 5000 if dtype == "bf16" else 1500)
        c.update(n_q=n, n_kv=n + rng.choice([0, 0, _log(rng, 1, 1500)]),
                 heads=kv * rng.choice([1, 2, 3, 4]) if kv < 8 else kv, docs=rng.randint(1, 8),
                 causal=rng.random() < 0.8, prefix=rng.random() < 0.5, cap=rng.choice([0.0, 20.0, 50.0]),
                 bias=rng.random() < 0.5, tail=rng.choice([0, 0, min(n, 33) - 1]))
    return c


# ---- sizes that follow from the case ---------------------------------------------------


def _lengths(case):
    """Per-sequence lengths: rows to append, or tokens cached; the first has the largest."""
    r = random.Random(case["sizes"])
    lo, hi = (case["rows_lo"], case["rows_hi"]) if case["op"] == "append" else (case["len_lo"], case["len_hi"])
    return [hi] + [r.randint(lo, hi) for _ in range(case["n_seq"] - 1)]


def _documents(case):
    """(starts, prefixes): document boundaries over the keys, the last ends before `tail` unused keys."""
    r = random.Random(case["sizes"])
    end = case["n_kv"] - case["tail"]
    cuts = sorted(r.randint(0, end) for _ in range(case["docs"] - 1))
    starts = [0] + cuts + [end]
    prefixes = [r.randint(0, b - a) if case["prefix"] else 0 for a, b in zip(starts, starts[1:])]
    return starts, prefixes


def _visible(case):
    """How many (query, key) pairs the bounds leave."""
    starts, prefixes = _documents(case)
    n, first = 0, case["n_kv"] - case["n_q"]
    for a, b, p in zip(starts, starts[1:], prefixes):
        for pos in range(max(a, first), b):
            n += (min(b, max(pos + 1, a + p)) if case["causal"] else b) - a
    return n


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    d, hk = case["dim"], case["kv_heads"]
    if case["op"] == "append":
        rows = sum(_lengths(case))
        return {"bytes": rows * hk * (4 * d * es + 8), "flops": 0}
    if case["op"] == "decode":
        n, h = sum(_lengths(case)), case["heads"]
        extra = (8 if case["weights"] else 0) + (4 if case["moved"] and case["bias"] else 0)
        return {"bytes": n * hk * (2 * d * es + extra) + 2 * case["n_seq"] * h * d * es, "flops": 4 * n * h * d}
    if case["op"] == "evict":
        keep, total = case["keep"], 0
        for n in _lengths(case):
            if n > keep:
                # kept rows behind the new length: the recent ones, and of the others there the
                # share that ranks among the kept
                recent = min(case["recent"], n - keep)
                share = (keep - case["recent"]) / max(1, n - case["recent"])
                moved = recent + (n - keep - recent) * share
                total += 8 * n + moved * (4 * d * es + 16)
        return {"bytes": max(1.0, total * hk), "flops": 0}
    n_q, n_kv, h = case["n_q"], case["n_kv"], case["heads"]
    return {"bytes": 2 * es * d * (n_q * h + n_kv * hk) + 8 * n_q, "flops": 4 * d * h * _visible(case)}


# ---- inputs ------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(case, g, tokens):
    """A pool a little larger than the sequences need, their pages in random order; table
    entries that no token uses are -1."""
    page, need = case["page"], [-(-t // case["page"]) for t in tokens]
    width = max(need) + 1
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(tokens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    shape = (total, page, case["kv_heads"], case["dim"])
    return table, shape


def _slopes(heads):
    """One slope per head, a geometric ladder from 1/2 to 1/256."""
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / heads) for i in range(heads)], dtype=torch.float32, device="cuda")


def _gapped(g, n_seq, kv, cap, moved):
    """Positions of cached tokens: the slot, or (moved) distinct ones in another order."""
    slots = torch.arange(cap, device="cuda", dtype=torch.int32)
    if not moved:
        return slots.expand(n_seq, kv, cap).contiguous()
    keys = torch.rand((n_seq, kv, cap), generator=g, device="cuda")
    return (keys.argsort(-1) * 2).to(torch.int32)


def prepare(case, seed):
    g, dt, op = _generator(seed), _DT[case["dtype"]], case["op"]
    d, hk = case["dim"], case["kv_heads"]
    st = {"case": dict(case)}
    if op == "masked":
        starts, prefixes = _documents(case)
        h = case["heads"]
        st["q"] = _randn(g, (case["n_q"], h, d), dt, 1.5)
        st["k"] = _randn(g, (case["n_kv"], hk, d), dt)
        st["v"] = _randn(g, (case["n_kv"], hk, d), dt)
        st["starts"], st["prefixes"] = _int(starts), _int(prefixes) if case["prefix"] else None
        st["slopes"] = _slopes(h) if case["bias"] else None
        return st
    lens = _lengths(case)
    n_seq = case["n_seq"]
    if op == "append":
        before = [case["cached"] - (s * 37) % case["cached"] for s in range(n_seq)]
        tokens = [a + b for a, b in zip(before, lens)]
        st["rows"] = sum(lens)
        st["k"] = _randn(g, (st["rows"], hk, d), dt)
        st["v"] = _randn(g, (st["rows"], hk, d), dt)
        st["starts"] = _int([sum(lens[:s]) for s in range(n_seq + 1)])
        st["lengths"] = _int(before)
        st["pos0"] = _int([2 * b for b in before])
    else:
        tokens = lens
        st["lengths"] = _int(lens)
    st["table"], shape = _pages(case, g, tokens)
    cap = max(tokens)
    if op == "append":
        st["k_pages"], st["v_pages"] = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))
        st["weights"] = torch.rand((n_seq, hk, cap), generator=g, device="cuda")
        st["positions"] = torch.zeros((n_seq, hk, cap), dtype=torch.int32, device="cuda")
        return st
    st["k_pages"], st["v_pages"] = (_randn(g, shape, dt) for _ in range(2))
    if op == "decode":
        h = case["heads"]
        st["q"] = _randn(g, (n_seq, h, d), dt, 1.5)
        st["slopes"] = _slopes(h) if case["bias"] else None
        st["positions"] = _gapped(g, n_seq, hk, cap, True) if case["moved"] else None
        st["q_positions"] = _int([2 * n for n in lens]) if case["moved"] else None
        # what earlier steps left: a little for most tokens, much for a few
        st["weights"] = torch.rand((n_seq, hk, cap), generator=g, device="cuda") ** 4 if case["weights"] else None
        return st
    # accumulated weights: heavy-tailed, a tenth still zero (new tokens; ties); the call works in
    # place, so a pass starts from a copy of them (one buffer: weights, then positions)
    w = torch.rand((n_seq, hk, cap), generator=g, device="cuda")
    w = torch.where(w < 0.1, torch.zeros_like(w), w ** 4)
    p = _gapped(g, n_seq, hk, cap, False)
    st["fresh"] = torch.stack([w.view(torch.int32), p])
    st["state"] = st["fresh"].clone()
    return st


# ---- one pass ------------------------------------------------------------------------------


def run(st):
    op = st["case"]["op"]
    if op == "append":
        return _run_append(st)
    if op == "decode":
        return _run_decode(st)
    if op == "evict":
        return _run_evict(st)
    return _run_masked(st)


def _run_append(st):
    if own:
        from streaming_flow_matching_b200 import paged_append
        paged_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lengths"],
                     row_starts=st["starts"], positions=st["positions"], weights=st["weights"], pos0=st["pos0"])
    else:
        page = st["k_pages"].shape[1]
        row = torch.arange(st["rows"], device="cuda")
        seq = torch.searchsorted(st["starts"][1:].long(), row, right=True)
        i = row - st["starts"].long()[seq]
        slot = st["lengths"].long()[seq] + i
        at = (st["table"].long()[seq, slot // page], slot % page)
        st["k_pages"][at] = st["k"]
        st["v_pages"][at] = st["v"]
        st["weights"][seq, :, slot] = 0.0
        st["positions"][seq, :, slot] = (st["pos0"].long()[seq] + i).to(torch.int32)[:, None]
    return st["k_pages"], st["v_pages"], st["positions"], st["weights"]


def _gather(pages, table, n):
    """The first n slots of every sequence: [n_seq][n][H][D] (unused table entries read page 0)."""
    page = pages.shape[1]
    slot = torch.arange(n, device=pages.device)
    rows = table.long().clamp(min=0)[:, slot // page] * page + slot % page
    return pages.reshape(-1, *pages.shape[2:])[rows]


def _run_decode(st):
    case = st["case"]
    if own:
        from streaming_flow_matching_b200 import paged_attention
        out = paged_attention(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lengths"],
                              softcap=case["cap"], slopes=st["slopes"], positions=st["positions"],
                              q_positions=st["q_positions"], weights=st["weights"])
        return (out, st["weights"]) if case["weights"] else (out,)
    n_seq, h, d = st["q"].shape
    hk, n = case["kv_heads"], case["len_hi"]
    k = _gather(st["k_pages"], st["table"], n).float().permute(0, 2, 3, 1)          # [S][Hk][D][n]
    v = _gather(st["v_pages"], st["table"], n).float().permute(0, 2, 1, 3)          # [S][Hk][n][D]
    s = (st["q"].float() / math.sqrt(d)).view(n_seq, hk, h // hk, d) @ k
    if case["cap"] > 0:
        s = case["cap"] * torch.tanh(s / case["cap"])
    slot = torch.arange(n, device="cuda")
    if case["bias"]:
        pos = slot[None, None] if st["positions"] is None else st["positions"][:, :, :n]
        here = (st["lengths"] - 1) if st["q_positions"] is None else st["q_positions"]
        far = (here[:, None, None] - pos).abs().float()
        s = s - st["slopes"].view(1, hk, h // hk, 1) * far[:, :, None]
    seen = (slot[None] < st["lengths"][:, None])[:, None, None]
    s = s.masked_fill(~seen, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = (p @ v).reshape(n_seq, h, d).to(st["q"].dtype)
    if not case["weights"]:
        return (out,)
    st["weights"][:, :, :n] += p.sum(2)
    return out, st["weights"]


def _run_evict(st):
    case, keep = st["case"], st["case"]["keep"]
    st["state"].copy_(st["fresh"])
    weights, positions = st["state"][0].view(torch.float32), st["state"][1]
    if own:
        from streaming_flow_matching_b200 import paged_evict
        paged_evict(st["k_pages"], st["v_pages"], st["table"], st["lengths"], weights, positions, keep,
                    n_first=case["first"], n_recent=case["recent"])
        return st["k_pages"], st["v_pages"], weights, positions
    n_seq, hk, cap = weights.shape
    slot = torch.arange(cap, device="cuda")
    there = (slot[None] < st["lengths"][:, None])[:, None].expand(n_seq, hk, cap)
    newest = positions.masked_fill(~there, -(1 << 30)).amax(-1, keepdim=True)
    guarded = (positions < case["first"]) | (positions > newest - case["recent"])
    rank = torch.where(guarded, torch.full_like(weights, float("inf")), weights)
    rank = rank.masked_fill(~there, float("-inf"))
    order = rank.argsort(dim=-1, descending=True, stable=True)                     # ties: lowest slot
    kept = torch.zeros_like(there).scatter(-1, order[..., :keep], True) & there
    cut = (st["lengths"] > keep)[:, None, None]
    hole = (slot < keep) & ~kept & cut
    mover = (slot >= keep) & kept & cut
    a, b = hole.nonzero(as_tuple=True), mover.nonzero(as_tuple=True)              # both in slot order
    page = st["k_pages"].shape[1]
    to = (st["table"].long()[a[0], a[2] // page], a[2] % page, a[1])
    fro = (st["table"].long()[b[0], b[2] // page], b[2] % page, b[1])
    st["k_pages"][to] = st["k_pages"][fro]
    st["v_pages"][to] = st["v_pages"][fro]
    weights[a] = weights[b]
    positions[a] = positions[b]
    return st["k_pages"], st["v_pages"], weights, positions


def _run_masked(st):
    case = st["case"]
    n_q, n_kv = case["n_q"], case["n_kv"]
    if own:
        from streaming_flow_matching_b200 import attention_bounds, attention_masked
        lo, hi = attention_bounds(n_q, n_kv, doc_starts=st["starts"], prefixes=st["prefixes"], causal=case["causal"])
        return (attention_masked(st["q"], st["k"], st["v"], lo, hi, softcap=case["cap"], slopes=st["slopes"]),)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    key = torch.arange(n_kv, device="cuda")
    at = key[n_kv - n_q:]
    doc = torch.searchsorted(st["starts"][1:], key.int(), right=True)               # past the last: n_docs
    q_doc, n_docs = doc[n_kv - n_q:], st["starts"].numel() - 1
    seen = (q_doc[:, None] == doc[None]) & (doc < n_docs)[None]
    if case["causal"]:
        ok = key[None] <= at[:, None]
        if st["prefixes"] is not None:
            start = st["starts"][doc.clamp(max=n_docs - 1)]
            ok = ok | (key - start < st["prefixes"][doc.clamp(max=n_docs - 1)])[None]
        seen = seen & ok
    q = (st["q"].float() / math.sqrt(d)).view(n_q, hk, h // hk, d).permute(1, 2, 0, 3)
    s = q @ st["k"].float().permute(1, 2, 0)[:, None]                               # [Hk][G][n_q][n_kv]
    if case["cap"] > 0:
        s = torch.tanh(s.div_(case["cap"])).mul_(case["cap"])
    if case["bias"]:
        far = (at[:, None] - key[None]).abs().float()
        s.sub_(st["slopes"].view(hk, h // hk, 1, 1) * far)
    s.masked_fill_(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top.masked_fill(top == float("-inf"), 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ st["v"].float().permute(1, 0, 2)[:, None]) / total.masked_fill(total == 0, 1.0)
    return (out.permute(2, 0, 1, 3).reshape(n_q, h, d).to(st["q"].dtype),)


# ---- 64 bits ---------------------------------------------------------------------------------


def _attend64(q, k, v, lo, hi, at, pos, cap, slopes):
    """One head: softmax over keys [lo, hi) of each query (q [n][D], k, v [m][D], at [n], pos [m]);
    returns the output and the softmax weights."""
    s = (q.double() @ k.double().t()) * (q.shape[-1] ** -0.5)
    if cap:
        s = torch.tanh(s / cap) * cap
    if slopes is not None:
        s = s - slopes.double()[:, None] * (at.double()[:, None] - pos.double()[None]).abs()
    j = torch.arange(k.shape[0], device=q.device)
    inside = (j[None] >= lo[:, None]) & (j[None] < hi[:, None])
    s = torch.where(inside, s, torch.full_like(s, -float("inf")))
    w = torch.where(inside, torch.exp(s - torch.logsumexp(s, 1, keepdim=True)), torch.zeros_like(s))
    return w @ v.double(), w


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "masked":
        return (_exact_masked(case, st),)
    table, lens = st["table"].tolist(), st["lengths"].tolist()
    page, hk = case["page"], case["kv_heads"]
    if op == "append":
        kp, vp, pos, w = (st[n].clone() for n in ("k_pages", "v_pages", "positions", "weights"))
        starts, pos0 = st["starts"].tolist(), st["pos0"].tolist()
        flat = [], []
        for s in range(case["n_seq"]):
            for i in range(starts[s + 1] - starts[s]):
                t = lens[s] + i
                flat[0].append(starts[s] + i)
                flat[1].append(table[s][t // page] * page + t % page)
            n = starts[s + 1] - starts[s]
            pos[s, :, lens[s]:lens[s] + n] = pos0[s] + torch.arange(n, device="cuda", dtype=torch.int32)
            w[s, :, lens[s]:lens[s] + n] = 0
        src, dst = (torch.tensor(f, device="cuda") for f in flat)
        for pages, new in ((kp, st["k"]), (vp, st["v"])):
            pages.view(-1, hk, case["dim"])[dst] = new[src]
        return kp.double(), vp.double(), pos, w.double()

    def rows(s):
        t = torch.arange(lens[s], device="cuda")
        return torch.tensor(table[s], device="cuda")[t // page] * page + t % page

    if op == "decode":
        g = case["heads"] // hk
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        w = st["weights"].double() if case["weights"] else None
        for s in range(case["n_seq"]):
            k, v = (st[n].view(-1, hk, case["dim"])[rows(s)] for n in ("k_pages", "v_pages"))
            n = lens[s]
            lo, hi = (torch.full((g,), x, device="cuda") for x in (0, n))
            here = n - 1 if st["q_positions"] is None else int(st["q_positions"][s])
            for x in range(hk):
                pos = torch.arange(n, device="cuda") if st["positions"] is None else st["positions"][s, x, :n]
                sl = st["slopes"][x * g:x * g + g] if case["bias"] else None
                o, p = _attend64(st["q"][s, x * g:x * g + g], k[:, x], v[:, x], lo, hi,
                                 torch.full((g,), here, device="cuda"), pos, case["cap"], sl)
                out[s, x * g:x * g + g] = o
                if w is not None:
                    w[s, x, :n] += p.sum(0)
        return (out, w) if case["weights"] else (out,)
    # evict: rank every slot of a head by (guarded, weight, slot)
    weights, positions = st["fresh"][0].view(torch.float32).clone(), st["fresh"][1].clone()
    kp, vp = st["k_pages"].clone(), st["v_pages"].clone()
    kf, vf = (x.view(-1, hk, case["dim"]) for x in (kp, vp))
    for s in range(case["n_seq"]):
        n, keep = lens[s], case["keep"]
        if n <= keep:
            continue
        at = rows(s)
        for x in range(hk):
            p, w = positions[s, x, :n].tolist(), weights[s, x, :n].tolist()
            newest = max(p)
            safe = [q < case["first"] or q > newest - case["recent"] for q in p]
            stay = set(sorted(range(n), key=lambda t: (not safe[t], -w[t] if not safe[t] else 0.0, t))[:keep])
            holes = [t for t in range(keep) if t not in stay]
            movers = [t for t in range(keep, n) if t in stay]
            if not holes:
                continue
            to, fro = torch.tensor(holes, device="cuda"), torch.tensor(movers, device="cuda")
            kf[at[to], x] = kf[at[fro], x]
            vf[at[to], x] = vf[at[fro], x]
            weights[s, x, to] = weights[s, x, fro]
            positions[s, x, to] = positions[s, x, fro]
    return kp.double(), vp.double(), weights.double(), positions


def _exact_masked(case, st):
    starts, prefixes = _documents(case)
    n_q, n_kv, g = case["n_q"], case["n_kv"], case["heads"] // case["kv_heads"]
    lo, hi = [0] * n_q, [0] * n_q
    for a, b, p in zip(starts, starts[1:], prefixes):
        for pos in range(max(a, n_kv - n_q), b):
            i = pos - (n_kv - n_q)
            lo[i], hi[i] = a, min(b, max(pos + 1, a + p)) if case["causal"] else b
    lo, hi = (torch.tensor(x, device="cuda") for x in (lo, hi))
    pos = torch.arange(n_kv, device="cuda")
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for x in range(case["heads"]):
        for r in range(0, n_q, 2048):
            rows = slice(r, min(n_q, r + 2048))
            q = st["q"][rows, x]
            sl = st["slopes"][x].expand(q.shape[0]) if case["bias"] else None
            out[rows, x] = _attend64(q, st["k"][:, x // g], st["v"][:, x // g], lo[rows], hi[rows],
                                     pos[n_kv - n_q:][rows], pos, case["cap"], sl)[0]
    return out
