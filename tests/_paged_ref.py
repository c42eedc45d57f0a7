"""Plain 64-bit forms of the paged cache and masked attention, written from the formulas."""
import math

import torch


def attend(q, k, v, lo, hi, *, cap=0.0, slopes=None, q_pos=None, k_pos=None):
    """One group of heads.  q [n][H][D], k, v [m][Hk][D], lo, hi [n] -> (out, mag, weights):
    out = softmax(q k^T) v over keys [lo, hi) per query, mag the same with |v| (the scale of
    rounding errors), weights [Hk][m] the softmax summed over queries and the heads of a key head.
    k_pos: [m] or [Hk][m]."""
    n, h, d = q.shape
    m, hk = k.shape[0], k.shape[1]
    g = h // hk
    out = torch.zeros(n, h, d, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    wts = torch.zeros(hk, m, dtype=torch.float64, device=q.device)
    j = torch.arange(m, device=q.device)
    seen = (j[None] >= lo[:, None].clamp(min=0)) & (j[None] < hi[:, None].clamp(max=m))
    for x in range(h):
        s = q[:, x].double() @ torch.nan_to_num(k[:, x // g].double(), 0.0, 0.0, 0.0).t() / math.sqrt(d)
        bad = ~torch.isfinite(k[:, x // g].double()).all(1)
        assert not (seen & bad[None]).any(), "the reference takes visible keys to be finite"
        if cap:
            s = cap * torch.tanh(s / cap)
        if slopes is not None:
            kp = j if k_pos is None else (k_pos if k_pos.dim() == 1 else k_pos[x // g])
            qp = (m - n + torch.arange(n, device=q.device)) if q_pos is None else q_pos
            s = s - slopes[x].double() * (qp.double()[:, None] - kp.double()[None]).abs()
        s = s.masked_fill(~seen, -math.inf)
        top = s.max(1, keepdim=True).values
        e = torch.where(seen, torch.exp(s - top.masked_fill(torch.isinf(top), 0.0)), torch.zeros_like(s))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
        vx = v[:, x // g].double()
        fin = torch.isfinite(vx)
        out[:, x] = p @ torch.where(fin, vx, torch.zeros_like(vx))
        mag[:, x] = p @ torch.where(fin, vx, torch.zeros_like(vx)).abs()
        for t in (~fin).any(1).nonzero().flatten().tolist():      # a visible non-finite element decides
            rows = seen[:, t]
            out[rows, x] = out[rows, x] + torch.where(fin[t], torch.zeros_like(vx[t]), vx[t])
        wts[x // g] += p.sum(0)
    return out, mag, wts


def rows_of(table, s, n, page, device):
    """Pool rows of the first n slots of sequence s."""
    t = torch.arange(n, device=device)
    return table[s].long()[t // page] * page + t % page


def evict(weights, positions, n, keep, n_first, n_recent):
    """One head (lists): (evicted slots < keep, kept slots >= keep), both ascending."""
    if n <= keep:
        return [], []
    newest = max(positions[:n])
    safe = [p < n_first or p > newest - n_recent for p in positions[:n]]

    def key(t):
        w = weights[t]
        if safe[t]:
            return (0, 0.0, t)
        return (2, 0.0, t) if w != w else (1, -w, t)

    stay = set(sorted(range(n), key=key)[:keep])
    return [t for t in range(keep) if t not in stay], [t for t in range(keep, n) if t in stay]


def bounds(n_q, n_kv, starts, prefixes, causal):
    """(lo, hi) lists of every query, by the definition."""
    lo, hi = [], []
    for i in range(n_q):
        pos = n_kv - n_q + i
        doc = [d for d in range(len(starts) - 1) if starts[d] <= pos < starts[d + 1]]
        if not doc:
            lo.append(0)
            hi.append(0)
            continue
        a, b = starts[doc[0]], starts[doc[0] + 1]
        seen = [j for j in range(a, b) if not causal or j <= pos or (prefixes and j - a < prefixes[doc[0]])]
        lo.append(a)
        hi.append(seen[-1] + 1)
    return lo, hi
