"""The paged K/V cache: append, one-token attention with weight accumulation, eviction, and a
run of them together, against plain 64-bit forms.

Tolerances (elementwise; A = sum_t p_t |v_t|):
  bf16 out: P enters as a bf16 pair (2^-15 of each term), the output is rounded once (2^-8),
            fp32 scores add at most a few 1e-4 of A:  2^-8 |o| + 5e-4 A
  fp32 out: as the masked attention's fp32 mode: 2e-4 A + 2^-23 |o|, relative L2 <= 1e-5
  weights:  fp32 sums of softmax terms, each off by at most 2e-4 of itself (scores as above):
            5e-4 of the step's weight + 2^-23 of the total, and 2^-126 for each query head (a
            term below that has no normal fp32 value and may become 0: 2^-126 is all it can lose)
Append and eviction move bits: exact.
"""
import random

import pytest
import torch

from streaming_flow_matching_b200 import _lib as L
from tests import _paged_ref as R
from tests._gpu_util import FP32_TOL, rel_l2

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ladder(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


class Cache:
    """A pool with every page of every sequence in random order; unused table entries are -1."""

    def __init__(self, tokens, page, hk, d, dtype, seed=0, spare=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-t // page) for t in tokens]
        n = sum(need) + spare
        order = torch.randperm(n, generator=g, device="cuda").tolist()
        width = max(max(need), 1) + 1
        rows, at = [], 0
        for x in need:
            rows.append(order[at:at + x] + [-1] * (width - x))
            at += x
        self.table = ints(rows)
        self.page, self.hk, self.d = page, hk, d
        self.k = torch.randn(n, page, hk, d, generator=g, device="cuda").to(dtype)
        self.v = torch.randn(n, page, hk, d, generator=g, device="cuda").to(dtype)

    def rows(self, s, n):
        return R.rows_of(self.table, s, n, self.page, "cuda")

    def gather(self, s, n):
        r = self.rows(s, n)
        return self.k.view(-1, self.hk, self.d)[r], self.v.view(-1, self.hk, self.d)[r]


# ---- append ------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32), (F32, 96)])
@pytest.mark.parametrize("page", [1, 7, 16, 100])
@pytest.mark.parametrize("hk,rows,before", [(1, [1], [0]), (3, [5, 0, 40, 1], [0, 9, 15, 63]),
                                            (8, [0, 300, 17], [100, 0, 1])])
def test_append(cuda_device, dtype, d, page, hk, rows, before):
    from streaming_flow_matching_b200 import paged_append
    n_seq = len(rows)
    c = Cache([a + b for a, b in zip(rows, before)], page, hk, d, dtype)
    cap = max(a + b for a, b in zip(rows, before)) + 3
    lead, tail = 2, 3                                        # rows of no sequence
    starts = [lead + sum(rows[:s]) for s in range(n_seq + 1)]
    n = starts[-1] + tail
    k, v = (torch.randn(n, hk, d, device="cuda").to(dtype) for _ in range(2))
    pos = torch.full((n_seq, hk, cap), -7, dtype=torch.int32, device="cuda")
    w = torch.rand(n_seq, hk, cap, device="cuda")
    pos0 = [1000 * s + 5 for s in range(n_seq)]
    ek, ev, ep, ew = c.k.clone(), c.v.clone(), pos.clone(), w.clone()
    for s in range(n_seq):
        at = c.rows(s, rows[s] + before[s])[before[s]:]
        ek.view(-1, hk, d)[at] = k[starts[s]:starts[s + 1]]
        ev.view(-1, hk, d)[at] = v[starts[s]:starts[s + 1]]
        sl = slice(before[s], before[s] + rows[s])
        ep[s, :, sl] = pos0[s] + torch.arange(rows[s], device="cuda", dtype=torch.int32)
        ew[s, :, sl] = 0
    paged_append(k, v, c.k, c.v, c.table, ints(before), row_starts=ints(starts), positions=pos,
                 weights=w, pos0=ints(pos0))
    torch.cuda.synchronize()
    assert L.check_call_error() == 0
    for a, b in ((c.k, ek), (c.v, ev), (pos, ep), (w, ew)):
        assert torch.equal(a, b)


def test_append_one_row_each_and_none(cuda_device):
    from streaming_flow_matching_b200 import paged_append
    c = Cache([10, 20, 33], 16, 2, 64, F32)
    k, v = torch.randn(3, 2, 64, device="cuda"), torch.randn(3, 2, 64, device="cuda")
    pos = torch.zeros(3, 2, 40, dtype=torch.int32, device="cuda")
    ek, ev = c.k.clone(), c.v.clone()
    for s, t in enumerate((9, 19, 32)):
        ek.view(-1, 2, 64)[c.rows(s, t + 1)[t]] = k[s]
        ev.view(-1, 2, 64)[c.rows(s, t + 1)[t]] = v[s]
    paged_append(k, v, c.k, c.v, c.table, ints([9, 19, 32]), positions=pos)
    assert torch.equal(c.k, ek) and torch.equal(c.v, ev)
    assert [int(pos[s, 1, t]) for s, t in enumerate((9, 19, 32))] == [9, 19, 32]
    paged_append(k[:0], v[:0], c.k, c.v, c.table, ints([9, 19, 32]), row_starts=ints([0, 0, 0, 0]))
    assert torch.equal(c.k, ek)
    assert L.check_call_error() == 0


def test_append_outside_the_cache_is_dropped_and_reported(cuda_device):
    from streaming_flow_matching_b200 import paged_append
    c = Cache([40, 40], 16, 2, 128, BF)
    k, v = (torch.randn(4, 2, 128, device="cuda").to(BF) for _ in range(2))
    ek, ev = c.k.clone(), c.v.clone()
    at = c.rows(0, 40)[38:]
    ek.view(-1, 2, 128)[at], ev.view(-1, 2, 128)[at] = k[:2], v[:2]
    # sequence 1's rows go past its last page, into entries that are -1
    paged_append(k, v, c.k, c.v, c.table, ints([38, 48]), row_starts=ints([0, 2, 4]))
    assert L.check_call_error() == 0x301
    assert torch.equal(c.k, ek) and torch.equal(c.v, ev)
    c.table[1, 0] = c.k.shape[0]                             # one past the pool
    paged_append(k[:2], v[:2], c.k, c.v, c.table, ints([0, 0]), row_starts=ints([0, 0, 2]))
    assert L.check_call_error() == 0x301
    for lens in ([0, 64], [0, -1], [0, 2 ** 31 - 1], [0, -2 ** 31]):  # past the table, or negative
        paged_append(k[:2], v[:2], c.k, c.v, c.table, ints(lens), row_starts=ints([0, 0, 2]))
        code = L.check_call_error()
        assert code in (0x301, 0x302) and (code == 0x302 or lens[1] == -1), (lens, hex(code))
    assert torch.equal(c.k, ek) and torch.equal(c.v, ev)


# ---- attention ---------------------------------------------------------------------------


def check_out(got, ref, mag, dtype):
    err = (got.double() - ref).abs()
    if dtype == BF:
        tol = 2.0 ** -8 * ref.abs() + 5e-4 * mag
    else:
        tol = 2e-4 * mag + 2.0 ** -23 * ref.abs()
        if float(ref.abs().max()) > 0:
            assert rel_l2(got.double().cpu().numpy(), ref.cpu().numpy()) <= FP32_TOL
    assert bool((err <= tol + 1e-30).all()), float((err / (tol + 1e-30)).max())


def reference(c, q, lens, *, cap=0.0, slopes=None, positions=None, q_positions=None):
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag, wts = torch.zeros_like(out), []
    for s, n in enumerate(lens):
        if n == 0:
            wts.append(torch.zeros(c.hk, 0, dtype=torch.float64, device="cuda"))
            continue
        k, v = c.gather(s, n)
        qp = ints([n - 1]) if q_positions is None else q_positions[s:s + 1]
        kp = None if positions is None else positions[s, :, :n]
        o, m, w = R.attend(q[s:s + 1], k, v, ints([0]), ints([n]), cap=cap, slopes=slopes, q_pos=qp, k_pos=kp)
        out[s], mag[s] = o[0], m[0]
        wts.append(w)
    return out, mag, wts


def run(c, q, lens, **kw):
    from streaming_flow_matching_b200 import paged_attention
    ref, mag, wts = reference(c, q, lens, cap=kw.get("softcap", 0.0),
                              **{n: kw[n] for n in ("slopes", "positions", "q_positions") if n in kw})
    before = kw["weights"].clone() if "weights" in kw else None
    out = paged_attention(q, c.k, c.v, c.table, ints(lens), **kw)
    torch.cuda.synchronize()
    assert L.check_call_error() == 0
    check_out(out, ref, mag, q.dtype)
    if before is not None:
        for s, n in enumerate(lens):
            got, want = kw["weights"][s, :, :n].double(), before[s, :, :n].double() + wts[s]
            assert bool(((got - want).abs() <= 5e-4 * wts[s] + 2.0 ** -23 * want + q.shape[1] * 2.0 ** -126).all())
            assert torch.equal(kw["weights"][s, :, n:], before[s, :, n:])     # past the length: as it was
    return out


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32), (F32, 64), (F32, 96), (F32, 128)])
@pytest.mark.parametrize("page", [1, 16, 37])
@pytest.mark.parametrize("h,hk", [(1, 1), (3, 1), (8, 2), (24, 2), (20, 1), (12, 12)])
def test_attention_lengths_and_heads(cuda_device, dtype, d, page, h, hk):
    lens = [1, 0, 63, 64, 65, 0, 300, 2]
    c = Cache(lens, page, hk, d, dtype, seed=h)
    q = (torch.randn(len(lens), h, d, device="cuda") * 1.5).to(dtype)
    out = run(c, q, lens)
    assert int(torch.count_nonzero(out[1])) == 0 and int(torch.count_nonzero(out[5])) == 0
    w = torch.rand(len(lens), hk, 310, device="cuda")
    run(c, q, lens, softcap=20.0, slopes=ladder(h), weights=w)
    # a table for far longer sequences: the form of long ones (a workspace, a second kernel)
    c.table = torch.cat([c.table, torch.full((len(lens), 40000 // page), -1, dtype=torch.int32, device="cuda")], 1)
    need = L.lib.sfm_paged_attention_workspace_bytes
    code = L.SFM_DTYPE_BF16 if dtype == BF else L.SFM_DTYPE_FP32
    assert need(len(lens), c.table.shape[1] * page, h, hk, d, code, 0) > 0
    out = run(c, q, lens)
    assert int(torch.count_nonzero(out[1])) == 0 and int(torch.count_nonzero(out[5])) == 0
    run(c, q, lens, softcap=20.0, slopes=ladder(h), weights=torch.rand(len(lens), hk, 40000, device="cuda"))


@pytest.mark.parametrize("dtype,d,h,hk,lens", [
    (BF, 128, 24, 8, [5000, 17, 3000, 1, 900]), (BF, 128, 4, 4, [20000]), (BF, 128, 16, 1, [7001, 7002]), (BF, 128, 300, 1, [500, 3]),
    (F32, 64, 8, 2, [4000, 10, 2500]), (BF, 128, 300, 300, [100, 65])])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (30.0, False), (30.0, True)])
def test_attention_splits(cuda_device, dtype, d, h, hk, lens, cap, bias):
    c = Cache(lens, 64, hk, d, dtype, seed=1)
    q = (torch.randn(len(lens), h, d, device="cuda") * 1.5).to(dtype)
    kw = dict(softcap=cap, weights=torch.zeros(len(lens), hk, max(lens), device="cuda"))
    if bias:
        kw["slopes"] = ladder(h)
    a = run(c, q, lens, **kw)
    kw["weights"] = torch.zeros_like(kw["weights"])
    b = run(c, q, lens, **kw)
    assert torch.equal(a, b)                                 # the same inputs, the same bits


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_attention_positions(cuda_device, dtype, d):
    # positions in any order, per key head; far queries
    lens, h, hk = [700, 64, 1], 6, 2
    c = Cache(lens, 16, hk, d, dtype, seed=4)
    q = torch.randn(3, h, d, device="cuda").to(dtype)
    pos = torch.stack([torch.stack([torch.randperm(705, device="cuda") * 3 for _ in range(hk)]) for _ in lens])
    pos = pos.to(torch.int32).contiguous()
    run(c, q, lens, slopes=ladder(h), positions=pos, q_positions=ints([2200, 0, 5]))
    run(c, q, lens, slopes=-0.01 * ladder(h), softcap=1000.0)
    run(c, q, lens, softcap=1e-3)
    run(c, q, lens, slopes=ladder(h), positions=pos, q_positions=ints([2200, 0, 5]), softcap=10.0,
        weights=torch.zeros(3, hk, 705, device="cuda"))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_positions_without_a_bias_change_nothing(cuda_device, dtype, d):
    from streaming_flow_matching_b200 import paged_attention
    lens = [300, 1, 77]
    c = Cache(lens, 16, 2, d, dtype, seed=8)
    q = torch.randn(3, 6, d, device="cuda").to(dtype)
    pos = torch.randint(0, 9999, (3, 2, 300), dtype=torch.int32, device="cuda")
    w = torch.zeros(3, 2, 300, device="cuda")
    a = paged_attention(q, c.k, c.v, c.table, ints(lens), positions=pos, q_positions=ints([9999] * 3), weights=w)
    assert torch.equal(a, run(c, q, lens, weights=torch.zeros_like(w)))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32), (F32, 128)])
@pytest.mark.parametrize("h,hk,lens", [
    (2, 1, [60, 64, 1]), (2, 1, [128, 65, 3]), (8, 2, [256, 1, 0, 129]), (4, 1, [512, 449, 70]), (16, 1, [1000]),
    (3, 3, [1500, 900]), (40, 1, [700, 500]), (5, 5, [1024] * 4)])
def test_attention_clusters(cuda_device, dtype, d, h, hk, lens):
    # one kernel for short sequences: 1, 2, 4 and 8 CTAs a sequence, some without a tile
    from streaming_flow_matching_b200 import paged_attention
    need = L.lib.sfm_paged_attention_workspace_bytes
    code = L.SFM_DTYPE_BF16 if dtype == BF else L.SFM_DTYPE_FP32
    c = Cache(lens, 16, hk, d, dtype, seed=h)
    assert h * hk == 40 or need(len(lens), c.table.shape[1] * 16, h, hk, d, code, 0) == 0
    q = (torch.randn(len(lens), h, d, device="cuda") * 1.5).to(dtype)
    w = torch.rand(len(lens), hk, max(lens), device="cuda")
    kw = dict(softcap=30.0, slopes=ladder(h))
    a = run(c, q, lens, **kw)
    run(c, q, lens, weights=w, **kw)
    assert torch.equal(a, run(c, q, lens, **kw))             # the same bits
    c.v.view(-1, hk, d)[c.rows(0, lens[0])[-1]] = float("inf")   # an infinity reaches its sequence's heads
    out = paged_attention(q, c.k, c.v, c.table, ints(lens))
    assert bool((out[0] == float("inf")).all()) and bool(torch.isfinite(out[1:]).all())


def test_attention_many_sequences(cuda_device):
    # more sequences than a warp scans at once, and than CTA slots; runs of empty ones
    r = random.Random(2)
    lens = [r.choice([0, 0, 1, 30, 64, 200]) for _ in range(150)]
    c = Cache(lens, 8, 2, 128, BF, seed=2)
    q = torch.randn(150, 4, 128, device="cuda").to(BF)
    run(c, q, lens, weights=torch.zeros(150, 2, 200, device="cuda"))
    run(c, q, [0] * 150)
    lens = [0] * 5000
    lens[3], lens[4000], lens[4999] = 700, 65, 1             # long runs of empty ones
    c = Cache(lens, 16, 1, 128, BF, seed=3)
    run(c, torch.randn(5000, 2, 128, device="cuda").to(BF), lens)
    c = Cache(lens, 16, 1, 32, F32, seed=3)
    run(c, torch.randn(5000, 2, 32, device="cuda"), lens)


def test_attention_unused_rows_may_hold_anything(cuda_device):
    lens = [70, 129]
    for dtype, d in ((BF, 128), (F32, 128)):
        c = Cache(lens, 16, 2, d, dtype, seed=6)
        used = torch.cat([c.rows(s, n) for s, n in enumerate(lens)])
        dead = torch.ones(c.k.shape[0] * 16, dtype=torch.bool, device="cuda")
        dead[used] = False
        c.k.view(-1, 2, d)[dead] = float("nan")
        c.v.view(-1, 2, d)[dead] = float("inf")
        run(c, torch.randn(2, 4, d, device="cuda").to(dtype), lens)


def test_attention_bad_pages_and_lengths(cuda_device):
    # slots on a bad page are left out, and reported; lengths are cut to the table
    from streaming_flow_matching_b200 import paged_attention
    for dtype, d in ((BF, 128), (F32, 64)):
        c = Cache([100, 64], 16, 1, d, dtype, seed=7)
        q = torch.randn(2, 2, d, device="cuda").to(dtype)
        keep = torch.tensor([t for t in range(100) if not 32 <= t < 48], device="cuda")
        k, v = c.gather(0, 100)
        ref, mag, _ = R.attend(q[:1], k[keep], v[keep], ints([0]), ints([84]))
        for bad in (-1, c.k.shape[0], 2 ** 31 - 1):
            t = c.table.clone()
            t[0, 2] = bad
            out = paged_attention(q, c.k, c.v, t, ints([100, 64]))
            assert L.check_call_error() == 0x301
            check_out(out[:1], ref, mag, dtype)
        t = torch.full_like(c.table, -1)
        out = paged_attention(q, c.k, c.v, t, ints([100, 64]), weights=torch.zeros(2, 1, 100, device="cuda"))
        assert L.check_call_error() == 0x301
        assert int(torch.count_nonzero(out)) == 0
        full = c.table.shape[1] * 16
        t = c.table.clone()
        t[t < 0] = 0
        good = paged_attention(q, c.k, c.v, t, ints([full, 0]))
        assert L.check_call_error() == 0
        out = paged_attention(q, c.k, c.v, t, ints([2 ** 31 - 1, -5]))
        assert L.check_call_error() == 0x302
        assert torch.equal(out, good)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_weights_of_slots_on_a_bad_page_stay(cuda_device, dtype, d):
    # all 16 slots that a warp takes lie on the bad page; the workspace holds anything
    from streaming_flow_matching_b200 import paged_attention
    c = Cache([100, 64], 16, 2, d, dtype, seed=7)
    q = torch.randn(2, 8, d, device="cuda").to(dtype)
    keep = torch.tensor([t for t in range(100) if not 32 <= t < 48], device="cuda")
    k, v = c.gather(0, 100)
    ref, mag, wts = R.attend(q[:1], k[keep], v[keep], ints([0]), ints([84]))
    t = c.table.clone()
    t[0, 2] = -1
    need = L.lib.sfm_paged_attention_workspace_bytes(2, 100, 8, 2, d, 0 if dtype == BF else 1, 1)
    for fill in (0x41, 0x7f, 0xff):                          # 12.1, 3.4e38, NaN
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        w = torch.full((2, 2, 100), 0.25, device="cuda")
        out = paged_attention(q, c.k, c.v, t, ints([100, 64]), weights=w, workspace=ws)
        assert L.check_call_error() == 0x301
        check_out(out[:1], ref, mag, dtype)
        assert bool((w[0, :, 32:48] == 0.25).all())
        err = (w[0, :, keep].double() - 0.25 - wts).abs()
        assert bool((err <= 5e-4 * wts + 2.0 ** -23 * (0.25 + wts) + 8 * 2.0 ** -126).all())


def test_attention_shared_pages_and_infinities(cuda_device):
    from streaming_flow_matching_b200 import paged_attention
    c = Cache([64, 64], 16, 1, 128, BF, seed=8)
    c.table[1] = c.table[0]                                  # one prefix, two readers
    q = torch.randn(2, 2, 128, device="cuda").to(BF)
    run(c, q, [64, 40])
    k0, v0 = c.rows(0, 64)[:2]
    c.v.view(-1, 128)[v0, 5] = float("inf")
    out = paged_attention(q, c.k, c.v, c.table, ints([64, 1]))
    assert torch.isinf(out[0, :, 5]).all() and torch.isfinite(out[0, :, 6:]).all()
    assert torch.isfinite(out[1]).all()                      # slot 1 is past its length
    c.k.view(-1, 128)[k0, 0] = float("nan")
    out = paged_attention(q, c.k, c.v, c.table, ints([64, 0]))
    assert torch.isnan(out[0]).all() and int(torch.count_nonzero(out[1])) == 0


def test_attention_far_pages(cuda_device):
    # element offsets past 2^31 and 2^32: the sequence's pages lie at the pool's end
    page, hk, d = 1024, 8, 128
    n_pages = 4600                                           # 4.8e9 elements of bf16 per pool
    k = torch.zeros(n_pages, page, hk, d, dtype=BF, device="cuda")
    v = torch.zeros(n_pages, page, hk, d, dtype=BF, device="cuda")
    ids = [4599, 2100, 0]
    g = torch.Generator(device="cuda").manual_seed(0)
    for i in ids:
        k[i] = torch.randn(page, hk, d, generator=g, device="cuda").to(BF)
        v[i] = torch.randn(page, hk, d, generator=g, device="cuda").to(BF)
    from streaming_flow_matching_b200 import paged_append, paged_attention, paged_evict
    q = torch.randn(1, 8, d, device="cuda").to(BF)
    n = 2500
    kk, vv = (torch.cat([x[i] for i in ids])[:n] for x in (k, v))
    ref, mag, _ = R.attend(q, kk, vv, ints([0]), ints([n]))
    check_out(paged_attention(q, k, v, ints([ids]), ints([n])), ref, mag, BF)
    new = torch.randn(1, hk, d, device="cuda").to(BF)
    paged_append(new, new, k, v, ints([ids]), ints([5]))
    assert torch.equal(k[4599, 5], new[0]) and torch.equal(v[4599, 5], new[0])
    w = torch.rand(1, hk, n, device="cuda")
    w[:, :, 2048:] += 1                                      # the last page's tokens stay
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, hk, n).contiguous()
    first = [R.evict(w[0, x].tolist(), pos[0, x].tolist(), n, 1000, 0, 0) for x in range(hk)]
    src = [[kk2[t // page][t % page, x].clone() for t in first[x][1]]
           for x in range(hk) for kk2 in [[k[i] for i in ids]]]
    paged_evict(k, v, ints([ids]), ints([n]), w, pos, 1000)
    for x in range(hk):
        assert torch.equal(torch.stack([k[4599, t, x] for t in first[x][0]]), torch.stack(src[x]))
    assert L.check_call_error() == 0


def test_attention_graph_follows_lengths(cuda_device):
    from streaming_flow_matching_b200 import paged_attention
    c = Cache([500, 400], 16, 2, 128, BF, seed=9)
    q = torch.randn(2, 6, 128, device="cuda").to(BF)
    lens = ints([500, 3])
    paged_attention(q, c.k, c.v, c.table, lens)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        w = torch.zeros(2, 2, 500, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = paged_attention(q, c.k, c.v, c.table, lens, weights=w)
        graphs.append((g, o, w))
    for now in ([500, 3], [1, 400], [0, 64], [130, 0]):
        lens.copy_(ints(now))
        for g, o, w in graphs:
            w.zero_()
            o.fill_(7)
            g.replay()
        torch.cuda.synchronize()
        ref, mag, wts = reference(c, q, now)
        for _, o, w in graphs:
            check_out(o, ref, mag, BF)
            for s, n in enumerate(now):
                assert bool(((w[s, :, :n].double() - wts[s]).abs() <= 5e-4 * wts[s] + 1e-12).all())
                assert int(torch.count_nonzero(w[s, :, n:])) == 0
    assert L.check_call_error() == 0


# ---- eviction ----------------------------------------------------------------------------


def evict_case(c, lens, w, pos, keep, n_first, n_recent):
    from streaming_flow_matching_b200 import paged_evict
    hk, d = c.hk, c.d
    ek, ev, ew, ep = c.k.clone(), c.v.clone(), w.clone(), pos.clone()
    moved = 0
    for s, n in enumerate(lens):
        if n <= keep:
            continue
        at = c.rows(s, n)
        for x in range(hk):
            to, fro = R.evict(w[s, x].tolist(), pos[s, x].tolist(), n, keep, n_first, n_recent)
            assert len(to) == len(fro)
            moved += len(to)
            for e in (ek, ev):
                e.view(-1, hk, d)[at[to], x] = e.view(-1, hk, d)[at[fro], x]
            ew[s, x, to], ep[s, x, to] = w[s, x, fro], pos[s, x, fro]
    paged_evict(c.k, c.v, c.table, ints(lens), w, pos, keep, n_first=n_first, n_recent=n_recent)
    torch.cuda.synchronize()
    assert L.check_call_error() == 0
    assert torch.equal(c.k.view(torch.uint8), ek.view(torch.uint8))
    assert torch.equal(c.v.view(torch.uint8), ev.view(torch.uint8))
    assert torch.equal(w.view(torch.int32), ew.view(torch.int32)) and torch.equal(pos, ep)
    return moved


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32), (F32, 96)])
@pytest.mark.parametrize("lens,keep,n_first,n_recent,page", [
    ([100], 64, 0, 0, 16), ([2], 1, 0, 1, 1), ([1, 0, 33, 32, 31], 32, 4, 8, 7), ([3000, 500, 1025], 900, 4, 300, 64),
    ([5000], 10, 2, 3, 100), ([700, 701], 699, 0, 699, 16), ([1500], 1400, 1400, 0, 32)])
def test_evict(cuda_device, dtype, d, lens, keep, n_first, n_recent, page):
    hk = 2
    c = Cache(lens, page, hk, d, dtype, seed=len(lens))
    cap = max(lens) + 5
    w = torch.rand(len(lens), hk, cap, device="cuda")
    w = torch.where(w < 0.2, torch.zeros_like(w), w ** 6)    # ties at zero
    pos = torch.arange(cap, device="cuda", dtype=torch.int32).expand(len(lens), hk, cap).contiguous()
    evict_case(c, lens, w, pos, keep, n_first, n_recent)


@pytest.mark.parametrize("kind", ["equal", "nan", "signs", "shuffled", "infinite", "dup_positions"])
def test_evict_odd_weights(cuda_device, kind):
    n, keep, hk = 2100, 1300, 3
    c = Cache([n], 16, hk, 128, BF, seed=3)
    w = torch.rand(1, hk, n, device="cuda")
    pos = torch.arange(n, device="cuda", dtype=torch.int32).expand(1, hk, n).contiguous()
    first, recent = 4, 100
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "nan":
        w[:, :, ::3] = float("nan")
        w[:, :, 1::3] = -float("inf")
    elif kind == "signs":
        w = (w * 4 - 2).round()
        w[w == 0] = torch.where(torch.rand_like(w[w == 0]) < 0.5, -0.0, 0.0)
    elif kind == "shuffled":
        pos = torch.stack([torch.randperm(n, device="cuda") - 50 for _ in range(hk)])[None].to(torch.int32)
    elif kind == "infinite":
        w[:, :, 5:2000:2] = float("inf")
    else:
        pos.fill_(7)                                         # all protected: the lowest slots stay
        recent = 1
    assert evict_case(c, [n], w, pos, keep, first, recent) >= 0


def test_evict_long(cuda_device):
    lens = [40000, 70000]
    c = Cache(lens, 128, 1, 32, F32, seed=3)
    w = torch.rand(2, 1, 70000, device="cuda") ** 8
    pos = torch.arange(70000, device="cuda", dtype=torch.int32).expand(2, 1, 70000).contiguous()
    assert evict_case(c, lens, w, pos, 35000, 4, 1000) > 0


@pytest.mark.parametrize("hk,lens,cap,keep", [
    # 2, 4 (short sequences beside a long one), 4, 2, 1 and 8 CTAs a head
    (1, [14000], 14000, 5000), (1, [26000, 3000, 13000, 12289], 26000, 2900), (2, [40000, 2100], 60000, 30000),
    (9, [14200], 14200, 4100), (40, [14001], 14001, 8999), (1, [250000], 250000, 200000)])
@pytest.mark.parametrize("kind", ["few values", "spread", "nan"])
def test_evict_in_clusters(cuda_device, hk, lens, cap, keep, kind):
    # several CTAs share a head's slots: ties that run over their borders, borders on both sides of keep
    c = Cache(lens, 64, hk, 32, F32, seed=4)
    g = torch.Generator(device="cuda").manual_seed(11)
    w = torch.rand(len(lens), hk, cap, generator=g, device="cuda")
    if kind == "few values":
        w = (w * 3).floor()
    elif kind == "nan":
        w[:, :, ::2] = float("nan")
    pos = torch.stack([torch.randperm(cap, generator=g, device="cuda") for _ in range(len(lens) * hk)])
    evict_case(c, lens, w, pos.view(len(lens), hk, cap).to(torch.int32), keep, 3, keep // 4)


@pytest.mark.parametrize("n_seq,hk,n,keep,alone", [
    (9, 8, 1024, 512, True), (20, 8, 300, 150, False), (2, 2, 640, 320, True), (2, 2, 650, 325, False),
    (3, 1, 7000, 6700, True)])
def test_evict_many_rows_in_one_kernel_or_two(cuda_device, n_seq, hk, n, keep, alone):
    assert (L.lib.sfm_paged_evict_workspace_bytes(n_seq, n, hk, keep) == 0) == alone
    lens = [n - 3 * s for s in range(n_seq)]
    for w in (torch.arange(n, device="cuda").expand(n_seq, hk, n).float().contiguous(),     # all that can move
              torch.rand(n_seq, hk, n, device="cuda")):
        c = Cache(lens, 16, hk, 128, BF, seed=6)
        pos = torch.arange(n, device="cuda", dtype=torch.int32).expand(n_seq, hk, n).contiguous()
        evict_case(c, lens, w, pos, keep, 0, 1)


def test_evict_more_than_clusters_hold(cuda_device):
    n = 400000                                               # 8 CTAs hold 393,216 ranks
    c = Cache([n], 512, 1, 32, F32, seed=5)
    w = torch.rand(1, 1, n, device="cuda")
    pos = torch.arange(n, device="cuda", dtype=torch.int32).view(1, 1, n).contiguous()
    assert evict_case(c, [n], w, pos, 390000, 4, 1000) > 0


def test_evict_bad_page_is_reported(cuda_device):
    from streaming_flow_matching_b200 import paged_evict
    c = Cache([64], 16, 1, 128, BF)
    w = torch.zeros(1, 1, 64, device="cuda")
    w[:, :, 48:] = 1.0
    pos = torch.arange(64, device="cuda", dtype=torch.int32).view(1, 1, 64).contiguous()
    k = c.k.clone()
    c.table[0, 3] = c.k.shape[0]
    paged_evict(c.k, c.v, c.table, ints([64]), w, pos, 48)
    assert L.check_call_error() == 0x301
    assert torch.equal(c.k, k)                               # no row could be read


# ---- together ----------------------------------------------------------------------------


def test_streaming_run(cuda_device):
    """A packed causal prefill, its K/V appended to pages, then steps of append, attention with
    weights and eviction: every attention against the 64-bit form over a list-based cache that
    is kept beside it."""
    from streaming_flow_matching_b200 import (attention_bounds, attention_masked, paged_append, paged_attention,
                                              paged_evict)
    h, hk, d, page, keep, cap = 6, 2, 128, 16, 160, 260
    slopes, softcap = ladder(h), 30.0
    lens = [150, 37, 200]
    n_seq, n = len(lens), sum(lens)
    starts = [0, 150, 187, 387]
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)      # noqa: E731
    c = Cache([cap] * n_seq, page, hk, d, BF)
    pos = torch.zeros(n_seq, hk, cap, dtype=torch.int32, device="cuda")
    w = torch.full((n_seq, hk, cap), 9.0, device="cuda")
    q, k, v = rnd(n, h, d), rnd(n, hk, d), rnd(n, hk, d)
    lo, hi = attention_bounds(n, n, doc_starts=ints(starts), causal=True)
    out = attention_masked(q, k, v, lo, hi, softcap=softcap, slopes=slopes)
    ref, mag, _ = R.attend(q, k, v, lo, hi, cap=softcap, slopes=slopes)
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + mag) + 5e-4 * mag).all())
    count = ints([0] * n_seq)
    paged_append(k, v, c.k, c.v, c.table, count, row_starts=ints(starts), positions=pos, weights=w)
    count = ints(lens)
    seen = list(lens)
    # per sequence and head: list of (position, k, v), the cache as the definition has it
    book = [[[(t, k[starts[s] + t, x], v[starts[s] + t, x]) for t in range(lens[s])] for x in range(hk)]
            for s in range(n_seq)]
    for step in range(6):
        k1, v1, q1 = rnd(n_seq, hk, d), rnd(n_seq, hk, d), rnd(n_seq, h, d)
        paged_append(k1, v1, c.k, c.v, c.table, count, positions=pos, weights=w, pos0=ints(seen))
        for s in range(n_seq):
            for x in range(hk):
                book[s][x].append((seen[s], k1[s, x], v1[s, x]))
        count = count + 1
        q_pos = ints(seen)
        seen = [t + 1 for t in seen]
        w0 = w.clone()
        out = paged_attention(q1, c.k, c.v, c.table, count, softcap=softcap, slopes=slopes, positions=pos,
                              q_positions=q_pos, weights=w)
        for s in range(n_seq):
            m = int(count[s])
            kk = torch.stack([torch.stack([e[1] for e in book[s][x]]) for x in range(hk)], 1)
            vv = torch.stack([torch.stack([e[2] for e in book[s][x]]) for x in range(hk)], 1)
            kp = torch.tensor([[e[0] for e in book[s][x]] for x in range(hk)], device="cuda")
            assert m == kk.shape[0]
            ref, mag, step_w = R.attend(q1[s:s + 1], kk, vv, ints([0]), ints([m]), cap=softcap, slopes=slopes,
                                        q_pos=q_pos[s:s + 1], k_pos=kp)
            check_out(out[s:s + 1], ref, mag, BF)
            want = w0[s, :, :m].double() + step_w
            tol = 5e-4 * step_w + 2.0 ** -23 * want + h * 2.0 ** -126
            assert bool(((w[s, :, :m].double() - want).abs() <= tol).all())
        if step % 2 == 1:
            for s in range(n_seq):
                for x in range(hk):
                    m = int(count[s])
                    to, fro = R.evict(w[s, x].tolist(), [e[0] for e in book[s][x]], m, keep, 4, 32)
                    for a, b in zip(to, fro):
                        book[s][x][a] = book[s][x][b]
                    del book[s][x][min(m, keep):]
            paged_evict(c.k, c.v, c.table, count, w, pos, keep, n_first=4, n_recent=32)
            count = count.clamp(max=keep)
    assert max(count.tolist()) == keep
    assert L.check_call_error() == 0


def test_two_streams(cuda_device):
    # two calls at once, each with its own workspace
    from streaming_flow_matching_b200 import paged_attention
    c = Cache([9000, 300], 64, 2, 128, BF, seed=12)
    q = [torch.randn(2, 8, 128, device="cuda").to(BF) for _ in range(2)]
    lens = ints([9000, 300])
    want = [paged_attention(x, c.k, c.v, c.table, lens) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(paged_attention(q[i], c.k, c.v, c.table, lens))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_refusals(cuda_device):
    from streaming_flow_matching_b200 import paged_append, paged_attention, paged_evict
    c = Cache([40, 30], 16, 2, 128, BF)
    lens = ints([40, 30])
    q = torch.randn(2, 4, 128, device="cuda").to(BF)
    w = torch.zeros(2, 2, 40, device="cuda")
    pos = torch.zeros(2, 2, 40, dtype=torch.int32, device="cuda")
    k = torch.randn(2, 2, 128, device="cuda").to(BF)
    sl = ladder(4)
    calls = [
        (lambda: paged_attention(q[:, :3].contiguous(), c.k, c.v, c.table, lens), L.SfmError),   # 3 over 2 heads
        (lambda: paged_attention(q.float(), c.k, c.v, c.table, lens), ValueError),
        (lambda: paged_attention(q[:1], c.k, c.v, c.table, lens), ValueError),
        (lambda: paged_attention(q, c.k, c.v, c.table.long(), lens), ValueError),
        (lambda: paged_attention(q, c.k, c.v, c.table, lens.long()), ValueError),
        (lambda: paged_attention(q, c.k, c.v, c.table[:, ::2], lens), ValueError),
        (lambda: paged_attention(q, c.k, c.v[:1], c.table, lens), ValueError),
        (lambda: paged_attention(q, c.k.transpose(0, 1), c.v, c.table, lens), ValueError),
        (lambda: paged_attention(q, c.k, c.v, c.table, lens, softcap=-2.0), L.SfmError),
        (lambda: paged_attention(q, c.k, c.v, c.table, lens, slopes=sl, positions=pos), L.SfmError),
        (lambda: paged_attention(q, c.k, c.v, c.table, lens, q_positions=lens), L.SfmError),
        (lambda: paged_attention(q, c.k, c.v, c.table, lens, weights=w[:, :1].contiguous()), ValueError),
        (lambda: paged_attention(q, c.k, c.v, c.table, lens, weights=w.double()), ValueError),
        (lambda: paged_attention(q, c.k, c.v, c.table.repeat(1, 400), lens,      # a long table needs more
                                 workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), L.SfmError),
        (lambda: paged_append(k, k, c.k, c.v, c.table, lens, row_starts=ints([0, 2])), ValueError),
        (lambda: paged_append(torch.cat([k, k]), torch.cat([k, k]), c.k, c.v, c.table, lens), L.SfmError),
        (lambda: paged_append(k, k, c.k, c.v, c.table, lens, pos0=lens), L.SfmError),
        (lambda: paged_append(k.float(), k.float(), c.k, c.v, c.table, lens), ValueError),
        (lambda: paged_evict(c.k, c.v, c.table, lens, w, pos, 0), L.SfmError),
        (lambda: paged_evict(c.k, c.v, c.table, lens, w, pos, 8, n_first=5, n_recent=4), L.SfmError),
        (lambda: paged_evict(c.k, c.v, c.table, lens, w, pos, 8, n_first=-1), L.SfmError),
        (lambda: paged_evict(c.k, c.v, c.table, lens, w, None, 8), ValueError),
        (lambda: paged_evict(c.k, c.v, c.table, lens, w, pos[:, :, :30].contiguous(), 8), ValueError),
    ]
    for i, (call, exc) in enumerate(calls):
        before = c.k.clone()
        with pytest.raises(exc):
            call()
            print("call", i, "was not refused")
        assert torch.equal(c.k, before), i
    assert L.check_call_error() == 0
