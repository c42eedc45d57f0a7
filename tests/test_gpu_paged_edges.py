"""The paged cache at its edges: calls from several threads, bad pages beside the state arrays, queries
far from every position, values that a vanishing weight could hide.

Tolerances as in test_gpu_paged.
"""
import sys
import threading

import pytest
import torch

from streaming_flow_matching_b200 import _lib as L
from tests import _paged_ref as R
from tests.test_gpu_paged import BF, F32, Cache, ints, ladder, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,h", [(BF, 128, 8), (BF, 128, 16), (F32, 64, 4)])
def test_two_host_threads(cuda_device, dtype, d, h):
    # calls of one kernel with different needs of shared memory (weights or none), from two threads at once
    lens = [100, 70]
    c = Cache(lens, 16, 1, d, dtype, seed=3)
    q = torch.randn(2, h, d, device="cuda").to(dtype)
    code = L.SFM_DTYPE_BF16 if dtype == BF else L.SFM_DTYPE_FP32
    n_pages, page = c.k.shape[:2]
    width, dev_lens = c.table.shape[1], ints(lens)
    for weights in (0, 1):
        assert L.lib.sfm_paged_attention_workspace_bytes(2, width * page, h, 1, d, code, weights) == 0
    w = torch.zeros(2, 1, 100, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = run(c, q, lens)
    torch.cuda.synchronize()
    codes, start = [set(), set()], threading.Barrier(2)

    def caller(i):
        args = (q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.table.data_ptr(), dev_lens.data_ptr(),
                outs[i].data_ptr(), 2, n_pages, page, width, h, 1, d, code, 0.0, None, None, None,
                w.data_ptr() if i else None, 100 if i else 0, None, 0, streams[i].cuda_stream)
        start.wait()
        for _ in range(20000):
            codes[i].add(L.lib.sfm_paged_attention(*args))

    every, threads = sys.getswitchinterval(), [threading.Thread(target=caller, args=(i,)) for i in range(2)]
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(every)
    torch.cuda.synchronize()
    assert codes == [{L.SFM_OK}, {L.SFM_OK}]
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert L.check_call_error() == 0


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32)])
@pytest.mark.parametrize("n,keep,alone", [(64, 48, True), (1500, 700, False)])
@pytest.mark.parametrize("where", ["from", "to", "both"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_evict_leaves_slots_on_a_bad_page_as_they_were(cuda_device, dtype, d, n, keep, alone, where, bad):
    from streaming_flow_matching_b200 import paged_evict
    hk, page = 2, 16
    c = Cache([n], page, hk, d, dtype, seed=2)
    assert (L.lib.sfm_paged_evict_workspace_bytes(1, n, hk, keep) == 0) == alone
    w = torch.arange(n, device="cuda").float().expand(1, hk, n).contiguous()      # the last `keep` stay
    pos = (torch.arange(n, device="cuda", dtype=torch.int32) + 5).expand(1, hk, n).contiguous()
    at = c.rows(0, n)
    dead = {"from": [(n - 3) // page], "to": [0], "both": [0, (n - 3) // page]}[where]
    ek, ev, ew, ep = c.k.clone(), c.v.clone(), w.clone(), pos.clone()
    moved = 0
    for x in range(hk):
        for a, b in zip(*R.evict(w[0, x].tolist(), pos[0, x].tolist(), n, keep, 0, 0)):
            if a // page in dead or b // page in dead:
                continue
            moved += 1
            for e, src in ((ek, c.k), (ev, c.v)):
                e.view(-1, hk, d)[at[a], x] = src.view(-1, hk, d)[at[b], x]
            ew[0, x, a], ep[0, x, a] = w[0, x, b], pos[0, x, b]
    for i in dead:
        c.table[0, i] = bad
    paged_evict(c.k, c.v, c.table, ints([n]), w, pos, keep)
    assert L.check_call_error() == 0x301
    assert moved > 0 or n == 64
    assert torch.equal(c.k, ek) and torch.equal(c.v, ev)
    assert torch.equal(w, ew) and torch.equal(pos, ep)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 96)])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("pos0", [None, [7, 900]])
def test_append_leaves_slots_on_a_bad_page_as_they_were(cuda_device, dtype, d, bad, pos0):
    from streaming_flow_matching_b200 import paged_append
    hk, page, cap = 3, 16, 100
    c = Cache([60, 90], page, hk, d, dtype, seed=4)
    before, rows = [5, 30], [55, 60]
    starts = [0, 55, 115]
    k, v = (torch.randn(115, hk, d, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(2, hk, cap, device="cuda")
    pos = torch.full((2, hk, cap), -7, dtype=torch.int32, device="cuda")
    ek, ev, ew, ep = c.k.clone(), c.v.clone(), w.clone(), pos.clone()
    dead = [(0, 1), (1, 3), (1, 4)]
    for s in range(2):
        at = c.rows(s, before[s] + rows[s])
        for i in range(rows[s]):
            t = before[s] + i
            if (s, t // page) in dead:
                continue
            ek.view(-1, hk, d)[at[t]], ev.view(-1, hk, d)[at[t]] = k[starts[s] + i], v[starts[s] + i]
            ew[s, :, t] = 0
            ep[s, :, t] = (pos0 or before)[s] + i
    for s, i in dead:
        c.table[s, i] = bad
    paged_append(k, v, c.k, c.v, c.table, ints(before), row_starts=ints(starts), positions=pos, weights=w,
                 pos0=None if pos0 is None else ints(pos0))
    assert L.check_call_error() == 0x301
    assert torch.equal(c.k, ek) and torch.equal(c.v, ev)
    assert torch.equal(w, ew) and torch.equal(pos, ep)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32), (F32, 64), (F32, 96), (F32, 128)])
@pytest.mark.parametrize("lens,h,hk", [([300, 64, 1], 6, 2), ([5000, 17, 3000], 8, 2), ([330] * 150 + [9, 0, 2000], 3, 1),
                                       ([700], 20, 1)])
@pytest.mark.parametrize("cap,sign", [(0.0, 1.0), (30.0, 1.0), (0.0, -1.0)])
def test_attention_far_from_every_position(cuda_device, dtype, d, lens, h, hk, cap, sign):
    n = max(lens)
    c = Cache(lens, 16, hk, d, dtype, seed=len(lens) + h)
    q = torch.randn(len(lens), h, d, device="cuda").to(dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    pos = torch.stack([torch.randperm(n + 5, generator=g, device="cuda") for _ in range(len(lens) * hk)])
    pos = (pos.view(len(lens), hk, n + 5) * 3).to(torch.int32).contiguous()
    for far in (57600, 1000003):
        kw = dict(softcap=cap, slopes=sign * ladder(h), positions=pos, q_positions=ints([far + s for s in range(len(lens))]))
        run(c, q, lens, weights=torch.rand(len(lens), hk, n + 5, device="cuda"), **kw)
        run(c, q, lens, **kw)
    kw["q_positions"] = ints([-9000] * len(lens))
    run(c, q, lens, weights=torch.zeros(len(lens), hk, n + 5, device="cuda"), **kw)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("lens,h,hk", [([330] * 150, 3, 1), ([1300, 7, 1300, 0] * 40, 8, 2), ([70] * 200, 20, 1)])
@pytest.mark.parametrize("cap,sign", [(0.0, 1.0), (30.0, -1.0)])
def test_attention_far_with_full_tables(cuda_device, dtype, d, lens, h, hk, cap, sign):
    # sequences as long as the state arrays, most of them finished by one CTA; ranks of positions and slots apart
    n = max(lens)
    c = Cache(lens, 16, hk, d, dtype, seed=len(lens))
    q = torch.randn(len(lens), h, d, device="cuda").to(dtype)
    g = torch.Generator(device="cuda").manual_seed(6)
    pos = torch.stack([torch.randperm(n, generator=g, device="cuda") for _ in range(len(lens) * hk)])
    pos = (pos.view(len(lens), hk, n) * 40).to(torch.int32).contiguous()
    for q_pos in (120000, -60000):
        run(c, q, lens, softcap=cap, slopes=sign * ladder(h), positions=pos, q_positions=ints([q_pos] * len(lens)),
            weights=torch.rand(len(lens), hk, n, device="cuda"))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_a_weight_that_vanishes_hides_nothing(cuda_device, dtype, d, what):
    # a non-finite element of V far away, in another CTA's share: the same in both forms
    from streaming_flow_matching_b200 import paged_attention
    lens = [500, 40]
    c = Cache(lens, 16, 1, d, dtype, seed=9)
    q = torch.randn(2, 2, d, device="cuda").to(dtype)
    c.v.view(-1, 1, d)[c.rows(0, 500)[3], 0, 5] = float(what)
    sl = torch.tensor([1.0, 0.5], device="cuda")              # 2^-717 and 2^-358 at the far end
    wide = torch.cat([c.table, torch.full((2, 2500), -1, dtype=torch.int32, device="cuda")], 1)
    code = L.SFM_DTYPE_BF16 if dtype == BF else L.SFM_DTYPE_FP32
    need = L.lib.sfm_paged_attention_workspace_bytes
    for t, big in ((c.table, False), (wide, True)):
        assert (need(2, t.shape[1] * 16, 2, 1, d, code, 0) > 0) == big
        out = paged_attention(q, c.k, c.v, t, ints(lens), slopes=sl)
        assert not bool(torch.isfinite(out[0, :, 5]).any())
        out[0, :, 5] = 0
        assert bool(torch.isfinite(out).all())
    assert L.check_call_error() == 0


def test_numbers_past_32_bits_are_refused(cuda_device):
    from streaming_flow_matching_b200 import attention_bounds, paged_evict
    c = Cache([64], 16, 1, 128, BF)
    w = torch.rand(1, 1, 64, device="cuda")
    pos = torch.arange(64, device="cuda", dtype=torch.int32).view(1, 1, 64).contiguous()
    ek, ew = c.k.clone(), w.clone()
    for kw in (dict(keep=2 ** 32 + 8), dict(keep=8, n_first=2 ** 32), dict(keep=8, n_recent=2 ** 32 + 1), dict(keep=-2 ** 32 + 8),
               dict(keep=2 ** 31)):
        with pytest.raises(ValueError):
            paged_evict(c.k, c.v, c.table, ints([64]), w, pos, **kw)
    for n_q, n_kv in ((4, 2 ** 32 + 8), (4, 2 ** 31)):
        with pytest.raises(ValueError):
            attention_bounds(n_q, n_kv)
    assert torch.equal(c.k, ek) and torch.equal(w, ew)
    paged_evict(c.k, c.v, c.table, ints([64]), w, pos, 2 ** 31 - 1)      # longer than any sequence: nothing to do
    assert torch.equal(c.k, ek) and torch.equal(w, ew)


def test_eviction_is_timed_on_the_same_state(cuda_device, monkeypatch):
    from streaming_flow_matching_b200 import microbench
    seen, real = [], microbench.paged_evict

    def spy(k, v, table, lengths, w, pos, keep, **kw):
        seen.append((w.clone(), pos.clone()))
        return real(k, v, table, lengths, w, pos, keep, **kw)

    monkeypatch.setattr(microbench, "paged_evict", spy)
    r = microbench.bench_paged(2, 300, 4, 2, 1, 3)
    assert r["evict_tenth_ms"] > 0 and len(seen) >= 4
    assert all(torch.equal(w, seen[0][0]) and torch.equal(p, seen[0][1]) for w, p in seen)
