"""Attention under per-query key ranges against its formula in 64 bits.

Tolerances (elementwise; A = sum_j p_j |v_j|, the scale of the sum's terms):
  bf16: P is rounded once for the product with V (at most 2^-8 of each term) and the output
        once (2^-8 of it), fp32 scores add at most a few 1e-4 of A:
        2^-8 (|o| + A) + 5e-4 A
  fp32: a score's dot product of D terms is off by at most D 2^-24 sum |q_d k_d| / sqrt(D)
        (<= 128 x 6e-8 x 11 = 9e-5 for the inputs here), which moves numerator and denominator
        of the softmax: 2e-4 A + 2^-23 |o|; and relative L2 <= 1e-5, the fp32 mode's tolerance.
"""
import ctypes as C
import math
import random

import pytest
import torch

from streaming_flow_matching_b200 import _lib as L
from tests import _paged_ref as R
from tests._gpu_util import FP32_TOL, rel_l2

pytestmark = pytest.mark.gpu


def make(n_q, n_kv, h, hk, d, dtype, seed=0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(n_q, h, d, generator=g, device="cuda") * scale).to(dtype)
    k = torch.randn(n_kv, hk, d, generator=g, device="cuda").to(dtype)
    v = torch.randn(n_kv, hk, d, generator=g, device="cuda").to(dtype)
    return q, k, v


def ladder(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


def check(got, ref, mag, dtype, far=False):
    """far: weights may underflow to 0, and 0 x infinity is NaN where the definition has infinity."""
    got, err = got.double(), None
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got))
    same = ~fin & ~torch.isnan(ref)
    if far:
        same = same & ~torch.isnan(got)
    else:
        assert torch.equal(torch.isnan(ref), torch.isnan(got))
    assert torch.equal(ref[same], got[same])
    err = (got - ref)[fin].abs()
    if dtype == torch.bfloat16:
        tol = 2.0 ** -8 * (ref.abs() + mag) + 5e-4 * mag
    else:
        tol = 2e-4 * mag + 2.0 ** -23 * ref.abs()
        if fin.all() and float(ref.abs().max()) > 0:
            assert rel_l2(got.cpu().numpy(), ref.cpu().numpy()) <= FP32_TOL
    assert bool((err <= tol[fin] + 1e-30).all()), float((err / (tol[fin] + 1e-30)).max())


def run(q, k, v, lo=None, hi=None, **kw):
    from streaming_flow_matching_b200 import attention_masked
    ref_kw = {n: kw[n] for n in ("slopes",) if n in kw}
    n_q, n_kv = q.shape[0], k.shape[0]
    out = attention_masked(q, k, v, lo, hi, **kw)
    torch.cuda.synchronize()
    assert L.check_call_error() == 0
    lo = torch.zeros(n_q, device="cuda", dtype=torch.int32) if lo is None else lo
    hi = torch.full((n_q,), n_kv, device="cuda", dtype=torch.int32) if hi is None else hi
    ref, mag, _ = R.attend(q, k, v, lo, hi, cap=kw.get("softcap", 0.0), **ref_kw)
    check(out, ref, mag, q.dtype, far="slopes" in kw)
    return out


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("n_q,n_kv,starts,prefixes,causal", [
    (1, 1, [0, 1], None, True),
    (5, 5, [0, 0, 3, 3, 5], [0, 9, 1, 0], True),            # empty documents, a prefix past the end
    (300, 300, [0, 100, 250, 290], None, True),             # padding behind the last
    (300, 700, [40, 450, 700], [30, 100], True),            # padding before the first, cached keys
    (300, 700, [0, 450, 450, 700], None, False),
    (257, 257, None, [100], True),
    (257, 300, None, None, True),
    (64, 100, None, None, False),
])
def test_bounds(cuda_device, n_q, n_kv, starts, prefixes, causal):
    from streaming_flow_matching_b200 import attention_bounds
    lo, hi = attention_bounds(n_q, n_kv, doc_starts=ints(starts) if starts else None,
                              prefixes=ints(prefixes) if prefixes else None, causal=causal)
    rl, rh = R.bounds(n_q, n_kv, starts or [0, n_kv], prefixes, causal)
    got = list(zip(lo.tolist(), hi.tolist()))
    assert got == [(a, b) if a < b else (a, b) for a, b in zip(rl, rh)]


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32), (F32, 64), (F32, 96), (F32, 128)])
@pytest.mark.parametrize("n_q,n_kv,h,hk", [
    (1, 1, 1, 1), (1, 129, 3, 1), (2, 640, 4, 4), (127, 127, 2, 1), (128, 128, 6, 3), (129, 257, 2, 2),
    (300, 1000, 8, 2), (513, 513, 3, 3)])
def test_causal(cuda_device, dtype, d, n_q, n_kv, h, hk):
    from streaming_flow_matching_b200 import attention_bounds
    q, k, v = make(n_q, n_kv, h, hk, d, dtype, seed=n_q + n_kv)
    lo, hi = attention_bounds(n_q, n_kv, causal=True)
    run(q, k, v, lo, hi)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("cap,bias", [(0.0, True), (20.0, False), (50.0, True)])
@pytest.mark.parametrize("n,docs,h,hk,seed", [(700, 6, 4, 2, 0), (1500, 3, 3, 3, 1), (400, 40, 6, 2, 2)])
def test_documents_cap_bias(cuda_device, dtype, d, cap, bias, n, docs, h, hk, seed):
    from streaming_flow_matching_b200 import attention_bounds
    r = random.Random(seed)
    end = n - 17
    starts = [0] + sorted(r.randint(0, end) for _ in range(docs - 1)) + [end]
    prefixes = [r.randint(0, b - a) for a, b in zip(starts, starts[1:])]
    q, k, v = make(n, n, h, hk, d, dtype, seed=seed, scale=4.0)
    if dtype == F32:
        q = q / 4                                           # keeps the derived score error
    lo, hi = attention_bounds(n, n, doc_starts=ints(starts), prefixes=ints(prefixes), causal=True)
    # padding holds what it holds
    k[end:], v[end:] = float("nan"), float("inf")
    kw = dict(softcap=cap)
    if bias:
        kw["slopes"] = ladder(h)
    out = run(q, k, v, lo, hi, **kw)
    assert int(torch.count_nonzero(out[end:])) == 0         # empty ranges: zeros


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("h,hk", [(4, 2), (3, 3)])
def test_masked_keys_may_hold_anything(cuda_device, dtype, d, h, hk):
    # non-finite K rows where a query may not look, non-finite V elements that some rows of a
    # tile see and others do not: they reach exactly the rows and dimensions that see them
    n = 400
    q, k, v = make(n, n, h, hk, d, dtype, seed=5)
    lo = ints([0] * 150 + [150] * 100 + [250] * 150)
    hi = ints([150] * 150 + [250] * 100 + [400] * 150)
    v[160, 0, 3] = float("inf")
    v[200, hk - 1, 7] = float("nan")
    v[201, 0, 3] = float("-inf")
    run(q, k, v, lo, hi)
    v = v.clone()
    v[150:250] = float("nan")
    k = k.clone()
    k[150:250] = float("nan")
    hi = ints([150] * 150 + [150] * 100 + [400] * 150)      # the middle document's rows see nothing
    out = run(q, k, v, lo, hi)
    assert int(torch.count_nonzero(out[150:250])) == 0


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32)])
def test_arbitrary_ranges(cuda_device, dtype, d):
    # ranges out of order, empty, reversed, outside [0, n_kv]
    r = random.Random(3)
    n_q, n_kv = 333, 900
    lo = [r.randint(-50, 950) for _ in range(n_q)]
    hi = [a + r.randint(-20, 300) for a in lo]
    q, k, v = make(n_q, n_kv, 4, 2, d, dtype, seed=8)
    run(q, k, v, ints(lo), ints(hi))
    run(q, k, v, ints(lo), None)
    run(q, k, v, None, ints(hi))
    run(q, k, v, ints([5] * n_q), ints([5] * n_q))          # every range empty


@pytest.mark.parametrize("h,hk", [(8, 2), (2, 2)])
@pytest.mark.parametrize("n_q,n_kv", [(300, 5000), (20000, 20000)])
def test_empty_blocks_write_zeros_whatever_q_holds(cuda_device, h, hk, n_q, n_kv):
    # blocks and query tiles without a key: nothing of Q, which is on its way then, may show
    from streaming_flow_matching_b200 import attention_masked
    q, k, v = make(n_q, n_kv, h, hk, 128, torch.bfloat16, seed=8)
    i = torch.arange(n_q, device="cuda", dtype=torch.int32)
    live = (i // 128) % 5 == 2                               # every fifth tile of 128 rows sees 3 keys
    hi = torch.where(live, 7, 4).to(torch.int32)
    lo = torch.full_like(hi, 4)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    seen = v[4:7].double().repeat_interleave(h // hk, 1)
    for qq in (q, torch.full_like(q, float("nan"))):
        flush.zero_()
        out = attention_masked(qq, k, v, lo, hi)
        assert int(torch.count_nonzero(out[~live])) == 0
    q0 = torch.zeros_like(q)                                 # equal weights: the mean of the three
    out = attention_masked(q0, k, v, lo, hi)
    assert int(torch.count_nonzero(out[~live])) == 0
    # P is 1, exact in bf16: the output's rounding, and a few of fp32 in the sum and its division
    tol = seen.mean(0).abs() * 2.0 ** -8 + seen.abs().sum(0) * 2.0 ** -21
    assert bool(((out[live].double() - seen.mean(0)).abs() <= tol).all())
    assert L.check_call_error() == 0


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32), (F32, 96), (F32, 128)])
@pytest.mark.parametrize("n_q,n_kv,h,hk", [(1, 20000, 2, 1), (3, 5000, 1, 1), (130, 9000, 4, 1)])
def test_key_splits_join(cuda_device, dtype, d, n_q, n_kv, h, hk):
    # few rows over many keys run in splits: rows that see no key of a split, or of any
    code = L.SFM_DTYPE_BF16 if dtype == BF else L.SFM_DTYPE_FP32
    assert L.lib.sfm_attention_masked_workspace_bytes(n_q, n_kv, h, hk, d, code) > 0
    q, k, v = make(n_q, n_kv, h, hk, d, dtype, seed=n_kv)
    run(q, k, v, softcap=30.0)
    hi = ints([0 if i % 3 == 2 else 100 + i for i in range(n_q)])
    out = run(q, k, v, None, hi)
    if n_q > 2:
        assert int(torch.count_nonzero(out[2])) == 0
    k[n_kv - 700:], v[n_kv - 700:] = float("nan"), float("inf")
    v[50, 0, 1] = float("-inf")
    hi = ints([n_kv - 700 - 300 * (i % 4) for i in range(n_q)])
    lo = ints([60 * (i % 2) for i in range(n_q)])
    run(q, k, v, lo, hi)


@pytest.mark.parametrize("n_q,n_kv,h,hk", [(924, 9000, 24, 8), (1848, 17000, 24, 24)])
def test_key_splits_over_several_waves(cuda_device, n_q, n_kv, h, hk):
    # more CTAs than SMs, and keys split all the same
    from streaming_flow_matching_b200 import attention_bounds, attention_masked
    need = L.lib.sfm_attention_masked_workspace_bytes(n_q, n_kv, h, hk, 128, L.SFM_DTYPE_BF16)
    splits = need // (n_q * h * 129 * 4)
    assert splits > 1 and splits * h * (n_q // 256) > 148
    q, k, v = make(n_q, n_kv, h, hk, 128, BF, seed=3)
    lo, hi = attention_bounds(n_q, n_kv, causal=True)
    out = attention_masked(q, k, v, lo, hi)
    assert L.check_call_error() == 0
    at = torch.cat([torch.arange(0, n_q, 97, device="cuda"), ints([n_q - 1]).long()])
    ref, mag, _ = R.attend(q[at], k, v, lo[at], hi[at])
    check(out[at], ref, mag, BF)


@pytest.mark.parametrize("h,hk", [(16, 16), (16, 8)])
def test_more_blocks_than_sms(cuda_device, h, hk):
    # several waves of query blocks: all keys, few, none
    n = 3000
    q, k, v = make(n, n, h, hk, 128, BF, seed=h + hk)
    run(q, k, v)
    hi = ints([n if i % 200 < 100 else 0 if i < 600 else 130 if i < 900 else i + 1 for i in range(n)])
    out = run(q, k, v, None, hi, softcap=20.0, slopes=ladder(h))
    assert int(torch.count_nonzero(out[100:200])) == 0
    out = run(q, k, v, None, ints([min(i, 400) for i in range(n)]))
    assert int(torch.count_nonzero(out[0])) == 0


@pytest.mark.parametrize("h,hk", [(3, 1), (6, 2), (5, 1), (14, 2), (7, 7)])
@pytest.mark.parametrize("n_q,n_kv", [(100, 700), (128, 128), (129, 129), (256, 900), (300, 300), (700, 700)])
def test_odd_groups(cuda_device, h, hk, n_q, n_kv):
    # pairs of heads and the odd one cover rows differently: every head and row once, in splits too
    from streaming_flow_matching_b200 import attention_bounds
    q, k, v = make(n_q, n_kv, h, hk, 128, BF, seed=h + n_q)
    lo, hi = attention_bounds(n_q, n_kv, doc_starts=ints([0, n_kv // 3, n_kv // 2, n_kv]), causal=True)
    run(q, k, v, lo, hi, softcap=20.0, slopes=ladder(h))


@pytest.mark.parametrize("h,hk", [(1, 1), (3, 1), (4, 2)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True)])
def test_query_tiles_with_their_own_keys(cuda_device, h, hk, cap, bias):
    # the 128-row tiles of one block see key tiles of their own: disjoint, one empty, one long
    # and one short, gaps, in either order; and non-finite values where only one of them looks
    n_kv = 2000
    spans = [((0, 300), (900, 2000)), ((1500, 2000), (0, 128)), ((0, 0), (256, 1300)), ((700, 1900), (5, 5)),
             ((0, 2000), (1000, 1001)), ((128, 256), (256, 384))]
    lo, hi = [], []
    for a, b in spans:
        for x, y in (a, b):
            lo += [x] * 128
            hi += [y] * 128
    lo, hi = lo[:-50], hi[:-50]
    q, k, v = make(len(lo), n_kv, h, hk, 128, BF, seed=h)
    kw = dict(softcap=cap, slopes=ladder(h)) if bias else dict(softcap=cap)
    run(q, k, v, ints(lo), ints(hi), **kw)
    v[310:890] = float("nan")
    v[1950, 0, 4] = float("inf")
    keep = [i for i in range(len(lo)) if not (lo[i] < 890 and hi[i] > 310)]
    lo = [lo[i] if i in set(keep) else 0 for i in range(len(lo))]
    hi = [hi[i] if i in set(keep) else 200 for i in range(len(hi))]
    run(q, k, v, ints(lo), ints(hi), **kw)


def test_all_keys_equals_attention_in_value(cuda_device):
    from streaming_flow_matching_b200 import attention, attention_masked
    q, k, v = make(500, 1200, 2, 2, 128, BF)
    a, b = attention(q, k, v).double(), attention_masked(q, k, v).double()
    assert rel_l2(b.cpu().numpy(), a.cpu().numpy()) <= 2.0 ** -7


def test_far_keys(cuda_device):
    # element offsets past 2^31 in K and V
    from streaming_flow_matching_b200 import attention_masked
    n, hk, far = 1100000, 16, 1098500
    q, _, _ = make(40, 1, hk, hk, 128, BF)
    k, v = (torch.zeros(n, hk, 128, dtype=BF, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    k[far:] = torch.randn(n - far, hk, 128, generator=g, device="cuda").to(BF)
    v[far:] = torch.randn(n - far, hk, 128, generator=g, device="cuda").to(BF)
    v[far + 3, 15, 7] = float("inf")
    out = attention_masked(q, k, v, ints([far + i for i in range(40)]), ints([n - i for i in range(40)]))
    ref, mag, _ = R.attend(q, k[far:], v[far:], ints(list(range(40))), ints([n - far - i for i in range(40)]))
    check(out, ref, mag, BF)
    assert L.check_call_error() == 0


def test_large_scores(cuda_device):
    # scores of hundreds, rising along the keys: the running max moves in every tile
    n = 700
    q, k, v = make(n, n, 2, 1, 128, BF, scale=1.0)
    k = (k.float() * torch.linspace(1, 40, n, device="cuda")[:, None, None]).to(BF)
    run(q, k, v)
    run(q, k, v, softcap=50.0)
    # caps far from the scores on either side, slopes that favour far keys
    run(q, k, v, softcap=1000.0)
    run(q, k, v, softcap=1e-3)
    run(q, k, v, softcap=1e20)
    run(q, k, v, slopes=-0.05 * ladder(2))
    run(q, k, v, slopes=-0.05 * ladder(2), softcap=5.0)


def test_infinite_scores(cuda_device):
    # a -inf score has weight 0; a row with nothing else gives zeros
    from streaming_flow_matching_b200 import attention_masked
    for dtype, d in ((BF, 128), (F32, 64)):
        q, k, v = make(40, 200, 2, 1, d, dtype)
        q[:, :, 0] = 1.0
        k[:150, :, 0] = float("-inf")
        ref = attention_masked(q, k[150:].contiguous(), v[150:].contiguous())
        out = attention_masked(q, k, v)
        check(out, ref.double(), ref.double().abs() + 1, dtype)
        out = attention_masked(q, k[:150].contiguous(), v[:150].contiguous())
        assert int(torch.count_nonzero(out)) == 0


def test_same_inputs_same_bits_and_graph(cuda_device):
    from streaming_flow_matching_b200 import attention_bounds, attention_masked
    q, k, v = make(600, 900, 4, 2, 128, BF)
    s = torch.cuda.Stream()
    lo, hi = attention_bounds(600, 900, causal=True)
    a = attention_masked(q, k, v, lo, hi, softcap=30.0)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = attention_masked(q, k, v, lo, hi, softcap=30.0)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bounds = attention_bounds(600, 900, causal=True)
        c = attention_masked(q, k, v, *bounds, softcap=30.0)
    q.copy_(torch.randn_like(q))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c, attention_masked(q, k, v, lo, hi, softcap=30.0))


def test_given_buffers_and_refusals(cuda_device):
    from streaming_flow_matching_b200 import attention_bounds, attention_masked
    q, k, v = make(2, 5000, 2, 1, 128, BF)
    need = L.lib.sfm_attention_masked_workspace_bytes(2, 5000, 2, 1, 128, L.SFM_DTYPE_BF16)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    assert attention_masked(q, k, v, out=out, workspace=ws) is out
    assert torch.equal(out, attention_masked(q, k, v))
    bad = [
        (dict(workspace=ws[:-16]), L.SfmError), (dict(softcap=-1.0), L.SfmError),
        (dict(softcap=math.inf), L.SfmError), (dict(softcap=math.nan), L.SfmError),
        (dict(slopes=torch.ones(3, device="cuda")), ValueError),
        (dict(key_lo=torch.zeros(2, dtype=torch.int64, device="cuda")), ValueError),
        (dict(key_lo=ints([0])), ValueError), (dict(out=out[:1]), ValueError),
    ]
    for kw, exc in bad:
        with pytest.raises(exc):
            attention_masked(q, k, v, **kw)
    with pytest.raises(ValueError):
        attention_masked(q, k.cpu(), v)
    with pytest.raises(ValueError):
        attention_masked(q.transpose(0, 1), k, v)
    with pytest.raises(L.SfmError):
        attention_masked(q, k.repeat(1, 3, 1), v.repeat(1, 3, 1))     # 2 heads over 3 key heads
    with pytest.raises(L.SfmError):
        attention_masked(q, k[:1].contiguous(), v[:1].contiguous(), slopes=ladder(2))
    with pytest.raises(L.SfmError):
        attention_bounds(5, 4)
    with pytest.raises(ValueError):
        attention_bounds(5, 5, doc_starts=ints([0, 5]), prefixes=ints([1, 2]))
    assert L.check_call_error() == 0


def test_a_wait_that_gives_up_is_reported(cuda_device):
    from streaming_flow_matching_b200 import attention_masked
    q, k, v = make(200, 300, 2, 1, 128, BF)
    good = attention_masked(q, k, v)
    L.set_call_fault(L.SFM_FAULT_ATTN_NO_LOADS, 20_000_000)
    try:
        attention_masked(q, k, v)
        code = L.check_call_error()
    finally:
        L.set_call_fault(0)
    assert code >> 8 == 4, hex(code)
    assert torch.equal(attention_masked(q, k, v), good)
    assert L.check_call_error() == 0
