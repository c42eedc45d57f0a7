"""The paged cache's and the masked attention's entry points refuse bad arguments on the
host, before anything touches a GPU; their workspace sizes are functions of the shape."""
import ctypes as C

import pytest

from streaming_flow_matching_b200 import _lib as L

P = 1 << 20          # an aligned address; no call below gets as far as using it
BF, F32 = L.SFM_DTYPE_BF16, L.SFM_DTYPE_FP32
INF, NAN = float("inf"), float("nan")


def append(**kw):
    a = dict(k=P, v=P, kp=P, vp=P, table=P, lengths=P, row_starts=P, n_rows=4, n_seq=2, n_pages=8, page=16,
             width=4, hk=2, d=128, dtype=BF, positions=P, pos0=P, weights=P, cap=64)
    a.update(kw)
    return L.lib.sfm_paged_append(*a.values(), None)


def attention(**kw):
    a = dict(q=P, kp=P, vp=P, table=P, lengths=P, o=2 * P, n_seq=2, n_pages=8, page=16, width=1024, h=4, hk=2,
             d=128, dtype=BF, cap=0.0, slopes=P, positions=P, q_positions=P, weights=P, room=1 << 14, ws=P,
             ws_bytes=1 << 40)
    a.update(kw)
    return L.lib.sfm_paged_attention(*a.values(), None)


def evict(**kw):
    a = dict(kp=P, vp=P, table=P, lengths=P, weights=P, positions=P, room=9000, n_seq=2, n_pages=8, page=16, width=600,
             hk=2, d=128, dtype=BF, keep=8000, first=0, recent=0, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return L.lib.sfm_paged_evict(*a.values(), None)


def masked(**kw):
    a = dict(q=P, k=P, v=P, o=2 * P, n_q=4, n_kv=8, h=4, hk=2, d=128, dtype=BF, lo=P, hi=P, cap=0.0, slopes=P, ws=P,
             ws_bytes=1 << 40)
    a.update(kw)
    return L.lib.sfm_attention_masked(*a.values(), None)


CACHE = [dict(kp=None), dict(vp=None), dict(table=None), dict(lengths=None), dict(kp=P + 8), dict(vp=P + 4),
         dict(table=P + 2), dict(lengths=P + 1), dict(n_seq=0), dict(n_pages=0), dict(page=0), dict(width=0),
         dict(hk=0), dict(dtype=7), dict(weights=P + 2), dict(positions=P + 1)]
UNSUPPORTED = [dict(d=64), dict(d=48, dtype=F32), dict(d=160, dtype=F32), dict(d=0, dtype=F32),
               dict(page=1 << 30, width=4), dict(page=1 << 20, n_pages=1 << 20), dict(n_seq=1 << 30, width=1 << 20)]


@pytest.mark.parametrize("call", [append, attention, evict])
@pytest.mark.parametrize("bad", CACHE)
def test_cache_arguments(call, bad):
    assert call(**bad) == L.SFM_EINVAL


@pytest.mark.parametrize("call", [append, attention, evict])
@pytest.mark.parametrize("bad", UNSUPPORTED)
def test_cache_shapes(call, bad):
    assert call(**bad) == L.SFM_EUNSUPPORTED


@pytest.mark.parametrize("bad", [dict(n_rows=-1), dict(k=None), dict(v=None), dict(k=P + 8), dict(cap=0),
                                 dict(positions=None, weights=None), dict(row_starts=None), dict(pos0=P + 2),
                                 dict(row_starts=P + 1)])
def test_append_arguments(bad):
    assert append(**bad) == L.SFM_EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(o=None), dict(o=P), dict(q=P + 8), dict(o=P + 2), dict(h=3), dict(h=0), dict(cap=-1.0),
    dict(cap=INF), dict(cap=1e-4), dict(cap=1e31),
    dict(cap=NAN), dict(positions=None), dict(q_positions=None), dict(room=0), dict(ws=None),
    dict(ws=P + 8), dict(ws_bytes=16), dict(slopes=P + 2)])
def test_attention_arguments(bad):
    assert attention(**bad) == L.SFM_EINVAL


@pytest.mark.parametrize("bad", [dict(keep=0), dict(first=-1), dict(recent=-1), dict(keep=8, first=5, recent=4),
                                 dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), dict(weights=None),
                                 dict(positions=None), dict(room=0), dict(ws=None), dict(ws_bytes=0)])
def test_evict_arguments(bad):
    assert evict(**bad) == L.SFM_EINVAL


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), L.SFM_EINVAL), (dict(k=None), L.SFM_EINVAL), (dict(v=None), L.SFM_EINVAL),
    (dict(o=None), L.SFM_EINVAL), (dict(o=P), L.SFM_EINVAL), (dict(n_q=0), L.SFM_EINVAL), (dict(n_kv=0), L.SFM_EINVAL),
    (dict(h=3), L.SFM_EINVAL), (dict(hk=0), L.SFM_EINVAL), (dict(dtype=3), L.SFM_EINVAL),
    (dict(d=64), L.SFM_EUNSUPPORTED), (dict(d=33, dtype=F32), L.SFM_EUNSUPPORTED),
    (dict(cap=-0.5), L.SFM_EINVAL), (dict(cap=1e-9), L.SFM_EINVAL), (dict(cap=NAN), L.SFM_EINVAL), (dict(cap=INF), L.SFM_EINVAL),
    (dict(n_q=9), L.SFM_EINVAL),                              # a bias needs n_kv >= n_q
    (dict(q=P + 2), L.SFM_EINVAL), (dict(lo=P + 2), L.SFM_EINVAL), (dict(slopes=P + 1), L.SFM_EINVAL),
    (dict(n_q=1, n_kv=4096, ws=None), L.SFM_EINVAL), (dict(n_q=1, n_kv=4096, ws_bytes=64), L.SFM_EINVAL),
    (dict(n_q=2 ** 31 - 1, n_kv=2 ** 31 - 1), L.SFM_EUNSUPPORTED)])
def test_masked_arguments(bad, code):
    assert masked(**bad) == code


@pytest.mark.parametrize("bad", [
    dict(n_q=0), dict(n_kv=3), dict(lo=None), dict(hi=None), dict(causal=2), dict(n_docs=0), dict(n_docs=-1),
    dict(starts=None, n_docs=2), dict(starts=None, prefixes=None, n_docs=1), dict(starts=None, n_docs=0)])
def test_bounds_arguments(bad):
    a = dict(n_q=4, n_kv=8, starts=P, prefixes=P, n_docs=2, causal=1, lo=P, hi=P)
    a.update(bad)
    assert L.lib.sfm_attention_bounds(*a.values(), None) == L.SFM_EINVAL


def test_sizes_past_what_32_bits_index():
    top = 2 ** 31 - 1
    assert append(n_rows=top) == L.SFM_EUNSUPPORTED
    assert L.lib.sfm_attention_bounds(top, top, P, P, 2, 1, P, P, None) == L.SFM_EUNSUPPORTED
    assert masked(n_q=4, n_kv=top) == L.SFM_EUNSUPPORTED
    assert L.lib.sfm_attention_masked_workspace_bytes(top, top, 4, 2, 128, BF) == 0
    assert L.lib.sfm_attention_masked_workspace_bytes(4, top, 4, 2, 32, F32) == 0
    assert L.lib.sfm_paged_attention_workspace_bytes(top, 100, 4, 2, 128, BF, 0) == 0
    assert attention(n_seq=top // 2, h=4) == L.SFM_EUNSUPPORTED
    # tiles of all sequences together, were every one as long as its table
    assert attention(n_seq=1 << 11, width=1 << 25, page=32, n_pages=1, weights=None, positions=None,
                     q_positions=None) == L.SFM_EUNSUPPORTED


def test_workspaces():
    att = L.lib.sfm_paged_attention_workspace_bytes
    assert att(4, 9000, 24, 8, 128, BF, 0) % 16 == 0
    # the raw scores of every slot and query head, when weights are accumulated
    assert att(4, 9000, 24, 8, 128, BF, 1) - att(4, 9000, 24, 8, 128, BF, 0) == 4 * 24 * 9000 * 4 + 4 * 24 * 4
    # without them it does not depend on the lengths
    assert att(4, 9000, 24, 8, 128, BF, 0) == att(400, 100000, 24, 8, 128, BF, 0)
    # small batches of short sequences need none, as long as one head group adds to the weights
    assert att(3, 1300, 24, 8, 128, BF, 0) == att(2, 300, 24, 8, 128, BF, 1) == att(2, 60, 8, 2, 64, F32, 1) == 0
    assert att(1, 100, 40, 1, 128, BF, 0) == 0 and att(1, 100, 40, 1, 128, BF, 1) > 0
    assert att(300, 100, 2, 1, 128, BF, 0) > 0
    for bad in ((0, 10, 4, 2, 128, BF, 0), (1, 0, 4, 2, 128, BF, 0), (1, 10, 4, 3, 128, BF, 0),
                (1, 10, 4, 2, 64, BF, 0), (1, 10, 4, 2, 128, 9, 0)):
        assert att(*bad) == 0
    ev = L.lib.sfm_paged_evict_workspace_bytes
    assert ev(2, 9000, 4, 8000) == (8 + 8 * 2 * 1000) * 4
    assert ev(2, 100, 4, 90) == ev(2, 100, 4, 100) == ev(16, 9000, 8, 8500) == 0      # few rows to move: none
    assert ev(0, 100, 4, 90) == 0 and ev(2, 100, 4, 0) == 0
    mk = L.lib.sfm_attention_masked_workspace_bytes
    assert mk(4096, 4096, 24, 8, 128, BF) == 0                # enough query blocks: no splits
    assert mk(1, 40000, 8, 8, 128, BF) > 0
    assert mk(1, 40000, 8, 8, 64, F32) > 0 and mk(1, 64, 8, 8, 64, F32) == 0
    assert C.sizeof(C.c_size_t) == 8


def test_one_buffer_for_two_results():
    assert append() == L.SFM_EINVAL                           # (kp and vp are one by default here)
    assert append(weights=None, positions=None, pos0=None) == L.SFM_EINVAL
    assert masked(k=2 * P) == L.SFM_EINVAL and masked(v=2 * P) == L.SFM_EINVAL
    assert L.lib.sfm_attention_bounds(4, 8, P, P, 2, 1, P, P, None) == L.SFM_EINVAL


def test_binding_without_the_raw_stream_call(monkeypatch):
    # a torch that lacks it: the stream's handle comes by way of its Stream object
    import importlib.util
    import types

    import torch

    import streaming_flow_matching_b200.paged as paged
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=40 + dev))
    spec = importlib.util.spec_from_file_location(paged.__name__ + "_again", paged.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._stream(2) == 42


def test_dependent_kernels_read_by_plain_loads():
    # a kernel that is set up while the one before still runs may not use the read-only path
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(L.__file__), "csrc")
    users = [f for f in glob.glob(os.path.join(csrc, "*.cu*"))
             if re.search(r"grid_dependency_wait|dependent\.cuh", open(f).read())]
    assert {"paged_attn.cu", "paged_cache.cu", "attn_masked.cu", "paged.cuh"} <= {os.path.basename(f) for f in users}
    for f in users:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        assert not re.search(r"__ldg|__restrict__|ld\.global\.nc", code), f
