"""Paged K/V cache and attention under per-query key ranges: thin binding over libsfm.

As in ``performer``: argument checks and marshalling only.  Tensors are contiguous
CUDA tensors of the current device; calls run on its current stream.  What only the
device knows (page tables, lengths) is checked there: ``_lib.check_call_error``
returns 0x301 / 0x302 after a bad page / a length that the cache does not hold.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .performer import _DT, _need


def _here(t, name):
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _raw_stream():
    return torch.cuda.current_stream().cuda_stream


def _opt(t, dtype, name, shape):
    """Data pointer of an optional tensor, checked; 0 where there is none."""
    if t is None:
        return 0
    _need(t, dtype, name, shape)
    _here(t, name)
    return t.data_ptr()


def _dtype(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DT:
        raise ValueError(f"{name} must be a bf16 or fp32 tensor")
    return _DT[t.dtype]


def _scratch(workspace, need, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _need(workspace, workspace.dtype, "workspace")
    _here(workspace, "workspace")
    return workspace


def _pools(k_pages, v_pages, table, lengths):
    """(dtype, n_seq, n_pages, page_size, max_pages, kv_heads, head_dim) of a cache."""
    dt = _dtype(k_pages, "k_pages")
    if k_pages.dim() != 4 or not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("k_pages must be [n_pages][page_size][kv_heads][head_dim] and table [n_seq][max_pages]")
    _need(k_pages, k_pages.dtype, "k_pages")
    _need(v_pages, k_pages.dtype, "v_pages", k_pages.shape)
    _need(table, torch.int32, "table")
    _need(lengths, torch.int32, "lengths", (table.shape[0],))
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages"), (table, "table"), (lengths, "lengths")):
        _here(t, name)
    return (dt, table.shape[0], k_pages.shape[0], k_pages.shape[1], table.shape[1], k_pages.shape[2],
            k_pages.shape[3])


def _capacity(positions, weights, n_seq, kv_heads):
    """Slots that the state arrays hold (their last dimension), 0 without any."""
    cap = 0
    for t, name in ((positions, "positions"), (weights, "weights")):
        if t is not None:
            if t.dim() != 3 or (cap and t.shape[2] != cap):
                raise ValueError(f"{name} must be [n_seq][kv_heads][cap], cap the same for both state arrays")
            cap = t.shape[2]
            if tuple(t.shape) != (n_seq, kv_heads, cap):
                raise ValueError(f"{name} must have shape {(n_seq, kv_heads, cap)}, got {tuple(t.shape)}")
    return cap


def paged_append(k, v, k_pages, v_pages, table, lengths, *, row_starts=None, positions=None,
                 weights=None, pos0=None):
    """Writes new K/V rows ([n_rows][kv_heads][head_dim]) behind each sequence's `lengths` slots.

    Sequence s owns rows [row_starts[s], row_starts[s + 1]) (None: row s); their positions
    become pos0[s] + i (None: lengths[s] + i) and their weights 0 where those arrays are
    given.  `lengths` is the count before the call and is not changed.
    """
    dt, n_seq, n_pages, page, width, hk, d = _pools(k_pages, v_pages, table, lengths)
    n_rows = k.shape[0]
    _need(k, k_pages.dtype, "k", (n_rows, hk, d))
    _need(v, k_pages.dtype, "v", k.shape)
    _here(k, "k")
    _here(v, "v")
    cap = _capacity(positions, weights, n_seq, hk)
    L.check(L.lib.sfm_paged_append(
        k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(),
        lengths.data_ptr(), _opt(row_starts, torch.int32, "row_starts", (n_seq + 1,)), n_rows, n_seq,
        n_pages, page, width, hk, d, dt, _opt(positions, torch.int32, "positions", None),
        _opt(pos0, torch.int32, "pos0", (n_seq,)), _opt(weights, torch.float32, "weights", None), cap,
        _raw_stream()), "sfm_paged_append")


def paged_attention(q, k_pages, v_pages, table, lengths, *, softcap=0.0, slopes=None, positions=None,
                    q_positions=None, weights=None, out=None, workspace=None):
    """Attention of one token per sequence (q [n_seq][heads][head_dim]) over its cached slots.

    softcap > 0 caps the scores (c tanh(s / c)); slopes ([heads] fp32) subtract
    slope |q_position - position| (positions default to the slots, q_positions to
    lengths - 1); weights, if given, gain each slot's softmax weight, summed over the query
    heads of its key head.
    """
    dt, n_seq, n_pages, page, width, hk, d = _pools(k_pages, v_pages, table, lengths)
    if q.dim() != 3:
        raise ValueError("q must be [n_seq][heads][head_dim]")
    h = q.shape[1]
    _need(q, k_pages.dtype, "q", (n_seq, h, d))
    _here(q, "q")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, q.dtype, "out", q.shape)
        _here(out, "out")
    cap = _capacity(positions, weights, n_seq, hk)
    tokens = min(width * page, cap) if cap else width * page
    need = L.lib.sfm_paged_attention_workspace_bytes(n_seq, tokens, h, hk, d, dt, weights is not None)
    ws = _scratch(workspace, need, q.device)
    L.check(L.lib.sfm_paged_attention(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lengths.data_ptr(),
        out.data_ptr(), n_seq, n_pages, page, width, h, hk, d, dt, softcap or 0.0,
        _opt(slopes, torch.float32, "slopes", (h,)), _opt(positions, torch.int32, "positions", None),
        _opt(q_positions, torch.int32, "q_positions", (n_seq,)),
        _opt(weights, torch.float32, "weights", None), cap, ws.data_ptr() if ws is not None else 0,
        ws.numel() * ws.element_size() if ws is not None else 0, _raw_stream()), "sfm_paged_attention")
    return out


def paged_evict(k_pages, v_pages, table, lengths, weights, positions, keep, *, n_first=0, n_recent=0,
                workspace=None):
    """Cuts every sequence longer than `keep` back to `keep` slots, key head by key head, in place.

    Kept: positions below n_first, the last n_recent positions, then the largest accumulated
    weights (ties: the lower slot).  Kept rows behind slot `keep` move into the evicted slots
    before it.  `lengths` is not changed; the new ones are lengths.clamp(max=keep).
    """
    dt, n_seq, n_pages, page, width, hk, d = _pools(k_pages, v_pages, table, lengths)
    if weights is None or positions is None:
        raise ValueError("paged_evict needs weights and positions")
    cap = _capacity(positions, weights, n_seq, hk)
    need = L.lib.sfm_paged_evict_workspace_bytes(n_seq, min(width * page, cap), hk, keep)
    ws = _scratch(workspace, need, k_pages.device)
    L.check(L.lib.sfm_paged_evict(
        k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lengths.data_ptr(),
        _opt(weights, torch.float32, "weights", None), _opt(positions, torch.int32, "positions", None), cap,
        n_seq, n_pages, page, width, hk, d, dt, keep, n_first, n_recent,
        ws.data_ptr() if ws is not None else 0, ws.numel() * ws.element_size() if ws is not None else 0,
        _raw_stream()), "sfm_paged_evict")


def attention_bounds(n_q, n_kv, *, doc_starts=None, prefixes=None, causal=False, out=None):
    """Key ranges (lo, hi), int32 [n_q] each, of n_q queries at the last n_q of n_kv keys.

    doc_starts (int32 [n_docs + 1]) are the documents' boundaries over the keys (None: one
    document of all); a query sees its own document, or (causal) its keys up to the query's own
    and its first prefixes[d].  Queries in no document get an empty range.
    """
    dev = torch.device("cuda", torch.cuda.current_device())
    n_docs = doc_starts.numel() - 1 if doc_starts is not None else (1 if prefixes is not None else 0)
    lo, hi = out if out is not None else torch.empty((2, n_q), dtype=torch.int32, device=dev)
    L.check(L.lib.sfm_attention_bounds(
        n_q, n_kv, _opt(doc_starts, torch.int32, "doc_starts", (n_docs + 1,)),
        _opt(prefixes, torch.int32, "prefixes", (n_docs,)), n_docs, 1 if causal else 0,
        _opt(lo, torch.int32, "lo", (n_q,)), _opt(hi, torch.int32, "hi", (n_q,)), _raw_stream()),
        "sfm_attention_bounds")
    return lo, hi


def attention_masked(q, k, v, key_lo=None, key_hi=None, *, softcap=0.0, slopes=None, out=None,
                     workspace=None):
    """Attention of q [n_q][heads][D] over k, v [n_kv][kv_heads][D], query i over keys
    [key_lo[i], key_hi[i]) (None: all); an empty range gives zeros.

    softcap > 0 caps the scores; slopes ([heads] fp32) subtract slope |n_kv - n_q + i - j|.
    """
    dt = _dtype(q, "q")
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q must be [n_q][heads][D] and k [n_kv][kv_heads][D]")
    n_q, h, d = q.shape
    n_kv, hk = k.shape[0], k.shape[1]
    _need(q, q.dtype, "q")
    _need(k, q.dtype, "k", (n_kv, hk, d))
    _need(v, q.dtype, "v", k.shape)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _here(t, name)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, q.dtype, "out", q.shape)
        _here(out, "out")
    need = L.lib.sfm_attention_masked_workspace_bytes(n_q, n_kv, h, hk, d, dt)
    ws = _scratch(workspace, need, q.device)
    L.check(L.lib.sfm_attention_masked(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), n_q, n_kv, h, hk, d, dt,
        _opt(key_lo, torch.int32, "key_lo", (n_q,)), _opt(key_hi, torch.int32, "key_hi", (n_q,)),
        softcap or 0.0, _opt(slopes, torch.float32, "slopes", (h,)),
        ws.data_ptr() if ws is not None else 0, ws.numel() * ws.element_size() if ws is not None else 0,
        _raw_stream()), "sfm_attention_masked")
    return out
