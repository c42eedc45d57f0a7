"""Paged K/V cache and attention under per-query key ranges: thin binding over libsfm.

As in ``performer``: argument checks and marshalling only.  Tensors are contiguous
CUDA tensors of the current device; calls run on its current stream.  What only the
device knows (page tables, lengths) is checked there: ``_lib.check_call_error``
returns 0x301 / 0x302 after a bad page / a length that the cache does not hold.
"""
from __future__ import annotations

from functools import lru_cache

import torch

from . import _lib as L
from .performer import _DT, _need

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
# pure functions of the shape, asked for by every call
_attention_bytes = lru_cache(4096)(L.lib.sfm_paged_attention_workspace_bytes)
_evict_bytes = lru_cache(4096)(L.lib.sfm_paged_evict_workspace_bytes)
_masked_bytes = lru_cache(4096)(L.lib.sfm_attention_masked_workspace_bytes)


# the entry points and the current stream's handle (without a Stream object around it): a call
# of a few rows takes less time on the GPU than in here, so lookups are made once
_append, _attention, _evict = L.lib.sfm_paged_append, L.lib.sfm_paged_attention, L.lib.sfm_paged_evict
_bounds, _masked = L.lib.sfm_attention_bounds, L.lib.sfm_attention_masked
_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
           or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
_device = torch.cuda.current_device
_Tensor, _empty, _U8 = torch.Tensor, torch.empty, torch.uint8


def _ptr(t, dtype, name, shape, dev):
    """Data pointer of a contiguous tensor of this type and shape on device `dev`."""
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev):
        return t.data_ptr()
    _need(t, dtype, name, shape)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _dims(t, n, name, what):
    if not isinstance(t, _Tensor) or t.dtype not in _DT:
        raise ValueError(f"{name} must be a bf16 or fp32 tensor")
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must be {what}")
    return shape


def _i32(x, name):
    """x, refused if a C int would take it for another number."""
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{name} must be a 32-bit number, got {x}")
    return x


def _scratch(workspace, need, dev):
    """(tensor to keep until the launch, pointer, bytes) of the caller's workspace or a new one."""
    if workspace is None:
        if not need:
            return None, 0, 0
        workspace = _empty(need, dtype=_U8, device=dev)
        return workspace, workspace.data_ptr(), need
    if not isinstance(workspace, _Tensor):
        raise ValueError("workspace must be a CUDA tensor")
    at = _ptr(workspace, workspace.dtype, "workspace", workspace.shape, dev)
    return workspace, at, workspace.numel() * workspace.element_size()


def _result(out, like, dev):
    """(output tensor, its pointer)"""
    if out is None:
        out = torch.empty_like(like)
        return out, out.data_ptr()
    return out, _ptr(out, like.dtype, "out", like.shape, dev)


def _width(table):
    if not isinstance(table, _Tensor) or table.dim() != 2:
        raise ValueError("table must be an int32 tensor [n_seq][max_pages]")
    return table.shape


def _capacity(positions, weights, n_seq, kv_heads, dev):
    """(slots that the state arrays hold, or 0 without any; positions' pointer; weights')."""
    if positions is None and weights is None:
        return 0, 0, 0
    cap = 0
    for t, name in ((positions, "positions"), (weights, "weights")):
        if t is not None:
            if not isinstance(t, _Tensor) or t.dim() != 3 or (cap and t.shape[2] != cap):
                raise ValueError(f"{name} must be [n_seq][kv_heads][cap], cap the same for both state arrays")
            cap = t.shape[2]
    shape = (n_seq, kv_heads, cap)
    return (cap, 0 if positions is None else _ptr(positions, _I32, "positions", shape, dev),
            0 if weights is None else _ptr(weights, _F32, "weights", shape, dev))


_POOL = "[n_pages][page_size][kv_heads][head_dim]"


def paged_append(k, v, k_pages, v_pages, table, lengths, *, row_starts=None, positions=None,
                 weights=None, pos0=None):
    """Writes new K/V rows ([n_rows][kv_heads][head_dim]) behind each sequence's `lengths` slots.

    Sequence s owns rows [row_starts[s], row_starts[s + 1]) (None: row s); their positions
    become pos0[s] + i (None: lengths[s] + i) and their weights 0 where those arrays are
    given.  `lengths` is the count before the call and is not changed.
    """
    dev = _device()
    n_pages, page, hk, d = pool = _dims(k_pages, 4, "k_pages", _POOL)
    dt = k_pages.dtype
    n_seq, width = _width(table)
    n_rows = _dims(k, 3, "k", "[n_rows][kv_heads][head_dim]")[0]
    rows = (n_rows, hk, d)
    cap, pos, wts = _capacity(positions, weights, n_seq, hk, dev)
    L.check(_append(
        _ptr(k, dt, "k", rows, dev), _ptr(v, dt, "v", rows, dev), _ptr(k_pages, dt, "k_pages", pool, dev),
        _ptr(v_pages, dt, "v_pages", pool, dev), _ptr(table, _I32, "table", (n_seq, width), dev),
        _ptr(lengths, _I32, "lengths", (n_seq,), dev),
        0 if row_starts is None else _ptr(row_starts, _I32, "row_starts", (n_seq + 1,), dev), n_rows, n_seq,
        n_pages, page, width, hk, d, _DT[dt], pos,
        0 if pos0 is None else _ptr(pos0, _I32, "pos0", (n_seq,), dev), wts, cap, _stream(dev)), "sfm_paged_append")


def paged_attention(q, k_pages, v_pages, table, lengths, *, softcap=0.0, slopes=None, positions=None,
                    q_positions=None, weights=None, out=None, workspace=None):
    """Attention of one token per sequence (q [n_seq][heads][head_dim]) over its cached slots.

    softcap > 0 caps the scores (c tanh(s / c)); slopes ([heads] fp32) subtract
    slope |q_position - position| (positions default to the slots, q_positions to
    lengths - 1); weights, if given, gain each slot's softmax weight, summed over the query
    heads of its key head.
    """
    dev = _device()
    n_pages, page, hk, d = pool = _dims(k_pages, 4, "k_pages", _POOL)
    dt = k_pages.dtype
    n_seq, width = _width(table)
    h = _dims(q, 3, "q", "[n_seq][heads][head_dim]")[1]
    pq = _ptr(q, dt, "q", (n_seq, h, d), dev)
    cap, pos, wts = _capacity(positions, weights, n_seq, hk, dev)
    args = (pq, _ptr(k_pages, dt, "k_pages", pool, dev), _ptr(v_pages, dt, "v_pages", pool, dev),
            _ptr(table, _I32, "table", (n_seq, width), dev), _ptr(lengths, _I32, "lengths", (n_seq,), dev))
    slp = 0 if slopes is None else _ptr(slopes, _F32, "slopes", (h,), dev)
    qpos = 0 if q_positions is None else _ptr(q_positions, _I32, "q_positions", (n_seq,), dev)
    out, po = _result(out, q, dev)
    tokens = width * page
    if cap and cap < tokens:
        tokens = cap
    ws, wp, wb = _scratch(workspace, _attention_bytes(n_seq, tokens, h, hk, d, _DT[dt], int(weights is not None)),
                          dev)
    L.check(_attention(*args, po, n_seq, n_pages, page, width, h, hk, d, _DT[dt], softcap or 0.0, slp, pos, qpos,
                       wts, cap, wp, wb, _stream(dev)), "sfm_paged_attention")
    return out


def paged_evict(k_pages, v_pages, table, lengths, weights, positions, keep, *, n_first=0, n_recent=0,
                workspace=None):
    """Cuts every sequence longer than `keep` back to `keep` slots, key head by key head, in place.

    Kept: positions below n_first, the last n_recent positions, then the largest accumulated
    weights (ties: the lower slot).  Kept rows behind slot `keep` move into the evicted slots
    before it.  `lengths` is not changed; the new ones are lengths.clamp(max=keep).
    """
    dev = _device()
    n_pages, page, hk, d = pool = _dims(k_pages, 4, "k_pages", _POOL)
    dt = k_pages.dtype
    n_seq, width = _width(table)
    if weights is None or positions is None:
        raise ValueError("paged_evict needs weights and positions")
    keep, n_first, n_recent = _i32(keep, "keep"), _i32(n_first, "n_first"), _i32(n_recent, "n_recent")
    cap, pos, wts = _capacity(positions, weights, n_seq, hk, dev)
    args = (_ptr(k_pages, dt, "k_pages", pool, dev), _ptr(v_pages, dt, "v_pages", pool, dev),
            _ptr(table, _I32, "table", (n_seq, width), dev), _ptr(lengths, _I32, "lengths", (n_seq,), dev))
    ws, wp, wb = _scratch(workspace, _evict_bytes(n_seq, min(width * page, cap), hk, keep), dev)
    L.check(_evict(*args, wts, pos, cap, n_seq, n_pages, page, width, hk, d, _DT[dt], keep, n_first, n_recent,
                   wp, wb, _stream(dev)), "sfm_paged_evict")


def attention_bounds(n_q, n_kv, *, doc_starts=None, prefixes=None, causal=False, out=None):
    """Key ranges (lo, hi), int32 [n_q] each, of n_q queries at the last n_q of n_kv keys.

    doc_starts (int32 [n_docs + 1]) are the documents' boundaries over the keys (None: one
    document of all); a query sees its own document, or (causal) its keys up to the query's own
    and its first prefixes[d].  Queries in no document get an empty range.
    """
    dev = _device()
    n_q, n_kv = _i32(n_q, "n_q"), _i32(n_kv, "n_kv")
    n_docs = doc_starts.numel() - 1 if doc_starts is not None else (1 if prefixes is not None else 0)
    lo, hi = (_empty(n_q, dtype=_I32, device=dev), _empty(n_q, dtype=_I32, device=dev)) if out is None else out
    L.check(_bounds(
        n_q, n_kv, 0 if doc_starts is None else _ptr(doc_starts, _I32, "doc_starts", (n_docs + 1,), dev),
        0 if prefixes is None else _ptr(prefixes, _I32, "prefixes", (n_docs,), dev), n_docs, 1 if causal else 0,
        _ptr(lo, _I32, "lo", (n_q,), dev), _ptr(hi, _I32, "hi", (n_q,), dev), _stream(dev)),
        "sfm_attention_bounds")
    return lo, hi


def attention_masked(q, k, v, key_lo=None, key_hi=None, *, softcap=0.0, slopes=None, out=None,
                     workspace=None):
    """Attention of q [n_q][heads][D] over k, v [n_kv][kv_heads][D], query i over keys
    [key_lo[i], key_hi[i]) (None: all); an empty range gives zeros.

    softcap > 0 caps the scores; slopes ([heads] fp32) subtract slope |n_kv - n_q + i - j|.
    """
    dev = _device()
    n_q, h, d = shape = _dims(q, 3, "q", "[n_q][heads][D]")
    n_kv, hk, _ = _dims(k, 3, "k", "[n_kv][kv_heads][D]")
    dt = q.dtype
    args = (_ptr(q, dt, "q", shape, dev), _ptr(k, dt, "k", (n_kv, hk, d), dev), _ptr(v, dt, "v", (n_kv, hk, d), dev))
    lo = 0 if key_lo is None else _ptr(key_lo, _I32, "key_lo", (n_q,), dev)
    hi = 0 if key_hi is None else _ptr(key_hi, _I32, "key_hi", (n_q,), dev)
    slp = 0 if slopes is None else _ptr(slopes, _F32, "slopes", (h,), dev)
    out, po = _result(out, q, dev)
    ws, wp, wb = _scratch(workspace, _masked_bytes(n_q, n_kv, h, hk, d, _DT[dt]), dev)
    L.check(_masked(*args, po, n_q, n_kv, h, hk, d, _DT[dt], lo, hi, softcap or 0.0, slp, wp, wb, _stream(dev)),
            "sfm_attention_masked")
    return out
