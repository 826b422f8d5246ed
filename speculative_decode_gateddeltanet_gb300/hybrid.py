"""Python binding of the hybrid-step operators (the C ABI in ``include/gdnhybrid.h``).

The rest of a Qwen3.5-style hybrid's verify step beside its GatedDeltaNet
layers: the paged cache's page map, the append of new K and V rows, the full
attention over the pages, and the acceptance of drafts against sampled tokens.
Argument marshalling only, as in ``gdn``: a ``make_*_args`` struct is filled once
from tensors and passed to its call as often as those buffers are used; the
tensors must stay alive while calls run.
"""
from __future__ import annotations

import ctypes

import torch

from .gdn import BF16, F32, _check, _lib, _ptr, _stream

STATUS_NO_PAGES, STATUS_TABLE_FULL, STATUS_BAD_PAGE, STATUS_BAD_LENGTH, STATUS_ROWS_FULL = 32, 64, 128, 256, 512
SAMPLE_MAX_V = 393216

_I32, _I64, _F32, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class GdnPageMapArgs(ctypes.Structure):
    """Mirror of ``gdn_page_map_args``."""

    _fields_ = [(f, _I32) for f in ("B", "R", "page_size", "n_pages", "max_pages", "table_stride", "n_slot_rows", "reserved")] + \
               [(f, _P) for f in ("ctx_len", "n_rows", "held_in", "free_ring", "free_in", "block_table", "held_out", "free_out",
                                  "rows_out", "row_start", "slot_map", "positions", "status")]


class GdnKvAppendArgs(ctypes.Structure):
    """Mirror of ``gdn_kv_append_args``."""

    _fields_ = [(f, _I32) for f in ("rows", "H_kv", "d", "page_size", "n_pages", "in_dtype")] + \
               [("k", _P), ("v", _P)] + \
               [(f, _I64) for f in ("k_row_stride", "k_head_stride", "v_row_stride", "v_head_stride")] + \
               [(f, _P) for f in ("slot_map", "k_cache", "v_cache")] + \
               [(f, _I64) for f in ("k_page_stride", "k_cache_head_stride", "k_token_stride",
                                    "v_page_stride", "v_cache_head_stride", "v_token_stride")] + [("status", _P)]


class GdnPagedAttnArgs(ctypes.Structure):
    """Mirror of ``gdn_paged_attn_args``."""

    _fields_ = [(f, _I32) for f in ("B", "R", "H_q", "H_kv", "d", "page_size", "n_pages", "max_pages", "table_stride",
                                    "n_q_rows", "in_dtype")] + [("scale", _F32)] + \
               [("q", _P), ("q_row_stride", _I64), ("q_head_stride", _I64)] + \
               [("k_cache", _P), ("k_page_stride", _I64), ("k_head_stride", _I64), ("k_token_stride", _I64)] + \
               [("v_cache", _P), ("v_page_stride", _I64), ("v_head_stride", _I64), ("v_token_stride", _I64)] + \
               [(f, _P) for f in ("block_table", "ctx_len", "n_rows", "row_start")] + \
               [("o", _P), ("o_row_stride", _I64), ("o_head_stride", _I64), ("work", _P), ("status", _P)]


class GdnSampleArgs(ctypes.Structure):
    """Mirror of ``gdn_sample_args``."""

    _fields_ = [(f, _I32) for f in ("B", "R", "V", "in_dtype")] + [("row_stride", _I64)] + \
               [(f, _P) for f in ("logits", "u", "temperature", "top_k", "top_p", "min_p", "drafts", "n_rows", "target",
                                  "prob", "accept_len", "status")]


for _name, _args in (("gdn_page_map", GdnPageMapArgs), ("gdn_kv_append", GdnKvAppendArgs),
                     ("gdn_paged_attention", GdnPagedAttnArgs), ("gdn_sample_accept", GdnSampleArgs)):
    getattr(_lib, _name).argtypes = [ctypes.POINTER(_args), _P]
    getattr(_lib, _name).restype = ctypes.c_int
_lib.gdn_paged_attention_work_bytes.argtypes = [ctypes.POINTER(GdnPagedAttnArgs)]
_lib.gdn_paged_attention_work_bytes.restype = ctypes.c_size_t


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported input dtype {t.dtype}")


def _same(dtype: torch.dtype, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.dtype != dtype:
            raise TypeError(f"{name}: {t.dtype} where {dtype} is needed")


def _shape(name: str, t, want: tuple) -> None:
    if t is not None and tuple(t.shape) != tuple(want):
        raise ValueError(f"{name}: shape {tuple(t.shape)} where {tuple(want)} is needed")


def _dense(**tensors) -> None:
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _rows(name: str, t) -> None:
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


def make_page_map_args(*, ctx_len, n_rows, held, free_ring, free_state, block_table, held_out, free_state_out, rows_out,
                       page_size: int, R: int, row_start=None, slot_map=None, positions=None, status=None) -> GdnPageMapArgs:
    """Fill a GdnPageMapArgs from int32 tensors: ctx_len, n_rows, held,
    held_out, rows_out [B], free_ring [n_pages], free_state and
    free_state_out [2], block_table [B][max_pages] (any row stride),
    row_start [B+1], slot_map and positions [rows].  R > 0: rows padded to R
    a request; R = 0: packed rows."""
    B, width = block_table.shape
    every = dict(ctx_len=ctx_len, n_rows=n_rows, held=held, free_ring=free_ring, free_state=free_state, held_out=held_out,
                 free_state_out=free_state_out, rows_out=rows_out, row_start=row_start, slot_map=slot_map,
                 positions=positions, status=status)
    _same(torch.int32, block_table=block_table, **every)
    _dense(**every)
    _rows("block_table", block_table)
    for name in ("ctx_len", "n_rows", "held", "held_out", "rows_out"):
        _shape(name, every[name], (B,))
    for name in ("free_state", "free_state_out"):
        _shape(name, every[name], (2,))
    _shape("row_start", row_start, (B + 1,))
    rows = slot_map if slot_map is not None else positions
    _shape("positions", positions, () if rows is None else rows.shape)
    return GdnPageMapArgs(
        B=B, R=R, page_size=page_size, n_pages=free_ring.numel(), max_pages=width,
        table_stride=block_table.stride(0) if B > 1 else width, n_slot_rows=B * R if rows is None else rows.numel(),
        ctx_len=_ptr(ctx_len), n_rows=_ptr(n_rows), held_in=_ptr(held), free_ring=_ptr(free_ring), free_in=_ptr(free_state),
        block_table=_ptr(block_table), held_out=_ptr(held_out), free_out=_ptr(free_state_out), rows_out=_ptr(rows_out),
        row_start=_ptr(row_start), slot_map=_ptr(slot_map), positions=_ptr(positions), status=_ptr(status))


def make_kv_append_args(*, k, v, slot_map, k_cache, v_cache, status=None) -> GdnKvAppendArgs:
    """Fill a GdnKvAppendArgs: k and v [rows][H_kv][d], pools seen as
    [pages][H_kv][page_size][d] (views with any strides, d contiguous),
    slot_map [rows] int32."""
    n_pages, H_kv, P, d = k_cache.shape
    rows = k.shape[0]
    _same(k.dtype, v=v, k_cache=k_cache, v_cache=v_cache)
    _same(torch.int32, slot_map=slot_map, status=status)
    _shape("v_cache", v_cache, k_cache.shape)
    _shape("k", k, (rows, H_kv, d))
    _shape("v", v, (rows, H_kv, d))
    _shape("slot_map", slot_map, (rows,))
    _dense(slot_map=slot_map)
    for name, t in (("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache)):
        _rows(name, t)
    return GdnKvAppendArgs(
        rows=rows, H_kv=H_kv, d=d, page_size=P, n_pages=n_pages, in_dtype=_dtype(k), k=_ptr(k), v=_ptr(v),
        k_row_stride=k.stride(0), k_head_stride=k.stride(1), v_row_stride=v.stride(0), v_head_stride=v.stride(1),
        slot_map=_ptr(slot_map), k_cache=_ptr(k_cache), v_cache=_ptr(v_cache),
        k_page_stride=k_cache.stride(0), k_cache_head_stride=k_cache.stride(1), k_token_stride=k_cache.stride(2),
        v_page_stride=v_cache.stride(0), v_cache_head_stride=v_cache.stride(1), v_token_stride=v_cache.stride(2),
        status=_ptr(status))


def make_paged_attention_args(*, q, k_cache, v_cache, block_table, ctx_len, n_rows, o, row_start=None, R: int = 0,
                              scale: float | None = None, work=None, status=None) -> GdnPagedAttnArgs:
    """Fill a GdnPagedAttnArgs: q and o [rows][H_q][d], pools seen as
    [pages][H_kv][page_size][d] (any strides, d contiguous), block_table
    [B][max_pages], ctx_len and n_rows [B].  row_start [B] (or [B+1]) names
    each request's first row; without it rows are padded, R to a request."""
    rows, H_q, d = q.shape
    n_pages, H_kv, P, _ = k_cache.shape
    B, width = block_table.shape
    _same(q.dtype, k_cache=k_cache, v_cache=v_cache, o=o)
    _same(torch.int32, block_table=block_table, ctx_len=ctx_len, n_rows=n_rows, row_start=row_start, status=status)
    _shape("k_cache", k_cache, (n_pages, H_kv, P, d))
    _shape("v_cache", v_cache, k_cache.shape)
    _shape("o", o, q.shape)
    _shape("ctx_len", ctx_len, (B,))
    _shape("n_rows", n_rows, (B,))
    if row_start is not None and tuple(row_start.shape) not in ((B,), (B + 1,)):
        raise ValueError(f"row_start: shape {tuple(row_start.shape)} where {(B,)} is needed")
    _dense(ctx_len=ctx_len, n_rows=n_rows, row_start=row_start)
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("o", o), ("block_table", block_table)):
        _rows(name, t)
    return GdnPagedAttnArgs(
        B=B, R=R, H_q=H_q, H_kv=H_kv, d=d, page_size=P, n_pages=n_pages, max_pages=width,
        table_stride=block_table.stride(0) if B > 1 else width, n_q_rows=rows, in_dtype=_dtype(q),
        scale=d ** -0.5 if scale is None else scale, q=_ptr(q), q_row_stride=q.stride(0), q_head_stride=q.stride(1),
        k_cache=_ptr(k_cache), k_page_stride=k_cache.stride(0), k_head_stride=k_cache.stride(1), k_token_stride=k_cache.stride(2),
        v_cache=_ptr(v_cache), v_page_stride=v_cache.stride(0), v_head_stride=v_cache.stride(1), v_token_stride=v_cache.stride(2),
        block_table=_ptr(block_table), ctx_len=_ptr(ctx_len), n_rows=_ptr(n_rows), row_start=_ptr(row_start),
        o=_ptr(o), o_row_stride=o.stride(0), o_head_stride=o.stride(1), work=_ptr(work), status=_ptr(status))


def paged_attention_work_bytes(args: GdnPagedAttnArgs) -> int:
    """Bytes of work an attention call of these sizes needs (0 if they are unsupported)."""
    return int(_lib.gdn_paged_attention_work_bytes(ctypes.byref(args)))


def make_sample_accept_args(*, logits, u, n_rows, target, drafts=None, accept_len=None, temperature=None, top_k=None,
                            top_p=None, min_p=None, prob=None, status=None) -> GdnSampleArgs:
    """Fill a GdnSampleArgs: logits [B][R][V] (rows a fixed stride apart), u
    and prob [B][R] fp32, temperature, top_p, min_p [B] fp32, top_k [B] int32,
    drafts [B][R-1], n_rows, accept_len [B], target [B][R] int32."""
    B, R, V = logits.shape
    row = logits.stride(1) if R > 1 else logits.stride(0) if B > 1 else V
    if V > 1 and logits.stride(2) != 1 or R > 1 and B > 1 and logits.stride(0) != R * row:
        raise ValueError("logits: rows must be contiguous and a fixed stride apart")
    _same(torch.float32, u=u, temperature=temperature, top_p=top_p, min_p=min_p, prob=prob)
    _same(torch.int32, top_k=top_k, drafts=drafts, n_rows=n_rows, target=target, accept_len=accept_len, status=status)
    for name, t in (("u", u), ("target", target), ("prob", prob)):
        _shape(name, t, (B, R))
    for name, t in (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p), ("n_rows", n_rows),
                    ("accept_len", accept_len)):
        _shape(name, t, (B,))
    if drafts is not None and R > 1:
        _shape("drafts", drafts, (B, R - 1))
    _dense(u=u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, drafts=drafts, n_rows=n_rows, target=target,
           prob=prob, accept_len=accept_len)
    return GdnSampleArgs(
        B=B, R=R, V=V, in_dtype=_dtype(logits), row_stride=row, logits=_ptr(logits), u=_ptr(u), temperature=_ptr(temperature),
        top_k=_ptr(top_k), top_p=_ptr(top_p), min_p=_ptr(min_p), drafts=_ptr(drafts), n_rows=_ptr(n_rows), target=_ptr(target),
        prob=_ptr(prob), accept_len=_ptr(accept_len), status=_ptr(status))


def gdn_page_map(args: GdnPageMapArgs, stream=None) -> None:
    """Tables, slots and positions of a step from its request lengths (``gdn_page_map``)."""
    _check(_lib.gdn_page_map(ctypes.byref(args), _stream(stream)), "gdn_page_map")


def gdn_kv_append(args: GdnKvAppendArgs, stream=None) -> None:
    """K and V rows of the new tokens to their slots (``gdn_kv_append``)."""
    _check(_lib.gdn_kv_append(ctypes.byref(args), _stream(stream)), "gdn_kv_append")


def gdn_paged_attention(args: GdnPagedAttnArgs, stream=None) -> None:
    """Attention of the new tokens over their requests' pages (``gdn_paged_attention``)."""
    _check(_lib.gdn_paged_attention(ctypes.byref(args), _stream(stream)), "gdn_paged_attention")


def gdn_sample_accept(args: GdnSampleArgs, stream=None) -> None:
    """Sampled target tokens and accept lengths (``gdn_sample_accept``)."""
    _check(_lib.gdn_sample_accept(ctypes.byref(args), _stream(stream)), "gdn_sample_accept")
