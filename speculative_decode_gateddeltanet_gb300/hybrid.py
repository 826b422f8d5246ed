"""Python binding of the hybrid-step operators (the C ABI in ``include/gdnhybrid.h``) and of
those for long contexts (``include/gdnlong.h``).

The rest of a Qwen3.5-style hybrid's verify step beside its GatedDeltaNet
layers: the paged cache's page map, the append of new K and V rows, the full
attention over the pages, and the acceptance of drafts against sampled tokens.
For long contexts: attention that reads a shared prefix once, the attention
weight of cached tokens, the choice of those that leave, and their moves.
Argument marshalling only, as in ``gdn``: a ``make_*_args`` struct is filled once
from tensors and passed to its call as often as those buffers are used; the
tensors must stay alive while calls run.
"""
from __future__ import annotations

import ctypes

import torch

from .gdn import BF16, F32, _check, _lib, _ptr, _stream

STATUS_NO_PAGES, STATUS_TABLE_FULL, STATUS_BAD_PAGE, STATUS_BAD_LENGTH, STATUS_ROWS_FULL = 32, 64, 128, 256, 512
STATUS_MOVES_FULL, STATUS_BAD_GROUP = 1024, 2048
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


class GdnSharedAttnArgs(ctypes.Structure):
    """Mirror of ``gdn_shared_attn_args``."""

    _fields_ = [("attn", GdnPagedAttnArgs), ("n_groups", _I32), ("reserved", _I32), ("group_start", _P), ("prefix_len", _P),
                ("lse", _P), ("lse_row_stride", _I64)]


class GdnAttnWeightArgs(ctypes.Structure):
    """Mirror of ``gdn_attn_weight_args``."""

    _fields_ = [(f, _I32) for f in ("B", "R", "H_q", "H_kv", "d", "page_size", "n_pages", "max_pages", "table_stride",
                                    "n_q_rows", "in_dtype", "fresh")] + [("scale", _F32), ("keep", _F32)] + \
               [("q", _P), ("q_row_stride", _I64), ("q_head_stride", _I64)] + \
               [("k_cache", _P), ("k_page_stride", _I64), ("k_head_stride", _I64), ("k_token_stride", _I64)] + \
               [("lse", _P), ("lse_row_stride", _I64)] + \
               [(f, _P) for f in ("block_table", "ctx_len", "n_rows", "row_start", "first", "position", "weight", "born", "work",
                                  "status")]


class GdnEvictArgs(ctypes.Structure):
    """Mirror of ``gdn_evict_args``."""

    _fields_ = [(f, _I32) for f in ("B", "page_size", "n_pages", "max_pages", "table_stride", "max_moves")] + \
               [(f, _P) for f in ("block_table", "ctx_len", "budget", "pinned", "keep_from", "weight", "born", "ctx_out", "n_moves",
                                  "move_from", "move_to", "status")]


class GdnKvMoveArgs(ctypes.Structure):
    """Mirror of ``gdn_kv_move_args``."""

    _fields_ = [(f, _I32) for f in ("B", "max_moves", "H_kv", "d", "page_size", "n_pages", "in_dtype", "reserved")] + \
               [(f, _P) for f in ("move_from", "move_to", "n_moves", "k_cache", "v_cache")] + \
               [(f, _I64) for f in ("k_page_stride", "k_head_stride", "k_token_stride",
                                    "v_page_stride", "v_head_stride", "v_token_stride")] + [("status", _P)]


for _name, _args in (("gdn_page_map", GdnPageMapArgs), ("gdn_kv_append", GdnKvAppendArgs),
                     ("gdn_paged_attention", GdnPagedAttnArgs), ("gdn_sample_accept", GdnSampleArgs),
                     ("gdn_shared_attention", GdnSharedAttnArgs), ("gdn_attn_weight", GdnAttnWeightArgs),
                     ("gdn_evict_select", GdnEvictArgs), ("gdn_kv_move", GdnKvMoveArgs)):
    getattr(_lib, _name).argtypes = [ctypes.POINTER(_args), _P]
    getattr(_lib, _name).restype = ctypes.c_int
for _name, _args in (("gdn_paged_attention_work_bytes", GdnPagedAttnArgs), ("gdn_shared_attention_work_bytes", GdnSharedAttnArgs),
                     ("gdn_attn_weight_work_bytes", GdnAttnWeightArgs)):
    getattr(_lib, _name).argtypes = [ctypes.POINTER(_args)]
    getattr(_lib, _name).restype = ctypes.c_size_t


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


def _lse(lse, rows: int, H_q: int) -> int:
    """Checks a [rows][H_q] fp32 array of log sums; its row stride."""
    _same(torch.float32, lse=lse)
    _shape("lse", lse, (rows, H_q))
    if H_q > 1 and lse.stride(1) != 1:
        raise ValueError("lse: the last dimension must be contiguous")
    return lse.stride(0) if rows > 1 else H_q


def make_shared_attention_args(*, q, k_cache, v_cache, block_table, ctx_len, n_rows, o, group_start=None, prefix_len=None,
                               lse=None, row_start=None, R: int = 0, scale: float | None = None, work=None,
                               status=None) -> GdnSharedAttnArgs:
    """Fill a GdnSharedAttnArgs: make_paged_attention_args' tensors, group_start
    [groups+1] and prefix_len [groups] int32, lse [rows][H_q] fp32 (any row
    stride).  Its work buffer is ``args.attn.work``."""
    if (group_start is None) != (prefix_len is None):
        raise ValueError("group_start and prefix_len go together")
    groups = 0 if prefix_len is None else prefix_len.numel()
    _same(torch.int32, group_start=group_start, prefix_len=prefix_len)
    _shape("prefix_len", prefix_len, (groups,))
    _shape("group_start", group_start, (groups + 1,))
    _dense(group_start=group_start, prefix_len=prefix_len)
    attn = make_paged_attention_args(q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, ctx_len=ctx_len, n_rows=n_rows,
                                     o=o, row_start=row_start, R=R, scale=scale, work=work, status=status)
    return GdnSharedAttnArgs(attn=attn, n_groups=groups, group_start=_ptr(group_start), prefix_len=_ptr(prefix_len), lse=_ptr(lse),
                             lse_row_stride=0 if lse is None else _lse(lse, q.shape[0], q.shape[1]))


def shared_attention_work_bytes(args: GdnSharedAttnArgs) -> int:
    """Bytes of work a shared-prefix attention call of these sizes needs (0 if they are unsupported)."""
    return int(_lib.gdn_shared_attention_work_bytes(ctypes.byref(args)))


def make_attn_weight_args(*, q, k_cache, lse, block_table, ctx_len, n_rows, weight, row_start=None, R: int = 0,
                          scale: float | None = None, keep: float = 1.0, fresh: bool = False, first=None, position=None,
                          born=None, work=None, status=None) -> GdnAttnWeightArgs:
    """Fill a GdnAttnWeightArgs: q [rows][H_q][d], the K pool as
    make_paged_attention_args takes it, lse [rows][H_q] fp32, weight fp32 and
    born int32 [pages*page_size], first and position [B] int32."""
    rows, H_q, d = q.shape
    n_pages, H_kv, P, _ = k_cache.shape
    B, width = block_table.shape
    _same(q.dtype, k_cache=k_cache)
    _same(torch.float32, weight=weight)
    _same(torch.int32, block_table=block_table, ctx_len=ctx_len, n_rows=n_rows, row_start=row_start, first=first, position=position,
          born=born, status=status)
    _shape("k_cache", k_cache, (n_pages, H_kv, P, d))
    for name, t in (("ctx_len", ctx_len), ("n_rows", n_rows), ("first", first), ("position", position)):
        _shape(name, t, (B,))
    for name, t in (("weight", weight), ("born", born)):
        _shape(name, t, (n_pages * P,))
    if row_start is not None and tuple(row_start.shape) not in ((B,), (B + 1,)):
        raise ValueError(f"row_start: shape {tuple(row_start.shape)} where {(B,)} is needed")
    _dense(ctx_len=ctx_len, n_rows=n_rows, row_start=row_start, first=first, position=position, weight=weight, born=born)
    for name, t in (("q", q), ("k_cache", k_cache), ("block_table", block_table)):
        _rows(name, t)
    return GdnAttnWeightArgs(
        B=B, R=R, H_q=H_q, H_kv=H_kv, d=d, page_size=P, n_pages=n_pages, max_pages=width,
        table_stride=block_table.stride(0) if B > 1 else width, n_q_rows=rows, in_dtype=_dtype(q), fresh=int(fresh),
        scale=d ** -0.5 if scale is None else scale, keep=keep, q=_ptr(q), q_row_stride=q.stride(0), q_head_stride=q.stride(1),
        k_cache=_ptr(k_cache), k_page_stride=k_cache.stride(0), k_head_stride=k_cache.stride(1), k_token_stride=k_cache.stride(2),
        lse=_ptr(lse), lse_row_stride=_lse(lse, rows, H_q), block_table=_ptr(block_table), ctx_len=_ptr(ctx_len), n_rows=_ptr(n_rows),
        row_start=_ptr(row_start), first=_ptr(first), position=_ptr(position), weight=_ptr(weight), born=_ptr(born), work=_ptr(work),
        status=_ptr(status))


def attn_weight_work_bytes(args: GdnAttnWeightArgs) -> int:
    """Bytes of work an attention-weight call of these sizes needs (0 if they are unsupported)."""
    return int(_lib.gdn_attn_weight_work_bytes(ctypes.byref(args)))


def make_evict_select_args(*, weight, block_table, ctx_len, budget, ctx_out, n_moves, move_from, move_to, page_size: int,
                           pinned=None, born=None, keep_from=None, status=None) -> GdnEvictArgs:
    """Fill a GdnEvictArgs: weight fp32 and born int32 [pages*page_size],
    block_table [B][max_pages], move_from and move_to [B][max_moves] int32, the
    others [B] int32.  ctx_out may be ctx_len."""
    B, width = block_table.shape
    _same(torch.float32, weight=weight)
    _same(torch.int32, block_table=block_table, ctx_len=ctx_len, budget=budget, ctx_out=ctx_out, n_moves=n_moves, move_from=move_from,
          move_to=move_to, pinned=pinned, born=born, keep_from=keep_from, status=status)
    for name, t in (("ctx_len", ctx_len), ("budget", budget), ("ctx_out", ctx_out), ("n_moves", n_moves), ("pinned", pinned),
                    ("keep_from", keep_from)):
        _shape(name, t, (B,))
    if weight.dim() != 1 or weight.numel() % page_size:
        raise ValueError(f"weight: shape {tuple(weight.shape)} where one value for each slot of whole pages is needed")
    _shape("born", born, weight.shape)
    _shape("move_from", move_from, (B, move_to.shape[-1]))
    _shape("move_to", move_to, move_from.shape)
    _dense(weight=weight, born=born, ctx_len=ctx_len, budget=budget, ctx_out=ctx_out, n_moves=n_moves, move_from=move_from,
           move_to=move_to, pinned=pinned, keep_from=keep_from)
    _rows("block_table", block_table)
    return GdnEvictArgs(
        B=B, page_size=page_size, n_pages=weight.numel() // page_size, max_pages=width,
        table_stride=block_table.stride(0) if B > 1 else width, max_moves=move_to.shape[1], block_table=_ptr(block_table),
        ctx_len=_ptr(ctx_len), budget=_ptr(budget), pinned=_ptr(pinned), keep_from=_ptr(keep_from), weight=_ptr(weight), born=_ptr(born),
        ctx_out=_ptr(ctx_out), n_moves=_ptr(n_moves), move_from=_ptr(move_from), move_to=_ptr(move_to), status=_ptr(status))


def make_kv_move_args(*, k_cache, v_cache, move_from, move_to, n_moves, status=None) -> GdnKvMoveArgs:
    """Fill a GdnKvMoveArgs: pools seen as [pages][H_kv][page_size][d] (views
    with any strides, d contiguous), move_from and move_to [B][max_moves],
    n_moves [B] int32."""
    n_pages, H_kv, P, d = k_cache.shape
    B, most = move_to.shape
    _same(k_cache.dtype, v_cache=v_cache)
    _same(torch.int32, move_from=move_from, move_to=move_to, n_moves=n_moves, status=status)
    _shape("v_cache", v_cache, k_cache.shape)
    _shape("move_from", move_from, (B, most))
    _shape("n_moves", n_moves, (B,))
    _dense(move_from=move_from, move_to=move_to, n_moves=n_moves)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _rows(name, t)
    return GdnKvMoveArgs(
        B=B, max_moves=most, H_kv=H_kv, d=d, page_size=P, n_pages=n_pages, in_dtype=_dtype(k_cache), move_from=_ptr(move_from),
        move_to=_ptr(move_to), n_moves=_ptr(n_moves), k_cache=_ptr(k_cache), v_cache=_ptr(v_cache),
        k_page_stride=k_cache.stride(0), k_head_stride=k_cache.stride(1), k_token_stride=k_cache.stride(2),
        v_page_stride=v_cache.stride(0), v_head_stride=v_cache.stride(1), v_token_stride=v_cache.stride(2), status=_ptr(status))


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


def gdn_shared_attention(args: GdnSharedAttnArgs, stream=None) -> None:
    """Attention of the new tokens, shared prefixes read once (``gdn_shared_attention``)."""
    _check(_lib.gdn_shared_attention(ctypes.byref(args), _stream(stream)), "gdn_shared_attention")


def gdn_attn_weight(args: GdnAttnWeightArgs, stream=None) -> None:
    """The rows' attention, added to the weights of the tokens it went to (``gdn_attn_weight``)."""
    _check(_lib.gdn_attn_weight(ctypes.byref(args), _stream(stream)), "gdn_attn_weight")


def gdn_evict_select(args: GdnEvictArgs, stream=None) -> None:
    """The tokens that leave, and the moves that close their gaps (``gdn_evict_select``)."""
    _check(_lib.gdn_evict_select(ctypes.byref(args), _stream(stream)), "gdn_evict_select")


def gdn_kv_move(args: GdnKvMoveArgs, stream=None) -> None:
    """K and V of the moved tokens (``gdn_kv_move``)."""
    _check(_lib.gdn_kv_move(ctypes.byref(args), _stream(stream)), "gdn_kv_move")
