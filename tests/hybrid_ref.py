"""Plain 64-bit forms of the hybrid-step operators, one request and row at a
time, and the inputs their tests share."""
from __future__ import annotations

import numpy as np
import torch


def page_map(ctx, n, held, ring, free, table, P, R, n_slot_rows):
    """The page map's definition, in request order on the host.  Returns a dict of arrays and the status bits."""
    B, N = len(ctx), len(ring)
    table, ring0 = table.copy(), ring.copy()
    ring = ring.copy()
    head, n_free = int(free[0]) % N, int(free[1])
    taken = given = demand = status = 0
    held_out, rows_out = held.copy(), np.zeros(B, np.int64)
    for b in range(B):
        need = -(-(int(ctx[b]) + int(n[b])) // P)
        why = (256 if ctx[b] < 0 else 0) | (4096 if n[b] < 0 or (R and n[b] > R) else 0)
        if held[b] < 0 or held[b] > table.shape[1] or (not why and need > table.shape[1]):
            why |= 64
        if why:
            status |= 2 if why & 4096 else 0
            status |= why & 0xFFF
            continue
        want = max(need - int(held[b]), 0)
        demand += want
        if want and demand > n_free:
            status |= 32
            continue
        for i in range(want):
            table[b, held[b] + i] = ring0[(head + taken) % N]
            taken += 1
        for i in range(need, int(held[b])):
            ring[(head + n_free + given) % N] = table[b, i]
            given += 1
        held_out[b], rows_out[b] = need, n[b]
    start, r = np.zeros(B + 1, np.int64), 0
    for b in range(B):
        start[b] = b * R if R else r
        r += rows_out[b]
        if not R and rows_out[b] and r > n_slot_rows:
            status |= 512
            rows_out[b] = 0
    start[B] = B * R if R else r
    slots, pos = np.full(n_slot_rows, -1), np.full(n_slot_rows, -1)
    for b in range(B):
        for t in range(int(rows_out[b])):
            j = int(ctx[b]) + t
            pos[start[b] + t] = j
            slots[start[b] + t] = table[b, j // P] * P + j % P
    return dict(table=table, ring=ring, held_out=held_out, rows_out=rows_out, row_start=start, slot_map=slots, positions=pos,
                free_out=np.array([(head + taken) % N, n_free - taken + given]), status=status)


def attention(q, k_cache, v_cache, table, ctx, n, start, scale):
    """o [rows][H_q][d] in float64 (NaN where no row is), and per row and head the largest |v| a row sees."""
    q, k_cache, v_cache = (t.double().cpu().numpy() for t in (q, k_cache, v_cache))
    H_kv, P, d = k_cache.shape[1:]
    G = q.shape[1] // H_kv
    o = np.full(q.shape, np.nan)
    vmax = np.zeros(q.shape[:2])
    for b in range(len(ctx)):
        L = int(ctx[b] + n[b])
        if n[b] <= 0:
            continue
        pages = table[b, :-(-L // P)]
        for h in range(H_kv):
            K = k_cache[pages, h].reshape(-1, d)[:L]
            V = v_cache[pages, h].reshape(-1, d)[:L]
            rows = slice(int(start[b]), int(start[b] + n[b]))
            for i in range(h * G, (h + 1) * G):
                z = q[rows, i] @ K.T * scale
                z[np.arange(L)[None] > ctx[b] + np.arange(n[b])[:, None]] = -np.inf
                p = np.exp(z - z.max(1, keepdims=True))
                o[rows, i] = p @ V / p.sum(1, keepdims=True)
                vmax[rows, i] = np.abs(V).max()
    return o, vmax


def make_attention(*, lens, H_q, H_kv, d, P, dtype, layout="heads", seed=0, R=0, pad_rows=0, spare=3, scale=None):
    """Inputs of one attention call.  lens: (ctx, n) pairs.  Every token slot that belongs to no request is NaN."""
    g = torch.Generator().manual_seed(seed)
    ctx, n = np.array([c for c, _ in lens]), np.array([m for _, m in lens])
    B = len(lens)
    need = -(-(ctx + n) // P) * (n > 0)
    n_pages = int(need.sum()) + spare
    ids = np.random.default_rng(seed).permutation(n_pages)
    width = max(int(need.max()), 1) + 2
    table = np.full((B, width), 2**31 - 1)  # entries past a request's pages are never used
    table[np.arange(width) < need[:, None]] = ids[:need.sum()]
    pool = torch.full((n_pages, 2, H_kv, P, d), float("nan"))
    for b in range(B):
        for j in range(0, int(ctx[b] + n[b]) if n[b] else 0, P):
            m = min(P, int(ctx[b] + n[b]) - j)
            pool[table[b, j // P], :, :, :m] = torch.randn((2, H_kv, m, d), generator=g)
    pool = pool.to(dtype)
    if layout == "tokens":
        pool = pool.transpose(2, 3).contiguous().transpose(2, 3)
    start = np.arange(B) * R if R else np.concatenate([[0], np.cumsum(n)[:-1]])
    rows = B * R if R else int(n.sum())
    x = torch.randn((rows + pad_rows, H_q + 2 * H_kv, d), generator=g).to(dtype)
    return dict(q=x[:, :H_q], k_cache=pool[:, 0], v_cache=pool[:, 1], table=table, ctx=ctx, n=n, start=start,
                scale=d ** -0.5 if scale is None else scale)


def sample_row(z, T, k, p, m, u, slack=0.0):
    """Token and probability of one row from the definition in float64 (weights not rounded to whole numbers).
    slack moves the drawn share and the nucleus' edge by that much of the total: where the answer for -slack and
    +slack is the same, rounding of the weights cannot change it."""
    z = np.asarray(z, np.float64)
    V = len(z)
    key = np.where(np.isnan(z), -np.inf, z)
    if np.isnan(z).all():
        return 0, 1.0
    order = np.lexsort((np.arange(V), -key, np.isnan(z)))
    live = int((~np.isnan(z)).sum())
    if not T > 0:
        return int(order[0]), 1.0
    top = key[order[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(key[order] == top, 1.0, np.exp((key[order] - top) / T))
    w[live:] = 0.0
    c = live if k <= 0 or k >= V else min(k, live)
    if p < 1:
        cum = np.cumsum(w[:c])
        before = cum - w[:c]
        c = max(1, int((before < (max(p, 0.0) + slack) * cum[-1]).sum()))
    keep = order[:c][w[:c] >= (min(m, 1.0) if m > 0 else 0.0)]
    full = np.zeros(V)
    full[order] = w
    mask = np.zeros(V, bool)
    mask[keep] = True
    full[~mask] = 0
    cum = np.cumsum(full)
    u = min(max(0.0 if np.isnan(u) else u, 0.0), 1 - 2.0**-24)
    i = int((cum <= max(0.0, u + slack) * cum[-1]).sum())
    i = min(i, int(np.flatnonzero(full)[-1]))
    return i, full[i] / cum[-1]
