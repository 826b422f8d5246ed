"""Plain 64-bit forms of the long-context operators, one request at a time, and the
inputs their tests share."""
from __future__ import annotations

import numpy as np
import torch

import hybrid_ref

U = 2.0 ** -24  # half a step of 32 bits, relative


def log_sums(q, k_cache, table, ctx, n, start, scale):
    """ln sum exp of every row and head in float64 (NaN where no row is), and the largest scale * sum |q||k| of a row."""
    q, k_cache = q.double().cpu().numpy(), k_cache.double().cpu().numpy()
    H_kv, P, d = k_cache.shape[1:]
    G = q.shape[1] // H_kv
    lse, size = np.full(q.shape[:2], np.nan), np.zeros(q.shape[:2])
    for b in range(len(ctx)):
        if n[b] <= 0:
            continue
        L = int(ctx[b] + n[b])
        rows = slice(int(start[b]), int(start[b] + n[b]))
        seen = np.arange(L)[None] <= ctx[b] + np.arange(n[b])[:, None]
        for h in range(H_kv):
            K = k_cache[table[b, :-(-L // P)], h].reshape(-1, d)[:L]
            for i in range(h * G, (h + 1) * G):
                z = np.where(seen, q[rows, i] @ K.T * scale, -np.inf)
                top = z.max(1)
                lse[rows, i] = top + np.log(np.exp(z - top[:, None]).sum(1))
                size[rows, i] = np.where(seen, np.abs(q[rows, i]) @ np.abs(K).T * abs(scale), 0).max(1)
    return lse, size


def weights(q, k_cache, lse, table, ctx, n, start, scale, keep, fresh, first, position, weight, born):
    """weight and born after a call, in float64 and int64, and how far 32 bits may be off in each weight."""
    q, k_cache, lse = q.double().cpu().numpy(), k_cache.double().cpu().numpy(), lse.double().cpu().numpy()
    H_kv, P, d = k_cache.shape[1:]
    H_q = q.shape[1]
    G = H_q // H_kv
    weight, born = weight.astype(np.float64), born.astype(np.int64)
    off = np.zeros_like(weight)
    for b in range(len(ctx)):
        if n[b] <= 0:
            continue
        L, lo = int(ctx[b] + n[b]), max(int(first[b]), 0)
        at = np.arange(L)
        slot = table[b, at // P].astype(np.int64) * P + at % P
        rows = slice(int(start[b]), int(start[b] + n[b]))
        seen = at[None] <= ctx[b] + np.arange(n[b])[:, None]
        got, slack = np.zeros(L), np.zeros(L)
        for h in range(H_kv):
            K = k_cache[table[b, :-(-L // P)], h].reshape(-1, d)[:L]
            for i in range(h * G, (h + 1) * G):
                x = q[rows, i] @ K.T * scale - lse[rows, i][:, None]
                p = np.where(seen, np.exp(x), 0)
                # a score's products and sums, its difference to lse, and the exponential: relative to p
                err = (2 * (d + 4) * (np.abs(q[rows, i]) @ np.abs(K).T) * abs(scale) + 4 * np.abs(x) + 4 * np.abs(lse[rows, i])[:, None] + 8) * U
                got += p.sum(0)
                slack += (p * err).sum(0)
        terms = int(n[b]) * H_q + 4
        old = np.where(at < ctx[b] if fresh else True, weight[slot] * keep, 0.0)
        new = np.where(at < ctx[b] if fresh else True, old + got, got)
        weight[slot[lo:]] = new[lo:]
        off[slot[lo:]] = (slack + terms * U * got + 2 * U * (np.abs(old) + got))[lo:]
        if fresh:
            born[slot[ctx[b]:]] = position[b] + np.arange(n[b])
    return weight, born, off


def weight_order(x):
    return np.where(np.isnan(x), -np.inf, x)


def select(weight, born, table, ctx, budget, pinned, keep_from, P, max_moves, n_pages, lists):
    """The choice's definition.  lists: (move_from, move_to) before the call.  Returns a dict of arrays and the status bits."""
    weight, born, status = weight.copy(), None if born is None else born.copy(), 0
    move_from, move_to = (x.copy() for x in lists)
    out, moves = ctx.copy(), np.zeros(len(ctx), np.int64)
    for b in range(len(ctx)):
        L = int(ctx[b])
        if L < 0 or L > table.shape[1] * P:
            status |= 256
            continue
        pages = table[b, :-(-L // P)]
        if ((pages < 0) | (pages >= n_pages)).any():
            status |= 128
            continue
        at = np.arange(L)
        slot = table[b, at // P].astype(np.int64) * P + at % P
        may = at >= pinned[b]
        if born is not None and keep_from is not None:
            may &= born[slot] < keep_from[b]
        may = np.flatnonzero(may)
        go = min(max(L - max(int(budget[b]), 0), 0), len(may))
        stays = np.ones(L, bool)
        stays[may[np.lexsort((-may, weight_order(weight[slot[may]])))[:go]]] = False
        K = L - go
        gaps, movers = np.flatnonzero(~stays[:K]), K + np.flatnonzero(stays[K:])
        assert len(gaps) == len(movers)
        if len(gaps) > max_moves:
            status |= 1024
            continue
        out[b], moves[b] = K, len(gaps)
        move_from[b, :len(gaps)], move_to[b, :len(gaps)] = slot[movers], slot[gaps]
        weight[slot[gaps]] = weight[slot[movers]]
        if born is not None:
            born[slot[gaps]] = born[slot[movers]]
    return dict(weight=weight, born=born, ctx_out=out, n_moves=moves, move_from=move_from, move_to=move_to, status=status)


def make_shared(*, groups, alone=(), H_q, H_kv, d, P, dtype, layout="heads", seed=0, R=0, scale=None, spare=3):
    """Inputs of one shared call.  groups: (prefix, [(own cached tokens, rows), ...]) each, then requests in no group as
    (cached tokens, rows).  Requests of a group share the prefix's whole pages and have copies of the one it ends in.
    Every token slot that belongs to no request is NaN."""
    lens, lead, prefix = [], [], []
    for length, members in groups:
        first = len(lens)
        for own, n in members:
            lens.append((length + own, n))
            lead.append(first)
            prefix.append(length)
    for ctx, n in alone:
        lead.append(len(lens))
        lens.append((ctx, n))
        prefix.append(0)
    case = hybrid_ref.make_attention(lens=lens, H_q=H_q, H_kv=H_kv, d=d, P=P, dtype=dtype, layout=layout, seed=seed, R=R, scale=scale,
                                     spare=spare)
    table = case["table"]
    for b, (a, length) in enumerate(zip(lead, prefix)):
        # the first request of the group with rows has pages; the prefix is what they hold
        while lens[a][1] == 0 and a < b:
            a += 1
        if a == b or lens[b][1] == 0:
            continue
        table[b, :length // P] = table[a, :length // P]
        if length % P:
            for c in ("k_cache", "v_cache"):
                case[c][table[b, length // P], :, :length % P] = case[c][table[a, length // P], :, :length % P]
    starts = np.cumsum([0] + [len(members) for _, members in groups])
    return case | dict(group_start=starts, prefix_len=np.array([length for length, _ in groups], dtype=np.int64))
