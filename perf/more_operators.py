"""Measured cases of the long-context operators: attention over shared prefixes, and
eviction from the paged cache by accumulated attention weight, each with its plain
form and its value in 64 bits.

A hybrid that serves long contexts keeps its attention layers' cache within bounds in
two ways: requests that begin alike read their common pages once, and tokens that few
rows attend to leave the cache.  One pass here is one call of one of four operators:

  shared   attention of a batch's new tokens whose requests share prefixes, with each
           row's log sum of exponentials
  weight   the attention that each cached token got from the step's rows, added to
           what it has
  select   which tokens leave: the lowest weights beyond a request's budget, and the
           moves that close their gaps
  move     K and V of the moved tokens
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

_BF16, _F32 = "bf16", "f32"


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == _BF16 else torch.float32


def _size(case):
    return 2 if case["dtype"] == _BF16 else 4


# ---- cases ------------------------------------------------------------------


def listed():
    return [
        # the smallest shared call: three short requests behind one short prefix, 32 bits
        {"name": "shared-small-f32", "op": "shared", "B": 3, "R": 5, "H_q": 6, "H_kv": 2, "d": 64, "P": 16, "groups": 1,
         "pre_lo": 300, "pre_hi": 300, "own_lo": 0, "own_hi": 200, "n_lo": 1, "n_hi": 5, "idle": 0, "layout": "tokens",
         "dtype": _F32, "lens": 1},
        # the verify step of 16 requests with three drafts behind one long instruction, the hybrid's own head shapes
        {"name": "shared-verify-B16", "op": "shared", "B": 16, "R": 4, "H_q": 16, "H_kv": 2, "d": 256, "P": 16, "groups": 1,
         "pre_lo": 8011, "pre_hi": 8011, "own_lo": 20, "own_hi": 1000, "n_lo": 4, "n_hi": 4, "idle": 0, "layout": "heads",
         "dtype": _BF16, "lens": 2},
        # single tokens of 64 samples drawn from one long document
        {"name": "shared-token-B64", "op": "shared", "B": 64, "R": 1, "H_q": 32, "H_kv": 8, "d": 128, "P": 64, "groups": 1,
         "pre_lo": 32768, "pre_hi": 32768, "own_lo": 0, "own_hi": 1000, "n_lo": 1, "n_hi": 1, "idle": 0, "layout": "heads",
         "dtype": _BF16, "lens": 3},
        # a wide ragged verify batch in five groups of unlike size and prefix, a tenth of the requests idle
        {"name": "shared-groups-B128", "op": "shared", "B": 128, "R": 9, "H_q": 32, "H_kv": 4, "d": 128, "P": 16, "groups": 5,
         "pre_lo": 400, "pre_hi": 6000, "own_lo": 1, "own_hi": 800, "n_lo": 2, "n_hi": 9, "idle": 10, "layout": "tokens",
         "dtype": _BF16, "lens": 4},
        # prompts of several hundred tokens behind a common instruction: bound by the products
        {"name": "shared-chunk", "op": "shared", "B": 4, "R": 0, "H_q": 32, "H_kv": 8, "d": 128, "P": 32, "groups": 1,
         "pre_lo": 8192, "pre_hi": 8192, "own_lo": 0, "own_hi": 300, "n_lo": 400, "n_hi": 1000, "idle": 0, "layout": "heads",
         "dtype": _BF16, "lens": 5},
        # the weights of a small step in 32 bits, behind pinned tokens
        {"name": "weight-small-f32", "op": "weight", "B": 3, "R": 5, "H_q": 6, "H_kv": 2, "d": 64, "P": 16, "first": 20,
         "ctx_lo": 30, "ctx_hi": 700, "n_lo": 1, "n_hi": 5, "idle": 0, "layout": "tokens", "dtype": _F32, "keep": 1.0, "lens": 6},
        # the weights of a verify step of 16 requests with three drafts, forgotten slowly
        {"name": "weight-verify-B16", "op": "weight", "B": 16, "R": 4, "H_q": 16, "H_kv": 2, "d": 256, "P": 16, "first": 0,
         "ctx_lo": 1000, "ctx_hi": 8000, "n_lo": 4, "n_hi": 4, "idle": 0, "layout": "heads", "dtype": _BF16, "keep": 0.99, "lens": 7},
        # the weights that whole prompts leave behind: bound by the products and exponentials
        {"name": "weight-prompt-4k", "op": "weight", "B": 2, "R": 0, "H_q": 32, "H_kv": 8, "d": 128, "P": 32, "first": 0,
         "ctx_lo": 0, "ctx_hi": 1000, "n_lo": 1500, "n_hi": 4096, "idle": 0, "layout": "heads", "dtype": _BF16, "keep": 1.0, "lens": 8},
        # 16 requests a little over their budgets: latency only
        {"name": "select-B16", "op": "select", "B": 16, "P": 16, "len_lo": 1000, "len_hi": 8000, "drop_lo": 4, "drop_hi": 64,
         "pinned": 16, "recent": 128, "lens": 9},
        # long contexts cut to a half, some of them not over their budgets
        {"name": "select-long-B8", "op": "select", "B": 8, "P": 64, "len_lo": 60000, "len_hi": 130000, "drop_lo": 0, "drop_hi": 60000,
         "pinned": 100, "recent": 1000, "lens": 10},
        # K and V of 16 requests' moves after a small eviction, two wide heads
        {"name": "move-verify-bf16", "op": "move", "B": 16, "moves_lo": 1, "moves_hi": 64, "H_kv": 2, "d": 256, "P": 16,
         "layout": "heads", "dtype": _BF16, "n_pages": 4096, "lens": 11},
        # a large eviction's moves, 32 bits, token-major pages, odd counts
        {"name": "move-large-f32", "op": "move", "B": 15, "moves_lo": 500, "moves_hi": 1999, "H_kv": 8, "d": 128, "P": 64,
         "layout": "tokens", "dtype": _F32, "n_pages": 1024, "lens": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "weight", "weight", "select", "move"])
    if op == "select":
        hi = _log(rng, 20, 130000)
        c = {"op": op, "B": _log(rng, 1, max(1, min(256, 1000000 // hi))), "P": rng.choice([16, 32, 48, 64, 128]),
             "len_lo": rng.randint(0, hi), "len_hi": hi, "drop_lo": 0, "drop_hi": _log(rng, 1, hi), "pinned": _log(rng, 1, 200) - 1,
             "recent": _log(rng, 1, 2000) - 1, "lens": rng.randrange(1 << 30)}
        return c
    if op == "move":
        h = rng.choice([1, 2, 4, 8])
        c = {"op": op, "B": _log(rng, 1, 200), "H_kv": h, "d": rng.choice([64, 128, 256]), "P": rng.choice([16, 32, 48, 64, 128]),
             "layout": rng.choice(["heads", "tokens"]), "dtype": rng.choice([_BF16, _F32]), "lens": rng.randrange(1 << 30)}
        c["moves_hi"] = _log(rng, 1, min(4000, 16000000 // (c["B"] * h * c["d"])))
        c["moves_lo"] = rng.randint(0, c["moves_hi"])
        c["n_pages"] = -(-2 * c["B"] * c["moves_hi"] // c["P"]) + rng.randint(1, 64)
        return c
    most = work(next(c for c in listed() if c["name"] == ("shared-chunk" if op == "shared" else "weight-prompt-4k")))["flops"]
    while True:
        h = rng.choice([1, 2, 4, 8])
        c = {"op": op, "H_q": h * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), "H_kv": h, "d": rng.choice([64, 128, 256]),
             "P": rng.choice([16, 32, 48, 64, 128]), "layout": rng.choice(["heads", "tokens"]),
             "dtype": rng.choice([_BF16, _BF16, _BF16, _F32]), "lens": rng.randrange(1 << 30)}
        kind = rng.choice(["token", "verify", "chunk"])
        B = _log(rng, 1, 128) if kind != "chunk" else rng.randint(1, 6)
        ctx = _log(rng, 16, {"token": 32768, "verify": 16384, "chunk": 8192}[kind])
        if kind == "token":
            c.update(B=B, R=1, n_lo=1, n_hi=1, idle=rng.choice([0, 10]))
        elif kind == "verify":
            c.update(B=B, R=rng.randint(2, 16), idle=rng.choice([0, 10]))
            c.update(n_lo=rng.randint(1, c["R"]), n_hi=c["R"])
        else:
            c.update(B=B, R=0, n_hi=_log(rng, 17, 2000 if op == "shared" else 4096), idle=0)
            c["n_lo"] = max(1, c["n_hi"] // 2)
        if op == "shared":
            c.update(groups=min(B, _log(rng, 1, 8)), pre_lo=rng.randint(0, ctx), pre_hi=ctx, own_lo=0, own_hi=_log(rng, 1, 1000))
            pre, own_ctx, n, _ = _shared_lengths(c)
            lens = [a + b + m for a, b, m in zip(pre, own_ctx, n)]
        else:
            c.update(ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, first=rng.choice([0, 0, 1, 17, 100]), keep=rng.choice([1.0, 0.95]))
            cached, n = _lengths(c)
            lens = [a + m for a, m in zip(cached, n)]
        # what the plain form holds at once stays within what the listed cases need
        keys, scores = c["B"] * max(lens) * h * c["d"], c["B"] * max(n) * max(lens) * c["H_q"]
        if (work(c)["flops"] <= most / (16 if c["dtype"] == _F32 else 1) and keys <= 2_100_000_000 and scores <= 1_500_000_000):
            return c


# ---- inputs -----------------------------------------------------------------


def _lengths(case):
    """Cached tokens and new rows of each request: they go with the case, not the seed, so that its work does too."""
    rng = random.Random(case["lens"])
    ctx, n = [], []
    for _ in range(case["B"]):
        ctx.append(rng.randint(case["ctx_lo"], case["ctx_hi"]))
        n.append(rng.randint(case["n_lo"], case["n_hi"]))
        if rng.random() * 100 < case["idle"]:
            n[-1] = 0
    if not any(n):
        n[0] = max(1, case["n_lo"])
    return ctx, n


def _shared_lengths(case):
    """Per request its group's prefix, its own cached tokens and its new rows; and where each group starts."""
    rng = random.Random(case["lens"])
    B, G = case["B"], case["groups"]
    cuts = sorted(rng.sample(range(1, B), G - 1)) if G > 1 else []
    start = [0] + cuts + [B]
    pre, own_ctx, n = [], [], []
    for g in range(G):
        length = rng.randint(case["pre_lo"], case["pre_hi"])
        for _ in range(start[g], start[g + 1]):
            pre.append(length)
            own_ctx.append(rng.randint(case["own_lo"], case["own_hi"]))
            n.append(rng.randint(case["n_lo"], case["n_hi"]))
            if rng.random() * 100 < case["idle"]:
                n[-1] = 0
    if not any(n):
        n[0] = max(1, case["n_lo"])
    return pre, own_ctx, n, start


def _select_lengths(case):
    """Tokens of each request, and how many of them are over its budget."""
    rng = random.Random(case["lens"])
    length = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["B"])]
    return length, [min(n, rng.randint(case["drop_lo"], case["drop_hi"])) for n in length]


def _move_counts(case):
    rng = random.Random(case["lens"])
    return [rng.randint(case["moves_lo"], case["moves_hi"]) for _ in range(case["B"])]


def _starts(case, n):
    """First row of each request: padded to R rows a request, or packed."""
    return [b * case["R"] for b in range(case["B"])] if case["R"] else [0] + list(np.cumsum(n)[:-1])


def _ints(v, shape=None):
    t = torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")
    return t if shape is None else t.reshape(shape)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pools(case, n_pages, g):
    """K and V pools as one allocation, seen as [pages][H_kv][P][d]: head-major or token-major pages."""
    H, P, d = case["H_kv"], case["P"], case["d"]
    shape = (n_pages, 2, H, P, d) if case["layout"] == "heads" else (n_pages, 2, P, H, d)
    pool = torch.randn(shape, device="cuda", generator=g, dtype=_dtype(case))
    if case["layout"] == "tokens":
        pool = pool.transpose(2, 3)
    return pool[:, 0], pool[:, 1]


def _tables(need, seed, spare=5):
    """Page tables of requests that need so many pages each, in no order of the pool; and the pool's pages."""
    need = np.asarray(need)
    n_pages = int(need.sum()) + spare
    ids = np.random.default_rng(seed).permutation(n_pages)
    table = np.full((len(need), int(need.max()) + 1), -1)
    table[np.arange(table.shape[1]) < need[:, None]] = ids[:need.sum()]
    return table, n_pages


def prepare(case, seed):
    return {"shared": _prepare_shared, "weight": _prepare_weight, "select": _prepare_select, "move": _prepare_move}[case["op"]](case, seed)


def _prepare_shared(case, seed):
    g = _gen(seed)
    pre, own_ctx, n, start = (np.array(v) for v in _shared_lengths(case))
    B, P, Hq, H, d = case["B"], case["P"], case["H_q"], case["H_kv"], case["d"]
    ctx = pre + own_ctx
    lead = np.repeat(start[:-1], np.diff(start))  # the request whose pages the group shares
    whole = pre // P
    table, n_pages = _tables(-(-(ctx + n) // P), seed)
    common = np.arange(table.shape[1]) < whole[:, None]
    table = np.where(common, table[lead], table)
    k_cache, v_cache = _pools(case, n_pages, g)
    for length in np.unique(pre[pre % P > 0]):  # a prefix that ends inside a page: each request has its own copy of that page
        b = np.flatnonzero(pre == length)
        at, src = table[b, length // P], table[lead[b], length // P]
        for c in (k_cache, v_cache):
            c[at, :, :length % P] = c[src, :, :length % P]
    rows = B * case["R"] if case["R"] else int(n.sum())
    x = torch.randn((rows, (Hq + 2 * H) * d), device="cuda", generator=g, dtype=_dtype(case))
    return {"case": case, "q": x[:, :Hq * d].unflatten(1, (Hq, d)), "k_cache": k_cache, "v_cache": v_cache, "table": _ints(table),
            "ctx_len": _ints(ctx), "n_rows": _ints(n), "row_start": _ints(_starts(case, n)), "scale": d ** -0.5,
            "group_start": _ints(start), "prefix_len": _ints(pre[start[:-1]]), "n_max": int(n.max()), "len_max": int((ctx + n).max()),
            "o": torch.zeros((rows, Hq, d), device="cuda", dtype=_dtype(case)), "lse": torch.zeros((rows, Hq), device="cuda")}


def _prepare_weight(case, seed):
    g = _gen(seed)
    ctx, n = (np.array(v) for v in _lengths(case))
    B, P, Hq, H, d = case["B"], case["P"], case["H_q"], case["H_kv"], case["d"]
    table, n_pages = _tables(-(-(ctx + n) // P), seed)
    k_cache, _ = _pools(case, n_pages, g)
    rows = B * case["R"] if case["R"] else int(n.sum())
    x = torch.randn((rows, (Hq + 2 * H) * d), device="cuda", generator=g, dtype=_dtype(case))
    s = {"case": case, "q": x[:, :Hq * d].unflatten(1, (Hq, d)), "k_cache": k_cache, "table": _ints(table), "ctx_len": _ints(ctx),
         "n_rows": _ints(n), "row_start": _ints(_starts(case, n)), "scale": d ** -0.5, "n_max": int(n.max()),
         "len_max": int((ctx + n).max()), "first": _ints([case["first"]] * B), "position": _ints(ctx + 1000),
         "weight": torch.rand(n_pages * P, device="cuda", generator=g) * 4, "born": torch.full((n_pages * P,), -1, dtype=torch.int32, device="cuda")}
    # what the step's attention gives beside its output: each row's log sum of exponentials
    s["lse"] = torch.zeros((rows, Hq), device="cuda")
    pos = torch.arange(s["len_max"], device="cuda")
    for b in range(B):
        if n[b] == 0:
            continue
        at = pos[:ctx[b] + n[b]]
        k = k_cache[s["table"][b].long()[at // P], :, at % P].float()
        r = slice(int(s["row_start"][b]), int(s["row_start"][b]) + int(n[b]))
        q = s["q"][r].float().reshape(int(n[b]), H, Hq // H, d)
        z = torch.einsum("thgd,lhd->thgl", q, k) * s["scale"]
        seen = at[None, :] <= ctx[b] + torch.arange(int(n[b]), device="cuda")[:, None]
        s["lse"][r] = torch.logsumexp(z.masked_fill(~seen[:, None, None], -math.inf), -1).reshape(int(n[b]), Hq)
    return s


def _prepare_select(case, seed):
    g = _gen(seed)
    length, over = (np.array(v) for v in _select_lengths(case))
    B, P = case["B"], case["P"]
    table, n_pages = _tables(np.maximum(-(-length // P), 1), seed)
    N = n_pages * P
    # few tokens hold most of the attention; new ones hold none yet
    weight = torch.exp(2.0 * torch.randn(N, device="cuda", generator=g))
    weight = torch.where(torch.rand(N, device="cuda", generator=g) < 0.03, 0.0, weight)
    t = _ints(table)
    pos = torch.arange(int(length.max()) + 1, device="cuda")
    live = pos[None, :] < _ints(length)[:, None]
    slot = t.long()[:, pos // P] * P + pos % P
    # tokens in the order they came, but for some that an earlier eviction moved
    moved = torch.rand(slot.shape, device="cuda", generator=g) < 0.05
    back = torch.randint(0, 1 << 20, slot.shape, device="cuda", generator=g) % (_ints(length).long()[:, None] + 1)
    when = torch.where(moved, back, pos[None, :].expand_as(back)) + 500
    born = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    born[slot[live]] = when[live].to(torch.int32)
    most = max(1, int(over.max()))
    new = lambda *shape: torch.full(shape, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": case, "weight": weight, "born": born, "table": t, "ctx_len": _ints(length), "budget": _ints(length - over),
            "pinned": _ints([case["pinned"]] * B), "keep_from": _ints(length + 500 - case["recent"]), "ctx_out": new(B), "n_moves": new(B),
            "move_from": new(B, most), "move_to": new(B, most), "len_max": int(length.max())}


def _prepare_move(case, seed):
    g = _gen(seed)
    n = np.array(_move_counts(case))
    k_cache, v_cache = _pools(case, case["n_pages"], g)
    most = max(1, int(n.max()))
    slots = torch.randperm(case["n_pages"] * case["P"], device="cuda", generator=g)[:2 * case["B"] * most].to(torch.int32)
    ends = slots.reshape(2, case["B"], most).sort(dim=2).values  # both lists rise along a request
    return {"case": case, "k_cache": k_cache, "v_cache": v_cache, "move_from": ends[0].contiguous(), "move_to": ends[1].contiguous(),
            "n_moves": _ints(n)}


# ---- one pass ---------------------------------------------------------------


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _own_shared(s):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    if "args" not in s:
        args = hybrid.make_shared_attention_args(
            q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], block_table=s["table"], ctx_len=s["ctx_len"], n_rows=s["n_rows"],
            row_start=s["row_start"], o=s["o"], scale=s["scale"], group_start=s["group_start"], prefix_len=s["prefix_len"], lse=s["lse"])
        s["work"] = torch.empty(hybrid.shared_attention_work_bytes(args), dtype=torch.uint8, device="cuda")
        args.attn.work = s["work"].data_ptr()
        s["args"] = args
    hybrid.gdn_shared_attention(s["args"])
    return [s["o"], s["lse"]]


def _own_weight(s):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    if "args" not in s:
        args = hybrid.make_attn_weight_args(
            q=s["q"], k_cache=s["k_cache"], lse=s["lse"], block_table=s["table"], ctx_len=s["ctx_len"], n_rows=s["n_rows"],
            row_start=s["row_start"], scale=s["scale"], weight=s["weight"], born=s["born"], first=s["first"], position=s["position"],
            keep=s["case"]["keep"], fresh=True)
        s["work"] = torch.empty(hybrid.attn_weight_work_bytes(args), dtype=torch.uint8, device="cuda")
        args.work = s["work"].data_ptr()
        s["args"] = args
    hybrid.gdn_attn_weight(s["args"])
    return [s["weight"], s["born"]]


def _own_select(s):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    if "args" not in s:
        s["args"] = hybrid.make_evict_select_args(
            weight=s["weight"], born=s["born"], block_table=s["table"], ctx_len=s["ctx_len"], budget=s["budget"], pinned=s["pinned"],
            keep_from=s["keep_from"], ctx_out=s["ctx_out"], n_moves=s["n_moves"], move_from=s["move_from"], move_to=s["move_to"],
            page_size=s["case"]["P"])
    hybrid.gdn_evict_select(s["args"])
    return _select_out(s)


def _own_move(s):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    if "args" not in s:
        s["args"] = hybrid.make_kv_move_args(k_cache=s["k_cache"], v_cache=s["v_cache"], move_from=s["move_from"], move_to=s["move_to"],
                                             n_moves=s["n_moves"])
    hybrid.gdn_kv_move(s["args"])
    return [s["k_cache"], s["v_cache"]]


def _select_out(s):
    return {k: s[k] for k in ("ctx_out", "n_moves", "move_from", "move_to", "weight", "born")}


def _scores(s):
    """Every new token's scaled products with its request's keys [b][h][g][t][l], the keys' places, and which pairs count."""
    case = s["case"]
    B, P, Hq, H, d = case["B"], case["P"], case["H_q"], case["H_kv"], case["d"]
    ctx, n = s["ctx_len"].long(), s["n_rows"].long()
    pos = torch.arange(s["len_max"], device="cuda")
    held = pos[None, :] < (ctx + n)[:, None]
    page = torch.where(held, s["table"].long()[:, pos // P], 0)
    k = s["k_cache"][page, :, pos % P].float()  # [B][L][H][d]
    t = torch.arange(s["n_max"], device="cuda")
    live = t[None, :] < n[:, None]
    row = torch.where(live, s["row_start"].long()[:, None] + t, 0)
    q = s["q"][row].float().reshape(B, -1, H, Hq // H, d)
    score = torch.einsum("bthgd,blhd->bhgtl", q, k) * s["scale"]
    seen = pos[None, None, :] <= (ctx[:, None] + t)[:, :, None]
    return score, seen, pos, held, page, row, live


def _plain_shared(s):
    case = s["case"]
    B, P, Hq = case["B"], case["P"], case["H_q"]
    score, seen, pos, held, page, row, live = _scores(s)
    v = torch.where(held[:, :, None, None], s["v_cache"][page, :, pos % P].float(), 0.0)
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp_()
    total = p.sum(-1)
    o = torch.einsum("bhgtl,blhd->bthgd", p, v) / total.permute(0, 3, 1, 2)[..., None]
    o = o.reshape(B, -1, Hq, case["d"]).to(_dtype(case))
    lse = (top[..., 0] + total.log()).permute(0, 3, 1, 2).reshape(B, -1, Hq)
    out, out_lse = torch.zeros_like(s["o"]), torch.zeros_like(s["lse"])
    out[row[live]] = o[live]
    out_lse[row[live]] = lse[live]
    return [out, out_lse]


def _plain_weight(s):
    case = s["case"]
    B, P, Hq, H = case["B"], case["P"], case["H_q"], case["H_kv"]
    score, seen, pos, held, page, row, live = _scores(s)
    lse = s["lse"][row].reshape(B, -1, H, Hq // H).permute(0, 2, 3, 1)[..., None]
    counts = (seen & live[:, :, None])[:, None, None]
    got = torch.where(counts, (score - lse).exp_(), 0.0).sum((1, 2, 3))  # [B][L]
    ctx, n = s["ctx_len"].long()[:, None], s["n_rows"].long()[:, None]
    slot = page * P + pos % P
    had = torch.where(pos[None, :] < ctx, s["weight"][slot] * case["keep"], 0.0)
    to = held & (n > 0) & (pos[None, :] >= s["first"].long()[:, None])
    s["weight"][slot[to]] = (had + got)[to]
    new = held & (n > 0) & (pos[None, :] >= ctx)
    s["born"][slot[new]] = (s["position"].long()[:, None] + pos[None, :] - ctx)[new].to(torch.int32)
    return [s["weight"], s["born"]]


def _plain_select(s):
    P, B = s["case"]["P"], s["case"]["B"]
    L, budget, pinned = (s[k].long()[:, None] for k in ("ctx_len", "budget", "pinned"))
    pos = torch.arange(s["len_max"], device="cuda")[None, :]
    live = pos < L
    slot = torch.where(live, s["table"].long()[:, pos[0] // P] * P + pos % P, 0)
    weight, born = s["weight"][slot], s["born"][slot].long()
    may_go = live & (pos >= pinned) & (born < s["keep_from"].long()[:, None])
    n_may = may_go.sum(1, keepdim=True)
    go = torch.minimum((L - budget.clamp(min=0)).clamp(min=0), n_may)
    # candidates by weight, the largest first, equal weights by the lowest index; the last `go` of them leave
    order = torch.where(may_go, weight, -math.inf).sort(dim=1, descending=True, stable=True).indices
    cand = torch.gather(may_go, 1, order)
    rank = cand.cumsum(1) - 1
    leaves = torch.zeros_like(may_go).scatter(1, order, cand & (rank >= n_may - go))
    K = L - go
    gap, mover = leaves & (pos < K), live & ~leaves & (pos >= K)
    n_moves = gap.sum(1)
    b = torch.arange(B, device="cuda")[:, None].expand_as(slot)
    s["move_to"][b[gap], (gap.cumsum(1) - 1)[gap]] = slot[gap].to(torch.int32)
    s["move_from"][b[mover], (mover.cumsum(1) - 1)[mover]] = slot[mover].to(torch.int32)
    s["weight"][slot[gap]] = s["weight"][slot[mover]]  # both in request and index order
    s["born"][slot[gap]] = s["born"][slot[mover]]
    s["ctx_out"].copy_(K[:, 0])
    s["n_moves"].copy_(n_moves)
    return _select_out(s)


def _plain_move(s):
    P = s["case"]["P"]
    live = torch.arange(s["move_to"].shape[1], device="cuda")[None, :] < s["n_moves"][:, None]
    src, dst = s["move_from"][live].long(), s["move_to"][live].long()
    for c in (s["k_cache"], s["v_cache"]):
        c[dst // P, :, dst % P] = c[src // P, :, src % P]
    return [s["k_cache"], s["v_cache"]]


_OWN = {"shared": _own_shared, "weight": _own_weight, "select": _own_select, "move": _own_move}
_PLAIN = {"shared": _plain_shared, "weight": _plain_weight, "select": _plain_select, "move": _plain_move}


# ---- what a pass cannot do without ------------------------------------------


def work(case):
    if case["op"] == "select":
        length, over = _select_lengths(case)
        # weight and age of every token, tables; at most as many moves as tokens that leave, each a pair of slots and its two values
        moves = sum(min(d, n - d) for n, d in zip(length, over))
        return {"bytes": 8.0 * sum(length) + 4.0 * sum(-(-n // case["P"]) for n in length) + 24.0 * moves / 2, "flops": 2.0 * sum(length)}
    if case["op"] == "move":
        return {"bytes": sum(_move_counts(case)) * (4.0 * case["H_kv"] * case["d"] * _size(case) + 8.0), "flops": 0.0}
    size, Hq, H, d = _size(case), case["H_q"], case["H_kv"], case["d"]
    if case["op"] == "shared":
        pre, own_ctx, n, start = _shared_lengths(case)
        # a group's prefix is read once, where any of its requests takes part
        keys = sum(pre[a] for a, z in zip(start, start[1:]) if any(n[a:z])) + sum(c + m for c, m in zip(own_ctx, n) if m)
        pairs = sum(m * (p + c) + m * (m + 1) // 2 for p, c, m in zip(pre, own_ctx, n))
        return {"bytes": 2.0 * keys * H * d * size + sum(n) * Hq * (2.0 * d * size + 4.0), "flops": 4.0 * pairs * Hq * d}
    ctx, n = _lengths(case)
    f = case["first"]
    keys = sum(max(a + m - f, 0) for a, m in zip(ctx, n) if m)
    pairs = sum(m * max(a - f, 0) + m * (m + 1) // 2 for a, m in zip(ctx, n))
    return {"bytes": keys * (1.0 * H * d * size + 8.0) + sum(n) * Hq * (1.0 * d * size + 4.0), "flops": 2.0 * pairs * Hq * d}


# ---- 64 bits, from the definitions ------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_shared, "weight": _exact_weight, "select": _exact_select, "move": _exact_move}[case["op"]](s)


def _requests(s):
    case = s["case"]
    for b, (ctx, n, start) in enumerate(zip(s["ctx_len"].tolist(), s["n_rows"].tolist(), s["row_start"].tolist())):
        if n:
            pages = s["table"][b, :-(-(ctx + n) // case["P"])].long()
            yield b, ctx, n, start, pages, torch.ones((n, ctx + n), dtype=torch.bool, device="cuda").triu(ctx + 1)


def _exact_shared(s):
    case = s["case"]
    G = case["H_q"] // case["H_kv"]
    out = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for _, ctx, n, start, pages, hidden in _requests(s):
        for h in range(case["H_kv"]):
            k, v = (c[pages, h].reshape(-1, case["d"])[:ctx + n].double() for c in (s["k_cache"], s["v_cache"]))
            for head in range(h * G, (h + 1) * G):
                z = (s["q"][start:start + n, head].double() @ k.T).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
                out[start:start + n, head] = torch.softmax(z, 1) @ v
                lse[start:start + n, head] = torch.logsumexp(z, 1)
    return [out, lse]


def _exact_weight(s):
    case = s["case"]
    P, G = case["P"], case["H_q"] // case["H_kv"]
    weight = s["weight"].double()
    for b, ctx, n, start, pages, hidden in _requests(s):
        got = torch.zeros(ctx + n, dtype=torch.float64, device="cuda")
        for h in range(case["H_kv"]):
            k = s["k_cache"][pages, h].reshape(-1, case["d"])[:ctx + n].double()
            for head in range(h * G, (h + 1) * G):
                z = (s["q"][start:start + n, head].double() @ k.T).mul_(s["scale"]) - s["lse"][start:start + n, head].double()[:, None]
                got += z.exp_().masked_fill_(hidden, 0.0).sum(0)
        at = torch.arange(ctx + n, device="cuda")
        slot = pages[at // P] * P + at % P
        had = weight[slot] * case["keep"]
        had[ctx:] = 0.0
        weight[slot[case["first"]:]] = (had + got)[case["first"]:]
    return [weight, None]


def _exact_select(s):
    P = s["case"]["P"]
    weight, born, table = (s[k].cpu().numpy() for k in ("weight", "born", "table"))
    out = weight.astype(np.float64)
    for b, (L, budget, pinned, keep_from) in enumerate(zip(*(s[k].tolist() for k in ("ctx_len", "budget", "pinned", "keep_from")))):
        at = np.arange(L)
        slot = table[b, at // P] * P + at % P
        may_go = np.flatnonzero((at >= pinned) & (born[slot] < keep_from))
        go = min(max(L - max(budget, 0), 0), len(may_go))
        by_weight = may_go[np.lexsort((-may_go, weight[slot[may_go]]))]  # the lightest first, among equals the last
        stays = np.ones(L, bool)
        stays[by_weight[:go]] = False
        K = L - go
        gaps, movers = np.flatnonzero(~stays[:K]), K + np.flatnonzero(stays[K:])
        out[slot[gaps]] = weight[slot[movers]]
    return {"ctx_out": None, "n_moves": None, "move_from": None, "move_to": None, "weight": torch.from_numpy(out), "born": None}


def _exact_move(s):
    P, out = s["case"]["P"], []
    for cache in (s["k_cache"], s["v_cache"]):
        c = cache.double().transpose(1, 2).flatten(0, 1)
        for b, n in enumerate(s["n_moves"].tolist()):
            c[s["move_to"][b, :n].long()] = c[s["move_from"][b, :n].long()]
        out.append(c.unflatten(0, (-1, P)).transpose(1, 2))
    return out
