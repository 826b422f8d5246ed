"""Measured cases of the hybrid-step operators: page maps, cache appends, paged
attention and sampled acceptance, each with its plain form and its value in 64 bits.

A Qwen3.5-style hybrid's verify step runs, beside the GatedDeltaNet layers, full
attention over a paged cache and, when requests sample, a sampled acceptance of the
drafts.  One pass here is one call of one of the four operators:

  pages    where the step's new tokens go: tables, slots and positions from lengths
  append   the new tokens' K and V rows written to those slots
  attend   every new token's attention over its request's pages
  sample   the target's sampled token per verify row, and the drafts it accepts
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
        # one verify step of 16 requests with three drafts each: the page map's usual call, latency only
        {"name": "pages-verify-B16", "op": "pages", "B": 16, "R": 4, "P": 16, "ctx_lo": 100, "ctx_hi": 8000, "n_lo": 4,
         "n_hi": 4, "idle": 0, "lens": 1},
        # a mixed step of a busy server: 1024 requests, most with a few rows, prompts among them, packed rows
        {"name": "pages-mixed-B1024", "op": "pages", "B": 1024, "R": 0, "P": 16, "ctx_lo": 0, "ctx_hi": 8000, "n_lo": 1,
         "n_hi": 255, "idle": 10, "lens": 2},
        # the K and V rows of a verify step, two wide heads, cut from the fused projection's rows
        {"name": "append-verify-bf16", "op": "append", "rows": 64, "H_q": 16, "H_kv": 2, "d": 256, "P": 16,
         "layout": "heads", "dtype": _BF16, "n_pages": 4096},
        # a prompt's rows, 32-bit, an odd count, token-major pages
        {"name": "append-prompt-f32", "op": "append", "rows": 16381, "H_q": 32, "H_kv": 8, "d": 128, "P": 64,
         "layout": "tokens", "dtype": _F32, "n_pages": 512},
        # the smallest attention call: three short requests in 32 bits
        {"name": "attend-small-f32", "op": "attend", "B": 3, "R": 5, "H_q": 6, "H_kv": 2, "d": 64, "P": 16, "ctx_lo": 0,
         "ctx_hi": 700, "n_lo": 1, "n_hi": 5, "idle": 0, "layout": "tokens", "dtype": _F32, "lens": 5},
        # the verify step of 16 requests with three drafts, the hybrid's own head shapes
        {"name": "attend-verify-B16", "op": "attend", "B": 16, "R": 4, "H_q": 16, "H_kv": 2, "d": 256, "P": 16,
         "ctx_lo": 1000, "ctx_hi": 8000, "n_lo": 4, "n_hi": 4, "idle": 0, "layout": "heads", "dtype": _BF16, "lens": 6},
        # one token of one request over a long context: the split along the keys is all the parallelism there is
        {"name": "attend-token-64k", "op": "attend", "B": 1, "R": 1, "H_q": 32, "H_kv": 8, "d": 128, "P": 64,
         "ctx_lo": 65537, "ctx_hi": 65537, "n_lo": 1, "n_hi": 1, "idle": 0, "layout": "heads", "dtype": _BF16, "lens": 7},
        # a wide ragged verify batch, two to nine rows, a tenth of the requests idle
        {"name": "attend-ragged-B256", "op": "attend", "B": 256, "R": 9, "H_q": 32, "H_kv": 4, "d": 128, "P": 16,
         "ctx_lo": 1, "ctx_hi": 4000, "n_lo": 2, "n_hi": 9, "idle": 10, "layout": "tokens", "dtype": _BF16, "lens": 8},
        # prompt chunks of up to 4096 new tokens behind cached ones: bound by the products
        {"name": "attend-chunk-4k", "op": "attend", "B": 3, "R": 0, "H_q": 32, "H_kv": 8, "d": 128, "P": 32, "ctx_lo": 0,
         "ctx_hi": 4096, "n_lo": 1500, "n_hi": 4096, "idle": 0, "layout": "heads", "dtype": _BF16, "lens": 9},
        # one request's sampled token over a small vocabulary, 32-bit logits
        {"name": "sample-one-f32", "op": "sample", "B": 1, "R": 1, "V": 32000, "dtype": _F32, "mix": "all", "idle": 0},
        # the verify step of 16 requests with three drafts over the hybrid's vocabulary, every filter in use
        {"name": "sample-verify-B16", "op": "sample", "B": 16, "R": 4, "V": 151936, "dtype": _BF16, "mix": "all", "idle": 0},
        # a wide ragged batch over an odd vocabulary: rows start off every alignment
        {"name": "sample-ragged-B128", "op": "sample", "B": 128, "R": 9, "V": 50001, "dtype": _BF16, "mix": "mixed", "idle": 10},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "append", "attend", "attend", "sample"])
    if op == "pages":
        packed = rng.random() < 0.5
        c = {"op": op, "B": _log(rng, 1, 1024), "R": 0 if packed else rng.randint(1, 16), "P": rng.choice([16, 32, 48, 64, 128]),
             "ctx_lo": 0, "ctx_hi": _log(rng, 10, 8000), "n_lo": rng.randint(0, 1), "idle": rng.choice([0, 10, 30]),
             "lens": rng.randrange(1 << 30)}
        c["n_hi"] = _log(rng, 1, 255) if packed else c["R"]
        return c
    if op == "append":
        h = rng.choice([1, 2, 4, 8])
        c = {"op": op, "rows": _log(rng, 1, 16000), "H_q": h * rng.randint(1, 4), "H_kv": h, "d": rng.choice([64, 128, 256]),
             "P": rng.choice([16, 32, 48, 64, 128]), "layout": rng.choice(["heads", "tokens"]), "dtype": rng.choice([_BF16, _F32])}
        if h * c["d"] * _size({"dtype": c["dtype"]}) > 4096:
            c["rows"] = min(c["rows"], 8000)
        c["n_pages"] = -(-c["rows"] // c["P"]) + rng.randint(1, 64)
        return c
    if op == "sample":
        return {"op": op, "B": _log(rng, 1, 64), "R": rng.randint(1, 9), "V": _log(rng, 64, 100000),
                "dtype": rng.choice([_BF16, _BF16, _F32]), "mix": rng.choice(["all", "mixed", "none"]), "idle": rng.choice([0, 10])}
    most = work(next(c for c in listed() if c["name"] == "attend-chunk-4k"))["flops"]
    while True:
        h = rng.choice([1, 2, 4, 8])
        c = {"op": op, "H_q": h * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), "H_kv": h, "d": rng.choice([64, 128, 256]),
             "P": rng.choice([16, 32, 48, 64, 128]), "layout": rng.choice(["heads", "tokens"]),
             "dtype": rng.choice([_BF16, _BF16, _BF16, _F32]), "lens": rng.randrange(1 << 30)}
        kind = rng.choice(["token", "verify", "chunk"])
        if kind == "token":
            c.update(B=_log(rng, 1, 256), R=1, n_lo=1, n_hi=1, ctx_lo=0, ctx_hi=_log(rng, 16, 65536), idle=rng.choice([0, 10]))
        elif kind == "verify":
            c.update(B=_log(rng, 1, 256), R=rng.randint(2, 16), ctx_lo=0, ctx_hi=_log(rng, 16, 16384), idle=rng.choice([0, 10]))
            c.update(n_lo=rng.randint(1, c["R"]), n_hi=c["R"])
        else:
            c.update(B=rng.randint(1, 4), R=0, n_hi=_log(rng, 17, 4096), ctx_lo=0, ctx_hi=_log(rng, 16, 8192), idle=0)
            c["n_lo"] = max(1, c["n_hi"] // 2)
        ctx, n = _lengths(c)
        keys = sum(a + b for a, b in zip(ctx, n))
        # what the plain form holds at once stays within what the listed cases need
        scores = c["B"] * max(n) * (max(ctx) + max(n)) * c["H_q"]
        if (work(c)["flops"] <= most / (16 if c["dtype"] == _F32 else 1) and keys * h * c["d"] <= 500_000_000
                and c["B"] * (max(ctx) + max(n)) * h * c["d"] <= 1_000_000_000 and scores <= 3_000_000_000):
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


def prepare(case, seed):
    return {"pages": _prepare_pages, "append": _prepare_append, "attend": _prepare_attend, "sample": _prepare_sample}[case["op"]](case, seed)


def _prepare_pages(case, seed):
    rng = np.random.default_rng(seed)
    ctx, n = (np.array(v) for v in _lengths(case))
    B, P = case["B"], case["P"]
    need = -(-(ctx + n) // P)
    # most requests hold the pages of their cached tokens; some still hold pages of drafts that were turned down
    cached = -(-ctx // P)
    held = cached + (rng.random(B) < 0.2) * rng.integers(0, 2, B)
    width = int(max(need.max(), cached.max() + 1)) + 3
    n_pages = int(np.maximum(need, cached + 1).sum()) + 37
    ids = rng.permutation(n_pages)
    table = np.full((B, width), -1)
    table[np.arange(width) < held[:, None]] = ids[:held.sum()]
    free = ids[held.sum():]
    head = int(rng.integers(0, n_pages))
    ring = np.full(n_pages, -1)
    ring[(head + np.arange(free.size)) % n_pages] = free
    rows = B * case["R"] if case["R"] else int(n.sum()) + 5
    new = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": case, "ctx_len": _ints(ctx), "n_rows": _ints(n), "held": _ints(held), "ring": _ints(ring),
            "free": _ints([head, free.size]), "table": _ints(table), "held_out": new(B), "free_out": new(2), "rows_out": new(B),
            "row_start": new(B + 1), "slots": new(rows), "positions": new(rows)}


def _prepare_append(case, seed):
    g = _gen(seed)
    T, Hq, H, d = case["rows"], case["H_q"], case["H_kv"], case["d"]
    k_cache, v_cache = _pools(case, case["n_pages"], g)
    x = torch.randn((T, (Hq + 2 * H) * d), device="cuda", generator=g, dtype=_dtype(case))
    slots = torch.randperm(case["n_pages"] * case["P"], device="cuda", generator=g)[:T].to(torch.int32)
    slots[torch.rand(T, device="cuda", generator=g) < 0.02] = -1  # padding rows
    return {"case": case, "k": x[:, Hq * d:(Hq + H) * d].unflatten(1, (H, d)), "v": x[:, (Hq + H) * d:].unflatten(1, (H, d)),
            "slots": slots, "k_cache": k_cache, "v_cache": v_cache}


def _prepare_attend(case, seed):
    g = _gen(seed)
    ctx, n = (np.array(v) for v in _lengths(case))
    B, P, Hq, H, d = case["B"], case["P"], case["H_q"], case["H_kv"], case["d"]
    need = -(-(ctx + n) // P)
    n_pages = int(need.sum()) + 5
    ids = np.random.default_rng(seed).permutation(n_pages)
    table = np.full((B, int(need.max()) + 1), -1)
    table[np.arange(table.shape[1]) < need[:, None]] = ids[:need.sum()]
    k_cache, v_cache = _pools(case, n_pages, g)
    rows = B * case["R"] if case["R"] else int(n.sum())
    x = torch.randn((rows, (Hq + 2 * H) * d), device="cuda", generator=g, dtype=_dtype(case))
    return {"case": case, "q": x[:, :Hq * d].unflatten(1, (Hq, d)), "k_cache": k_cache, "v_cache": v_cache, "table": _ints(table),
            "ctx_len": _ints(ctx), "n_rows": _ints(n), "row_start": _ints(_starts(case, n)), "scale": d ** -0.5,
            "n_max": int(n.max()), "len_max": int((ctx + n).max()), "o": torch.zeros((rows, Hq, d), device="cuda", dtype=_dtype(case))}


def _prepare_sample(case, seed):
    g = _gen(seed)
    B, R, V = case["B"], case["R"], case["V"]
    rand = lambda *s: torch.rand(s, device="cuda", generator=g)  # noqa: E731
    # a head of likely tokens above a wide floor, as a trained model's logits have
    logits = 2.0 * torch.randn((B, R, V), device="cuda", generator=g)
    at = torch.randint(0, V, (B, R, 24), device="cuda", generator=g)
    logits.scatter_add_(2, at, 6.0 + 4.0 * rand(B, R, 24))
    logits = logits.to(_dtype(case))
    pick = torch.randint(0, 4, (B,), device="cuda", generator=g)
    every = torch.ones(B, dtype=torch.bool, device="cuda") if case["mix"] == "all" else pick > 0
    temperature, top_k = 0.3 + rand(B), torch.randint(1, min(V, 200) + 1, (B,), device="cuda", generator=g).to(torch.int32)
    top_p, min_p = 0.5 + 0.5 * rand(B), 0.1 * rand(B)
    if case["mix"] == "mixed":  # greedy requests and requests without some filter among the others
        temperature = torch.where(pick == 0, 0.0, temperature)
        top_k = torch.where(pick == 1, 0, top_k)
        top_p = torch.where(pick == 2, 1.0, top_p)
        min_p = torch.where(pick == 3, 0.0, min_p)
    if case["mix"] == "none":  # temperature alone
        top_k, top_p, min_p = torch.zeros_like(top_k), torch.ones_like(top_p), torch.zeros_like(min_p)
    n = torch.randint(1, R + 1, (B,), device="cuda", generator=g)
    n = torch.where(rand(B) * 100 < case["idle"], 0, n)
    n[0] = R
    # drafts that are often the target's likeliest token
    best = logits.float().argmax(2)[:, :max(R - 1, 1)]
    drafts = torch.where(rand(*best.shape) < 0.7, best, torch.randint(0, V, best.shape, device="cuda", generator=g))
    return {"case": case, "logits": logits, "u": rand(B, R), "temperature": temperature.float(), "top_k": top_k.to(torch.int32),
            "top_p": top_p, "min_p": min_p, "drafts": drafts[:, :R - 1].to(torch.int32).contiguous(), "n_rows": n.to(torch.int32),
            "target": torch.full((B, R), -1, dtype=torch.int32, device="cuda"), "prob": torch.zeros((B, R), device="cuda"),
            "accept_len": torch.full((B,), -1, dtype=torch.int32, device="cuda")}


# ---- one pass ---------------------------------------------------------------


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _own_pages(s):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    if "args" not in s:
        s["args"] = hybrid.make_page_map_args(
            ctx_len=s["ctx_len"], n_rows=s["n_rows"], held=s["held"], free_ring=s["ring"], free_state=s["free"],
            block_table=s["table"], held_out=s["held_out"], free_state_out=s["free_out"], rows_out=s["rows_out"],
            row_start=s["row_start"], slot_map=s["slots"], positions=s["positions"], page_size=s["case"]["P"], R=s["case"]["R"])
    hybrid.gdn_page_map(s["args"])
    return _pages_out(s)


def _own_append(s):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    if "args" not in s:
        s["args"] = hybrid.make_kv_append_args(k=s["k"], v=s["v"], slot_map=s["slots"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    hybrid.gdn_kv_append(s["args"])
    return [s["k_cache"], s["v_cache"]]


def _own_attend(s):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    if "args" not in s:
        args = hybrid.make_paged_attention_args(
            q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], block_table=s["table"], ctx_len=s["ctx_len"], n_rows=s["n_rows"],
            row_start=s["row_start"], o=s["o"], scale=s["scale"])
        s["work"] = torch.empty(hybrid.paged_attention_work_bytes(args), dtype=torch.uint8, device="cuda")
        args.work = s["work"].data_ptr()
        s["args"] = args
    hybrid.gdn_paged_attention(s["args"])
    return s["o"]


def _own_sample(s):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    if "args" not in s:
        s["args"] = hybrid.make_sample_accept_args(
            logits=s["logits"], u=s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
            drafts=s["drafts"], n_rows=s["n_rows"], target=s["target"], prob=s["prob"], accept_len=s["accept_len"])
    hybrid.gdn_sample_accept(s["args"])
    return [s["target"], s["prob"], s["accept_len"]]


def _pages_out(s):
    return {k: s[k] for k in ("table", "ring", "held_out", "free_out", "rows_out", "row_start", "slots", "positions")}


def _plain_pages(s):
    P, R, B = s["case"]["P"], s["case"]["R"], s["case"]["B"]
    ctx, n, held, table, ring = (s[k].long() for k in ("ctx_len", "n_rows", "held", "table", "ring"))
    N, width, rows = ring.numel(), table.shape[1], s["slots"].numel()
    head, n_free = s["free"][0].long(), s["free"][1].long()
    need = (ctx + n + P - 1) // P
    want = (need - held).clamp(min=0)
    served = (want == 0) | (want.cumsum(0) <= n_free)
    take = torch.where(served, want, 0)
    back = torch.where(served, (held - need).clamp(min=0), 0)
    n = torch.where(served, n, 0)
    held_new = torch.where(served, need, held)
    col = torch.arange(width, device="cuda")[None, :]
    # pages given back go behind the free ones, pages taken come off the ring's head, both in request order
    give = (col >= need[:, None]) & (col < (need + back)[:, None])
    at = torch.where(give, (head + n_free + (back.cumsum(0) - back)[:, None] + col - need[:, None]) % N, N)
    new_ring = torch.cat([ring, ring[:1]]).scatter(0, at.reshape(-1), table.reshape(-1))[:N]
    got = (col >= held[:, None]) & (col < (held + take)[:, None])
    new_table = torch.where(got, ring[(head + (take.cumsum(0) - take)[:, None] + col - held[:, None]) % N], table)
    start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    r = torch.arange(rows, device="cuda")
    b = r // R if R else torch.searchsorted(start[1:].contiguous(), r, right=True).clamp(max=B - 1)
    first = b * R if R else start[b]
    live = (r - first) < n[b]
    pos = torch.where(live, ctx[b] + r - first, -1)
    slots = torch.where(live, new_table[b, pos.clamp(min=0) // P] * P + pos % P, -1)
    out = {"table": new_table, "ring": new_ring, "held_out": held_new, "rows_out": n, "slots": slots, "positions": pos,
           "free_out": torch.stack([(head + take.sum()) % N, n_free - take.sum() + back.sum()]),
           "row_start": torch.cat([torch.arange(B, device="cuda") * R, start[-1:] * 0 + B * R]) if R else start}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_append(s):
    P, slots = s["case"]["P"], s["slots"].long()
    # a padding row writes what the first live row writes, to the same place
    row = torch.arange(slots.numel(), device="cuda")
    row = torch.where(slots >= 0, row, (slots >= 0).to(torch.int32).argmax())
    slots = slots[row].clamp(min=0)
    s["k_cache"][slots // P, :, slots % P] = s["k"][row]
    s["v_cache"][slots // P, :, slots % P] = s["v"][row]
    return [s["k_cache"], s["v_cache"]]


def _plain_attend(s):
    case = s["case"]
    B, P, Hq, H, d = case["B"], case["P"], case["H_q"], case["H_kv"], case["d"]
    ctx, n = s["ctx_len"].long(), s["n_rows"].long()
    pos = torch.arange(s["len_max"], device="cuda")
    held = pos[None, :] < (ctx + n)[:, None]
    page = torch.where(held, s["table"].long()[:, pos // P], 0)
    k = s["k_cache"][page, :, pos % P].float()  # [B][L][H][d]
    v = torch.where(held[:, :, None, None], s["v_cache"][page, :, pos % P].float(), 0.0)
    t = torch.arange(s["n_max"], device="cuda")
    live = t[None, :] < n[:, None]
    row = torch.where(live, s["row_start"].long()[:, None] + t, 0)
    q = s["q"][row].float().reshape(B, -1, H, Hq // H, d)
    score = torch.einsum("bthgd,blhd->bhgtl", q, k) * s["scale"]
    seen = pos[None, None, :] <= (ctx[:, None] + t)[:, :, None]
    score = torch.where(seen[:, None, None], score, -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp_()
    o = torch.einsum("bhgtl,blhd->bthgd", p, v) / p.sum(-1).permute(0, 3, 1, 2)[..., None]
    o = o.reshape(B, -1, Hq, d).to(_dtype(case))
    out = torch.zeros_like(s["o"])
    out[row[live]] = o[live]
    return out


def _shift_mul(total, frac):
    """floor(total * frac / 2^24) of whole numbers, with no product over 62 bits."""
    return (total >> 24) * frac + (((total & 0xFFFFFF) * frac) >> 24)


def _plain_sample(s):
    case = s["case"]
    B, R, V = case["B"], case["R"], case["V"]
    per_row = lambda v: v[:, None].expand(B, R).reshape(B * R, 1)  # noqa: E731
    T, k, p, mp = (per_row(s[key]) for key in ("temperature", "top_k", "top_p", "min_p"))
    lg = s["logits"].reshape(B * R, V).float()
    lg, index = lg.sort(dim=1, descending=True, stable=True)  # equal logits: the lowest index first
    x = torch.where(lg == lg[:, :1], 0.0, (lg - lg[:, :1]) * (1.0 / torch.where(T > 0, T, 1.0)))
    w = x.exp()
    W = (w * 2147483648.0).round().to(torch.int64)
    rank = torch.arange(V, device="cuda")[None, :]
    kept = (k <= 0) | (rank < k)
    total = torch.where(kept, W, 0).sum(1, keepdim=True)
    limit = _shift_mul(total, (p.clamp(0, 1) * 16777216.0).floor().to(torch.int64))
    before = W.cumsum(1) - W
    kept &= (p >= 1) | (before < limit) | (rank == 0)
    kept &= (mp <= 0) | (w >= mp.clamp(max=1.0))
    kept = torch.where(T > 0, kept, rank == 0)  # no temperature: the largest logit
    W = torch.where(kept, W, 0)
    total = W.sum(1, keepdim=True)
    # the kept tokens in index order, and the first whose running sum passes the drawn share of the total
    run_sum = torch.zeros_like(W).scatter(1, index, W).cumsum(1)
    r = _shift_mul(total, (s["u"].reshape(B * R, 1).clamp(0, 1 - 2.0 ** -24) * 16777216.0).floor().to(torch.int64))
    token = (run_sum > r).to(torch.int8).argmax(1, keepdim=True)
    prob = (torch.where(index == token, w, 0.0).sum(1, keepdim=True) * 2147483648.0) / total.float()
    live = torch.arange(R, device="cuda")[None, :] < s["n_rows"][:, None]
    token, prob = token.reshape(B, R), prob.reshape(B, R)
    same = (token[:, :R - 1] == s["drafts"]) & live[:, 1:]
    accept = same.to(torch.int32).cumprod(1).sum(1)
    return [torch.where(live, token, -1).to(torch.int32), torch.where(live, prob, 0.0), accept.to(torch.int32)]


_OWN = {"pages": _own_pages, "append": _own_append, "attend": _own_attend, "sample": _own_sample}
_PLAIN = {"pages": _plain_pages, "append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}


# ---- what a pass cannot do without ------------------------------------------


def work(case):
    if case["op"] == "pages":
        ctx, n = (np.array(v) for v in _lengths(case))
        need, held = -(-(ctx + n) // case["P"]), -(-ctx // case["P"])
        rows = case["B"] * case["R"] if case["R"] else int(n.sum()) + 5
        touched = int((need - ctx // case["P"])[n > 0].sum())  # pages that new rows lie on
        ints = 6 * case["B"] + 2 * int((need - held).sum()) + touched + 2 * rows
        return {"bytes": 4.0 * ints, "flops": 4.0 * rows}
    if case["op"] == "append":
        return {"bytes": 4.0 * case["rows"] * case["H_kv"] * case["d"] * _size(case) + 4.0 * case["rows"], "flops": 0.0}
    if case["op"] == "sample":
        # row counts come with the seed: between 1 and R, R for the first request
        rows = case["R"] + (case["B"] - 1) * (1 - case["idle"] / 100) * (case["R"] + 1) / 2
        return {"bytes": rows * (case["V"] * _size(case) + 16), "flops": 4.0 * rows * case["V"]}
    ctx, n = _lengths(case)
    keys = sum(a + b for a, b in zip(ctx, n) if b)
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(ctx, n))
    size = _size(case)
    return {"bytes": 2.0 * keys * case["H_kv"] * case["d"] * size + 2.0 * sum(n) * case["H_q"] * case["d"] * size,
            "flops": 4.0 * pairs * case["H_q"] * case["d"]}


# ---- 64 bits, from the definitions ------------------------------------------


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers alone
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s)


def _exact_append(s):
    P, out = s["case"]["P"], []
    live = [i for i, v in enumerate(s["slots"].tolist()) if v >= 0]
    to = s["slots"][live].long()
    for rows, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        c = cache.double().transpose(1, 2).reshape(-1, *rows.shape[1:])
        c.index_copy_(0, to, rows[live].double())
        out.append(c.unflatten(0, (-1, P)).transpose(1, 2))
    return out


def _exact_attend(s):
    case = s["case"]
    P, G = case["P"], case["H_q"] // case["H_kv"]
    out = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    for b, (ctx, n, start) in enumerate(zip(s["ctx_len"].tolist(), s["n_rows"].tolist(), s["row_start"].tolist())):
        if n == 0:
            continue
        pages = s["table"][b, :-(-(ctx + n) // P)].long()
        hidden = torch.ones((n, ctx + n), dtype=torch.bool, device="cuda").triu(ctx + 1)
        for h in range(case["H_kv"]):
            k, v = (c[pages, h].reshape(-1, case["d"])[:ctx + n].double() for c in (s["k_cache"], s["v_cache"]))
            for head in range(h * G, (h + 1) * G):
                z = (s["q"][start:start + n, head].double() @ k.T).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
                out[start:start + n, head] = torch.softmax(z, 1) @ v
    return out


def _exact_sample(s):
    case = s["case"]
    B, R, V = case["B"], case["R"], case["V"]
    prob = np.zeros((B, R))
    n = s["n_rows"].tolist()
    if sum(n) * V > 100_000_000:
        return None
    T, k, p, mp, u = (s[key].double().cpu().numpy() for key in ("temperature", "top_k", "top_p", "min_p", "u"))
    for b in range(B):
        for t in range(n[b]):
            z = s["logits"][b, t].double().cpu().numpy()
            if not T[b] > 0:
                prob[b, t] = 1.0
                continue
            order = np.argsort(-z, kind="stable")
            w = np.exp((z[order] - z[order[0]]) / T[b])
            m = V if k[b] <= 0 else min(V, int(k[b]))
            if p[b] < 1:
                c = np.cumsum(w[:m])
                m = min(m, 1 + int(np.searchsorted(c, p[b] * c[-1], side="left")))
            keep = np.zeros(V, bool)
            keep[order[:m][w[:m] >= min(mp[b], 1.0)]] = True
            full = np.zeros(V)
            full[order] = w
            full[~keep] = 0.0
            c = np.cumsum(full)
            token = int(np.searchsorted(c, u[b, t] * c[-1], side="right"))
            prob[b, t] = full[min(token, V - 1)] / c[-1]
    return [None, torch.from_numpy(prob), None]
