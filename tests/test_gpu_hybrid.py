"""The hybrid-step operators on the GPU against their plain 64-bit forms, at the
lengths, shapes, strides and values where they can go wrong.

Tolerances, from the arithmetic each call promises.  Page maps, appends and
sampled tokens are exact.  32-bit attention: a score is a sum of d <= 256 products
of size up to ~4, so its error stays under d * 2^-24 * 4 * sqrt(d) * scale < 2e-5 in
the worst case and far below on average; 1e-5 of the result's 2-norm.  bf16
attention: every weight p is rounded to 8 bits (2^-9 of itself), so an output moves
by at most 2^-9 of the largest |v| its row sees; rounding o adds 2^-9 of |o|, and the
32-bit part of the work 1e-5 of that |v|."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import hybrid_ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def hy(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_gateddeltanet_gb300 import hybrid

    return hybrid


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


# ---- page map ------------------------------------------------------------------


def run_page_map(hy, ctx, n, held, ring, free, table, P, R, rows):
    t = dict(ctx_len=ints(ctx), n_rows=ints(n), held=ints(held), free_ring=ints(ring), free_state=ints(free), block_table=ints(table))
    new = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    B = len(ctx)
    out = dict(held_out=new(B), free_state_out=new(2), rows_out=new(B), row_start=new(B + 1), slot_map=new(rows), positions=new(rows),
               status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    hy.gdn_page_map(hy.make_page_map_args(**t, **out, page_size=P, R=R))
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in (t | out).items()}
    return dict(table=got["block_table"], ring=got["free_ring"], free_out=got["free_state_out"], status=int(got["status"][0]),
                **{k: got[k] for k in ("held_out", "rows_out", "row_start", "slot_map", "positions")})


def page_case(B, P, R, seed, ctx_hi=300, n_hi=40, scarce=0.0, idle=0.2):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, B)
    n = rng.integers(0, (R or n_hi) + 1, B)
    done = rng.random(B) < idle
    ctx[done] = n[done] = 0
    held = -(-ctx // P) + rng.integers(0, 3, B)
    need = -(-(ctx + n) // P)
    width = int(max(need.max(), held.max(), 1)) + 1
    demand = int(np.maximum(need - held, 0).sum())
    n_free = int(demand * (1 - scarce)) + (2 if not scarce else 0)
    N = int(held.sum()) + n_free + 5
    ids = rng.permutation(N)
    table = np.full((B, width), -1)
    table[np.arange(width) < held[:, None]] = ids[:held.sum()]
    head = int(rng.integers(0, N))
    ring = np.full(N, -1)
    ring[(head + np.arange(n_free)) % N] = ids[held.sum():held.sum() + n_free]
    return ctx, n, held, ring, np.array([head, n_free]), table, P, R, B * R if R else int(n.sum()) + 3


@pytest.mark.parametrize("B,P,R,scarce,seed", [(1, 16, 1, 0, 0), (16, 16, 4, 0, 1), (7, 48, 9, 0, 2), (513, 16, 0, 0, 3),
                                               (4096, 32, 3, 0, 4), (100, 1, 5, 0, 5), (64, 16, 0, 0.5, 6), (1000, 16, 16, 0.3, 7)])
def test_page_map_matches_the_definition(hy, B, P, R, scarce, seed):
    case = page_case(B, P, R, seed, scarce=scarce)
    ref = hybrid_ref.page_map(*case)
    got = run_page_map(hy, *case)
    assert (ref["status"] == 32) == (scarce > 0)
    for key, want in ref.items():
        assert np.array_equal(got[key], want), key


def test_page_map_refuses_bad_requests_alone(hy):
    ctx, n, held, ring, free, table, P, R, rows = page_case(12, 16, 4, 11, idle=0)
    ctx[1] = -1
    n[2] = 5
    n[3] = -2
    held[4] = table.shape[1] + 1
    ctx[5] = 16 * table.shape[1]
    n[5] = 3
    case = (ctx, n, held, ring, free, table, P, R, rows)
    ref, got = hybrid_ref.page_map(*case), run_page_map(hy, *case)
    assert ref["status"] == 256 | 2 | 64
    for key, want in ref.items():
        assert np.array_equal(got[key], want), key


def test_page_map_packed_rows_that_do_not_fit(hy):
    ctx, n, held, ring, free, table, P, R, rows = page_case(20, 16, 0, 12, idle=0)
    case = (ctx, n, held, ring, free, table, P, R, int(n[:12].sum()) + 1)
    ref, got = hybrid_ref.page_map(*case), run_page_map(hy, *case)
    assert ref["status"] == 512
    for key, want in ref.items():
        assert np.array_equal(got[key], want), key


def test_page_map_steps_keep_every_page_once(hy):
    """Twenty steps of growth, turned-down drafts and finished requests, the counts alternating between two buffers:
    at every step each page is in one table row or free, never both."""
    rng = np.random.default_rng(5)
    B, P, R, N = 9, 16, 4, 64
    new = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, ring = new(B, 20), ints(rng.permutation(N))
    held, free = [new(B), new(B)], [ints([5, N]), new(2)]
    rows, slots, status = new(B), new(B * R), new(1)
    ctx = np.zeros(B, np.int64)
    for step in range(20):
        n = rng.integers(0, R + 1, B)
        ctx[rng.random(B) < 0.05] = 0
        a, b = step % 2, 1 - step % 2
        hy.gdn_page_map(hy.make_page_map_args(
            ctx_len=ints(ctx), n_rows=ints(n), held=held[a], free_ring=ring, free_state=free[a], block_table=table, held_out=held[b],
            free_state_out=free[b], rows_out=rows, slot_map=slots, page_size=P, R=R, status=status))
        torch.cuda.synchronize()
        h, (head, count) = held[b].cpu().numpy(), free[b].cpu().numpy()
        tab, rg = table.cpu().numpy(), ring.cpu().numpy()
        pages = [int(x) for r in range(B) for x in tab[r, :h[r]]] + [int(rg[(head + i) % N]) for i in range(count)]
        assert sorted(pages) == list(range(N))
        live = slots.cpu().numpy()
        live = live[live >= 0]
        assert len(set(live.tolist())) == len(live) == int(rows.sum())
        ctx += np.minimum(n, rng.integers(0, R + 1, B))


# ---- append --------------------------------------------------------------------


@pytest.mark.parametrize("rows,H,d,P,layout,dtype", [(1, 1, 64, 16, "heads", BF16), (37, 3, 128, 48, "tokens", BF16),
                                                     (500, 2, 256, 16, "heads", F32), (1023, 8, 64, 32, "tokens", F32),
                                                     (9, 2, 40, 7, "heads", BF16)])
def test_append_writes_the_slots_alone(hy, rows, H, d, P, layout, dtype):
    g = torch.Generator().manual_seed(rows)
    n_pages = -(-rows // P) + 4
    pool = torch.randn((n_pages, 2, H, P, d) if layout == "heads" else (n_pages, 2, P, H, d), generator=g).to(dtype)
    x = torch.randn((rows, 3 * H + 1, d), generator=g).to(dtype)
    slots = torch.randperm(n_pages * P, generator=g)[:rows].to(torch.int32)
    slots[::5] = -1
    if rows > 20:
        slots[7] = n_pages * P  # beyond the pool: skipped and flagged
        slots[8] = 2**31 - 1
    dev = pool.cuda()
    view = lambda p: p if layout == "heads" else p.transpose(2, 3)  # noqa: E731
    xc = x.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hy.gdn_kv_append(hy.make_kv_append_args(k=xc[:, H:2 * H], v=xc[:, 2 * H:3 * H], slot_map=slots.cuda(), k_cache=view(dev)[:, 0],
                                            v_cache=view(dev)[:, 1], status=status))
    torch.cuda.synchronize()
    want = view(pool)
    for r, s in enumerate(slots.tolist()):
        if 0 <= s < n_pages * P:
            want[s // P, 0, :, s % P] = x[r, H:2 * H]
            want[s // P, 1, :, s % P] = x[r, 2 * H:3 * H]
    assert torch.equal(dev.cpu(), pool)
    assert int(status.item()) == (hy.STATUS_BAD_PAGE if rows > 20 else 0)


# ---- attention -----------------------------------------------------------------


def run_attention(hy, case, R=0, o_pad=2, calls=1, stream=None, status=None):
    q = case["q"].cuda()
    k, v = case["k_cache"].cuda(), case["v_cache"].cuda()
    if case["k_cache"].stride(2) > case["k_cache"].stride(1):  # token-major pages keep their strides
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    out = torch.full((q.shape[0], q.shape[1] + o_pad, q.shape[2]), 7.0, device="cuda", dtype=q.dtype)
    args = hy.make_paged_attention_args(
        q=q, k_cache=k, v_cache=v, block_table=ints(case["table"]), ctx_len=ints(case["ctx"]), n_rows=ints(case["n"]),
        row_start=None if R else ints(case["start"]), R=R, o=out[:, :q.shape[1]], scale=case["scale"], status=status)
    tensors = [ints(case["table"]), ints(case["ctx"]), ints(case["n"]), ints(case["start"])]
    args.block_table, args.ctx_len, args.n_rows = (t.data_ptr() for t in tensors[:3])
    args.row_start = None if R else tensors[3].data_ptr()
    work = torch.full((hy.paged_attention_work_bytes(args),), 255, dtype=torch.uint8, device="cuda")
    args.work = work.data_ptr()
    torch.cuda.synchronize()
    for _ in range(calls):
        hy.gdn_paged_attention(args, stream=stream)
    torch.cuda.synchronize()
    assert bool((out[:, q.shape[1]:] == 7.0).all()), "elements between the rows were written"
    return out[:, :q.shape[1]]


def check_attention(case, o):
    ref, vmax = hybrid_ref.attention(case["q"], case["k_cache"], case["v_cache"], case["table"], case["ctx"], case["n"], case["start"],
                                     case["scale"])
    got = o.double().cpu().numpy()
    live = ~np.isnan(ref[..., 0])
    assert (got[~live] == 7.0).all(), "rows of no request were written"
    if o.dtype == F32:
        assert np.linalg.norm(got[live] - ref[live]) <= 1e-5 * np.linalg.norm(ref[live])
    else:
        bound = 2.0**-9 * (vmax[live][:, None] + np.abs(ref[live])) + 1e-5 * vmax[live][:, None]
        err = np.abs(got[live] - ref[live])
        assert np.isfinite(got[live]).all()
        assert (err <= bound).all(), f"worst {np.max(err / bound):.2f} of the bound"


ONE = [(0, 1)]
RAGGED = [(0, 3), (1, 9), (127, 2), (128, 1), (500, 0), (129, 5), (1000, 7), (15, 1), (16, 4), (2047, 9)]
ATTENTION = [
    # lens, H_q, H_kv, d, P, layout, R
    (ONE, 1, 1, 64, 16, "heads", 0),
    (ONE, 8, 2, 128, 16, "tokens", 1),
    ([(0, 0), (0, 0)], 4, 2, 64, 16, "heads", 1),              # nothing to do
    ([(4096, 1)], 32, 8, 128, 64, "heads", 1),                 # one token, split over many blocks
    ([(3001, 1)], 16, 2, 256, 16, "heads", 1),
    (RAGGED, 8, 2, 128, 16, "heads", 9),
    (RAGGED, 16, 2, 256, 32, "tokens", 0),
    (RAGGED, 10, 2, 64, 48, "heads", 0),                       # groups of five: tokens straddle the row tiles
    (RAGGED, 7, 1, 128, 128, "tokens", 9),
    ([(300, 1), (5, 1), (64, 1)], 128, 1, 64, 16, "heads", 0),  # one token's heads fill a row tile
    ([(777, 1)], 96, 1, 128, 1024, "heads", 0),
    ([(0, 300), (200, 131), (63, 64)], 4, 4, 128, 16, "heads", 0),   # prompts, no sharing of heads
    ([(0, 257), (1000, 100)], 12, 4, 64, 64, "tokens", 0),
    ([(31, 200), (0, 1), (400, 17)], 6, 2, 256, 16, "tokens", 0),
    ([(0, 1500)], 5, 1, 128, 32, "heads", 0),
    ([(3, 2)] * 200, 8, 4, 128, 16, "heads", 2),               # more tiles than blocks
    ([(700 + 3 * i, 1 + i % 5) for i in range(150)], 32, 4, 128, 16, "tokens", 0),  # several long tiles a block, of 8 to 40 rows
    ([(900 - 5 * i, 1 + i % 9) for i in range(100)], 32, 4, 64, 32, "heads", 9),
    ([(600 + i, 1 + i % 12) for i in range(90)], 32, 4, 256, 64, "heads", 0),       # 8 to 96 rows
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,H_q,H_kv,d,P,layout,R", ATTENTION, ids=[f"{i}" for i in range(len(ATTENTION))])
def test_attention_matches_the_definition(hy, lens, H_q, H_kv, d, P, layout, R, dtype):
    case = hybrid_ref.make_attention(lens=lens, H_q=H_q, H_kv=H_kv, d=d, P=P, dtype=dtype, layout=layout, R=R, seed=len(lens) + d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_attention(case, run_attention(hy, case, R=R, status=status))
    assert int(status.item()) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_attention_of_few_rows(hy, dtype, d):
    """One to 33 rows a tile, each split over several blocks."""
    lens = [(1500 - 7 * n, n) for n in (1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33)]
    case = hybrid_ref.make_attention(lens=lens, H_q=2, H_kv=2, d=d, P=16, dtype=dtype, seed=d)
    check_attention(case, run_attention(hy, case))


@pytest.mark.parametrize("P", [1, 7, 24, 3000])
def test_attention_f32_with_any_page_size(hy, P):
    case = hybrid_ref.make_attention(lens=[(100, 3), (0, 40)], H_q=4, H_kv=2, d=64, P=P, dtype=F32, seed=P)
    check_attention(case, run_attention(hy, case))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_attention_of_wide_scores(hy, dtype):
    """Scores far apart (the running maximum grows along the keys, weights underflow) and a negative scale."""
    for scale, grow in ((0.5, True), (-0.3, False), (0.0, False)):
        case = hybrid_ref.make_attention(lens=[(700, 6), (0, 40)], H_q=8, H_kv=2, d=128, P=16, dtype=dtype, seed=3, scale=scale)
        if grow:
            k = case["k_cache"]
            for b in range(2):
                for i, page in enumerate(case["table"][b, :-(-int(case["ctx"][b] + case["n"][b]) // 16)]):
                    k[page] *= 0.2 * (1 + i)
        o = run_attention(hy, case)
        ref, vmax = hybrid_ref.attention(*(case[k] for k in ("q", "k_cache", "v_cache", "table", "ctx", "n", "start", "scale")))
        # scores reach ~2000 here, and 32-bit sums of them are off by up to d * 2^-24 of the products' size: 2e-3 in the exponent
        tol = (2.0**-9 if dtype == BF16 else 0.0) * (vmax[..., None] + np.abs(ref)) + 4e-3 * vmax[..., None]
        assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_attention_takes_infinite_and_nan_values_as_the_definition_does(hy, dtype):
    """A NaN key spoils the rows that see it and no others; a key of -inf score has no weight."""
    case = hybrid_ref.make_attention(lens=[(40, 4), (40, 4)], H_q=4, H_kv=1, d=64, P=16, dtype=dtype, seed=9)
    page = case["table"][0]
    case["k_cache"][page[42 // 16], 0, 42 % 16, 5] = float("nan")  # position 42: seen by rows 2 and 3 of request 0
    case["q"][4:, :, 0] = 1.0
    case["k_cache"][case["table"][1][0], 0, 3, 0] = float("-inf")
    o = run_attention(hy, case).double().cpu().numpy()
    assert np.isnan(o[2:4]).all() and np.isfinite(o[:2]).all() and np.isfinite(o[4:]).all()
    clean = dict(case, k_cache=case["k_cache"].clone())
    clean["k_cache"][page[42 // 16], 0, 42 % 16] = 0
    ref, vmax = hybrid_ref.attention(*(clean[k] for k in ("q", "k_cache", "v_cache", "table", "ctx", "n", "start", "scale")))
    tol = 2.0**-8 * vmax[..., None] + 1e-5
    assert (np.abs(o - ref)[[0, 1, 4, 5, 6, 7]] <= tol[[0, 1, 4, 5, 6, 7]]).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_attention_skips_bad_requests_and_flags_them(hy, dtype):
    case = hybrid_ref.make_attention(lens=[(20, 2), (30, 2), (40, 2), (50, 2), (60, 2)], H_q=4, H_kv=2, d=128, P=16, dtype=dtype, R=2, seed=4)
    good = run_attention(hy, case, R=2).clone()
    for change, bit in ((dict(n=3), 2), (dict(n=-1), 2), (dict(ctx=-1), 256), (dict(ctx=16 * case["table"].shape[1] - 1), 256)):
        bad = dict(case, ctx=case["ctx"].copy(), n=case["n"].copy())
        for key, v in change.items():
            bad[key][1] = v
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = run_attention(hy, bad, R=2, status=status)
        assert int(status.item()) == bit, change
        assert bool((o[2:4] == 7.0).all())
        assert torch.equal(o[[0, 1, 4, 5, 6, 7, 8, 9]], good[[0, 1, 4, 5, 6, 7, 8, 9]])
    bad = dict(case, table=case["table"].copy())
    bad["table"][2, 1] = 10**6  # a page outside the pool reads as zeros and is flagged
    bad["table"][3, 0] = -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = run_attention(hy, bad, R=2, status=status)
    assert int(status.item()) == 128
    assert torch.equal(o[[0, 1, 2, 3, 8, 9]], good[[0, 1, 2, 3, 8, 9]]) and bool(torch.isfinite(o).all())
    zero = dict(case, table=bad["table"].copy(), k_cache=case["k_cache"].clone(), v_cache=case["v_cache"].clone())
    for b, i in ((2, 1), (3, 0)):
        page = case["table"][b, i]
        zero["table"][b, i] = page
        zero["k_cache"][page] = 0
        zero["v_cache"][page] = 0
    assert torch.equal(o, run_attention(hy, zero, R=2))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_attention_repeats_its_bits_on_any_stream(hy, dtype):
    case = hybrid_ref.make_attention(lens=RAGGED, H_q=8, H_kv=2, d=128, P=16, dtype=dtype, seed=21)
    first = run_attention(hy, case)
    assert torch.equal(first, run_attention(hy, case, calls=3))
    assert torch.equal(first, run_attention(hy, case, stream=torch.cuda.Stream()))


# ---- sampling ------------------------------------------------------------------


def sample_case(B, R, V, dtype, seed, ties=False, pad=0):
    g = torch.Generator().manual_seed(seed)
    logits = 2.0 * torch.randn((B, R, V), generator=g)
    if ties:
        logits = logits.round()
    else:
        logits[:, :, :: max(V // 20, 1)] += 5.0
    logits = torch.nn.functional.pad(logits, (0, pad), value=50.0).to(dtype)[:, :, :V]
    rand = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    n = torch.randint(0, R + 1, (B,), generator=g).to(torch.int32)
    n[0] = R
    return dict(logits=logits, u=rand(B, R), temperature=0.3 + rand(B), top_k=torch.randint(1, V + 1, (B,), generator=g).to(torch.int32),
                top_p=0.3 + 0.7 * rand(B), min_p=0.1 * rand(B), drafts=torch.randint(0, V, (B, max(R - 1, 0)), generator=g).to(torch.int32),
                n_rows=n)


def run_sample(hy, case, off=()):
    B, R, V = case["logits"].shape
    store = case["logits"].as_strided((B, R, case["logits"].stride(1)), case["logits"].stride())
    dev = {k: v.cuda() for k, v in case.items() if k != "logits" and k not in off}
    dev["logits"] = store.cuda()[:, :, :V]
    out = dict(target=torch.full((B, R), -5, dtype=torch.int32, device="cuda"), prob=torch.full((B, R), -5.0, device="cuda"),
               accept_len=torch.full((B,), -5, dtype=torch.int32, device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    hy.gdn_sample_accept(hy.make_sample_accept_args(**dev, **out))
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def whole_number_token(z, T, k, p, m, u):
    """The definition in whole numbers, from a device row z and 32-bit weights: its token, exactly."""
    V = z.numel()
    z = z.float()
    live = ~torch.isnan(z)
    if not bool(live.any()):
        return 0
    key = torch.where(live, z, -np.inf)
    top = key.max()
    order = np.lexsort((np.arange(V), -key.double().cpu().numpy(), ~live.cpu().numpy()))
    if not T > 0:
        return int(order[0])
    inv = torch.tensor(1.0, device="cuda") / torch.tensor(T, dtype=F32, device="cuda")
    w = torch.where(z == top, 1.0, ((z - top) * inv).exp())
    w = torch.where(live, w, 0.0).cpu().numpy()
    W = np.rint(w.astype(np.float64) * 2.0**31).astype(object)[order]
    c = int(live.sum())
    c = c if k <= 0 or k >= V else min(k, c)
    frac = lambda x, most: int(np.floor(np.float64(min(max(np.float32(0 if np.isnan(x) else x), 0), most)) * 2**24))  # noqa: E731
    if p < 1:
        limit = int(W[:c].sum()) * frac(p, 1.0) >> 24
        before = np.concatenate([[0], np.cumsum(W[:c])[:-1]])
        c = max(1, int((before < limit).sum()))
    floor_w = min(np.float32(m), np.float32(1)) if m > 0 else 0
    keep = order[:c][w[order[:c]] >= floor_w]
    full = np.zeros(V, object)
    full[order] = W
    kept = np.zeros(V, object)
    kept[keep] = full[keep]
    cum = np.cumsum(kept)
    return int((cum <= (int(cum[-1]) * frac(u, 1 - 2.0**-24) >> 24)).sum())


def check_sample(case, got, off=()):
    """Tokens equal the whole-number definition's always, and the 64-bit definition's wherever rounding the weights to
    2^-31 (and exp to 32 bits: 2^-22 of a weight) cannot decide: where a shift of the drawn share and of the nucleus by
    V * 2^-32 + 2^-21 gives the same token."""
    B, R, V = case["logits"].shape
    slack = V * 2.0**-32 + 2.0**-21
    none = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    n = case["n_rows"].numpy()
    z = case["logits"].float().numpy()
    dev = case["logits"].cuda()
    for b in range(B):
        par = [none[k] if k in off else case[k][b].item() for k in ("temperature", "top_k", "top_p", "min_p")]
        for t in range(R):
            if t >= n[b]:
                assert got["target"][b, t] == -5 and got["prob"][b, t] == -5.0
                continue
            u = case["u"][b, t].item()
            assert got["target"][b, t] == whole_number_token(dev[b, t], *par, u), (b, t)
            u = np.floor(u * 2**24) / 2**24
            lo, hi = (hybrid_ref.sample_row(z[b, t], *par, u, s)[0] for s in (-slack, slack))
            token, prob = hybrid_ref.sample_row(z[b, t], *par, u)
            if lo == hi:
                assert got["target"][b, t] == token, (b, t)
                assert abs(got["prob"][b, t] - prob) <= 2.0**-20 * prob + V * 2.0**-32
    for b in range(B):
        a = 0
        while a < n[b] - 1 and case["drafts"][b, a] == got["target"][b, a]:
            a += 1
        assert got["accept_len"][b] == a
    assert got["status"][0] == 0


SAMPLE = [(1, 1, 64, F32, False, 0), (3, 4, 1000, BF16, False, 0), (5, 3, 777, BF16, True, 0), (4, 2, 4097, F32, False, 3),
          (9, 5, 32000, BF16, False, 0), (2, 2, 151936, BF16, False, 0), (2, 1, 100001, F32, True, 0), (6, 2, 1, BF16, False, 0),
          (8, 4, 3, F32, True, 5), (3, 2, 50257, BF16, True, 7)]


@pytest.mark.parametrize("B,R,V,dtype,ties,pad", SAMPLE, ids=[f"{i}" for i in range(len(SAMPLE))])
def test_sampling_matches_the_definition(hy, B, R, V, dtype, ties, pad):
    case = sample_case(B, R, V, dtype, seed=V, ties=ties, pad=pad)
    check_sample(case, run_sample(hy, case))
    for off in (("temperature", "top_k", "top_p", "min_p"), ("top_k",), ("top_p", "min_p"), ("top_k", "top_p")):
        check_sample(case, run_sample(hy, case, off), off)


@pytest.mark.parametrize("B,R,V,dtype", [(160, 4, 1500, BF16), (77, 4, 14001, F32)])
def test_sampling_of_more_rows_than_the_gpu_holds(hy, B, R, V, dtype):
    case = sample_case(B, R, V, dtype, seed=B)
    check_sample(case, run_sample(hy, case))
    check_sample(case, run_sample(hy, case, ("top_k",)), ("top_k",))


@pytest.mark.parametrize("V,k", [(5000, 300), (40000, 700), (40000, 20), (3000, 512), (3000, 513), (700, 699)])
def test_sampling_with_many_equal_logits(hy, V, k):
    """Far more tokens at the k-th largest logit than k: they enter by index, whichever way the k-th is found."""
    case = sample_case(3, 2, V, BF16, seed=k)
    case["logits"] = (case["logits"] / 4).round()  # a handful of values
    case["top_k"][:] = k
    check_sample(case, run_sample(hy, case))
    check_sample(case, run_sample(hy, case, ("top_p", "min_p")), ("top_p", "min_p"))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_sampling_parameters_at_their_edges(hy, dtype):
    """Requests with a parameter at or past its edge against the definition with that filter's plain meaning."""
    V = 500
    edges = [dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(top_k=1), dict(top_k=-3),
             dict(top_k=V), dict(top_k=V + 7), dict(top_p=0.0), dict(top_p=-1.0), dict(top_p=1.5), dict(top_p=1e-9), dict(min_p=1.0),
             dict(min_p=3.0), dict(min_p=-1.0), dict(temperature=1e-6), dict(temperature=1e6), dict(top_p=float("nan")),
             dict(min_p=float("nan")), dict(temperature=float("inf"))]
    case = sample_case(len(edges), 3, V, dtype, seed=2)
    case["n_rows"][:] = 3
    for b, e in enumerate(edges):
        for k, v in e.items():
            case[k][b] = v
    case["u"][:, 0] = 0.0
    case["u"][:, 1] = 1.0  # clamped below one
    got = run_sample(hy, case)
    plain = {k: v.clone() for k, v in case.items()}
    plain["top_p"] = torch.nan_to_num(plain["top_p"], nan=1.0)
    plain["min_p"] = torch.nan_to_num(plain["min_p"], nan=0.0)
    plain["u"].clamp_(max=1 - 2.0**-24)
    check_sample(plain, got)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_sampling_of_infinite_and_nan_logits(hy, dtype):
    nan, inf, low = float("nan"), float("inf"), torch.finfo(dtype).min
    case = sample_case(9, 1, 300, dtype, seed=5)
    case["n_rows"][:] = 1
    z = case["logits"]
    z[0] = nan
    z[1] = -inf
    z[2, 0, 5:] = -inf
    z[3, 0, 7:] = low
    z[4, 0, ::2] = nan
    z[5, 0, 11] = inf
    z[6, 0, [3, 200]] = inf
    z[7, 0, 1:] = nan
    z[8, 0, :] = -0.0
    z[8, 0, ::2] = 0.0
    case["top_k"][2] = 100  # more than the tokens that are not masked
    case["top_k"][8] = 150
    got = run_sample(hy, case)
    check_sample(case, got)
    assert got["target"][0, 0] == 0 and got["prob"][0, 0] == 1.0 and got["target"][2, 0] < 5 and got["target"][3, 0] < 7
    assert got["target"][4, 0] % 2 == 1 and got["target"][5, 0] == 11 and got["target"][6, 0] in (3, 200) and got["target"][7, 0] == 0


def test_sampling_flags_a_bad_row_count(hy):
    case = sample_case(4, 3, 100, F32, seed=1)
    case["n_rows"] = torch.tensor([3, 4, -1, 2], dtype=torch.int32)
    got = run_sample(hy, case)
    assert got["status"][0] == 2 and (got["target"][1:3] == -5).all() and got["accept_len"][1] == 0 and got["accept_len"][2] == 0


def test_greedy_requests_agree_with_greedy_acceptance(hy):
    from speculative_decode_gateddeltanet_gb300 import gdn

    case = sample_case(16, 4, 4096, BF16, seed=8, ties=True)
    got = run_sample(hy, dict(case, temperature=torch.zeros(16)))
    target = torch.full((16, 4), -5, dtype=torch.int32, device="cuda")
    acc = torch.empty(16, dtype=torch.int32, device="cuda")
    gdn.greedy_accept(case["logits"].cuda(), case["drafts"].cuda(), case["n_rows"].cuda(), target, acc)
    assert np.array_equal(target.cpu().numpy(), got["target"]) and np.array_equal(acc.cpu().numpy(), got["accept_len"])


def test_sampled_shares_follow_the_weights(hy):
    """Evenly spaced random numbers draw every token in proportion to its weight, to one draw."""
    w = np.array([0.4, 0.1, 0.25, 0.05, 0.2])
    B, R = 100, 100
    logits = torch.tensor(np.log(w), dtype=F32, device="cuda").expand(B, R, 5).contiguous()
    u = ((torch.arange(B * R, dtype=torch.float64) + 0.5) / (B * R)).float().reshape(B, R).cuda()
    target = torch.zeros((B, R), dtype=torch.int32, device="cuda")
    hy.gdn_sample_accept(hy.make_sample_accept_args(logits=logits, u=u, n_rows=torch.full((B,), R, dtype=torch.int32, device="cuda"), target=target))
    torch.cuda.synchronize()
    assert np.abs(np.bincount(target.cpu().numpy().ravel(), minlength=5) - w * B * R).max() <= 1


# ---- together ------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_step_chained_on_one_stream_and_in_a_graph(hy, dtype):
    """Page map, append and attention back to back with no synchronisation, eager and as one captured graph: the
    attention sees what the two before it wrote."""
    B, R, P, Hq, H, d = 5, 4, 16, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    ctx, n = np.array([0, 17, 31, 100, 64]), np.array([4, 1, 4, 0, 3])
    held = -(-ctx // P)
    N = 40
    ids = np.random.default_rng(0).permutation(N)
    table = np.full((B, 9), -1)
    table[np.arange(9) < held[:, None]] = ids[:held.sum()]
    ring = np.concatenate([ids[held.sum():], np.zeros(held.sum(), int)])
    pool = torch.randn((N, 2, H, P, d), device="cuda", generator=g).to(dtype)
    x = torch.randn((B * R, Hq + 2 * H, d), device="cuda", generator=g).to(dtype)
    new = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dict(ctx_len=ints(ctx), n_rows=ints(n), held=ints(held), free_ring=ints(ring), free_state=ints([0, N - held.sum()]),
             block_table=ints(table), held_out=new(B), free_state_out=new(2), rows_out=new(B), row_start=new(B + 1), slot_map=new(B * R))
    o = torch.full((B * R, Hq, d), 7.0, device="cuda", dtype=dtype)
    maps = hy.make_page_map_args(**t, page_size=P, R=R)
    app = hy.make_kv_append_args(k=x[:, Hq:Hq + H], v=x[:, Hq + H:], slot_map=t["slot_map"], k_cache=pool[:, 0], v_cache=pool[:, 1])
    att = hy.make_paged_attention_args(q=x[:, :Hq], k_cache=pool[:, 0], v_cache=pool[:, 1], block_table=t["block_table"],
                                       ctx_len=t["ctx_len"], n_rows=t["rows_out"], row_start=t["row_start"], o=o)
    work = torch.empty(hy.paged_attention_work_bytes(att), dtype=torch.uint8, device="cuda")
    att.work = work.data_ptr()

    def step():
        hy.gdn_page_map(maps)
        hy.gdn_kv_append(app)
        hy.gdn_paged_attention(att)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    case = dict(q=x[:, :Hq], k_cache=pool[:, 0], v_cache=pool[:, 1], table=t["block_table"].cpu().numpy(), ctx=ctx, n=n,
                start=np.arange(B) * R, scale=d ** -0.5)
    slots = t["slot_map"].cpu().numpy()
    for r in range(B * R):
        if slots[r] >= 0:
            assert torch.equal(pool[slots[r] // P, 0, :, slots[r] % P], x[r, Hq:Hq + H])
    assert (slots >= 0).sum() == n.sum()
    check_attention(case, o)
    first = o.clone()
    o.fill_(7.0)
    step()
    torch.cuda.synchronize()
    assert torch.equal(first, o)
