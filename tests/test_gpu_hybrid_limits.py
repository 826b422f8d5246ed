"""Calls of the hybrid-step operators at the ends of what they take."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import hybrid_ref
import test_gpu_hybrid as base
from test_gpu_hybrid import BF16, F32, ints

pytestmark = pytest.mark.gpu
hy = base.hy  # the module-wide fixture

# ---- page map ------------------------------------------------------------------

FRESH = """
import numpy as np, hybrid_ref, test_gpu_hybrid as base
from speculative_decode_gateddeltanet_gb300 import hybrid
for B in (2031, 2032, 2040, 2047, 2048):
    case = base.page_case(B, 16, 2, B)
    got = base.run_page_map(hybrid, *case)
    for key, want in hybrid_ref.page_map(*case).items():
        assert np.array_equal(got[key], want), (B, key)
"""


def test_page_map_batches_around_the_default_shared_memory_limit():
    """In a process of its own: a larger call before them would have raised the limit for good."""
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([os.path.dirname(here), here, os.environ.get("PYTHONPATH", "")])
    run = subprocess.run([sys.executable, "-c", FRESH], env=dict(os.environ, PYTHONPATH=path), capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


@pytest.mark.parametrize("arrays", [(), ("positions",)], ids=["none", "positions"])
def test_packed_page_map_without_row_arrays_serves_every_request(hy, arrays):
    ctx, n, held, ring, free, table, P, R, rows = base.page_case(40, 16, 0, 3)
    ref = hybrid_ref.page_map(ctx, n, held, ring, free, table, P, R, rows)
    t = dict(ctx_len=ints(ctx), n_rows=ints(n), held=ints(held), free_ring=ints(ring), free_state=ints(free), block_table=ints(table))
    new = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    out = dict(held_out=new(40), free_state_out=new(2), rows_out=new(40), row_start=new(41), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    out |= {name: new(rows) for name in arrays}
    hy.gdn_page_map(hy.make_page_map_args(**t, **out, page_size=P, R=R))
    torch.cuda.synchronize()
    assert int(out["status"].item()) == 0 and ref["status"] == 0
    for key in ("held_out", "rows_out", "row_start", *arrays):
        assert np.array_equal(out[key].cpu().numpy(), ref[key]), key
    assert np.array_equal(t["block_table"].cpu().numpy(), ref["table"])


@pytest.mark.parametrize("R", [0, 4])
def test_empty_page_map_hands_the_counts_on(hy, R):
    """A step without requests is a turn of the two copies of the counts like any other."""
    new = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = 0 if R else 5
    out = dict(held_out=new(0), free_state_out=new(2), rows_out=new(0), row_start=new(1), slot_map=new(rows), positions=new(rows), status=new(1))
    out["status"].zero_()
    ring = ints(np.arange(20)[::-1].copy())
    free = ints([17, 9])
    hy.gdn_page_map(hy.make_page_map_args(ctx_len=new(0), n_rows=new(0), held=new(0), free_ring=ring, free_state=free,
                                          block_table=new(0, 6), **out, page_size=16, R=R))
    torch.cuda.synchronize()
    assert out["free_state_out"].tolist() == [17, 9] and out["row_start"].tolist() == [0] and int(out["status"].item()) == 0
    assert out["slot_map"].tolist() == out["positions"].tolist() == [-1] * rows
    assert ring.tolist() == list(range(19, -1, -1))


def test_page_map_returns_no_more_pages_than_there_are(hy):
    """Counts that do not add up: every request holds all pages and needs none.  Their sum passes 2^32; the ring takes
    one turn, and nothing outside it or the tables is touched."""
    B, N = 4096, 1 << 20
    table = torch.arange(N, dtype=torch.int32, device="cuda")  # row 0; no other row is read
    store = torch.full((N + 64,), -9, dtype=torch.int32, device="cuda")
    new = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    out = dict(held_out=new(B), free_state_out=new(2), rows_out=new(B), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    zero, held, free = ints(np.zeros(B)), ints(np.full(B, N)), ints([5, 0])
    args = hy.make_page_map_args(ctx_len=zero, n_rows=zero, held=held, free_ring=store[:N], free_state=free,
                                 block_table=table[:4].expand(B, 4), **out, page_size=16, R=1)
    args.max_pages = args.table_stride = N
    hy.gdn_page_map(args)
    torch.cuda.synchronize()
    assert out["free_state_out"].tolist() == [5, N] and int(out["held_out"].max().item()) == 0
    assert torch.equal(store[:N].roll(-5), table) and bool((store[N:] == -9).all())


@pytest.mark.parametrize("B,R", [(3, 0), (4096, 524287)], ids=["packed", "padded"])
def test_page_map_of_almost_2_31_rows(hy, B, R):
    """A slot array that ends within one step of the blocks of 2^31: 8.6 GB."""
    rows = B * R if R else 2**31 - 1
    ctx, n = np.zeros(B, np.int64), np.zeros(B, np.int64)
    ctx[:3], n[:3] = (5, 0, 31), (2, 1, 4)
    held = -(-ctx // 16)
    ids = np.arange(40)[::-1].copy()
    table = np.full((B, 4), -1)
    table[np.arange(4) < held[:, None]] = ids[:held.sum()]
    ring = np.concatenate([ids[held.sum():], np.zeros(held.sum(), np.int64)])
    free = [0, 40 - held.sum()]
    # the plain form at a width it can hold: a request's rows stand at the front of its own
    ref = hybrid_ref.page_map(ctx, n, held, ring, free, table, 16, 4 if R else 0, 4 * B if R else 16)
    slots = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    new = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dict(ctx_len=ints(ctx), n_rows=ints(n), held=ints(held), free_ring=ints(ring), free_state=ints(free), block_table=ints(table))
    out = dict(held_out=new(B), free_state_out=new(2), rows_out=new(B), row_start=new(B + 1), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    hy.gdn_page_map(hy.make_page_map_args(**t, **out, slot_map=slots, page_size=16, R=R))
    torch.cuda.synchronize()
    assert int(out["status"].item()) == 0 and np.array_equal(out["rows_out"].cpu().numpy(), n)
    assert out["free_state_out"].tolist() == ref["free_out"].tolist()
    if R:
        for b in range(3):
            assert slots[b * R:b * R + 4].tolist() == ref["slot_map"][4 * b:4 * b + 4].tolist()
            slots[b * R:b * R + 4] = -1
    else:
        assert slots[:16].tolist() == ref["slot_map"].tolist()
        slots[:16] = -1
    assert int(slots.max().item()) == int(slots.min().item()) == -1


def test_page_map_refuses_more_pages_than_there_are(hy):
    """Counts above the pool's pages, and lengths above its tokens (with a position past 2^31 among them), in table rows
    wide enough for both.  The widest are so by their stride alone: a call that used one would read out of range."""
    new = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    for ctx, n, held, want in (([3, 40], [2, 1], [1, 65], 64), ([2**31 - 4], [8], [2**27], 64), ([2**31 - 4], [8], [60], 32),
                               ([64 * 16 - 1], [2], [63], 32)):
        B = len(ctx)
        table = ints(np.arange(B * 70).reshape(B, 70) % 64)
        ring = ints(np.arange(64))
        lengths = dict(ctx_len=ints(ctx), n_rows=ints(n), held=ints(held), free_state=ints([3, 64]))
        out = dict(held_out=new(B), free_state_out=new(2), rows_out=new(B), row_start=new(B + 1), slot_map=new(B * 8), positions=new(B * 8),
                   status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        before = table.clone()
        args = hy.make_page_map_args(**lengths, free_ring=ring, block_table=table, **out, page_size=16, R=8)
        if B == 1:
            args.max_pages = args.table_stride = 2**27 + 1
        hy.gdn_page_map(args)
        torch.cuda.synchronize()
        assert int(out["status"].item()) == want
        assert out["rows_out"].tolist() == ([2, 0] if B == 2 else [0]) and out["held_out"].tolist() == held
        assert out["free_state_out"].tolist() == [3, 64] and torch.equal(table, before) and ring.tolist() == list(range(64))
        assert int((out["slot_map"] >= 0).sum()) == (2 if B == 2 else 0)


# ---- sampling ------------------------------------------------------------------


@pytest.mark.parametrize("R", [1, 3])
def test_sampling_without_accept_lengths_flags_a_bad_row_count(hy, R):
    for bad in (R + 1, -1):
        case = base.sample_case(3, R, 100, F32, seed=1)
        case["n_rows"] = torch.tensor([R, bad, 1], dtype=torch.int32)
        dev = {k: v.cuda() for k, v in case.items() if k != "drafts"}
        target, status = torch.full((3, R), -5, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        hy.gdn_sample_accept(hy.make_sample_accept_args(**dev, target=target, status=status))
        torch.cuda.synchronize()
        assert int(status.item()) == 2
        assert (target[1] == -5).all() and int(target[0].min()) >= 0 and int(target[2, 0]) >= 0


# ---- attention -----------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ctx,n", [(2**31 - 2, 1), (2**31 - 1, 1), (2**31 - 1000, 7), (0, 2**31 // 128), (0, 2**31 - 5)])
def test_attention_of_numbers_past_32_bits_is_flagged(hy, dtype, ctx, n):
    """Positions up to 2^31, and rows (tokens times query heads of a kv head) of as many, in a table row and a q that are
    wide enough by their sizes alone: the request is skipped with its bit, the one beside it is served."""
    case = hybrid_ref.make_attention(lens=[(20, 2), (30, 2)], H_q=128, H_kv=1, d=64, P=16, dtype=dtype, seed=4)
    good = base.run_attention(hy, dict(case, n=np.array([2, 0])))
    q, k, v = (case[x].cuda() for x in ("q", "k_cache", "v_cache"))
    out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    t = dict(block_table=ints(case["table"]), ctx_len=ints([20, ctx]), n_rows=ints([2, n]), row_start=ints([0, 0]))
    args = hy.make_paged_attention_args(q=q, k_cache=k, v_cache=v, **t, o=out, scale=case["scale"], status=status)
    args.max_pages = args.table_stride = 2**27 + 100  # the second row is never read
    args.n_q_rows = 2**31 - 1
    work = torch.empty(hy.paged_attention_work_bytes(args), dtype=torch.uint8, device="cuda")
    args.work = work.data_ptr()
    hy.gdn_paged_attention(args)
    torch.cuda.synchronize()
    assert int(status.item()) == 256
    assert torch.equal(out[:2], good[:2]) and bool((out[2:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 1e-37, -1e-37, 2e-39])
def test_attention_with_scales_near_zero(hy, dtype, scale):
    """Scores of 1e37 times these scales are moderate numbers, or 0: every key counts.  A 32-bit sum of 64 products of
    some 1e36 is off by at most 64 * 2^-24 of 1e38, 4e-5 in the exponent here; a denormal scale of 2e-39 is one of 1.4e6
    steps, and 3e-7 off in itself."""
    case = hybrid_ref.make_attention(lens=[(300, 3), (0, 20)], H_q=4, H_kv=2, d=64, P=16, dtype=dtype, seed=6, scale=scale)
    case["q"] = case["q"] * 1e18
    case["k_cache"].mul_(1e18)
    o = base.run_attention(hy, case).double().cpu().numpy()
    ref, vmax = hybrid_ref.attention(*(case[k] for k in ("q", "k_cache", "v_cache", "table", "ctx", "n", "start", "scale")))
    tol = (2.0**-9 if dtype == BF16 else 0.0) * (vmax[..., None] + np.abs(ref)) + 1e-3 * vmax[..., None]
    assert (np.abs(o - ref) <= tol).all()
