"""The pages of a shared prefix through the lives of the requests that hold it: they join, grow, lose
tokens to the budget and end, the one that wrote the prefix among the first.  Every page is in one
place after each page map, the prefix stays as it was, and each request attends to what it holds.
Tolerances are those of test_gpu_long's step by step test."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import long_ref
from test_gpu_long import BF16, F32, always, hy, ints, status_word  # noqa: F401

pytestmark = pytest.mark.gpu

P, LENGTH = 16, 37          # page size; a prefix that ends inside its third page
W = LENGTH // P             # its whole pages, which the requests share
JOIN = {0: 0, 4: 0, 1: 1, 2: 4, 3: 4}  # table row -> step; 4 is in no group
END = {0: 6, 2: 12, 1: 20, 4: 25, 3: 30}
AGAIN = {0: 9, 2: 15}       # rows that serve another request later
END_AGAIN = {0: 27, 2: 18}


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_requests_of_a_prefix_join_grow_and_end(hy, always, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(11)
    B, H_q, H_kv, d, N, ROWS, MOVES, budget, recent = 5, 8, 2, 64, 40, 64, 16, 50, 6
    new = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.full((N, 2, H_kv, P, d), float("nan"), dtype=dtype, device="cuda")
    kc, vc = pool[:, 0], pool[:, 1]
    ring, table = ints(np.random.default_rng(1).permutation(N)), new(B, 8) - 1
    free, held = [ints([3, N]), new(2)], [new(B), new(B)]
    ctx, text, rows, starts, slots, status = new(B), new(B), new(B), new(B + 1), new(ROWS), status_word()
    weight, born = torch.full((N * P,), 5.0, device="cuda"), new(N * P) - 1
    n_moves, lists = new(B), [new(B, MOVES), new(B, MOVES)]
    pinned = ints([LENGTH] * 4 + [2])
    groups = dict(group_start=ints([0, 4]), prefix_len=ints([LENGTH]))
    model, prefix = [[] for _ in range(B)], None  # each request's tokens as (K, V) in cache order
    live, shared, moved, forced = set(), None, 0, 0
    for step in range(32):
        a, b_ = step % 2, 1 - step % 2
        n = torch.randint(0, 4, (B,), generator=g)
        joins = [b for when in (JOIN, AGAIN) for b in when if when[b] == step]
        ends = [b for when in (END, END_AGAIN) for b in when if when[b] == step]
        for b in joins:
            live.add(b)
            if b < 4 and prefix is None:
                n[b] = LENGTH  # the first of the group writes the prefix
                continue
            if b < 4:  # the prefix's whole pages, which it does not get from the page map
                table[b, :W] = ints(shared)
                held[a][b], ctx[b], text[b] = W, LENGTH, LENGTH
                model[b] = list(prefix)
        for b in range(B):
            if b not in live:
                n[b] = 0
        for b in ends:
            n[b] = 0
            live.remove(b)
            others = b < 4 and any(x < 4 for x in live)
            ctx[b] = W * P if others else 0  # what the page map must not see as given back
            model[b] = []
        hy.gdn_page_map(hy.make_page_map_args(
            ctx_len=ctx, n_rows=n.to(torch.int32).cuda(), held=held[a], free_ring=ring, free_state=free[a], block_table=table,
            held_out=held[b_], free_state_out=free[b_], rows_out=rows, row_start=starts, slot_map=slots, page_size=P, R=0, status=status))
        for b in joins:
            if b < 4 and prefix is not None:  # the rest of the prefix into the request's own page
                source = next(x for x in sorted(live) if x < 4 and x not in joins)
                at = torch.arange(LENGTH - W * P, dtype=torch.int32, device="cuda")
                hy.gdn_kv_move(hy.make_kv_move_args(
                    k_cache=kc, v_cache=vc, move_from=(table[source, W] * P + at)[None], move_to=(table[b, W] * P + at)[None],
                    n_moves=(held[b_][b:b + 1] > W).int() * len(at), status=status))  # none where no page was left for it
        for b in ends:
            held[b_][b], ctx[b], text[b] = 0, 0, 0
        torch.cuda.synchronize()
        # every page is in the ring, in one request, or one of the prefix's
        ring_, (head, n_free), tab, count = ring.cpu().numpy(), free[b_].tolist(), table.cpu().numpy(), held[b_].tolist()
        places = [int(ring_[(head + i) % N]) for i in range(n_free)]
        members = [b for b in live if b < 4]
        for b in live:
            places += tab[b, W if b < 4 else 0:count[b]].tolist()
        if members:
            shared = tab[members[0], :W].tolist()
            places += shared
        assert sorted(places) == list(range(N)), step
        assert all(tab[b, :W].tolist() == shared for b in members) and rows.tolist() == n.tolist()
        x = torch.randn((ROWS, H_q + 2 * H_kv, d), generator=g).to(dtype).cuda()
        q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
        hy.gdn_kv_append(hy.make_kv_append_args(k=k, v=v, slot_map=slots, k_cache=kc, v_cache=vc, status=status))
        o, lse = torch.zeros((ROWS, H_q, d), dtype=dtype, device="cuda"), torch.zeros((ROWS, H_q), device="cuda")
        args = hy.make_shared_attention_args(q=q, k_cache=kc, v_cache=vc, block_table=table, ctx_len=ctx, n_rows=rows, row_start=starts,
                                             o=o, lse=lse, status=status, **groups)
        work = torch.empty(hy.shared_attention_work_bytes(args), dtype=torch.uint8, device="cuda")
        args.attn.work = work.data_ptr()
        start = starts.tolist()
        for b in live:
            model[b] += [(k[start[b] + t], v[start[b] + t]) for t in range(int(n[b]))]
        for lib in (None, always):
            o.fill_(7.0)
            if lib is None:
                hy.gdn_shared_attention(args)
            else:
                assert lib.gdn_shared_attention(args, torch.cuda.current_stream().cuda_stream or None) == 0
                forced += len(members) > 1
            torch.cuda.synchronize()
            for b in live:
                m = int(n[b])
                if m == 0:
                    continue
                K, V = (torch.stack([tok[i] for tok in model[b]]).double().repeat_interleave(H_q // H_kv, 1) for i in (0, 1))
                z = torch.einsum("thd,lhd->htl", q[start[b]:start[b] + m].double(), K) * d ** -0.5
                z = z.masked_fill(torch.ones(m, len(model[b]), device="cuda").triu(len(model[b]) - m + 1).bool(), -float("inf"))
                ref = torch.einsum("htl,lhd->thd", torch.softmax(z, 2), V)
                top = V.abs().max()
                off = (o[start[b]:start[b] + m].double() - ref).abs().max()
                assert off <= (2.0 ** -8 * (top + ref.abs().max()) if dtype == BF16 else 0) + 1e-5 * top
            assert (o[start[B]:] == 7.0).all()
        wargs = hy.make_attn_weight_args(q=q, k_cache=kc, lse=lse, block_table=table, ctx_len=ctx, n_rows=rows, row_start=starts, weight=weight,
                                         born=born, position=text, first=pinned, fresh=True, keep=0.9, status=status)
        wwork = torch.empty(hy.attn_weight_work_bytes(wargs), dtype=torch.uint8, device="cuda")
        wargs.work = wwork.data_ptr()
        hy.gdn_attn_weight(wargs)
        ctx += rows
        text += rows
        lens = ctx.cpu().numpy()
        assert lens.tolist() == [len(m) for m in model]
        old_weight, old_born, keep_from = weight.cpu().numpy(), born.cpu().numpy(), text - recent
        hy.gdn_evict_select(hy.make_evict_select_args(
            weight=weight, born=born, block_table=table, ctx_len=ctx, budget=ints([budget] * B), ctx_out=ctx, n_moves=n_moves,
            move_from=lists[0], move_to=lists[1], page_size=P, pinned=pinned, keep_from=keep_from, status=status))
        hy.gdn_kv_move(hy.make_kv_move_args(k_cache=kc, v_cache=vc, move_from=lists[0], move_to=lists[1], n_moves=n_moves, status=status))
        torch.cuda.synchronize()
        want = long_ref.select(old_weight, old_born, tab, lens, np.array([budget] * B), pinned.cpu().numpy(), keep_from.cpu().numpy(), P, MOVES,
                               N, [np.zeros((B, MOVES), int)] * 2)
        assert ctx.tolist() == want["ctx_out"].tolist() and n_moves.tolist() == want["n_moves"].tolist()
        for b in range(B):
            where = {tab[b, j // P] * P + j % P: j for j in range(lens[b])}
            for i in range(int(want["n_moves"][b])):
                model[b][where[want["move_to"][b, i]]] = model[b][where[want["move_from"][b, i]]]
                moved += 1
            del model[b][int(want["ctx_out"][b]):]
        if prefix is None:
            prefix = model[0][:LENGTH]
            before = pool[shared].clone()
        if members:  # neither the weights nor the cache of the prefix's pages were touched
            assert torch.equal(pool[shared].view(torch.int16), before.view(torch.int16))
            assert (weight.view(N, P)[shared] == 5.0).all()
        assert int(status.item()) == 0
    assert not live and moved > 10 and forced > 20
    assert free[b_].tolist()[1] == N and sorted(ring.tolist()) == list(range(N))
