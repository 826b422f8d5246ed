"""The long-context calls at the largest batch that may share, and their chain captured in a graph.
Tolerances are those of test_gpu_long; the captured chain gives the eager one's bits."""
from __future__ import annotations

import pytest
import torch

import long_ref
from test_gpu_long import BF16, F32, Shared, always, hy, ints, status_word  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 256), (F32, 64), (F32, 256)])
def test_the_most_requests_and_groups(hy, always, dtype, d):  # noqa: F811
    groups = [(17 + g % 5, [(i % 3, 1) for i in range(8)]) for g in range(512)]
    case = long_ref.make_shared(groups=groups, alone=[], H_q=2, H_kv=1, d=d, P=16, dtype=dtype, R=1)
    s = Shared(hy, case, 1)
    assert s.args.attn.B == 4096 and s.args.n_groups == 512
    s.run().check()
    s.again(always).check()


class Chain:
    """A layer's cache of three requests: attention, weights, the choice and its moves, one after the other."""

    def __init__(self, hy, dtype, pages_a_request):  # noqa: F811
        g = torch.Generator().manual_seed(5)
        B, R, P, H_q, H_kv, d, N = 3, 2, 16, 4, 2, 64, 64
        new = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.hy = hy
        self.pool = torch.randn((N, 2, H_kv, P, d), generator=g).to(dtype).cuda()
        self.q = torch.randn((B * R, H_q, d), generator=g).to(dtype).cuda()
        self.table = torch.full((B, pages_a_request), -1, dtype=torch.int32, device="cuda")
        self.table[:, :20] = torch.randperm(N, generator=g)[:60].reshape(3, 20).to(torch.int32).cuda()
        self.ctx, self.n, self.text = ints([300, 17, 64]), ints([2, 1, 0]), ints([300, 17, 64])
        self.weight, self.born = torch.rand(N * P, generator=g).cuda(), torch.randint(0, 300, (N * P,), generator=g).to(torch.int32).cuda()
        self.budget, self.pinned, self.keep_from = ints([250, 16, 64]), ints([3, 0, 1]), ints([280, 400, 64])
        self.n_moves, self.lists = new(B), [new(B, 64), new(B, 64)]
        self.o, self.lse, self.status = torch.zeros_like(self.q), torch.zeros((B * R, H_q), device="cuda"), status_word()
        cache = dict(k_cache=self.pool[:, 0], v_cache=self.pool[:, 1])
        step = dict(block_table=self.table, ctx_len=self.ctx, n_rows=self.n, R=R, status=self.status)
        self.attend = hy.make_shared_attention_args(q=self.q, **cache, **step, o=self.o, lse=self.lse)
        self.weigh = hy.make_attn_weight_args(q=self.q, k_cache=self.pool[:, 0], lse=self.lse, **step, weight=self.weight, born=self.born,
                                              position=self.text, fresh=True, keep=0.5)
        self.works = [torch.empty(b, dtype=torch.uint8, device="cuda")
                      for b in (hy.shared_attention_work_bytes(self.attend), hy.attn_weight_work_bytes(self.weigh))]
        self.attend.attn.work, self.weigh.work = (w.data_ptr() for w in self.works)
        self.choose = hy.make_evict_select_args(
            weight=self.weight, born=self.born, block_table=self.table, ctx_len=self.ctx, budget=self.budget, ctx_out=self.ctx,
            n_moves=self.n_moves, move_from=self.lists[0], move_to=self.lists[1], page_size=P, pinned=self.pinned, keep_from=self.keep_from,
            status=self.status)
        self.move = hy.make_kv_move_args(**cache, move_from=self.lists[0], move_to=self.lists[1], n_moves=self.n_moves, status=self.status)

    def step(self):
        self.hy.gdn_shared_attention(self.attend)
        self.hy.gdn_attn_weight(self.weigh)
        self.ctx.add_(self.n)
        self.text.add_(self.n)
        self.keep_from.add_(self.n)
        self.hy.gdn_evict_select(self.choose)
        self.hy.gdn_kv_move(self.move)

    def all(self):
        return [self.pool, self.ctx, self.text, self.weight, self.born, self.n_moves, self.o, self.lse, self.status]


@pytest.mark.parametrize("dtype,pages", [(BF16, 20), (F32, 20), (BF16, 2000)])  # 2000 pages: the choice by clusters
def test_the_chain_in_a_graph_gives_the_eager_chains_bits(hy, dtype, pages):  # noqa: F811
    a, b = Chain(hy, dtype, pages), Chain(hy, dtype, pages)
    start = [x.clone() for x in b.all()]
    keep = b.keep_from.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        b.step()  # before the capture, so that nothing is loaded within it
        with torch.cuda.graph(graph, stream=stream):
            b.step()
        for x, y in zip(b.all() + [b.keep_from], start + [keep]):
            x.copy_(y)
    torch.cuda.current_stream().wait_stream(stream)
    moved = 0
    for _ in range(4):
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.all(), b.all()):
            assert torch.equal(x, y)
        moved += int(a.n_moves.sum())
    assert int(a.status.item()) == 0 and moved > 0 and a.ctx.tolist() == [250, 16, 64]
