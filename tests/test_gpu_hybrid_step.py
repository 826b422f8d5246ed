"""The hybrid-step operators as one step: captured in a graph with the sampled acceptance among them, called from several
host threads at once, and in the example's loop with sampling in bf16."""
from __future__ import annotations

import os
import sys
import threading

import numpy as np
import pytest
import torch

import test_gpu_hybrid as base
from test_gpu_hybrid import BF16, F32, ints

pytestmark = pytest.mark.gpu
hy = base.hy  # the module-wide fixture
B, R, P, H_Q, H_KV, D, V, N = 6, 4, 16, 8, 2, 128, 1000, 60


class Step:
    """Buffers and arguments of one step of all four calls; its inputs are drawn anew in place."""

    def __init__(self, hy, dtype, seed):
        self.hy, self.g = hy, torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s, fill=0: torch.full(s, fill, dtype=torch.int32, device="cuda")  # noqa: E731
        ctx = np.array([0, 17, 31, 100, 64, 5]) + seed
        held = -(-ctx // P)
        ids = np.random.default_rng(seed).permutation(N)
        table = np.full((B, 10), -1)
        table[np.arange(10) < held[:, None]] = ids[:held.sum()]
        self.start = dict(block_table=ints(table), free_ring=ints(np.concatenate([ids[held.sum():], np.zeros(held.sum(), int)])))
        self.t = dict(ctx_len=ints(ctx), n_rows=ints([4, 1, 4, 0, 3, 2]), held=ints(held), free_state=ints([0, N - held.sum()]),
                      **{k: v.clone() for k, v in self.start.items()}, held_out=new(B), free_state_out=new(2), rows_out=new(B),
                      row_start=new(B + 1), slot_map=new(B * R), positions=new(B * R))
        self.pool = torch.randn((N, 2, H_KV, P, D), device="cuda", generator=self.g).to(dtype)
        self.x = torch.zeros((B * R, H_Q + 2 * H_KV, D), device="cuda", dtype=dtype)
        self.o = torch.zeros((B * R, H_Q, D), device="cuda", dtype=dtype)
        self.w = (torch.randn((H_Q * D, V), device="cuda", generator=self.g) * 0.1).to(dtype)
        self.logits = torch.zeros((B * R, V), device="cuda", dtype=dtype)
        self.s = dict(u=torch.zeros((B, R), device="cuda"), temperature=torch.tensor([0.7, 0.0, 1.0, 1.0, 1.3, 0.9], device="cuda"),
                      top_k=ints([40, 0, 0, 7, 900, 0]), top_p=torch.tensor([0.9, 1.0, 0.8, 1.0, 0.95, 1.0], device="cuda"),
                      drafts=new(B, R - 1))
        self.out = dict(target=new(B, R, fill=-5), prob=torch.zeros((B, R), device="cuda"), accept_len=new(B, fill=-5), status=new(1))
        self.map = hy.make_page_map_args(**self.t, page_size=P, R=R, status=self.out["status"])
        self.append = hy.make_kv_append_args(k=self.x[:, H_Q:H_Q + H_KV], v=self.x[:, H_Q + H_KV:], slot_map=self.t["slot_map"],
                                             k_cache=self.pool[:, 0], v_cache=self.pool[:, 1])
        self.attend = hy.make_paged_attention_args(
            q=self.x[:, :H_Q], k_cache=self.pool[:, 0], v_cache=self.pool[:, 1], block_table=self.t["block_table"],
            ctx_len=self.t["ctx_len"], n_rows=self.t["rows_out"], row_start=self.t["row_start"], R=R, o=self.o, status=self.out["status"])
        self.work = torch.empty(hy.paged_attention_work_bytes(self.attend), dtype=torch.uint8, device="cuda")
        self.attend.work = self.work.data_ptr()
        self.sample = hy.make_sample_accept_args(logits=self.logits.reshape(B, R, V), n_rows=self.t["rows_out"], **self.s, **self.out)

    def draw(self):
        """New inputs of one step; the tables as they were."""
        for name, t in self.start.items():
            self.t[name].copy_(t)
        self.x.normal_(generator=self.g)
        self.s["u"].uniform_(generator=self.g)
        self.s["drafts"].random_(0, V, generator=self.g)

    def run(self):
        self.hy.gdn_page_map(self.map)
        self.hy.gdn_kv_append(self.append)
        self.hy.gdn_paged_attention(self.attend)
        torch.matmul(self.o.reshape(B * R, -1), self.w, out=self.logits)
        self.hy.gdn_sample_accept(self.sample)

    def results(self):
        names = ("block_table", "free_ring", "held_out", "free_state_out", "rows_out", "slot_map")
        return [t.clone() for t in (self.pool, self.o, self.logits, *self.out.values(), *(self.t[n] for n in names))]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_captured_step_with_sampling(hy, dtype):
    """The step with its sampled acceptance as one graph: what eager calls give, for every replay's inputs, and the tokens
    that the definition draws from its logits."""
    step = Step(hy, dtype, 1)
    step.draw()
    step.run()  # loads the product's library before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for _ in range(3):
        step.draw()
        graph.replay()
        torch.cuda.synchronize()
        got = step.results()
        for name, t in step.start.items():
            step.t[name].copy_(t)
        step.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step.results()))
        assert int(step.out["status"].item()) == 0
        n, par = step.t["n_rows"].tolist(), {k: step.s[k].tolist() for k in ("temperature", "top_k", "top_p")}
        target = step.out["target"].tolist()
        for b in range(B):
            for t in range(n[b]):
                assert target[b][t] == base.whole_number_token(step.logits[b * R + t], *(par[k][b] for k in par), 0.0, step.s["u"][b, t].item())
            drafts, a = step.s["drafts"][b].tolist(), 0
            while a < n[b] - 1 and drafts[a] == target[b][a]:
                a += 1
            assert int(step.out["accept_len"][b]) == a


def test_steps_of_four_host_threads(hy):
    """Four threads, each with buffers and a stream of its own, give what one thread alone gives."""
    steps = [Step(hy, (BF16, F32)[i % 2], i) for i in range(4)]
    torch.cuda.synchronize()
    rounds, failed = 12, []

    def work(step, out):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(rounds):
                    step.draw()
                    step.run()
                    out.append(step.results())
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    together = [[] for _ in steps]
    threads = [threading.Thread(target=work, args=(s, o)) for s, o in zip(steps, together)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for i, first in enumerate(together):
        alone, step = [], Step(hy, (BF16, F32)[i % 2], i)
        torch.cuda.synchronize()
        work(step, alone)
        assert not failed and len(alone) == len(first) == rounds
        for a, b in zip(first, alone):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_the_example_in_bf16(hy, temperature):
    """Every step accepts what its tokens confirm, contexts grow by what was accepted, and every page is in one table row
    or free."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_decode as example

    dec = example.Decoder(example.Model(), [3, 1, 4, 1, 5], 3, temperature=temperature)
    done = [dec.step() for _ in range(40)]
    torch.cuda.synchronize()
    assert int(dec.status.item()) == 0
    accepted = torch.stack([n for _, n in done])
    assert int(accepted.min()) >= 0 and int(accepted.max()) <= 3
    assert dec.ctx.tolist() == (accepted + 1).sum(0).tolist()
    assert all(0 <= int(t.min()) and int(t.max()) < example.V for t, _ in done)
    held, (head, free) = dec.held[dec.steps % 2].tolist(), dec.free[dec.steps % 2].tolist()
    pages = [p for b, h in enumerate(held) for p in dec.table[b, :h].tolist()]
    pages += [int(dec.ring[(head + i) % 512]) for i in range(free)]
    assert sorted(pages) == list(range(512))
