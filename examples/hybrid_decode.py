"""Speculative decoding of a toy hybrid: one GatedDeltaNet layer and one full-attention
layer over a paged cache, random weights, everything decided on the device.

    python examples/hybrid_decode.py [--drafts 3] [--steps 64] [--temperature 0.0] [--budget 0]

One step verifies the rows [pending, d1..dk] of every request:

  gdn_verify_deferred   the GatedDeltaNet layer, committing the step before from its carry
  gdn_page_map          pages, slots and positions of the rows from the request lengths
  gdn_kv_append         the rows' K and V to those slots
  gdn_paged_attention   the rows over their requests' pages
  gdn_sample_accept     the target's sampled tokens, and how many drafts they confirm

With a budget the attention layer's cache keeps at most so many tokens of a request:

  gdn_shared_attention  in place of gdn_paged_attention: it also gives each row's log sum of exponentials
  gdn_attn_weight       what the accepted rows gave to each cached token
  gdn_evict_select      the lightest tokens beyond the budget leave, but for a request's first ones and its latest
  gdn_kv_move           K and V of the tokens that take their places

The projections between them are plain matrix products.  Drafts come from a table of the last
seen successor of each token.  No step reads anything back to the host.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decode_gateddeltanet_gb300 import gdn, hybrid  # noqa: E402

V, D = 512, 256                             # vocabulary, model width
H_QK, H_V, D_K, D_V, W = 2, 4, 64, 64, 4    # GatedDeltaNet layer
H_Q, H_KV, D_H, PAGE = 8, 2, 64, 16         # attention layer
C = 2 * H_QK * D_K + H_V * D_V


def i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


class Model:
    def __init__(self, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        w = lambda i, o: (torch.randn(i, o, generator=g) * i ** -0.5).to("cuda", dtype)  # noqa: E731
        self.dtype = dtype
        self.emb, self.out = torch.randn(V, D, generator=g).to("cuda", dtype), w(D, V)
        self.x, self.gate, self.o1 = w(D, C), w(D, 2 * H_V), w(H_V * D_V, D)
        self.qkv, self.o2 = w(D, (H_Q + 2 * H_KV) * D_H), w(H_Q * D_H, D)
        self.conv = (torch.randn(C, W, generator=g) * 0.5).to("cuda", dtype)
        self.A_log = torch.rand(H_V, generator=g).cuda()


class Decoder:
    """Caches and call arguments of B requests, each starting from one token."""

    def __init__(self, model: Model, first, drafts: int, pages: int = 512, temperature=0.0, seed=0, budget: int = 0):
        self.m, self.k, self.B, self.R, self.budget = model, drafts, len(first), drafts + 1, budget
        B, R, dt = self.B, self.R, model.dtype
        self.rng = torch.Generator(device="cuda").manual_seed(seed)
        self.pending = torch.tensor(first, dtype=torch.int32, device="cuda")
        self.guess = torch.zeros(V, dtype=torch.int32, device="cuda")
        self.n_rows, self.status = i32(B, fill=R), i32(1)
        self.temperature = torch.full((B,), float(temperature), device="cuda")
        self.target, self.accept_len = i32(B, R), [i32(B), i32(B)]
        # GatedDeltaNet layer: states, and rows and carries for two steps in turn
        self.state = torch.zeros((B, H_V, D_V, D_K), device="cuda")
        self.window = torch.zeros((B, C, W - 1), device="cuda", dtype=dt)
        self.slots = torch.arange(B, dtype=torch.int32, device="cuda")
        self.o1 = torch.zeros((B, R, H_V, D_V), device="cuda")
        self.x = [torch.zeros((B, R, C), device="cuda", dtype=dt) for _ in range(2)]
        args = self.gdn_args(0, self.x[0], None, None, None)
        self.gdn_work = torch.empty(gdn.work_bytes(args) // 4, device="cuda")
        self.carry = [torch.empty(gdn.carry_bytes(args) // 4, device="cuda") for _ in range(2)]
        # attention layer: the pool, its free ring (all pages), tables and two turns of the counts
        self.pool = torch.zeros((pages, 2, H_KV, PAGE, D_H), device="cuda", dtype=dt)
        self.ctx = i32(B)
        self.ring = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.free = [torch.tensor([0, pages], dtype=torch.int32, device="cuda"), i32(2)]
        self.held = [i32(B), i32(B)]
        self.table = i32(B, pages // B, fill=-1)
        self.rows, self.starts, self.slot_map, self.positions = i32(B), i32(B + 1), i32(B * R), i32(B * R)
        self.qkv = torch.zeros((B * R, H_Q + 2 * H_KV, D_H), device="cuda", dtype=dt)
        self.o2 = torch.zeros((B * R, H_Q, D_H), device="cuda", dtype=dt)
        self.attn = hybrid.make_paged_attention_args(
            q=self.qkv[:, :H_Q], k_cache=self.pool[:, 0], v_cache=self.pool[:, 1], block_table=self.table, ctx_len=self.ctx,
            n_rows=self.rows, row_start=self.starts, R=R, o=self.o2, status=self.status)
        self.attn_work = torch.empty(hybrid.paged_attention_work_bytes(self.attn), dtype=torch.uint8, device="cuda")
        self.attn.work = self.attn_work.data_ptr()
        self.append = hybrid.make_kv_append_args(k=self.qkv[:, H_Q:H_Q + H_KV], v=self.qkv[:, H_Q + H_KV:], slot_map=self.slot_map,
                                                 k_cache=self.pool[:, 0], v_cache=self.pool[:, 1], status=self.status)
        self.map = [hybrid.make_page_map_args(
            ctx_len=self.ctx, n_rows=self.n_rows, held=self.held[i], free_ring=self.ring, free_state=self.free[i],
            block_table=self.table, held_out=self.held[1 - i], free_state_out=self.free[1 - i], rows_out=self.rows,
            row_start=self.starts, slot_map=self.slot_map, positions=self.positions, page_size=PAGE, R=R, status=self.status)
            for i in range(2)]
        self.steps = 0
        if budget:
            self.make_eviction(pages)

    def make_eviction(self, pages):
        """Arguments of the calls that keep the cache within the budget."""
        B, R = self.B, self.R
        self.text, self.count, self.keep_from = i32(B), i32(B), i32(B)  # tokens of the text, rows that count, ages that stay
        self.lse = torch.zeros((B * R, H_Q), device="cuda")
        self.weight, self.born = torch.zeros(pages * PAGE, device="cuda"), i32(pages * PAGE)
        self.n_moves, self.move_from, self.move_to = i32(B), i32(B, R), i32(B, R)  # a step adds at most R tokens
        self.most, self.pinned = i32(B, fill=self.budget), i32(B, fill=4)
        cache = dict(k_cache=self.pool[:, 0], v_cache=self.pool[:, 1])
        self.shared = hybrid.make_shared_attention_args(
            q=self.qkv[:, :H_Q], **cache, block_table=self.table, ctx_len=self.ctx, n_rows=self.rows, row_start=self.starts, R=R, o=self.o2,
            lse=self.lse, status=self.status)
        self.shared_work = torch.empty(hybrid.shared_attention_work_bytes(self.shared), dtype=torch.uint8, device="cuda")
        self.shared.attn.work = self.shared_work.data_ptr()
        self.weigh = hybrid.make_attn_weight_args(
            q=self.qkv[:, :H_Q], k_cache=self.pool[:, 0], lse=self.lse, block_table=self.table, ctx_len=self.ctx, n_rows=self.count,
            row_start=self.starts, R=R, weight=self.weight, born=self.born, position=self.text, fresh=True, status=self.status)
        self.weigh_work = torch.empty(hybrid.attn_weight_work_bytes(self.weigh), dtype=torch.uint8, device="cuda")
        self.weigh.work = self.weigh_work.data_ptr()
        self.select = hybrid.make_evict_select_args(
            weight=self.weight, born=self.born, block_table=self.table, ctx_len=self.ctx, budget=self.most, ctx_out=self.ctx,
            n_moves=self.n_moves, move_from=self.move_from, move_to=self.move_to, page_size=PAGE, pinned=self.pinned,
            keep_from=self.keep_from, status=self.status)
        self.move = hybrid.make_kv_move_args(**cache, move_from=self.move_from, move_to=self.move_to, n_moves=self.n_moves, status=self.status)

    def evict(self, accept):
        """After a step: the accepted rows' weights, and the tokens beyond the budget out of the cache."""
        torch.add(accept, 1, out=self.count)
        hybrid.gdn_attn_weight(self.weigh)
        self.ctx += self.count
        self.text += self.count
        torch.sub(self.text, self.budget // 2, out=self.keep_from)
        hybrid.gdn_evict_select(self.select)
        hybrid.gdn_kv_move(self.move)

    def gdn_args(self, turn, x, a, b, carry):
        return gdn.make_args(x=x, g=a, beta=b, conv_w=self.m.conv, conv_state=self.window, ssm_state=self.state, slot_ids=self.slots,
                             n_rows=self.n_rows, o=self.o1, work=getattr(self, "gdn_work", None), status=self.status, H_qk=H_QK,
                             A_log=self.m.A_log, carry=carry)

    def step(self):
        """One verify step.  Returns the target's tokens [B][R] and accept lengths [B], on the device: request b's new
        tokens are its first accept_len + 1."""
        m, turn = self.m, self.steps % 2
        drafts, last = [], self.pending
        for _ in range(self.k):
            last = self.guess[last.long()]
            drafts.append(last)
        tokens = torch.stack([self.pending, *drafts], 1)
        drafts = tokens[:, 1:].contiguous()
        h = m.emb[tokens.long()]
        # the GatedDeltaNet layer; the rows of the step before are committed from their carry
        torch.matmul(h, m.x, out=self.x[turn])
        gate = (h @ m.gate).float().reshape(self.B, self.R, 2, H_V)
        a, b = gate[:, :, 0].contiguous(), gate[:, :, 1].contiguous()
        prev = None
        if self.steps:
            prev = gdn.make_prev(x=self.x[1 - turn], n_rows=self.n_rows, accept_len=self.accept_len[1 - turn], carry=self.carry[1 - turn])
        gdn.gdn_verify_deferred(self.gdn_args(turn, self.x[turn], a, b, self.carry[turn]), prev)
        h = h + self.o1.reshape(self.B, self.R, -1).to(m.dtype) @ m.o1
        # the attention layer
        hybrid.gdn_page_map(self.map[turn])
        torch.matmul(h.reshape(self.B * self.R, D), m.qkv, out=self.qkv.reshape(self.B * self.R, -1))
        hybrid.gdn_kv_append(self.append)
        if self.budget:
            hybrid.gdn_shared_attention(self.shared)
        else:
            hybrid.gdn_paged_attention(self.attn)
        h = h + (self.o2.reshape(self.B, self.R, -1) @ m.o2)
        # the target's tokens, and the drafts they confirm
        logits = h @ m.out
        u = torch.rand((self.B, self.R), device="cuda", generator=self.rng)
        accept = self.accept_len[turn]
        hybrid.gdn_sample_accept(hybrid.make_sample_accept_args(
            logits=logits, u=u, n_rows=self.n_rows, target=self.target, drafts=drafts if self.k else None, accept_len=accept,
            temperature=self.temperature, status=self.status))
        target = self.target.clone()
        self.guess.scatter_(0, tokens[:, 0].long(), target[:, 0])
        self.pending = target.gather(1, accept.long()[:, None])[:, 0]
        if self.budget:
            self.evict(accept)
        else:
            self.ctx += accept + 1
        self.steps += 1
        return target, accept.clone()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--budget", type=int, default=0, help="tokens of a request that the attention layer's cache keeps (0: all)")
    a = ap.parse_args()
    dec = Decoder(Model(), list(range(1, a.batch + 1)), a.drafts, temperature=a.temperature, budget=a.budget)
    done = [dec.step() for _ in range(a.steps)]
    torch.cuda.synchronize()
    counts = torch.stack([n + 1 for _, n in done]).float()
    print(f"{a.batch} requests, {a.steps} steps of {a.drafts} drafts: {counts.mean().item():.2f} tokens a step, "
          f"status {int(dec.status.item())}")
    for b in range(a.batch):
        out = [t for target, n in done for t in target[b, :int(n[b]) + 1].tolist()]
        print(f"request {b}: {' '.join(map(str, out[:24]))} ...")


if __name__ == "__main__":
    main()
