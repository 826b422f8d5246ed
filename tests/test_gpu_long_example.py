"""The example's decode loop with a budget: the cache stays within it, and nothing changes before it is reached."""
from __future__ import annotations

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_decode

    return hybrid_decode


def run(example, dtype, budget, drafts, steps):
    dec = example.Decoder(example.Model(dtype), list(range(1, 6)), drafts, budget=budget)
    done = [dec.step() for _ in range(steps)]
    torch.cuda.synchronize()
    assert int(dec.status.item()) == 0
    return dec, [[t for target, n in done for t in target[b, :int(n[b]) + 1].tolist()] for b in range(5)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_cache_stays_within_its_budget(example, dtype):
    dec, out = run(example, dtype, 24, 3, 50)
    lengths = torch.tensor([len(o) for o in out])
    assert dec.text.tolist() == lengths.tolist()
    assert dec.ctx.tolist() == lengths.clamp(max=24).tolist() and min(lengths) >= 50
    slots = [[int(dec.table[b, j // 16]) * 16 + j % 16 for j in range(int(dec.ctx[b]))] for b in range(5)]
    for b, at in enumerate(slots):
        ages = dec.born[at].tolist()
        n = int(lengths[b])
        assert len(set(ages)) == len(ages) and ages[:4] == [0, 1, 2, 3]           # pinned tokens stay where they are
        assert set(range(n - 12, n)) <= set(ages)                               # and the latest ones stay
        assert torch.isfinite(dec.weight[at]).all() and (dec.weight[at] >= 0).all()
    held, (head, free) = dec.held[dec.steps % 2].tolist(), dec.free[dec.steps % 2].tolist()
    pages = [p for b, h in enumerate(held) for p in dec.table[b, :h].tolist()]
    pages += [int(dec.ring[(head + i) % 512]) for i in range(free)]
    assert sorted(pages) == list(range(512))


def test_a_budget_that_is_not_reached_changes_nothing(example):
    _, plain = run(example, torch.float32, 0, 3, 20)
    dec, kept = run(example, torch.float32, 400, 3, 20)
    assert kept == plain and int(dec.n_moves.sum()) == 0
