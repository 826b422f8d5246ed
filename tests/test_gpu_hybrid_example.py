"""The example's decode loop: drafts change how fast tokens come, not which."""
from __future__ import annotations

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


def tokens(example, drafts, steps, batch=5, **kw):
    dec = example.Decoder(example.Model(torch.float32), list(range(1, batch + 1)), drafts, **kw)
    done = [dec.step() for _ in range(steps)]
    torch.cuda.synchronize()
    assert int(dec.status.item()) == 0
    out = [[t for target, n in done for t in target[b, :int(n[b]) + 1].tolist()] for b in range(batch)]
    assert [len(o) for o in out] == dec.ctx.tolist()
    return out, dec


def test_speculative_and_single_token_decoding_agree(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_decode as example

    one, _ = tokens(example, 0, 60)
    many, dec = tokens(example, 3, 40)
    assert sum(map(len, many)) > 5 * 40  # some drafts were accepted
    for a, b in zip(one, many):
        n = min(len(a), len(b))
        assert n >= 40 and a[:n] == b[:n]
    # every page is in one table row or free
    held, (head, free) = dec.held[dec.steps % 2].tolist(), dec.free[dec.steps % 2].tolist()
    pages = [p for b, h in enumerate(held) for p in dec.table[b, :h].tolist()]
    pages += [int(dec.ring[(head + i) % 512]) for i in range(free)]
    assert sorted(pages) == list(range(512))
