"""Strides of dimensions with one entry are never used, whatever they are.
Tolerances are those of test_gpu_long."""
from __future__ import annotations

import pytest

import long_ref
from test_gpu_long import BF16, F32, Shared, Weight, always, hy  # noqa: F401

pytestmark = pytest.mark.gpu
FAR = 1 << 39


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_of_single_entries_do_not_matter(hy, always, dtype):  # noqa: F811
    case = long_ref.make_shared(groups=[], alone=[(9, 1)], H_q=1, H_kv=1, d=64, P=16, dtype=dtype, R=1, spare=0)
    s, w = Shared(hy, case, 1, groups=False), Weight(hy, case, 1)
    assert s.k.shape[:2] == (1, 1) and s.q.shape[:2] == (1, 1)
    for a in (s.args.attn, w.args):
        a.k_page_stride = a.k_head_stride = a.q_row_stride = a.q_head_stride = FAR
    s.args.attn.v_page_stride = s.args.attn.v_head_stride = FAR
    s.run().check()
    s.again(always).check()
    w.run().check()
