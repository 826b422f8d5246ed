"""Strides that no tensor map can have are an unsupported argument, not a failed launch.  No GPU."""
from __future__ import annotations

import ctypes

import pytest

from test_hybrid_abi_cpu import attn_args
from test_long_abi_cpu import hy, shared_args, weight_args  # noqa: F401

FAR = 1 << 39  # elements of two bytes
POOLS = ["k_page_stride", "k_head_stride", "k_token_stride", "v_page_stride", "v_head_stride", "v_token_stride"]
CALLS = [("gdn_paged_attention", attn_args, s) for s in POOLS] + [("gdn_shared_attention", shared_args, s) for s in POOLS] + \
        [("gdn_attn_weight", weight_args, s) for s in POOLS[:3] + ["q_row_stride", "q_head_stride"]]


@pytest.mark.parametrize("call,make,stride", CALLS, ids=[f"{c}-{s}" for c, _, s in CALLS])
def test_a_stride_beyond_a_tensor_map_is_unsupported(hy, cuda_lib, call, make, stride):  # noqa: F811
    run = getattr(cuda_lib._lib, call)
    assert run(ctypes.byref(make(hy, **{stride: FAR})), None) == cuda_lib.ERR_UNSUPPORTED
    assert run(ctypes.byref(make(hy, **{stride: FAR + (1 << 60)})), None) == cuda_lib.ERR_UNSUPPORTED
    # refused for its alignment or sign first
    assert run(ctypes.byref(make(hy, **{stride: FAR + 1})), None) == cuda_lib.ERR_MISALIGNED
