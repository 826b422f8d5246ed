"""Arguments at the ends of their ranges, refused on the host."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import pytest

import test_hybrid_abi_cpu as base
from test_hybrid_abi_cpu import append_args, attn_args

hy = base.hy  # the module-wide fixture
HERE = os.path.dirname(os.path.abspath(__file__))


def fresh(code):
    """The code in a process of its own, which a fault of the host's would end."""
    path = os.pathsep.join([os.path.dirname(HERE), HERE, os.environ.get("PYTHONPATH", "")])
    run = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, PYTHONPATH=path), capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.returncode, run.stderr[-2000:])


def test_append_of_sizes_whose_product_passes_64_bits(hy, cuda_lib):
    """2^30 rows of 2^30 heads of 32: 2^66 bytes.  And a row of 2^32 chunks, and rows of the largest sizes there are."""
    fresh("import ctypes, test_hybrid_abi_cpu as t\n"
          "from speculative_decode_gateddeltanet_gb300 import gdn, hybrid\n"
          "for over in (dict(rows=1 << 30, H_kv=1 << 30, d=32), dict(rows=1, H_kv=1 << 30, d=32),\n"
          "             dict(rows=2**31 - 1, H_kv=2**31 - 1, d=2**31 - 8)):\n"
          "    assert gdn._lib.gdn_kv_append(ctypes.byref(t.append_args(hybrid, **over)), None) == 2, over\n")
    assert cuda_lib._lib.gdn_kv_append(ctypes.byref(append_args(hy, rows=0)), None) == 0


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_attention_scales_beyond_the_exponent_of_two_are_refused(hy, cuda_lib, dtype, scale):
    """Scores are kept in the exponent of 2: a scale that log2(e) carries past the 32-bit range would be infinite there."""
    args = attn_args(hy, in_dtype=dtype, scale=scale)
    assert cuda_lib._lib.gdn_paged_attention(ctypes.byref(args), None) == cuda_lib.ERR_UNSUPPORTED


@pytest.mark.parametrize("call,make,names", [
    ("gdn_kv_append", append_args, ("k_page_stride", "k_cache_head_stride", "k_token_stride", "v_page_stride", "v_cache_head_stride", "v_token_stride")),
    ("gdn_paged_attention", attn_args, ("k_page_stride", "k_head_stride", "k_token_stride", "v_page_stride", "v_head_stride", "v_token_stride"))])
def test_negative_pool_strides_are_refused(hy, cuda_lib, call, make, names):
    """Both calls mark a token without a place by a negative offset."""
    for name in names:
        for dtype in (0, 1):
            args = make(hy, in_dtype=dtype)
            setattr(args, name, -getattr(args, name))
            assert getattr(cuda_lib._lib, call)(ctypes.byref(args), None) == cuda_lib.ERR_INVALID_ARG, (name, dtype)


def test_the_bindings_load_where_pytorch_has_no_cuda():
    """PyTorch builds without CUDA lack the private functions that a call looks its stream up with."""
    fresh("import torch\n"
          "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
          "    if hasattr(torch._C, name):\n"
          "        delattr(torch._C, name)\n"
          "from speculative_decode_gateddeltanet_gb300 import gdn, hybrid\n"
          "assert hybrid._stream is gdn._stream and gdn._stream(5) == 5 and gdn._stream(0) is None\n")
