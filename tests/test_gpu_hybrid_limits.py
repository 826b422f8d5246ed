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
