"""The attention kernel's bounded waits, made to run out on the GPU: a test-only
build (GDN_TEST_HOOKS, 2 ms limit) declares one block's first K copy on its
barrier and never issues it.  No copy is in flight; the block gives up, the
status says so, every row it had no part in is right, and the same context
serves a correct call afterwards."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import hybrid_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_gateddeltanet_gb300 import build as pkg_build
    from speculative_decode_gateddeltanet_gb300 import hybrid

    lib = ctypes.CDLL(str(pkg_build.build_attn_test_hooks()))
    lib.gdn_paged_attention.argtypes = [ctypes.POINTER(hybrid.GdnPagedAttnArgs), ctypes.c_void_p]
    lib.gdn_paged_attention.restype = ctypes.c_int
    lib.gdn_test_drop_attention_copy.argtypes = [ctypes.c_int]
    lib.gdn_test_drop_attention_copy.restype = ctypes.c_int
    yield lib
    lib.gdn_test_drop_attention_copy(-1)


def test_a_wait_that_runs_out_ends_the_block_and_no_other(hooks, cuda_lib):
    from speculative_decode_gateddeltanet_gb300 import hybrid as hy

    case = hybrid_ref.make_attention(lens=[(300, 1)] * 40, H_q=16, H_kv=8, d=128, P=16, dtype=torch.bfloat16, R=1, seed=1)
    t = {k: torch.tensor(np.asarray(case[k], np.int32), device="cuda") for k in ("table", "ctx", "n")}
    q, k, v = (case[x].cuda() for x in ("q", "k_cache", "v_cache"))
    o, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = hy.make_paged_attention_args(q=q, k_cache=k, v_cache=v, block_table=t["table"], ctx_len=t["ctx"], n_rows=t["n"], R=1, o=o,
                                        status=status)
    work = torch.empty(hy.paged_attention_work_bytes(args), dtype=torch.uint8, device="cuda")
    args.work = work.data_ptr()
    torch.cuda.synchronize()
    ref, vmax = hybrid_ref.attention(*(case[x] for x in ("q", "k_cache", "v_cache", "table", "ctx", "n", "start", "scale")))
    bound = 2.0**-9 * (vmax[..., None] + np.abs(ref)) + 1e-5 * vmax[..., None]

    assert hooks.gdn_test_drop_attention_copy(0) == 0
    assert hooks.gdn_paged_attention(ctypes.byref(args), None) == 0
    torch.cuda.synchronize()  # returns: no wait is without bound
    assert int(status.item()) == cuda_lib.STATUS_TIMEOUT
    # 320 tiles of three key blocks and three units of their own over 152 blocks: block 0 has thirteen units, which lie in
    # the first three kv heads of request 0
    got = o.double().cpu().numpy()
    assert (np.abs(got - ref)[1:] <= bound[1:]).all() and (np.abs(got - ref)[0, 6:] <= bound[0, 6:]).all()

    assert hooks.gdn_test_drop_attention_copy(-1) == 0
    status.zero_()
    assert hooks.gdn_paged_attention(ctypes.byref(args), None) == 0
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert (np.abs(o.double().cpu().numpy() - ref) <= bound).all()
