"""The work buffer of the attention over shared prefixes, filled to its last place: nothing behind it
is written, whatever the rows of q.  Tolerances are those of test_gpu_long."""
from __future__ import annotations

import pytest
import torch

import long_ref
from test_gpu_long import BF16, F32, Shared, always, hy  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,H_q,H_kv,d,most", [(BF16, 8, 2, 64, 31), (BF16, 16, 2, 256, 15), (BF16, 2, 2, 128, 127), (F32, 8, 2, 64, 7),
                                                   (F32, 3, 3, 128, 31)])
def test_every_request_has_as_many_rows_as_may_share(hy, always, dtype, H_q, H_kv, d, most):  # noqa: F811
    R = most + 9  # padded: more rows than places
    groups = [(200, [(3, most), (0, most)]), (33, [(1, most), (70, most), (0, most)])]
    case = long_ref.make_shared(groups=groups, H_q=H_q, H_kv=H_kv, d=d, P=16, dtype=dtype, R=R, seed=most)
    s = Shared(hy, case, R)
    size = hy.shared_attention_work_bytes(s.args)
    s.work = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    s.args.attn.work = s.work.data_ptr()
    for lib in (None, always):
        s.again(lib).check()
        assert (s.work[size:] == 255).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompts_beside_rows_that_share(hy, always, dtype):  # noqa: F811
    """The rows of q are far more than the places: a prompt lies between requests that share, and none of its rows has one."""
    groups = [(150, [(3, 2), (40, 600), (0, 3)]), (20, [(0, 1), (7, 300), (2, 1)])]
    case = long_ref.make_shared(groups=groups, H_q=8, H_kv=2, d=64, P=16, dtype=dtype, seed=2)
    s = Shared(hy, case)
    size = hy.shared_attention_work_bytes(s.args)
    s.work = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    s.args.attn.work = s.work.data_ptr()
    for lib in (None, always):
        s.again(lib).check()
        assert (s.work[size:] == 255).all()
