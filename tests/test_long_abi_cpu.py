"""The long-context C ABI without a GPU: declared symbols are exported, the ctypes
mirrors match the C structs, host checks refuse bad calls before anything is
launched, and the plain forms the GPU tests compare with hold on cases that can
be worked out by hand."""
from __future__ import annotations

import ctypes
import re
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

import hybrid_ref
import long_ref
from test_hybrid_abi_cpu import FAKE, attn_args, fill

ROOT = Path(__file__).resolve().parents[1]
HEADER = ROOT / "include" / "gdnlong.h"


@pytest.fixture(scope="module")
def hy(cuda_lib):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    return hybrid


def test_declared_symbols_are_exported(cuda_lib):
    names = re.findall(r"^GDN_API\s+[\w\s\*]+?\b(\w+)\s*\(", HEADER.read_text(), flags=re.M)
    assert set(names) == {"gdn_shared_attention", "gdn_shared_attention_work_bytes", "gdn_attn_weight", "gdn_attn_weight_work_bytes",
                          "gdn_evict_select", "gdn_kv_move"}
    lib = ctypes.CDLL(str(cuda_lib.LIB_PATH))
    import speculative_decode_gateddeltanet_gb300 as pkg
    for name in names:
        assert hasattr(lib, name), name
        assert getattr(pkg, name.removeprefix("gdn_") if name.endswith("_bytes") else name)


def test_status_bits_match_header_and_are_distinct(hy, cuda_lib):
    bits = {m.group(1): int(m.group(2)) for m in re.finditer(r"GDN_(STATUS_[A-Z_]+)\s*=\s*(\d+)", HEADER.read_text())}
    assert len(bits) == 2
    for name, value in bits.items():
        assert getattr(hy, name) == value, name
    every = {n: getattr(m, n) for m in (hy, cuda_lib) for n in dir(m) if n.startswith("STATUS_")}
    assert len(set(every.values())) == len(every)


@pytest.mark.parametrize("mirror,cname", [("GdnSharedAttnArgs", "gdn_shared_attn_args"), ("GdnAttnWeightArgs", "gdn_attn_weight_args"),
                                           ("GdnEvictArgs", "gdn_evict_args"), ("GdnKvMoveArgs", "gdn_kv_move_args")])
def test_struct_layout_matches_header(hy, tmp_path, mirror, cname):
    cls = getattr(hy, mirror)
    fields = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdnlong.h"\nint main(void){\n'
                   + f'printf("%zu\\n", sizeof({cname}));\n'
                   + "".join(f'printf("%zu\\n", offsetof({cname}, {f}));\n' for f in fields) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", str(HEADER.parent), str(src), "-o", str(exe)], check=True)
    vals = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(cls)
    for f, off in zip(fields, vals[1:]):
        assert getattr(cls, f).offset == off, f


def shared_args(hy, **over):
    own = {k: over.pop(k) for k in list(over) if k in ("n_groups", "reserved", "group_start", "prefix_len", "lse", "lse_row_stride")}
    a = hy.GdnSharedAttnArgs(attn=attn_args(hy, **over), n_groups=1, group_start=FAKE, prefix_len=FAKE, lse=FAKE, lse_row_stride=8)
    for k, v in own.items():
        setattr(a, k, v)
    return a


def weight_args(hy, **over):
    ints = dict(B=2, R=4, H_q=8, H_kv=2, d=64, page_size=16, n_pages=8, max_pages=4, table_stride=4, n_q_rows=8, in_dtype=0, fresh=1,
                scale=0.125, keep=1.0, q_row_stride=512, q_head_stride=64, k_page_stride=2048, k_head_stride=1024, k_token_stride=64,
                lse_row_stride=8)
    return fill(hy.GdnAttnWeightArgs, ints, [f for f, t in hy.GdnAttnWeightArgs._fields_ if t is ctypes.c_void_p], over)


def evict_args(hy, **over):
    ints = dict(B=2, page_size=16, n_pages=8, max_pages=4, table_stride=4, max_moves=8)
    return fill(hy.GdnEvictArgs, ints, [f for f, t in hy.GdnEvictArgs._fields_ if t is ctypes.c_void_p], over)


def move_args(hy, **over):
    ints = dict(B=2, max_moves=8, H_kv=2, d=64, page_size=16, n_pages=8, in_dtype=0, k_page_stride=2048, k_head_stride=1024,
                k_token_stride=64, v_page_stride=2048, v_head_stride=1024, v_token_stride=64)
    return fill(hy.GdnKvMoveArgs, ints, [f for f, t in hy.GdnKvMoveArgs._fields_ if t is ctypes.c_void_p], over)


INF, NAN = float("inf"), float("nan")
REFUSED = [
    ("gdn_shared_attention", shared_args, dict(B=-1), 1), ("gdn_shared_attention", shared_args, dict(H_q=9), 2),
    ("gdn_shared_attention", shared_args, dict(d=96), 2), ("gdn_shared_attention", shared_args, dict(page_size=24), 2),
    ("gdn_shared_attention", shared_args, dict(scale=NAN), 1), ("gdn_shared_attention", shared_args, dict(work=None), 1),
    ("gdn_shared_attention", shared_args, dict(q=FAKE + 4), 3), ("gdn_shared_attention", shared_args, dict(v_token_stride=-64), 1),
    ("gdn_shared_attention", shared_args, dict(R=0, row_start=None), 1), ("gdn_shared_attention", shared_args, dict(scale=3e38), 2),
    ("gdn_shared_attention", shared_args, dict(n_groups=-1), 1), ("gdn_shared_attention", shared_args, dict(n_groups=513), 2),
    ("gdn_shared_attention", shared_args, dict(B=4097), 2), ("gdn_shared_attention", shared_args, dict(group_start=None), 1),
    ("gdn_shared_attention", shared_args, dict(prefix_len=None), 1), ("gdn_shared_attention", shared_args, dict(lse_row_stride=7), 1),
    ("gdn_shared_attention", shared_args, dict(reserved=1), 1), ("gdn_shared_attention", shared_args, dict(group_start=FAKE + 2), 3),
    ("gdn_shared_attention", shared_args, dict(prefix_len=FAKE + 1), 3), ("gdn_shared_attention", shared_args, dict(lse=FAKE + 2), 3),
    ("gdn_attn_weight", weight_args, dict(B=-1), 1), ("gdn_attn_weight", weight_args, dict(H_q=258), 2),
    ("gdn_attn_weight", weight_args, dict(in_dtype=7), 2), ("gdn_attn_weight", weight_args, dict(page_size=2048), 2),
    ("gdn_attn_weight", weight_args, dict(scale=INF), 1), ("gdn_attn_weight", weight_args, dict(keep=INF), 1),
    ("gdn_attn_weight", weight_args, dict(keep=NAN), 1), ("gdn_attn_weight", weight_args, dict(fresh=2), 1),
    ("gdn_attn_weight", weight_args, dict(lse=None), 1), ("gdn_attn_weight", weight_args, dict(weight=None), 1),
    ("gdn_attn_weight", weight_args, dict(work=None), 1), ("gdn_attn_weight", weight_args, dict(lse_row_stride=7), 1),
    ("gdn_attn_weight", weight_args, dict(k_cache=FAKE + 8), 3), ("gdn_attn_weight", weight_args, dict(k_token_stride=65), 3),
    ("gdn_attn_weight", weight_args, dict(k_page_stride=-2048), 1), ("gdn_attn_weight", weight_args, dict(first=FAKE + 2), 3),
    ("gdn_attn_weight", weight_args, dict(weight=FAKE + 1), 3), ("gdn_attn_weight", weight_args, dict(born=FAKE + 2), 3),
    ("gdn_attn_weight", weight_args, dict(R=0, row_start=None), 1), ("gdn_attn_weight", weight_args, dict(work=FAKE + 8), 3),
    ("gdn_evict_select", evict_args, dict(B=-1), 1), ("gdn_evict_select", evict_args, dict(page_size=0), 1),
    ("gdn_evict_select", evict_args, dict(table_stride=3), 1), ("gdn_evict_select", evict_args, dict(max_moves=-1), 1),
    ("gdn_evict_select", evict_args, dict(B=65536), 2), ("gdn_evict_select", evict_args, dict(n_pages=1 << 28), 2),
    ("gdn_evict_select", evict_args, dict(B=60000, max_moves=60000), 2), ("gdn_evict_select", evict_args, dict(budget=None), 1),
    ("gdn_evict_select", evict_args, dict(weight=None), 1), ("gdn_evict_select", evict_args, dict(move_to=None), 1),
    ("gdn_evict_select", evict_args, dict(weight=FAKE + 2), 3), ("gdn_evict_select", evict_args, dict(ctx_out=FAKE + 1), 3),
    ("gdn_kv_move", move_args, dict(B=-1), 1), ("gdn_kv_move", move_args, dict(max_moves=-1), 1),
    ("gdn_kv_move", move_args, dict(in_dtype=4), 2), ("gdn_kv_move", move_args, dict(d=36), 2),
    ("gdn_kv_move", move_args, dict(B=60000, max_moves=60000), 2), ("gdn_kv_move", move_args, dict(B=65536), 2),
    ("gdn_kv_move", move_args, dict(move_from=None), 1), ("gdn_kv_move", move_args, dict(k_cache=FAKE + 8), 3),
    ("gdn_kv_move", move_args, dict(v_head_stride=1020), 3), ("gdn_kv_move", move_args, dict(k_page_stride=-2048), 1),
    ("gdn_kv_move", move_args, dict(n_moves=FAKE + 2), 3), ("gdn_kv_move", move_args, dict(reserved=1), 1),
    ("gdn_kv_move", move_args, dict(n_pages=1 << 28), 2),
]


@pytest.mark.parametrize("call,make,over,code", REFUSED, ids=[f"{c}-{'-'.join(o)}-{i}" for i, (c, _, o, _) in enumerate(REFUSED)])
def test_bad_arguments_are_refused(hy, cuda_lib, call, make, over, code):
    assert getattr(cuda_lib._lib, call)(ctypes.byref(make(hy, **over)), None) == code


def test_null_and_empty_calls(hy, cuda_lib):
    lib = cuda_lib._lib
    for call in ("gdn_shared_attention", "gdn_attn_weight", "gdn_evict_select", "gdn_kv_move"):
        assert getattr(lib, call)(None, None) == cuda_lib.ERR_INVALID_ARG
    assert lib.gdn_shared_attention_work_bytes(None) == lib.gdn_attn_weight_work_bytes(None) == 0
    assert lib.gdn_shared_attention(ctypes.byref(shared_args(hy, B=0, q=None)), None) == 0
    assert lib.gdn_shared_attention(ctypes.byref(shared_args(hy, n_q_rows=0, q=None)), None) == 0
    assert lib.gdn_attn_weight(ctypes.byref(weight_args(hy, B=0, q=None)), None) == 0
    assert lib.gdn_attn_weight(ctypes.byref(weight_args(hy, n_q_rows=0, lse=None)), None) == 0
    assert lib.gdn_evict_select(ctypes.byref(evict_args(hy, B=0, weight=None)), None) == 0
    assert lib.gdn_kv_move(ctypes.byref(move_args(hy, B=0, k_cache=None)), None) == 0
    assert lib.gdn_kv_move(ctypes.byref(move_args(hy, max_moves=0, k_cache=None)), None) == 0


def test_work_bytes(hy):
    assert hy.shared_attention_work_bytes(shared_args(hy)) > 0 and hy.attn_weight_work_bytes(weight_args(hy)) > 0
    assert hy.shared_attention_work_bytes(shared_args(hy, B=9)) == hy.shared_attention_work_bytes(shared_args(hy, n_groups=0))
    assert hy.attn_weight_work_bytes(weight_args(hy, B=9)) == hy.attn_weight_work_bytes(weight_args(hy))
    for a in (shared_args(hy, d=80), shared_args(hy, n_groups=-1), shared_args(hy, B=5000)):
        assert hy.shared_attention_work_bytes(a) == 0
    assert hy.attn_weight_work_bytes(weight_args(hy, H_q=7)) == 0


def test_binding_refuses_wrong_tensors(hy):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool, q = torch.zeros(4, 2, 16, 64), torch.zeros(3, 4, 64)
    attn = dict(q=q, k_cache=pool, v_cache=pool, block_table=i32(2, 4), ctx_len=i32(2), n_rows=i32(2), o=q, R=2)
    for error, over in ((ValueError, dict(group_start=i32(2))), (ValueError, dict(group_start=i32(2), prefix_len=i32(2))),
                        (TypeError, dict(group_start=i32(2).long(), prefix_len=i32(1))), (TypeError, dict(lse=torch.zeros(3, 4).double())),
                        (ValueError, dict(lse=torch.zeros(3, 5))), (ValueError, dict(lse=torch.zeros(4, 3).T))):
        with pytest.raises(error):
            hy.make_shared_attention_args(**attn, **over)
    weight = dict(q=q, k_cache=pool, lse=torch.zeros(3, 4), block_table=i32(2, 4), ctx_len=i32(2), n_rows=i32(2), R=2, weight=torch.zeros(64))
    assert hy.make_attn_weight_args(**weight).lse_row_stride == 4
    for error, over in ((ValueError, dict(weight=torch.zeros(63))), (TypeError, dict(weight=torch.zeros(64).double())),
                        (ValueError, dict(born=i32(65))), (ValueError, dict(first=i32(3))), (TypeError, dict(position=i32(2).long())),
                        (ValueError, dict(lse=torch.zeros(2, 4))), (TypeError, dict(k_cache=pool.bfloat16()))):
        with pytest.raises(error):
            hy.make_attn_weight_args(**(weight | over))
    evict = dict(weight=torch.zeros(64), block_table=i32(2, 4), ctx_len=i32(2), budget=i32(2), ctx_out=i32(2), n_moves=i32(2),
                 move_from=i32(2, 5), move_to=i32(2, 5), page_size=16)
    assert hy.make_evict_select_args(**evict).n_pages == 4
    for error, over in ((ValueError, dict(page_size=15)), (ValueError, dict(move_to=i32(2, 6))), (ValueError, dict(budget=i32(3))),
                        (TypeError, dict(born=i32(64).long())), (ValueError, dict(born=i32(60))), (ValueError, dict(pinned=i32(4)[::2]))):
        with pytest.raises(error):
            hy.make_evict_select_args(**(evict | over))
    move = dict(k_cache=pool, v_cache=pool, move_from=i32(2, 5), move_to=i32(2, 5), n_moves=i32(2))
    for error, over in ((ValueError, dict(n_moves=i32(3))), (ValueError, dict(move_from=i32(2, 4))), (TypeError, dict(v_cache=pool.bfloat16())),
                        (TypeError, dict(k_cache=pool.double(), v_cache=pool.double()))):
        with pytest.raises(error):
            hy.make_kv_move_args(**(move | over))


def test_plain_log_sums_by_hand():
    """Equal keys: lse is the logarithm of the keys a row sees plus the common score."""
    k = torch.ones(1, 1, 16, 64)
    lse, size = long_ref.log_sums(torch.ones(2, 1, 64), k, np.array([[0]]), np.array([3]), np.array([2]), np.array([0]), 0.5)
    assert np.allclose(lse[:, 0], 32 + np.log([4, 5])) and np.allclose(size, 32)


def test_plain_weights_by_hand():
    """Equal keys share each row's weight evenly among the tokens that it sees."""
    k, q = torch.zeros(2, 1, 16, 64), torch.ones(2, 1, 64)
    lse = torch.tensor(np.log([[4.0], [5.0]]))
    weight, born, off = long_ref.weights(q, k, lse, np.array([[1, 0]]), np.array([3]), np.array([2]), np.array([0]), 1.0, 0.5, True,
                                         np.array([1]), np.array([100]), np.ones(32), np.full(32, -1))
    assert np.allclose(weight[16:21], [1.0, 0.5 + 0.45, 0.5 + 0.45, 0.45, 0.2])
    assert np.allclose(weight[:16], 1) and born[16:21].tolist() == [-1, -1, -1, 100, 101] and off[16] == 0 and off[17] > 0


def test_plain_select_by_hand():
    """Six tokens, four to keep: the two lightest may not be pinned or young; their gaps take the last that stay."""
    weight = np.array([0.1, 0.5, 0.2, 0.2, 0.0, 0.9], np.float32)
    born = np.array([0, 1, 2, 3, 9, 5])
    lists = [np.full((1, 2), -7)] * 2
    out = long_ref.select(weight, born, np.array([[0]]), np.array([6]), np.array([4]), np.array([1]), np.array([9]), 16, 2, 1, lists)
    # candidates 1, 2, 3, 5: of the equal ones at 2 and 3 both go; 4 and 5 move into their places
    assert out["ctx_out"][0] == 4 and out["move_to"][0].tolist() == [2, 3] and out["move_from"][0].tolist() == [4, 5]
    assert np.allclose(out["weight"][:4], [0.1, 0.5, 0.0, 0.9]) and out["born"][:4].tolist() == [0, 1, 9, 5] and out["status"] == 0
    out = long_ref.select(weight, born, np.array([[0]]), np.array([6]), np.array([5]), np.array([1]), np.array([9]), 16, 2, 1, lists)
    assert out["move_to"][0].tolist() == [3, -7] and out["move_from"][0].tolist() == [5, -7]  # of equal weights the last goes


def test_shared_cases_share_what_they_say():
    case = long_ref.make_shared(groups=[(40, [(0, 0), (3, 1), (9, 2)])], alone=[(5, 1)], H_q=2, H_kv=1, d=64, P=16, dtype=torch.float32)
    t = case["table"]
    assert t[1, :2].tolist() == t[2, :2].tolist() and t[1, 2] != t[2, 2]
    assert torch.equal(case["k_cache"][t[1, 2], :, :8], case["k_cache"][t[2, 2], :, :8])
    assert not torch.equal(case["k_cache"][t[1, 2], :, 8], case["k_cache"][t[2, 2], :, 8])
    plain = [case[x] for x in ("q", "k_cache", "v_cache", "table", "ctx", "n", "start", "scale")]
    o, _ = hybrid_ref.attention(*plain)
    assert not np.isnan(o).any()
