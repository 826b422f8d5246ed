"""The hybrid-step C ABI without a GPU: declared symbols are exported, the
ctypes mirrors match the C structs, host checks refuse bad calls before anything
is launched, and the plain forms the GPU tests compare with hold on cases that
can be worked out by hand."""
from __future__ import annotations

import ctypes
import re
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

import hybrid_ref

ROOT = Path(__file__).resolve().parents[1]
HEADER = ROOT / "include" / "gdnhybrid.h"
FAKE = 1 << 20  # an aligned stand-in address; never dereferenced on these paths


@pytest.fixture(scope="module")
def hy(cuda_lib):
    from speculative_decode_gateddeltanet_gb300 import hybrid

    return hybrid


def test_declared_symbols_are_exported(cuda_lib):
    names = re.findall(r"^GDN_API\s+[\w\s\*]+?\b(\w+)\s*\(", HEADER.read_text(), flags=re.M)
    assert set(names) == {"gdn_page_map", "gdn_kv_append", "gdn_paged_attention", "gdn_paged_attention_work_bytes",
                          "gdn_sample_accept"}
    lib = ctypes.CDLL(str(cuda_lib.LIB_PATH))
    for name in names:
        assert hasattr(lib, name), name


def test_status_bits_match_header_and_are_distinct(hy, cuda_lib):
    bits = {m.group(1): int(m.group(2)) for m in re.finditer(r"GDN_(STATUS_[A-Z_]+)\s*=\s*(\d+)", HEADER.read_text())}
    assert len(bits) == 5
    for name, value in bits.items():
        assert getattr(hy, name) == value, name
    old = [getattr(cuda_lib, n) for n in dir(cuda_lib) if n.startswith("STATUS_")]
    assert len(set(bits.values()) | set(old)) == len(bits) + len(set(old))


@pytest.mark.parametrize("mirror,cname", [("GdnPageMapArgs", "gdn_page_map_args"), ("GdnKvAppendArgs", "gdn_kv_append_args"),
                                           ("GdnPagedAttnArgs", "gdn_paged_attn_args"), ("GdnSampleArgs", "gdn_sample_args")])
def test_struct_layout_matches_header(hy, tmp_path, mirror, cname):
    cls = getattr(hy, mirror)
    fields = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdnhybrid.h"\nint main(void){\n'
                   + f'printf("%zu\\n", sizeof({cname}));\n'
                   + "".join(f'printf("%zu\\n", offsetof({cname}, {f}));\n' for f in fields) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", str(HEADER.parent), str(src), "-o", str(exe)], check=True)
    vals = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(cls)
    for f, off in zip(fields, vals[1:]):
        assert getattr(cls, f).offset == off, f


def fill(cls, ints, pointers, over):
    a = cls(**ints)
    for i, f in enumerate(pointers):
        setattr(a, f, FAKE * (i + 1))
    for k, v in over.items():
        setattr(a, k, v)
    return a


def page_map_args(hy, **over):
    ints = dict(B=4, R=2, page_size=16, n_pages=64, max_pages=8, table_stride=8, n_slot_rows=8)
    return fill(hy.GdnPageMapArgs, ints, [f for f, t in hy.GdnPageMapArgs._fields_ if t is ctypes.c_void_p], over)


def append_args(hy, **over):
    ints = dict(rows=8, H_kv=2, d=64, page_size=16, n_pages=8, in_dtype=0, k_row_stride=128, k_head_stride=64, v_row_stride=128,
                v_head_stride=64, k_page_stride=2048, k_cache_head_stride=1024, k_token_stride=64, v_page_stride=2048,
                v_cache_head_stride=1024, v_token_stride=64)
    return fill(hy.GdnKvAppendArgs, ints, [f for f, t in hy.GdnKvAppendArgs._fields_ if t is ctypes.c_void_p], over)


def attn_args(hy, **over):
    ints = dict(B=2, R=4, H_q=8, H_kv=2, d=64, page_size=16, n_pages=8, max_pages=4, table_stride=4, n_q_rows=8, in_dtype=0,
                scale=0.125, q_row_stride=512, q_head_stride=64, k_page_stride=2048, k_head_stride=1024, k_token_stride=64,
                v_page_stride=2048, v_head_stride=1024, v_token_stride=64, o_row_stride=512, o_head_stride=64)
    return fill(hy.GdnPagedAttnArgs, ints, [f for f, t in hy.GdnPagedAttnArgs._fields_ if t is ctypes.c_void_p], over)


def sample_args(hy, **over):
    ints = dict(B=2, R=3, V=100, in_dtype=0, row_stride=100)
    return fill(hy.GdnSampleArgs, ints, [f for f, t in hy.GdnSampleArgs._fields_ if t is ctypes.c_void_p], over)


REFUSED = [
    ("gdn_page_map", page_map_args, dict(B=-1), 1), ("gdn_page_map", page_map_args, dict(page_size=0), 1),
    ("gdn_page_map", page_map_args, dict(table_stride=7), 1), ("gdn_page_map", page_map_args, dict(n_slot_rows=7), 1),
    ("gdn_page_map", page_map_args, dict(B=5000, n_slot_rows=10000), 2), ("gdn_page_map", page_map_args, dict(n_pages=1 << 28), 2),
    ("gdn_page_map", page_map_args, dict(held_in=None), 1), ("gdn_page_map", page_map_args, dict(free_ring=FAKE + 2), 3),
    ("gdn_page_map", page_map_args, dict(held_in=FAKE, held_out=FAKE), 1), ("gdn_page_map", page_map_args, dict(reserved=1), 1),
    ("gdn_page_map", page_map_args, dict(free_in=FAKE, free_out=FAKE + 4), 1),
    ("gdn_page_map", page_map_args, dict(n_rows=FAKE, rows_out=FAKE + 8), 1),
    ("gdn_kv_append", append_args, dict(rows=-1), 1), ("gdn_kv_append", append_args, dict(in_dtype=5), 2),
    ("gdn_kv_append", append_args, dict(d=36), 2), ("gdn_kv_append", append_args, dict(k=None), 1),
    ("gdn_kv_append", append_args, dict(k=FAKE + 8), 3), ("gdn_kv_append", append_args, dict(v_token_stride=68), 3),
    ("gdn_kv_append", append_args, dict(rows=1 << 30), 2),
    ("gdn_paged_attention", attn_args, dict(B=-1), 1), ("gdn_paged_attention", attn_args, dict(H_q=9), 2),
    ("gdn_paged_attention", attn_args, dict(H_q=258), 2), ("gdn_paged_attention", attn_args, dict(d=96), 2),
    ("gdn_paged_attention", attn_args, dict(page_size=24), 2), ("gdn_paged_attention", attn_args, dict(page_size=2048), 2),
    ("gdn_paged_attention", attn_args, dict(in_dtype=3), 2), ("gdn_paged_attention", attn_args, dict(scale=float("nan")), 1),
    ("gdn_paged_attention", attn_args, dict(scale=float("inf")), 1), ("gdn_paged_attention", attn_args, dict(work=None), 1),
    ("gdn_paged_attention", attn_args, dict(R=0, row_start=None), 1), ("gdn_paged_attention", attn_args, dict(q=FAKE + 4), 3),
    ("gdn_paged_attention", attn_args, dict(k_token_stride=65), 3), ("gdn_paged_attention", attn_args, dict(o_head_stride=60), 3),
    ("gdn_paged_attention", attn_args, dict(block_table=FAKE + 1), 3), ("gdn_paged_attention", attn_args, dict(table_stride=3), 1),
    ("gdn_sample_accept", sample_args, dict(V=0), 1), ("gdn_sample_accept", sample_args, dict(row_stride=99), 1),
    ("gdn_sample_accept", sample_args, dict(in_dtype=2), 2), ("gdn_sample_accept", sample_args, dict(V=1 << 21, row_stride=1 << 21), 2),
    ("gdn_sample_accept", sample_args, dict(u=None), 1), ("gdn_sample_accept", sample_args, dict(drafts=None), 1),
    ("gdn_sample_accept", sample_args, dict(logits=FAKE + 1), 3), ("gdn_sample_accept", sample_args, dict(prob=FAKE + 2), 3),
    ("gdn_sample_accept", sample_args, dict(B=70000), 2),
]


@pytest.mark.parametrize("call,make,over,code", REFUSED, ids=[f"{c}-{'-'.join(o)}" for c, _, o, _ in REFUSED])
def test_bad_arguments_are_refused(hy, cuda_lib, call, make, over, code):
    assert getattr(cuda_lib._lib, call)(ctypes.byref(make(hy, **over)), None) == code


def test_null_and_empty_calls(hy, cuda_lib):
    for call in ("gdn_page_map", "gdn_kv_append", "gdn_paged_attention", "gdn_sample_accept"):
        assert getattr(cuda_lib._lib, call)(None, None) == cuda_lib.ERR_INVALID_ARG
    lib = cuda_lib._lib
    assert lib.gdn_page_map(ctypes.byref(hy.GdnPageMapArgs(page_size=16, n_pages=4)), None) == 0
    assert lib.gdn_kv_append(ctypes.byref(append_args(hy, rows=0, k=None)), None) == 0
    assert lib.gdn_paged_attention(ctypes.byref(attn_args(hy, B=0, q=None)), None) == 0
    assert lib.gdn_paged_attention(ctypes.byref(attn_args(hy, n_q_rows=0, q=None)), None) == 0
    assert lib.gdn_sample_accept(ctypes.byref(sample_args(hy, B=0, u=None)), None) == 0


def test_work_bytes(hy):
    assert hy.paged_attention_work_bytes(attn_args(hy)) > 0
    assert hy.paged_attention_work_bytes(attn_args(hy, B=9999)) == hy.paged_attention_work_bytes(attn_args(hy))
    assert hy.paged_attention_work_bytes(attn_args(hy, d=80)) == 0


def test_binding_refuses_wrong_tensors(hy):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros(4, 2, 16, 64)
    with pytest.raises(TypeError):
        hy.make_kv_append_args(k=torch.zeros(3, 2, 64).half(), v=torch.zeros(3, 2, 64).half(), slot_map=i32(3),
                               k_cache=pool.half(), v_cache=pool.half())
    with pytest.raises(TypeError):
        hy.make_kv_append_args(k=torch.zeros(3, 2, 64), v=torch.zeros(3, 2, 64), slot_map=i32(3).long(), k_cache=pool, v_cache=pool)
    with pytest.raises(ValueError):
        hy.make_kv_append_args(k=torch.zeros(3, 2, 64), v=torch.zeros(3, 1, 64), slot_map=i32(3), k_cache=pool, v_cache=pool)
    with pytest.raises(ValueError):  # d must be contiguous
        hy.make_kv_append_args(k=torch.zeros(3, 64, 2).transpose(1, 2), v=torch.zeros(3, 2, 64), slot_map=i32(3), k_cache=pool, v_cache=pool)
    with pytest.raises(ValueError):
        hy.make_paged_attention_args(q=torch.zeros(3, 4, 64), k_cache=pool, v_cache=pool, block_table=i32(2, 4), ctx_len=i32(2),
                                     n_rows=i32(3), o=torch.zeros(3, 4, 64))
    with pytest.raises(ValueError):
        hy.make_sample_accept_args(logits=torch.zeros(2, 3, 50)[:, :, ::2], u=torch.zeros(2, 3), n_rows=i32(2), target=i32(2, 3))
    with pytest.raises(TypeError):
        hy.make_sample_accept_args(logits=torch.zeros(2, 3, 50), u=torch.zeros(2, 3).double(), n_rows=i32(2), target=i32(2, 3))


def test_plain_page_map_by_hand():
    out = hybrid_ref.page_map(np.array([20, 0, 5]), np.array([13, 0, 1]), np.array([2, 3, 1]), np.array([7, 8, 0, 0, 0, 0, 0, 0, 9]),
                              np.array([8, 3]), np.array([[1, 2, -1], [3, 4, 5], [6, -1, -1]]), 16, 0, 16)
    # 33 tokens need a third page: the ring's head, 9; the finished request's pages go to the tail; 6 tokens fit one page
    assert out["table"][0].tolist() == [1, 2, 9] and out["held_out"].tolist() == [3, 0, 1]
    assert out["ring"].tolist() == [7, 8, 3, 4, 5, 0, 0, 0, 9] and out["free_out"].tolist() == [0, 5]
    assert out["row_start"].tolist() == [0, 13, 13, 14] and out["status"] == 0
    assert out["slot_map"][:14].tolist() == [2 * 16 + i for i in range(4, 16)] + [9 * 16, 6 * 16 + 5]
    assert out["positions"][14:].tolist() == [-1, -1]


def test_plain_attention_by_hand():
    """Equal keys average the values a row sees; one dominant key picks its value."""
    k = torch.zeros(1, 1, 16, 64)
    v = torch.arange(16.0)[None, None, :, None].expand(1, 1, 16, 64)
    o, _ = hybrid_ref.attention(torch.ones(2, 1, 64), k, v, np.array([[0]]), np.array([3]), np.array([2]), np.array([0]), 1.0)
    assert np.allclose(o[0], 1.5) and np.allclose(o[1], 2.0)
    k[0, 0, 2] = 10.0
    o, _ = hybrid_ref.attention(torch.ones(2, 1, 64), k, v, np.array([[0]]), np.array([3]), np.array([2]), np.array([0]), 1.0)
    assert np.allclose(o, 2.0)


def test_plain_sampling_by_hand():
    z = np.log([0.5, 0.25, 0.125, 0.125])
    assert [hybrid_ref.sample_row(z, 1, 0, 1, 0, u)[0] for u in (0.0, 0.49, 0.51, 0.74, 0.76, 0.9)] == [0, 0, 1, 1, 2, 3]
    assert [hybrid_ref.sample_row(z, 1, 2, 1, 0, u)[0] for u in (0.6, 0.7, 0.999)] == [0, 1, 1]
    assert hybrid_ref.sample_row(z, 1, 0, 0.6, 0, 0.999) == (1, pytest.approx(1 / 3))
    assert hybrid_ref.sample_row(z, 1, 3, 1, 0, 0.999)[0] == 2  # of equal logits the lower index is in the first three
    assert hybrid_ref.sample_row(z, 1, 0, 1, 0.6, 0.999)[0] == 0
    assert hybrid_ref.sample_row(z, 0, 0, 1, 0, 0.999) == (0, 1.0)
    assert hybrid_ref.sample_row([np.nan, np.nan], 1, 0, 1, 0, 0.5) == (0, 1.0)
