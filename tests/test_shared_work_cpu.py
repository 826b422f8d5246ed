"""The work buffer of the attention over shared prefixes: as large as the rows that can share need,
and no larger, up to sizes whose products come near 64 bits.  No GPU."""
from __future__ import annotations

import pytest

from test_long_abi_cpu import hy, shared_args  # noqa: F401

COLUMN, ENTRY = 4, 16  # a part has its columns in 32 bits, and a maximum, a sum, a block and where it is in its tile


def parts(rows, H_q, d):
    return 2 * rows * H_q * (COLUMN * d + ENTRY)


def work(hy, **over):  # noqa: F811
    return hy.shared_attention_work_bytes(shared_args(hy, **over))


# rows of a tile less one, over the query heads of a kv head: behind more of them a request reads apart
MOST = [(0, 32, 8, 31), (0, 16, 2, 15), (0, 8, 8, 127), (0, 128, 1, 0), (1, 32, 8, 7), (1, 40, 1, 0)]


@pytest.mark.parametrize("dtype,H_q,H_kv,most", MOST)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,rows", [(1, 1), (4, 8192), (4096, 4096), (16, 64), (4, 2 ** 31 - 1)])
def test_places_are_for_the_rows_that_can_share(hy, dtype, H_q, H_kv, most, d, B, rows):  # noqa: F811
    over = dict(in_dtype=dtype, H_q=H_q, H_kv=H_kv, d=d, R=0)
    share = min(rows, B * most)
    got = work(hy, B=B, n_q_rows=rows, **over) - work(hy, B=0, n_q_rows=0, **over)
    assert got == parts(share, H_q, d) + 4 * share  # and each rank's row


def test_products_that_come_near_64_bits(hy):  # noqa: F811
    for H_q, rows in ((2 ** 30, 2 ** 30), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 27, 2 ** 26)):
        got = work(hy, in_dtype=0, H_q=H_q, H_kv=H_q, d=256, R=0, B=4096, n_q_rows=rows)
        assert got >= parts(4096 * 127, H_q, 256)
