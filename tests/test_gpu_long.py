"""The long-context operators on the GPU against their plain 64-bit forms, at the
lengths, shapes, strides and values where they can go wrong.

Tolerances, from the arithmetic each call promises (u = 2^-24, half a step of 32 bits).
A score is a sum of d products whose rounding is off by at most (d + 4) u of the sum of
their sizes, twice that where the tensor cores drop bits instead of rounding; call it s.
It moves a weight's share by a factor 1 + s.  lse is off by s, by the (L + 16) u of a sum
of L terms, and by the roundings of its own size.  An output is off by 2 s and 2 (L + 16) u
of the largest |v| its row sees; in bf16 also by the weights' rounding, 2^-8 of that |v|, and
its own, 2^-8 of itself.  Choices, moves and ages are exact."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import hybrid_ref
import long_ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = long_ref.U


@pytest.fixture(scope="module", autouse=True)
def hy(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_gateddeltanet_gb300 import hybrid

    return hybrid


@pytest.fixture(scope="module")
def always(hy):
    """The attention built for tests: it shares prefixes whatever that costs (and drops no copy unless told to)."""
    import ctypes

    from speculative_decode_gateddeltanet_gb300 import build as pkg_build

    lib = ctypes.CDLL(str(pkg_build.build_attn_test_hooks()))
    lib.gdn_shared_attention.argtypes = [ctypes.POINTER(hy.GdnSharedAttnArgs), ctypes.c_void_p]
    lib.gdn_attn_weight.argtypes = [ctypes.POINTER(hy.GdnAttnWeightArgs), ctypes.c_void_p]
    yield lib
    lib.gdn_test_drop_shared_copy(-1)
    lib.gdn_test_drop_weight_copy(-1)


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- shared prefixes -----------------------------------------------------------


class Shared:
    """A shared call's tensors on the GPU, and its check against 64 bits."""

    def __init__(self, hy, case, R=0, groups=True, lse=True):
        self.hy, self.case = hy, case
        self.q, self.k, self.v = (case[x].cuda() for x in ("q", "k_cache", "v_cache"))
        if case["k_cache"].stride(1) == case["k_cache"].shape[3]:  # token-major pools keep their strides
            self.k, self.v = (case[x].transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in ("k_cache", "v_cache"))
        self.t = {k: ints(case[k]) for k in ("table", "ctx", "n", "start", "group_start", "prefix_len")}
        self.o, self.status = torch.full_like(self.q, 7.0), status_word()
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda") if lse else None
        self.args = hy.make_shared_attention_args(
            q=self.q, k_cache=self.k, v_cache=self.v, block_table=self.t["table"], ctx_len=self.t["ctx"], n_rows=self.t["n"],
            row_start=self.t["start"], R=R, o=self.o, scale=case["scale"], lse=self.lse, status=self.status,
            group_start=self.t["group_start"] if groups else None, prefix_len=self.t["prefix_len"] if groups else None)
        self.work = torch.full((hy.shared_attention_work_bytes(self.args),), 255, dtype=torch.uint8, device="cuda")  # NaN
        self.args.attn.work = self.work.data_ptr()

    def run(self, lib=None):
        if lib is None:
            self.hy.gdn_shared_attention(self.args)
        else:
            assert lib.gdn_shared_attention(self.args, torch.cuda.current_stream().cuda_stream or None) == 0
        return self

    def again(self, lib):
        self.o.fill_(7.0)
        if self.lse is not None:
            self.lse.fill_(7.0)
        self.status.zero_()
        self.work.fill_(255)
        return self.run(lib)

    def check(self, n=None, status=0):
        torch.cuda.synchronize()
        c = dict(self.case)
        if n is not None:
            c["n"] = n
        plain = [c[x] for x in ("q", "k_cache", "v_cache", "table", "ctx", "n", "start", "scale")]
        ref, vmax = hybrid_ref.attention(*plain)
        want, size = long_ref.log_sums(*plain[:2], *plain[3:])
        live = ~np.isnan(want)
        d, L = self.q.shape[2], int((c["ctx"] + c["n"]).max())
        s = (2 * (d + 4) * size * U)[..., None]
        bound = (2 * s + 2 * (L + 16) * U + 2 ** -20) * vmax[..., None]
        if self.q.dtype == BF16:
            bound = bound + 2.0 ** -8 * (vmax[..., None] + np.abs(ref))
        got = self.o.double().cpu().numpy()
        assert int(self.status.item()) == status
        assert (np.abs(got - ref)[live] <= bound[live]).all(), np.nanmax((np.abs(got - ref) / bound)[live])
        assert (got[~live] == 7.0).all()  # rows of no request
        if self.lse is not None:
            got = self.lse.double().cpu().numpy()
            bound = s[..., 0] + (L + 16) * U + 8 * U * (np.abs(want) + size)
            assert (np.abs(got - want)[live] <= bound[live]).all()
            assert (got[~live] == 7.0).all()


SHARED = [
    # groups, alone, H_q, H_kv, d, P, dtype, layout, R
    ([(300, [(0, 1), (5, 1), (130, 1)])], [], 6, 2, 64, 16, F32, "tokens", 1),
    ([(77, [(0, 3), (5, 1), (40, 5)]), (1, [(1, 1), (2, 2)])], [(9, 4)], 4, 4, 128, 7, F32, "heads", 5),
    ([(500, [(3, 30), (0, 41)])], [], 8, 2, 256, 48, F32, "heads", 0),
    ([(300, [(0, 1), (5, 1), (130, 1)])], [], 6, 2, 64, 16, BF16, "tokens", 1),
    ([(301, [(0, 4), (5, 4), (130, 4)]), (128, [(0, 4), (1, 4)])], [(3, 4), (400, 4)], 16, 2, 256, 16, BF16, "heads", 4),
    ([(1000, [(i, 1) for i in range(9)])], [], 32, 8, 128, 64, BF16, "heads", 1),
    ([(129, [(0, 2), (300, 9), (17, 0), (1, 5)]), (640, [(64, 3)]), (15, [(0, 1), (0, 1)])], [], 28, 4, 128, 32, BF16, "tokens", 9),
    ([(2000, [(0, 0), (10, 3), (0, 2)]), (0, [(100, 2), (30, 1)])], [(0, 1)], 8, 8, 64, 48, BF16, "heads", 3),
    ([(257, [(0, 200), (33, 150)]), (90, [(0, 1), (0, 300)])], [(70, 130)], 10, 2, 128, 16, BF16, "heads", 0),
    ([(700, [(5, 130), (0, 77), (200, 1)])], [], 16, 1, 256, 128, BF16, "tokens", 0),
    ([(5000, [(50, 2), (0, 1)])], [], 5, 1, 64, 64, BF16, "heads", 2),
    ([(16, [(0, 1)] * 40), (33, [(0, 2)] * 30)], [(0, 1)] * 5, 4, 2, 128, 16, BF16, "heads", 2),
    ([(64, [(0, 3), (9, 3)])], [], 128, 1, 128, 16, BF16, "heads", 3),
    ([(8193, [(0, 1)])], [(8200, 1)], 16, 2, 256, 16, BF16, "heads", 1),
]


@pytest.mark.parametrize("groups,alone,H_q,H_kv,d,P,dtype,layout,R", SHARED, ids=range(len(SHARED)))
def test_shared_attention_matches_the_plain_form(hy, always, groups, alone, H_q, H_kv, d, P, dtype, layout, R):
    case = long_ref.make_shared(groups=groups, alone=alone, H_q=H_q, H_kv=H_kv, d=d, P=P, dtype=dtype, layout=layout, R=R, seed=len(groups))
    s = Shared(hy, case, R).run()
    s.check()
    first = s.o.clone(), s.lse.clone()
    s.run()
    torch.cuda.synchronize()
    assert torch.equal(s.o, first[0]) and torch.equal(s.lse, first[1])  # the same bits again
    s.again(always).check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_attention_without_groups_or_log_sums(hy, dtype):
    case = long_ref.make_shared(groups=[], alone=[(300, 3), (0, 3), (77, 1), (500, 2)], H_q=8, H_kv=2, d=128, P=16, dtype=dtype, R=3)
    Shared(hy, case, 3, groups=False).run().check()
    Shared(hy, case, 3, groups=False, lse=False).run().check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_attention_with_scales_of_either_sign_and_large_scores(hy, always, dtype):
    for scale in (-0.1, 0.0, 1.0):
        case = long_ref.make_shared(groups=[(200, [(3, 2), (60, 2)])], H_q=8, H_kv=2, d=64, P=16, dtype=dtype, R=2, scale=scale)
        s = Shared(hy, case, 2).run()
        s.check()
        s.again(always).check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("start", [[0, 3, 2], [0, 2, 9], [-1, 2, 4], [0, -(2 ** 31), 2 ** 31 - 1]])
def test_groups_that_do_not_rise_share_nothing(hy, always, dtype, start):
    case = long_ref.make_shared(groups=[(100, [(0, 1), (5, 1)]), (60, [(1, 1), (2, 1)])], H_q=4, H_kv=2, d=64, P=16, dtype=dtype, R=1)
    case["group_start"] = np.array(start)
    s = Shared(hy, case, 1).run()
    s.check(status=hy.STATUS_BAD_GROUP)
    s.again(always).check(status=hy.STATUS_BAD_GROUP)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_requests_shorter_than_their_groups_prefix_read_their_own_pages(hy, always, dtype):
    """A request with fewer cached tokens than the prefix takes no part in it; a negative or huge prefix is none."""
    case = long_ref.make_shared(groups=[(100, [(0, 2), (5, 2), (30, 2)]), (60, [(1, 2), (2, 2)]), (20, [(1, 1), (2, 2)])], H_q=4, H_kv=2,
                                d=64, P=16, dtype=dtype, R=2)
    for cut in (False, True):
        if cut:
            case["ctx"] = case["ctx"] - np.array([20, 0, 0, 40, 0, 0, 0])  # the first of two groups
        for prefix in ([100, 60, 20], [-5, 2 ** 31 - 1, -(2 ** 31)], [99, 59, 19], [16, 15, 1], [106, 62, 22]):
            case["prefix_len"] = np.array(prefix)
            s = Shared(hy, case, 2).run()
            s.check()
            s.again(always).check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_attention_skips_bad_requests_alone(hy, always, dtype):
    case = long_ref.make_shared(groups=[(100, [(0, 2), (5, 2), (30, 2), (1, 2), (4, 1)])], alone=[(20, 2)], H_q=4, H_kv=2, d=64, P=16,
                                dtype=dtype, R=2)
    s = Shared(hy, case, 2)
    s.t["n"][1] = 3            # more rows than R
    s.t["ctx"][0] = -1         # the first request of the group
    s.t["ctx"][3] = 2 ** 31 - 1
    s.run()
    n = case["n"].copy()
    n[[0, 1, 3]] = 0
    s.check(n=n, status=hy.STATUS_BAD_LENGTH | 2)
    s.again(always).check(n=n, status=hy.STATUS_BAD_LENGTH | 2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_attention_reads_bad_pages_as_zeros(hy, always, dtype):
    case = long_ref.make_shared(groups=[(100, [(0, 2), (5, 2)])], alone=[(40, 2)], H_q=4, H_kv=2, d=64, P=16, dtype=dtype, R=2)
    bad = case["table"][0, 1]
    case["k_cache"][bad] = 0
    case["v_cache"][bad] = 0
    s = Shared(hy, case, 2)
    for b, page in ((0, -3), (1, case["k_cache"].shape[0])):
        s.t["table"][b, 1] = page
    s.run().check(status=hy.STATUS_BAD_PAGE)
    s.again(always).check(status=hy.STATUS_BAD_PAGE)


@pytest.mark.parametrize("forced", [False, True])
def test_shared_attention_in_a_graph_follows_lengths_and_groups(hy, always, forced):
    """One captured graph serves other lengths, rows, groups and prefixes."""
    case = long_ref.make_shared(groups=[(400, [(0, 4), (50, 4), (9, 4)]), (100, [(7, 4), (8, 4)])], alone=[(30, 4)], H_q=16, H_kv=2, d=128,
                                P=16, dtype=BF16, R=4)
    lib = always if forced else None
    s = Shared(hy, case, 4).run(lib)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.run(lib)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.run(lib)
    for n, starts, prefix in (([4, 4, 4, 4, 4, 4], [0, 3, 5], [400, 100]), ([1, 0, 4, 2, 3, 1], [0, 3, 5], [400, 100]),
                              ([2, 2, 2, 2, 2, 2], [0, 2, 3], [384, 100]), ([4, 1, 1, 1, 1, 4], [3, 3, 5], [0, 100])):
        s.t["n"].copy_(ints(n))
        s.t["group_start"].copy_(ints(starts))
        s.t["prefix_len"].copy_(ints(prefix))
        s.o.fill_(7.0)
        s.lse.fill_(7.0)
        graph.replay()
        s.check(n=np.array(n))


def test_shared_attention_with_far_pages_and_strided_rows(hy, always):
    """Element offsets beyond 2^31, q and o as slices of wider rows, lse with a row stride."""
    case = long_ref.make_shared(groups=[(40, [(0, 2), (25, 2)])], H_q=4, H_kv=2, d=64, P=16, dtype=BF16, R=2, spare=1)
    s = Shared(hy, case, 2)
    pages, far = case["k_cache"].shape[0], 2 ** 29
    pool = torch.empty(pages * far + 4096, dtype=BF16, device="cuda")
    k = pool.as_strided((pages, 2, 16, 64), (far, 1024, 64, 1))
    v = pool.as_strided((pages, 2, 16, 64), (far, 1024, 64, 1), 2048)
    k.copy_(s.k)
    v.copy_(s.v)
    wide = torch.full((case["q"].shape[0], 9, 64), 7.0, dtype=BF16, device="cuda")
    q = wide[:, 2:6]
    q.copy_(s.q)
    lse = torch.full((q.shape[0], 11), 7.0, device="cuda")
    args = hy.make_shared_attention_args(q=q, k_cache=k, v_cache=v, block_table=s.t["table"], ctx_len=s.t["ctx"], n_rows=s.t["n"],
                                         row_start=s.t["start"], R=2, o=s.o, scale=case["scale"], lse=lse[:, :4], status=s.status,
                                         group_start=s.t["group_start"], prefix_len=s.t["prefix_len"])
    args.attn.work = s.work.data_ptr()
    for lib in (None, always):
        if lib is None:
            hy.gdn_shared_attention(args)
        else:
            s.o.fill_(7.0)
            lse.fill_(7.0)
            assert lib.gdn_shared_attention(args, torch.cuda.current_stream().cuda_stream or None) == 0
        s.lse.copy_(lse[:, :4])
        assert (lse[:, 4:] == 7.0).all()
        s.check()


@pytest.mark.parametrize("dtype,d,own", [(BF16, 128, 300), (BF16, 256, 20), (F32, 64, 40)])
def test_a_wide_batch_shares_by_itself(hy, dtype, d, own):
    """Calls in which sharing pays, with many parts a prefix, several groups, and one that does not pay among them."""
    groups = [(2500, [(own * i // 40, 1 + i % 3) for i in range(40)]), (1700, [(i, 2) for i in range(30)]), (60, [(5, 1), (900, 2)])]
    case = long_ref.make_shared(groups=groups, alone=[(700, 3)], H_q=16, H_kv=4, d=d, P=32, dtype=dtype, R=3)
    s = Shared(hy, case, 3).run()
    s.check()
    first = s.o.clone(), s.lse.clone()
    s.run()
    torch.cuda.synchronize()
    assert torch.equal(s.o, first[0]) and torch.equal(s.lse, first[1])
    # half of the prefix's tokens moved to other pages: the table rows of requests behind the first are not asked for them
    table = s.t["table"].clone()
    s.t["table"][1:40, :2500 // 32] = s.t["table"][1:40, 2500 // 32, None]
    s.again(None)
    torch.cuda.synchronize()
    s.t["table"].copy_(table)
    s.check()


@pytest.mark.parametrize("d,P", [(64, 16), (128, 48), (256, 16)])
def test_shared_attention_of_pools_whose_pages_are_no_whole_number_of_heads(hy, always, d, P):
    case = long_ref.make_shared(groups=[(140, [(0, 2), (25, 2)])], alone=[(33, 2)], H_q=4, H_kv=2, d=d, P=P, dtype=BF16, R=2)
    s = Shared(hy, case, 2)
    pages, stride = case["k_cache"].shape[0], 2 * P * d + 24
    k, v = (torch.full((pages * stride,), float("nan"), dtype=BF16, device="cuda").as_strided((pages, 2, P, d), (stride, P * d, d, 1))
            for _ in range(2))
    k.copy_(s.k)
    v.copy_(s.v)
    args = hy.make_shared_attention_args(q=s.q, k_cache=k, v_cache=v, block_table=s.t["table"], ctx_len=s.t["ctx"], n_rows=s.t["n"],
                                         row_start=s.t["start"], R=2, o=s.o, scale=case["scale"], lse=s.lse, status=s.status,
                                         group_start=s.t["group_start"], prefix_len=s.t["prefix_len"])
    args.attn.work = s.work.data_ptr()
    hy.gdn_shared_attention(args)
    s.check()
    s.args = args
    s.again(always).check()


# ---- weights -------------------------------------------------------------------


class Weight:
    def __init__(self, hy, case, R=0, keep=1.0, fresh=True, first=None, position=None, born=True, seed=0):
        self.hy, self.case, self.opts = hy, case, (keep, fresh)
        g = np.random.default_rng(seed)
        self.q, self.k = (case[x].cuda() for x in ("q", "k_cache"))
        if case["k_cache"].stride(1) == case["k_cache"].shape[3]:
            self.k = case["k_cache"].transpose(1, 2).contiguous().cuda().transpose(1, 2)
        n_pages, H_kv, P, d = self.k.shape
        lse, _ = long_ref.log_sums(*(case[x] for x in ("q", "k_cache", "table", "ctx", "n", "start", "scale")))
        self.lse = torch.tensor(np.where(np.isnan(lse), 1e30, lse), dtype=F32)
        B = len(case["ctx"])
        self.first = np.zeros(B, np.int64) if first is None else np.array(first)
        self.position = case["ctx"] if position is None else np.array(position)
        self.weight0 = g.random(n_pages * P).astype(np.float32)
        if fresh:  # slots of the step's own tokens may hold anything
            for b in range(B):
                for j in range(int(case["ctx"][b]), int(case["ctx"][b] + case["n"][b])):
                    self.weight0[case["table"][b, j // P] * P + j % P] = np.nan
        self.born0 = np.full(n_pages * P, -9)
        self.t = {k: ints(case[k]) for k in ("table", "ctx", "n", "start")}
        self.weight, self.born = torch.tensor(self.weight0, device="cuda"), ints(self.born0)
        self.status = status_word()
        self.tensors = dict(q=self.q, k_cache=self.k, lse=self.lse.cuda(), block_table=self.t["table"], ctx_len=self.t["ctx"],
                            n_rows=self.t["n"], row_start=self.t["start"], weight=self.weight, first=None if first is None else ints(first),
                            position=None if position is None else ints(position), born=self.born if born else None, status=self.status)
        self.args = hy.make_attn_weight_args(**self.tensors, R=R, scale=case["scale"], keep=keep, fresh=fresh)
        self.work = torch.full((hy.attn_weight_work_bytes(self.args),), 255, dtype=torch.uint8, device="cuda")
        self.args.work = self.work.data_ptr()

    def run(self):
        self.hy.gdn_attn_weight(self.args)
        return self

    def expected(self, n=None):
        c, (keep, fresh) = self.case, self.opts
        return long_ref.weights(c["q"], c["k_cache"], self.lse, c["table"], c["ctx"], c["n"] if n is None else n, c["start"], c["scale"], keep,
                                fresh, self.first, self.position, self.weight0, self.born0)

    def check(self, n=None, status=0):
        torch.cuda.synchronize()
        want, born, off = self.expected(n)
        got = self.weight.double().cpu().numpy()
        assert int(self.status.item()) == status
        same = np.isnan(want) == np.isnan(got)
        assert same.all()
        bad = np.abs(got - want) > off
        assert not bad.any(), (np.flatnonzero(bad)[:5], np.nanmax(np.abs(got - want)))
        if self.args.born:
            assert np.array_equal(self.born.cpu().numpy(), born)


WEIGHT = [
    # lens, H_q, H_kv, d, P, dtype, layout, R, first, keep, fresh
    ([(0, 1)], 1, 1, 64, 16, F32, "heads", 1, None, 1.0, True),
    ([(100, 3), (0, 5), (33, 1), (5, 0)], 6, 2, 64, 7, F32, "tokens", 5, [20, 0, 33, 0], 0.5, True),
    ([(300, 70), (0, 130)], 8, 4, 128, 48, F32, "heads", 0, None, 1.0, False),
    ([(64, 2)], 2, 1, 256, 16, F32, "heads", 2, [-5], 1.0, True),
    ([(0, 1)], 1, 1, 64, 16, BF16, "heads", 1, None, 1.0, True),
    ([(100, 3), (0, 5), (33, 1), (5, 0)], 6, 2, 64, 16, BF16, "tokens", 5, [20, 0, 33, 0], 0.5, True),
    ([(1000, 4), (129, 4), (127, 4), (128, 4), (4000, 4)], 16, 2, 256, 16, BF16, "heads", 4, None, 0.99, True),
    ([(3000, 1)], 32, 8, 128, 64, BF16, "heads", 1, [129], 1.0, True),
    ([(300, 70), (0, 130), (511, 257)], 28, 4, 128, 48, BF16, "tokens", 0, [256, 0, 511], 1.0, True),
    ([(40, 200), (0, 1), (700, 3)], 10, 2, 64, 32, BF16, "heads", 0, [300, 0, 0], 0.0, True),
    ([(0, 600)], 8, 1, 256, 128, BF16, "heads", 0, None, 1.0, True),
    ([(5, 1)] * 200 + [(600, 2)], 4, 2, 128, 16, BF16, "heads", 2, None, 1.0, False),
    ([(60, 3), (2, 2)], 128, 1, 64, 16, BF16, "heads", 3, None, 1.0, True),
    ([(700, 16), (20, 7)], 24, 2, 128, 16, BF16, "tokens", 16, None, 1.0, False),
    ([(0, 90), (2000, 33)], 5, 5, 64, 16, BF16, "heads", 0, [40, 17], 1.0, True),
    ([(200, 3), (0, 5)], 128, 1, 256, 16, BF16, "heads", 0, None, 1.0, True),   # heads of a token over two tiles
    ([(130, 2), (300, 1)], 144, 2, 256, 32, BF16, "tokens", 2, [3, 0], 1.0, False),
    ([(70, 3), (0, 2)], 80, 2, 64, 16, F32, "heads", 3, None, 1.0, True),
    ([(3, 2), (0, 0), (1, 1)], 2, 2, 128, 16, BF16, "heads", 2, [5, 0, 2 ** 31 - 1], 1.0, True),  # firsts at and past the end
    ([(2, 40)], 6, 1, 64, 5, F32, "heads", 0, [42], 1.0, True),
]


@pytest.mark.parametrize("lens,H_q,H_kv,d,P,dtype,layout,R,first,keep,fresh", WEIGHT, ids=range(len(WEIGHT)))
def test_weights_match_the_plain_form(hy, lens, H_q, H_kv, d, P, dtype, layout, R, first, keep, fresh):
    case = hybrid_ref.make_attention(lens=lens, H_q=H_q, H_kv=H_kv, d=d, P=P, dtype=dtype, layout=layout, R=R, seed=len(lens))
    position = [1000 + 7 * b for b in range(len(lens))] if R % 2 else None
    w = Weight(hy, case, R, keep, fresh, first, position).run()
    w.check()
    again = Weight(hy, case, R, keep, fresh, first, position).run()
    torch.cuda.synchronize()
    assert torch.equal(again.weight.view(torch.int32), w.weight.view(torch.int32))  # the same bits


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_step_hands_out_one_weight_for_each_row_and_head(hy, dtype):
    """The weights of a request's first step sum to its rows times heads: with the lse that the attention gave."""
    case = long_ref.make_shared(groups=[], alone=[(0, 150), (0, 1), (0, 40)], H_q=8, H_kv=2, d=128, P=16, dtype=dtype)
    s = Shared(hy, case, groups=False).run()
    w = Weight(hy, case)
    w.tensors["lse"] = s.lse
    args = hy.make_attn_weight_args(**w.tensors, scale=case["scale"], fresh=True)
    args.work = w.work.data_ptr()
    hy.gdn_attn_weight(args)
    torch.cuda.synchronize()
    P = 16
    for b, n in enumerate((150, 1, 40)):
        slots = [case["table"][b, j // P] * P + j % P for j in range(n)]
        total = w.weight[slots].double().sum().item()
        # each share is off by at most 2 (d + 4) u of a score's size (below 40 here), lse by as much again
        assert abs(total - n * 8) <= n * 8 * (2 * 2 * 132 * 40 * U + 2 ** -18)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weights_skip_bad_requests_and_pages(hy, dtype):
    case = hybrid_ref.make_attention(lens=[(100, 2), (30, 2), (200, 2), (20, 2)], H_q=4, H_kv=2, d=64, P=16, dtype=dtype, R=2)
    w = Weight(hy, case, 2)
    w.t["n"][1] = -1
    w.t["ctx"][3] = 2 ** 31 - 1
    w.run()
    n = case["n"].copy()
    n[[1, 3]] = 0
    w.check(n=n, status=hy.STATUS_BAD_LENGTH | 2)
    w = Weight(hy, case, 2)
    page = int(case["table"][2, 3])
    w.t["table"][2, 3] = case["k_cache"].shape[0]
    w.run()
    torch.cuda.synchronize()
    want, born, off = w.expected()
    want[page * 16:page * 16 + 16], born[page * 16:page * 16 + 16] = w.weight0[page * 16:page * 16 + 16], -9
    got = w.weight.double().cpu().numpy()
    assert int(w.status.item()) == hy.STATUS_BAD_PAGE
    assert (np.abs(got - want)[~np.isnan(want)] <= off[~np.isnan(want)]).all()
    assert np.array_equal(w.born.cpu().numpy(), born)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weights_with_far_pages_strided_rows_and_a_negative_scale(hy, dtype):
    case = hybrid_ref.make_attention(lens=[(100, 2), (30, 2)], H_q=4, H_kv=2, d=64, P=16, dtype=dtype, R=2, scale=-0.2)
    w = Weight(hy, case, 2)
    pages, far = case["k_cache"].shape[0], 2 ** 29
    pool = torch.empty(pages * far + 4096, dtype=dtype, device="cuda")
    k = pool.as_strided((pages, 2, 16, 64), (far, 1024, 64, 1))
    k.copy_(w.k)
    wide = torch.full((case["q"].shape[0], 9, 64), float("nan"), dtype=dtype, device="cuda")
    wide[:, 2:6] = w.q
    lse = torch.full((w.q.shape[0], 11), float("nan"), device="cuda")
    lse[:, :4] = w.tensors["lse"]
    args = hy.make_attn_weight_args(**(w.tensors | dict(q=wide[:, 2:6], k_cache=k, lse=lse[:, :4])), R=2, scale=-0.2, fresh=True)
    args.work = w.work.data_ptr()
    hy.gdn_attn_weight(args)
    w.check()


@pytest.mark.parametrize("dtype,d,P", [(BF16, 64, 16), (BF16, 256, 48), (F32, 128, 16)])
def test_weights_of_pools_whose_pages_are_no_whole_number_of_heads(hy, dtype, d, P):
    case = hybrid_ref.make_attention(lens=[(300, 2), (30, 2), (5, 1)], H_q=4, H_kv=2, d=d, P=P, dtype=dtype, R=2)
    w = Weight(hy, case, 2)
    pages, stride = case["k_cache"].shape[0], 2 * P * d + 24
    k = torch.full((pages * stride,), float("nan"), dtype=dtype, device="cuda").as_strided((pages, 2, P, d), (stride, P * d, d, 1))
    k.copy_(w.k)
    args = hy.make_attn_weight_args(**(w.tensors | dict(k_cache=k)), R=2, scale=case["scale"], fresh=True)
    args.work = w.work.data_ptr()
    hy.gdn_attn_weight(args)
    w.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weights_of_one_page_and_one_head(hy, dtype):
    for H_kv, P, lens in ((1, 128, [(100, 2)]), (3, 64, [(40, 5)]), (1, 16, [(100, 2), (3, 1)])):
        case = hybrid_ref.make_attention(lens=lens, H_q=3 * H_kv, H_kv=H_kv, d=64, P=P, dtype=dtype, spare=0)
        Weight(hy, case).run().check()


def test_weights_in_a_graph_follow_lengths(hy):
    case = hybrid_ref.make_attention(lens=[(400, 4), (50, 4), (1000, 4)], H_q=16, H_kv=2, d=128, P=16, dtype=BF16, R=4)
    w = Weight(hy, case, 4)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            w.run()
    for n in ([4, 4, 4], [1, 0, 3], [0, 2, 1]):
        w.t["n"].copy_(ints(n))
        w.weight.copy_(torch.tensor(w.weight0))
        w.born.copy_(ints(w.born0))
        graph.replay()
        w.check(n=np.array(n))


# ---- choice and moves ----------------------------------------------------------


def run_select(hy, weight, born, table, ctx, budget, pinned, keep_from, P, max_moves, in_place=False):
    B = len(ctx)
    new = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dict(weight=torch.tensor(weight, device="cuda"), born=None if born is None else ints(born), ctx_len=ints(ctx),
             n_moves=new(B), move_from=new(B, max_moves), move_to=new(B, max_moves), status=status_word())
    t["ctx_out"] = t["ctx_len"] if in_place else new(B)
    hy.gdn_evict_select(hy.make_evict_select_args(**t, block_table=ints(table), budget=ints(budget), page_size=P,
                                                  pinned=None if pinned is None else ints(pinned),
                                                  keep_from=None if keep_from is None else ints(keep_from)))
    torch.cuda.synchronize()
    return {k: None if v is None else v.cpu().numpy() for k, v in t.items()}


def select_case(lens, P, seed, kind):
    g = np.random.default_rng(seed)
    lens = np.array(lens)
    need = np.maximum(-(-lens // P), 0)
    n_pages = int(need.sum()) + 2
    table = np.full((len(lens), int(need.max(initial=0)) + 1), 2 ** 31 - 1)
    table[np.arange(table.shape[1]) < need[:, None]] = g.permutation(n_pages)[:need.sum()]
    N = n_pages * P
    weight = {"plain": lambda: g.exponential(size=N), "ties": lambda: g.integers(-2, 3, N) * 1.0, "same": lambda: np.full(N, 0.25),
              "odd": lambda: g.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0, 1e-45, -1e-45, 3.4e38, -3.4e38], N),
              "close": lambda: 1.0 + g.integers(0, 4000, N) * 2.0 ** -23}[kind]().astype(np.float32)
    return weight, g.integers(0, 2000, N), table, n_pages


SELECT = [
    # lens, P, kind, over, pinned, recent
    ([0, 1, 2, 31, 33, 1023, 1024, 1025], 16, "plain", 0.3, False, False),
    ([0, 1, 2, 31, 33, 1023, 1024, 1025], 16, "ties", 0.5, True, True),
    ([5000, 4097, 3, 20000], 64, "plain", 0.02, True, True),
    ([5000, 4097, 3, 20000], 48, "odd", 0.7, True, False),
    ([3000] * 40, 16, "close", 0.4, False, True),
    ([777] * 300, 7, "ties", 0.1, True, True),
    ([100000, 70000], 128, "plain", 0.5, True, True),
    ([300000], 64, "ties", 0.3, False, True),
    ([9000, 100], 1, "same", 0.9, False, False),
    ([600000], 64, "close", 0.001, True, True),
]


@pytest.mark.parametrize("lens,P,kind,over,pinned,recent", SELECT, ids=range(len(SELECT)))
def test_select_matches_the_definition(hy, lens, P, kind, over, pinned, recent):
    weight, born, table, n_pages = select_case(lens, P, len(lens), kind)
    g = np.random.default_rng(3)
    ctx = np.array(lens)
    budget = (ctx * (1 - over * g.random(len(lens)) * 1.2)).astype(int) - (g.random(len(lens)) < 0.1) * 10
    pins = g.integers(-2, 40, len(lens)) if pinned else None
    keep_from = g.integers(500, 2100, len(lens)) if recent else None
    most = max(int((ctx - np.minimum(budget, ctx)).max()), 1)
    lists = (np.full((len(lens), most), -7), np.full((len(lens), most), -7))
    want = long_ref.select(weight, born if recent else None, table, ctx, budget, np.zeros(len(lens), int) if pins is None else pins, keep_from,
                           P, most, n_pages, lists)
    got = run_select(hy, weight, born if recent else None, table, ctx, budget, pins, keep_from, P, most)
    for key in ("ctx_out", "n_moves", "move_from", "move_to", "born"):
        assert want[key] is None or np.array_equal(got[key], want[key]), key
    assert int(got["status"][0]) == want["status"] == 0
    assert np.array_equal(got["weight"].view(np.int32), want["weight"].view(np.int32))


def test_select_corner_requests(hy):
    """Budgets of nothing, below nothing and above the length, all pinned, all young, nothing over: in place."""
    lens = [50] * 9
    weight, born, table, n_pages = select_case(lens, 16, 1, "plain")
    ctx, budget = np.array(lens), np.array([0, -5, 50, 51, 2 ** 31 - 1, 20, 20, 20, -(2 ** 31)])
    pins = np.array([0, 10, 0, 0, 0, 50, 2 ** 31 - 1, 0, 49])
    keep_from = np.array([3000, 3000, 0, 0, 0, 3000, 3000, -(2 ** 31), 2 ** 31 - 1])
    lists = (np.full((9, 50), -7), np.full((9, 50), -7))
    want = long_ref.select(weight, born, table, ctx, budget, pins, keep_from, 16, 50, n_pages, lists)
    assert want["ctx_out"].tolist() == [0, 10, 50, 50, 50, 50, 50, 50, 49]
    got = run_select(hy, weight, born, table, ctx, budget, pins, keep_from, 16, 50, in_place=True)
    for key in ("ctx_out", "n_moves", "move_from", "move_to", "born"):
        assert np.array_equal(got[key], want[key]), key


def test_select_leaves_bad_requests_as_they_are(hy):
    lens = [100, 100, 100, 100, 100, 100]
    weight, born, table, n_pages = select_case(lens, 16, 2, "plain")
    ctx = np.array(lens)
    ctx[0], ctx[1] = -1, 16 * table.shape[1] + 1
    table[2, 3], table[3, 0] = n_pages, -1
    budget = np.array([10, 10, 10, 10, 50, 97])
    lists = (np.full((6, 7), -7), np.full((6, 7), -7))
    want = long_ref.select(weight, born, table, ctx, budget, np.zeros(6, int), None, 16, 7, n_pages, lists)
    assert want["status"] == 256 | 128 | 1024 and want["ctx_out"][5] == 97
    got = run_select(hy, weight, born, table, ctx, budget, None, None, 16, 7)
    for key in ("ctx_out", "n_moves", "move_from", "move_to", "born"):
        assert np.array_equal(got[key], want[key]), key
    assert int(got["status"][0]) == want["status"]
    assert np.array_equal(got["weight"].view(np.int32), want["weight"].view(np.int32))


def test_select_without_room_for_moves(hy):
    """max_moves 0 serves requests whose last tokens are their lightest."""
    lens = [40, 40]
    weight, born, table, n_pages = select_case(lens, 16, 2, "plain")
    for j in range(40):
        weight[table[0, j // 16] * 16 + j % 16] = 100 - j
        weight[table[1, j // 16] * 16 + j % 16] = j
    got = run_select(hy, weight, None, table, np.array(lens), np.array([30, 30]), None, None, 16, 0)
    assert got["ctx_out"].tolist() == [30, 40] and got["n_moves"].tolist() == [0, 0] and int(got["status"][0]) == hy.STATUS_MOVES_FULL


@pytest.mark.parametrize("B,most,H,d,P,layout,dtype", [(1, 1, 1, 64, 16, "heads", BF16), (5, 70, 3, 128, 48, "tokens", BF16),
                                                       (16, 64, 2, 256, 16, "heads", F32), (3, 900, 8, 64, 7, "tokens", F32),
                                                       (300, 3, 2, 8, 16, "heads", BF16), (2, 1500, 8, 128, 64, "heads", BF16)])
def test_moves_match_the_definition(hy, B, most, H, d, P, layout, dtype):
    g = torch.Generator().manual_seed(B)
    n = torch.randint(0, most + 1, (B,), generator=g)
    n[0] = most
    n_pages = -(-2 * B * most // P) + 3
    pool = torch.randn((n_pages, 2, H, P, d) if layout == "heads" else (n_pages, 2, P, H, d), generator=g).to(dtype).cuda()
    ends = torch.randperm(n_pages * P, generator=g)[:2 * B * most].reshape(2, B, most).to(torch.int32).cuda()
    want = pool.clone()
    view = lambda x: (x if layout == "heads" else x.transpose(2, 3))  # noqa: E731
    flat = view(want).movedim(3, 1).flatten(0, 1) if layout == "tokens" else view(want).movedim(3, 1).reshape(-1, 2, H, d)
    for b in range(B):
        src, dst = (ends[i, b, :n[b]].long() for i in (0, 1))
        got = view(want)[src // P, :, :, src % P]
        view(want)[dst // P, :, :, dst % P] = got
    assert flat.shape[0] == n_pages * P
    status = status_word()
    hy.gdn_kv_move(hy.make_kv_move_args(k_cache=view(pool)[:, 0], v_cache=view(pool)[:, 1], move_from=ends[0].contiguous(),
                                        move_to=ends[1].contiguous(), n_moves=n.to(torch.int32).cuda(), status=status))
    torch.cuda.synchronize()
    assert torch.equal(pool, want) and int(status.item()) == 0


def test_moves_skip_bad_slots_and_counts(hy):
    k, v = (torch.randn((4, 2, 16, 64), device="cuda") for _ in range(2))
    want = [k.clone(), v.clone()]
    src = ints([[0, 64, -1, 3], [4, 5, 6, 7], [8, 9, 10, 11]])
    dst = ints([[20, 21, 22, 64], [24, 25, 26, 27], [28, 29, 30, 31]])
    for x in want:
        x[1, :, 4] = x[0, :, 0]
    status = status_word()
    hy.gdn_kv_move(hy.make_kv_move_args(k_cache=k, v_cache=v, move_from=src, move_to=dst, n_moves=ints([4, 5, -1]), status=status))
    torch.cuda.synchronize()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert int(status.item()) == hy.STATUS_BAD_PAGE | hy.STATUS_BAD_LENGTH


def test_moves_between_far_pages(hy):
    pages, far = 9, 2 ** 29
    pool = torch.empty(pages * far + 4096, dtype=BF16, device="cuda")
    k = pool.as_strided((pages, 2, 16, 64), (far, 1024, 64, 1))
    v = pool.as_strided((pages, 2, 16, 64), (far, 1024, 64, 1), 2048)
    k.normal_()
    v.normal_()
    want = k[8, :, 15].clone(), v[8, :, 15].clone(), k[0, :, 3].clone()
    hy.gdn_kv_move(hy.make_kv_move_args(k_cache=k, v_cache=v, move_from=ints([[8 * 16 + 15, 3]]), move_to=ints([[5 * 16 + 2, 7 * 16]]),
                                        n_moves=ints([2])))
    torch.cuda.synchronize()
    assert torch.equal(k[5, :, 2], want[0]) and torch.equal(v[5, :, 2], want[1]) and torch.equal(k[7, :, 0], want[2])


# ---- all of them, as a step uses them --------------------------------------------


def test_a_request_keeps_attending_to_the_tokens_that_stay(hy):
    """Sixty steps of three requests in two layers' pools with a shared table: pages, append, attention, weights, eviction,
    moves.  A host model keeps each request's tokens as (text position, K, V) in cache order and makes every choice from its own
    64-bit weights where those are not within rounding of each other."""
    g = torch.Generator().manual_seed(3)
    B, R, P, H_q, H_kv, d, N, budget, recent = 3, 4, 16, 8, 2, 64, 64, 60, 8
    new = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    pools = [torch.full((N, 2, H_kv, P, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2)]
    ring, free, held, table = ints(np.random.default_rng(1).permutation(N)), [ints([3, N]), new(2)], [new(B), new(B)], new(B, 20)
    ctx, text, rows, slots, positions, status = new(B), new(B), new(B), new(B * R), new(B * R), status_word()
    weight, born = torch.full((N * P,), float("nan"), device="cuda"), new(N * P) - 5
    n_moves, lists, out_ctx = new(B), [new(B, 16), new(B, 16)], new(B)
    model = [[] for _ in range(B)]  # per request: (position, [(k, v) of each layer])
    seen_moves = seen_pages_back = 0
    for step in range(60):  # some 120 tokens a request, twice its budget
        n = torch.randint(0, R + 1, (B,), generator=g)
        a, b_ = step % 2, 1 - step % 2
        hy.gdn_page_map(hy.make_page_map_args(
            ctx_len=ctx, n_rows=n.to(torch.int32).cuda(), held=held[a], free_ring=ring, free_state=free[a], block_table=table,
            held_out=held[b_], free_state_out=free[b_], rows_out=rows, slot_map=slots, positions=positions, page_size=P, R=R, status=status))
        for layer in range(2):
            x = torch.randn((B * R, H_q + 2 * H_kv, d), generator=g).to(BF16).cuda()
            k, v = x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
            kc, vc = pools[layer][:, 0], pools[layer][:, 1]
            hy.gdn_kv_append(hy.make_kv_append_args(k=k, v=v, slot_map=slots, k_cache=kc, v_cache=vc, status=status))
            o, lse = torch.zeros_like(x[:, :H_q]).contiguous(), torch.zeros((B * R, H_q), device="cuda")
            args = hy.make_shared_attention_args(q=x[:, :H_q], k_cache=kc, v_cache=vc, block_table=table, ctx_len=ctx, n_rows=rows, R=R,
                                                 o=o, lse=lse, status=status)
            work = torch.empty(hy.shared_attention_work_bytes(args), dtype=torch.uint8, device="cuda")
            args.attn.work = work.data_ptr()
            hy.gdn_shared_attention(args)
            wargs = hy.make_attn_weight_args(q=x[:, :H_q], k_cache=kc, lse=lse, block_table=table, ctx_len=ctx, n_rows=rows, R=R, weight=weight,
                                             born=born, position=text, fresh=layer == 0, keep=0.9 if layer == 0 else 1.0, status=status)
            wwork = torch.empty(hy.attn_weight_work_bytes(wargs), dtype=torch.uint8, device="cuda")
            wargs.work = wwork.data_ptr()
            hy.gdn_attn_weight(wargs)
            torch.cuda.synchronize()
            for b in range(B):
                m = int(n[b])
                if layer == 0:
                    model[b] += [[int(text[b]) + t, []] for t in range(m)]
                for t in range(m):
                    model[b][len(model[b]) - m + t][1].append((k[b * R + t], v[b * R + t]))
                if m == 0:
                    continue
                K, V = (torch.stack([tok[1][layer][i] for tok in model[b]]).double().repeat_interleave(H_q // H_kv, 1) for i in (0, 1))
                z = torch.einsum("thd,lhd->htl", x[b * R:b * R + m, :H_q].double(), K) * d ** -0.5
                z = z.masked_fill(torch.ones(m, len(model[b]), device="cuda").triu(len(model[b]) - m + 1).bool(), -float("inf"))
                ref = torch.einsum("htl,lhd->thd", torch.softmax(z, 2), V)
                top = V.abs().max()
                assert (o[b * R:b * R + m].double() - ref).abs().max() <= 2.0 ** -8 * (top + ref.abs().max()) + 1e-5 * top
        ctx += rows
        text += rows
        lens = ctx.cpu().numpy()
        assert lens.tolist() == [len(m) for m in model]
        old_weight, old_born = weight.cpu().numpy(), born.cpu().numpy()
        tab = table.cpu().numpy()
        at = [[tab[b, j // P] * P + j % P for j in range(lens[b])] for b in range(B)]
        for b in range(B):  # each token's text position travelled with it
            assert old_born[at[b]].tolist() == [tok[0] for tok in model[b]]
        keep_from = text - recent
        hy.gdn_evict_select(hy.make_evict_select_args(weight=weight, born=born, block_table=table, ctx_len=ctx, budget=ints([budget] * B),
                                                      ctx_out=ctx, n_moves=n_moves, move_from=lists[0], move_to=lists[1], page_size=P,
                                                      pinned=ints([0, 4, 17]), keep_from=keep_from, status=status))
        for pool in pools:
            hy.gdn_kv_move(hy.make_kv_move_args(k_cache=pool[:, 0], v_cache=pool[:, 1], move_from=lists[0], move_to=lists[1], n_moves=n_moves,
                                                status=status))
        torch.cuda.synchronize()
        want = long_ref.select(old_weight, old_born, tab, lens, np.array([budget] * B), np.array([0, 4, 17]), keep_from.cpu().numpy(), P, 16, N,
                               [np.zeros((B, 16), int)] * 2)
        assert ctx.cpu().numpy().tolist() == want["ctx_out"].tolist() and n_moves.cpu().numpy().tolist() == want["n_moves"].tolist()
        for b in range(B):
            where = {s: j for j, s in enumerate(at[b])}
            for i in range(int(want["n_moves"][b])):
                model[b][where[want["move_to"][b, i]]] = model[b][where[want["move_from"][b, i]]]
                seen_moves += 1
            seen_pages_back += -(-len(model[b]) // P) - -(-int(want["ctx_out"][b]) // P)
            del model[b][int(want["ctx_out"][b]):]
        assert int(status.item()) == 0
    assert seen_moves > 20 and seen_pages_back >= 0 and all(len(m) <= budget for m in model)


# ---- bounded waits, streams ------------------------------------------------------


def test_a_wait_that_runs_out_ends_the_shared_attention(hy, always):
    """A block whose first K copy never lands gives up; rows that it had no part in are right, and the context serves the next
    call.  No copy is in flight: it was declared on its barrier and not issued."""
    case = long_ref.make_shared(groups=[(300, [(i, 1) for i in range(20)])], alone=[(200, 1)] * 20, H_q=16, H_kv=8, d=128, P=16,
                                dtype=BF16, R=1)
    s = Shared(hy, case, 1)
    assert always.gdn_test_drop_shared_copy(0) == 0
    s.run(always)
    torch.cuda.synchronize()  # returns: no wait is without bound
    assert int(s.status.item()) == 8
    # block 0 begins with request 0's own keys
    ref, vmax = hybrid_ref.attention(*(case[x] for x in ("q", "k_cache", "v_cache", "table", "ctx", "n", "start", "scale")))
    bound = 2.0 ** -8 * (vmax[..., None] + np.abs(ref)) + 1e-5 * vmax[..., None]
    assert (np.abs(s.o.double().cpu().numpy() - ref)[25:] <= bound[25:]).all()
    assert always.gdn_test_drop_shared_copy(-1) == 0
    s.again(always).check()


def test_a_wait_that_runs_out_ends_the_weights(hy, always):
    case = hybrid_ref.make_attention(lens=[(1500, 2)] * 30, H_q=16, H_kv=4, d=128, P=16, dtype=BF16, R=2)
    w = Weight(hy, case, 2)
    assert always.gdn_test_drop_weight_copy(3) == 0
    assert always.gdn_attn_weight(w.args, torch.cuda.current_stream().cuda_stream or None) == 0
    torch.cuda.synchronize()
    assert int(w.status.item()) == 8
    # 30 requests of 12 key blocks and 4 heads, three units each, over 152 blocks: block 3 has units of request 0 and 1 alone
    want, _, off = w.expected()
    slots = (case["table"][2:, :94, None] * 16 + np.arange(16)).reshape(28, -1)[:, :1500]
    got = w.weight.double().cpu().numpy()
    assert (np.abs(got - want)[slots] <= off[slots]).all()
    assert always.gdn_test_drop_weight_copy(-1) == 0
    w.weight.copy_(torch.tensor(w.weight0))
    w.born.copy_(ints(w.born0))
    w.status.zero_()
    assert always.gdn_attn_weight(w.args, torch.cuda.current_stream().cuda_stream or None) == 0
    w.check()


def test_calls_on_two_streams_with_buffers_of_their_own(hy):
    case = long_ref.make_shared(groups=[(900, [(5 * i, 2) for i in range(12)])], alone=[(400, 2)], H_q=16, H_kv=4, d=128, P=16, dtype=BF16, R=2)
    attend = [Shared(hy, case, 2) for _ in range(2)]
    weigh = [Weight(hy, case, 2, first=case["ctx"] - 3) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, w, stream in zip(attend, weigh, streams):
            hy.gdn_shared_attention(s.args, stream)
            w.weight.record_stream(stream)
            with torch.cuda.stream(stream):
                w.weight.copy_(torch.tensor(w.weight0), non_blocking=False)
            hy.gdn_attn_weight(w.args, stream)
    torch.cuda.synchronize()
    for s, w in zip(attend, weigh):
        s.check()
        w.check()
