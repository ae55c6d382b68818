"""w4_attn_decode_shared against attention in 64 bits over each request's prefix and own tokens in one row."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from oracle import kv_oracle as KO
from oracle import kv_share_oracle as SO
from tests.kv_cases import DEV, bf16_tensor, gpu, paged, values

pytestmark = pytest.mark.gpu

HEADS = [(16, 4, 256), (40, 8, 128), (64, 8, 128), (7, 1, 64), (6, 3, 80), (4, 4, 112), (8, 2, 192), (5, 1, 16), (36, 2, 96)]


class Case:
    """Groups of requests over shared prefixes; NaN in every place of the cache that no request reads.

    groups: (prefix length, [(own tokens, rows) of each request]); `alone` requests before and after them.
    whole: (group, request) whose own length is shorter than that: they lie within the prefix, on pages of their own.
    """

    def __init__(self, groups, Hq, H, D, P, before=(), after=(), whole=(), order="token", format=16, seed=0, std=1.0):
        self.P, self.format = P, format
        rng = np.random.default_rng(seed)
        lens, fresh, prefix_of, starts = [], [], [], []
        for own, n in before:
            lens.append(own), fresh.append(n), prefix_of.append(None)
        for g, (m, members) in enumerate(groups):
            starts.append(len(lens))
            for own, n in members:
                lens.append(m + own), fresh.append(n), prefix_of.append((g, m))
        starts.append(len(lens))
        for own, n in after:
            lens.append(own), fresh.append(n), prefix_of.append(None)
        for g, i, n in whole:
            lens[starts[g] + i] = n
        for b, p in enumerate(prefix_of):
            if p is not None and lens[b] - fresh[b] < p[1]:
                prefix_of[b] = None
        self.lens, self.fresh, self.prefix_of = lens, fresh, prefix_of
        self.group_starts = np.array(starts, np.int32)
        self.prefix_lens = np.array([m for m, _ in groups], np.int32)
        self.starts = np.concatenate([[0], np.cumsum(fresh)]).astype(np.int32)
        T = int(self.starts[-1])
        have_p = [-(-m // P) for m, _ in groups]
        # own pages: from the page on that the prefix ends in; all, where a request is read on its own
        first = [p[1] // P if p is not None else 0 for p in prefix_of]
        have = [-(-n // P) for n in lens]
        pages = sum(have_p) + sum(h - f for h, f in zip(have, first)) + 3
        ids = rng.permutation(pages)
        self.prefix_table = np.full((len(groups), max(have_p, default=0) + 2), -1, np.int32)
        self.table = np.full((len(lens), max(have, default=0) + 2), -1, np.int32)
        at = 0
        for g, h in enumerate(have_p):
            self.prefix_table[g, :h] = ids[at:at + h]
            at += h
        for b, (h, f) in enumerate(zip(have, first)):
            # (entries of shared pages are never read: page 0 or none at all)
            self.table[b, :f] = rng.choice([-1, 0])
            self.table[b, f:h] = ids[at:at + h - f]
            at += h - f
        self.rows = SO.token_rows(self.table, lens, P, prefix_of, self.prefix_table)
        read = np.zeros(pages * P, bool)
        read[self.rows[self.rows >= 0]] = True
        for g, (m, _) in enumerate(groups):  # rows of a prefix are read even where no request stands behind it
            p = np.arange(m)
            read[self.prefix_table[g, p // P].astype(np.int64) * P + p % P] = True
        free = torch.tensor(~read.reshape(pages, P))
        kd, vd = bf16_tensor((pages, P, H, D), seed + 1, std), bf16_tensor((pages, P, H, D), seed + 2)
        self.q = bf16_tensor((T, Hq, D), seed + 3, 1.5)
        self.scales = {}
        self.k, self.v = paged(pages, P, H, D, order, 0.0, 0)
        if format == 16:
            kd[free], vd[free] = float("nan"), float("nan")
            self.k.copy_(kd), self.v.copy_(vd)
            self.kv, self.vv = values(kd), values(vd)
        else:
            out = []
            for x in (kd, vd):
                codes, scale = KO.rtn8(values(x))
                scale[free.numpy()] = np.nan
                out.append((torch.tensor(codes), torch.tensor(scale, dtype=torch.bfloat16).transpose(1, 2).contiguous().to(DEV), codes * scale[..., None]))
            like = self.k
            self.k, self.v = (torch.empty_strided(like.shape, like.stride(), dtype=torch.int8, device=DEV).copy_(x[0]) for x in out)
            self.scales = {"k_scales": out[0][1], "v_scales": out[1][1]}
            self.kv, self.vv = out[0][2], out[1][2]

    def args(self):
        return dict(q=self.q.to(DEV), k_cache=self.k, v_cache=self.v, block_table=gpu(self.table), lens=gpu(self.lens),
                    group_starts=gpu(self.group_starts), prefix_table=gpu(self.prefix_table), prefix_lens=gpu(self.prefix_lens),
                    starts=gpu(self.starts), **self.scales)

    def run(self, status=0, **more):
        out = w4.w4_attn_decode_shared(**{**self.args(), **more})
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == status
        return out

    def check(self, out, scale=None, rows=slice(None)):
        D = self.q.shape[2]
        flat = [x.reshape(-1, 1, *x.shape[2:]) for x in (self.kv, self.vv)]
        ref, spread, largest = KO.attention(values(self.q), *flat, self.rows, self.lens, self.starts, D ** -0.5 if scale is None else scale)
        bound = KO.attention_bound(ref, spread, largest, D, max(self.lens, default=1), self.format)
        got, ref, bound = (x[rows] for x in (values(out), ref, bound))
        assert np.isfinite(got).all(), f"{np.count_nonzero(~np.isfinite(got))} values are not finite"
        worst = (np.abs(got - ref) / np.maximum(bound, 1e-300)).max() if got.size else 0.0
        assert worst <= 1.0, f"largest error is {worst:.3g} of the bound"


def members(*own, n=1):
    return [(o, n) for o in own]


FEW = [(77, members(1, 2, 17, 40)), (1, members(1, 33)), (0, members(5, 1)), (160, members(3)), (16, members(16, 1, 64, 9, 130))]


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D", HEADS)
def test_heads(cuda_lib, Hq, H, D, format):
    case = Case(FEW, Hq, H, D, 16, before=members(7, 70), after=members(1), format=format, seed=D + Hq)
    case.check(case.run())


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("order,P", [("token", 1), ("token", 3), ("head", 16), ("pair", 24), ("head", 64), ("token", 700)])
def test_page_sizes_and_orders(cuda_lib, order, P, format):
    case = Case(FEW, 10, 2, 128, P, after=members(50, 8), order=order, format=format, seed=P)
    case.check(case.run())


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257, 500, 1025])
def test_prefix_lengths(cuda_lib, length, format):
    for Hq, H, D in ((8, 2, 128), (16, 2, 64)):
        case = Case([(length, members(1, 5, 30))], Hq, H, D, 16, format=format, seed=length)
        case.check(case.run(starts=None))


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D", [(16, 4, 256), (40, 8, 128), (64, 8, 64), (6, 3, 80), (36, 2, 96), (8, 2, 192)])
@pytest.mark.parametrize("count", [9, 30, 70])
def test_many_requests_behind_a_prefix(cuda_lib, Hq, H, D, count, format):
    """Rows to a head from a few to many hundreds: every kernel of the first pass, the few-row one of the second."""
    rng = np.random.default_rng(count)
    groups = [(300, members(*rng.integers(1, 40, count))), (129, members(*rng.integers(1, 40, 3)))]
    case = Case(groups, Hq, H, D, 16, after=members(5), format=format, seed=count)
    case.check(case.run())


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D", [(16, 4, 256), (64, 8, 128), (16, 1, 64), (12, 2, 112)])
@pytest.mark.parametrize("rows", [2, 5, 13])
def test_verify_passes(cuda_lib, Hq, H, D, rows, format):
    """Many rows to a request: the many-row kernel in both passes (13 rows of 8 query heads), requests without rows."""
    groups = [(200, [(rows, rows), (rows + 9, rows), (60, rows)]), (65, [(30, 0), (rows, rows), (14, 1)]), (40, [(3, 0)])]
    case = Case(groups, Hq, H, D, 16, before=[(rows, rows), (3, 0)], after=[(100, rows)], format=format, seed=rows)
    case.check(case.run())


@pytest.mark.parametrize("format", [16, 8])
def test_long_prefixes_and_own_tokens(cuda_lib, format):
    """Parts of many CTAs in both passes."""
    case = Case([(6000, members(3000, 17, 1)), (2500, members(1, 900))], 8, 2, 128, 16, format=format, seed=1)
    case.check(case.run())
    case = Case([(5000, [(40, 13)] * 8)], 16, 2, 128, 32, format=format, seed=2)
    case.check(case.run())


@pytest.mark.parametrize("format", [16, 8])
def test_requests_within_the_prefix_are_read_on_their_own(cuda_lib, format):
    groups = [(100, [(5, 1), (5, 2), (9, 5), (30, 5)]), (50, [(5, 1), (1, 1)])]
    # lengths below the prefix, at its end, and with the first of their new tokens inside of it
    case = Case(groups, 8, 2, 128, 16, whole=[(0, 0, 60), (0, 1, 101), (0, 2, 103), (1, 0, 50)], format=format, seed=3)
    assert [p is None for p in case.prefix_of] == [True, True, True, False, True, False]
    case.check(case.run())


def test_rows_that_see_nothing_are_zeros(cuda_lib):
    """Padded requests (length 0 with a row) and more rows than tokens, inside and outside of a group."""
    groups = [(64, [(5, 1), (5, 1), (5, 3), (20, 1)])]
    case = Case(groups, 8, 2, 128, 16, after=[(0, 1), (1, 3)], whole=[(0, 1, 0), (0, 2, 1)], seed=4)
    out = case.run()
    case.check(out)
    assert (out[1] == 0).all() and (out[2:4] == 0).all() and (out[6] == 0).all() and (out[7:9] == 0).all()


def test_no_groups_is_the_other_call(cuda_lib):
    case = Case([], 8, 2, 128, 16, after=members(70, 5, 300), seed=5)
    out = case.run()
    case.check(out)
    kw = case.args()
    for name in ("group_starts", "prefix_table", "prefix_lens"):
        del kw[name]
    assert torch.equal(out.view(torch.int16), w4.w4_attn_decode(**kw).view(torch.int16))


def test_scores_far_apart(cuda_lib):
    """The weights of one of the two passes vanish beside the other's; scales of both signs and zero."""
    for std in (0.01, 20.0):
        for scale in (None, -0.3, 0.0):
            case = Case(FEW, 8, 2, 128, 16, seed=6, std=std)
            case.check(case.run(scale=scale), scale=scale)
    case = Case([(200, members(*[50] * 40))], 8, 2, 128, 16, seed=7)
    for part in (0, 1):  # own keys, or the prefix's, a hundred times as large
        for x in (case.k,):
            ids = torch.tensor(np.unique(case.prefix_table[case.prefix_table >= 0]), device=DEV)
            mask = torch.zeros(x.shape[0], dtype=torch.bool, device=DEV)
            mask[ids] = True
            x[mask if part else ~mask] *= 100 if part == 0 else 1e4
        case.kv = values(case.k)
        case.check(case.run())


def test_rows_behind_the_last_are_left_as_they_were(cuda_lib):
    case = Case(FEW, 8, 2, 128, 16, seed=8)
    T = case.q.shape[0]
    q = torch.cat([case.q, torch.full((5, 8, 128), float("nan"), dtype=torch.bfloat16)]).to(DEV)
    out = torch.full_like(q, 7.0)
    case.run(q=q, out=out)
    assert (out[T:] == 7).all()
    case.check(out[:T])


def test_in_place_strided_and_with_a_workspace(cuda_lib):
    case = Case(FEW, 8, 2, 128, 16, seed=9)
    first = case.run()
    T = case.q.shape[0]
    wide = torch.zeros((T, 12, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, :8] = case.q.to(DEV)
    out = case.run(q=wide[:, :8], out=wide[:, :8])
    assert torch.equal(out.contiguous().view(torch.int16), first.view(torch.int16))
    size = w4.w4_attn_decode_shared_workspace_bytes(case.q.to(DEV), case.k, len(case.lens), len(case.prefix_lens))
    for fill in (0, 255, 77):  # what the workspace holds before does not matter
        scratch = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        for _ in range(2):
            assert torch.equal(case.run(workspace=scratch).view(torch.int16), first.view(torch.int16))
    with pytest.raises(w4.W4Error):
        case.run(workspace=torch.empty(size - 1, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("rows", [1, 13])
def test_the_same_bits_in_every_run_and_in_graphs(cuda_lib, rows):
    case = Case([(3000, [(50, rows)] * 9), (700, [(300, rows)] * 2)], 16, 2, 128, 16, seed=10)
    first = case.run()
    size = w4.w4_attn_decode_shared_workspace_bytes(case.q.to(DEV), case.k, len(case.lens), len(case.prefix_lens))
    scratch = torch.empty(size, dtype=torch.uint8, device=DEV)
    kw, outs = case.args(), [torch.zeros_like(first) for _ in range(2)]
    graphs = []
    for out in outs:  # two graphs over one workspace, one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w4.w4_attn_decode_shared(**kw, out=out, workspace=scratch)
        graphs.append(graph)
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0
        for out in outs:
            assert torch.equal(out.view(torch.int16), first.view(torch.int16))


def test_a_graph_follows_its_lengths(cuda_lib):
    """Lengths, tables and groups are read at replay."""
    cases = [Case([(m, members(*own)) for m, own in groups], 8, 2, 128, 16, after=members(9), seed=20 + i)
             for i, groups in enumerate([((100, (5, 30, 1)), (33, (2, 8))), ((7, (90,)), (64, (1, 1, 1, 50))), ((300, (1, 1, 1, 1)), (0, (70,)))])]
    width = max(c.table.shape[1] for c in cases)
    prefix_width = max(c.prefix_table.shape[1] for c in cases)
    for c in cases:
        c.table = np.pad(c.table, ((0, 0), (0, width - c.table.shape[1])), constant_values=-1)
        c.prefix_table = np.pad(c.prefix_table, ((0, 0), (0, prefix_width - c.prefix_table.shape[1])), constant_values=-1)
    pages = max(c.k.shape[0] for c in cases)
    kw = cases[0].args()
    kw["k_cache"], kw["v_cache"] = (torch.zeros((pages, 16, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.empty_like(kw["q"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4_attn_decode_shared(**kw, out=out)
    for c in cases:
        for name, x in c.args().items():
            (kw[name][:x.shape[0]] if name.endswith("cache") else kw[name]).copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0
        c.check(out)


def test_calls_on_two_streams_at_once(cuda_lib):
    cases = [Case([(2000, members(*[30 + i] * 12))], 8, 2, 128, 16, seed=30 + i) for i in range(2)]
    kws = [c.args() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (s, kw) in enumerate(zip(streams, kws)):
            with torch.cuda.stream(s):
                outs[i].append(w4.w4_attn_decode_shared(**kw))
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        c.check(out[0])
        assert all(torch.equal(x.view(torch.int16), out[0].view(torch.int16)) for x in out)


def test_not_finite_values_that_a_row_sees(cuda_lib):
    """A NaN in a prefix reaches the rows behind it, in its column, and no other row."""
    case = Case([(90, members(5, 30)), (40, members(6, 2))], 8, 2, 128, 16, after=members(12), seed=11)
    clean = case.run()
    page = int(case.prefix_table[0, 2])
    case.v[page, 3, 1, 77] = float("nan")
    got = case.run()
    spoilt = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
    spoilt[:2, 4:, 77] = True
    assert torch.isnan(got[spoilt]).all()
    assert torch.equal(got[~spoilt].view(torch.int16), clean[~spoilt].view(torch.int16))


def test_numbers_out_of_range(cuda_lib):
    """Reported, and nothing out of bounds is read: rows that do not depend on them are as ever."""
    case = Case(FEW, 8, 2, 128, 16, before=members(20), after=members(30), seed=12)
    bad = w4.W4_ERR_INVALID_ARG
    table = case.prefix_table.copy()
    table[0, 1], table[0, 2] = 10 ** 6, -1
    last = slice(int(case.starts[case.group_starts[1]]), None)
    case.check(case.run(status=bad, prefix_table=gpu(table)), rows=last)
    lens = case.prefix_lens.copy()
    lens[0] = 10 ** 9
    case.check(case.run(status=bad, prefix_lens=gpu(lens)), rows=last)
    lens[0] = -3
    out = case.run(status=bad, prefix_lens=gpu(lens))
    case.check(out, rows=slice(0, 1))
    # requests of no group where group_starts fall or pass the batch
    for starts in ([-5, 4, 4, 4, 4, 4], [0, 99, 99, 99, 99, 99], [9, 7, 5, 3, 1, 0]):
        torch.cuda.synchronize()
        w4.w4_attn_decode_shared(**{**case.args(), "group_starts": gpu(starts)})
        torch.cuda.synchronize()
        w4.w4_last_device_status()
    case.check(case.run())


def test_a_cache_past_2_to_the_32_bytes(cuda_lib):
    """Prefix and own pages at the far end of a cache of 4.6 GB."""
    case = Case([(200, members(5, 60, 33))], 8, 2, 128, 16, seed=13)
    pages, far = case.k.shape[0], 280000
    both = torch.zeros((2, far, 16, 2, 128), dtype=torch.bfloat16, device=DEV)
    both[0, far - pages:], both[1, far - pages:] = case.k, case.v
    shift = lambda t: gpu(np.where(t >= 0, t + far - pages, -1))  # noqa: E731
    out = case.run(k_cache=both[0], v_cache=both[1], block_table=shift(case.table), prefix_table=shift(case.prefix_table))
    case.check(out)


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("order,P", [("token", 1), ("token", 3), ("token", 8), ("head", 8), ("head", 16), ("pair", 24), ("pair", 32), ("head", 64),
                                     ("token", 128), ("head", 256), ("pair", 256), ("token", 384), ("token", 700)])
def test_page_sizes_and_orders_of_many_rows(cuda_lib, order, P, format):
    """Whole tiles in boxes, where pages divide tiles or tiles pages, and by rows; ends inside of a page and of a tile."""
    groups = [(300, members(*range(1, 41))), (512, members(*range(20, 50))), (97, members(*[3] * 30))]
    for Hq, H, D in ((10, 2, 128), (24, 3, 64), (8, 1, 80)):
        case = Case(groups, Hq, H, D, P, after=members(50, 8), order=order, format=format, seed=P + D)
        case.check(case.run())


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("length", [1, 8, 127, 128, 129, 256, 384, 385, 511, 512, 513, 640, 900])
def test_prefix_lengths_of_many_rows(cuda_lib, length, format):
    """One to eight tiles, for each of the two groups of rows that take them in turn."""
    for Hq, H, D in ((16, 2, 128), (8, 1, 64), (8, 1, 256)):
        case = Case([(length, members(*[1, 5, 30] * 12))], Hq, H, D, 16, format=format, seed=length)
        case.check(case.run(starts=None))


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("P", [16, 24])
def test_numbers_out_of_range_under_many_rows(cuda_lib, P, format):
    case = Case([(300, members(*[9] * 40)), (300, members(*[9] * 40))], 8, 1, 128, P, after=members(30), format=format, seed=15)
    table = case.prefix_table.copy()
    table[0, 1], table[0, 2], table[0, 5] = 10 ** 6, -1, case.k.shape[0]
    last = slice(int(case.starts[case.group_starts[1]]), None)
    case.check(case.run(status=w4.W4_ERR_INVALID_ARG, prefix_table=gpu(table)), rows=last)
    case.check(case.run())


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_values_under_many_rows(cuda_lib, where, value):
    """They reach every row behind their prefix, through its head, and no other row."""
    case = Case([(300, members(*[5] * 40)), (200, members(*[6] * 40))], 16, 2, 128, 16, after=members(12), seed=16)
    clean = case.run()
    (case.k if where == "k" else case.v)[int(case.prefix_table[0, 9]), 3, 1, 77] = value
    got = case.run()
    spoilt = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
    spoilt[:40, 8:, :] = where == "k"
    spoilt[:40, 8:, 77] = True
    if where == "v" or value != value:
        assert (~torch.isfinite(got[spoilt])).all()
    assert torch.equal(got[~spoilt].view(torch.int16), clean[~spoilt].view(torch.int16))


def test_a_cache_past_2_to_the_32_bytes_under_many_rows(cuda_lib):
    """Tiles in boxes and by rows, at the far end of a cache of 4.6 GB."""
    for P in (16, 24):
        case = Case([(300, members(*range(3, 43)))], 8, 1, 128, P, seed=17)
        pages, far = case.k.shape[0], 280000 * 32 // P
        both = torch.zeros((2, far, P, 1, 128), dtype=torch.bfloat16, device=DEV)
        both[0, far - pages:], both[1, far - pages:] = case.k, case.v
        shift = lambda t: gpu(np.where(t >= 0, t + far - pages, -1))  # noqa: E731
        case.check(case.run(k_cache=both[0], v_cache=both[1], block_table=shift(case.table), prefix_table=shift(case.prefix_table)))


def test_checks_of_the_binding(cuda_lib):
    case = Case(FEW, 8, 2, 128, 16, seed=14)
    kw = case.args()
    for name, value, error in (("group_starts", kw["group_starts"][:-1], ValueError), ("prefix_lens", kw["prefix_lens"].long(), TypeError),
                               ("prefix_table", kw["prefix_table"].t(), ValueError), ("prefix_table", kw["prefix_table"][0], ValueError),
                               ("lens", kw["lens"].cpu(), TypeError), ("starts", kw["starts"][1:], ValueError)):
        with pytest.raises(error):
            w4.w4_attn_decode_shared(**{**kw, name: value})


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D", [(16, 1, 128), (16, 2, 64), (48, 2, 128)])
def test_long_prefixes_of_many_rows_in_every_run(cuda_lib, Hq, H, D, format):
    """Scores and weights of dozens of tiles take turns in tensor memory: the same bits each time, and the right ones."""
    case = Case([(9000, members(*[3] * 9)), (4000, members(*[2] * 12)), (257, members(*[1] * 10))], Hq, H, D, 16, format=format, seed=D + Hq)
    first = case.run()
    case.check(first)
    for _ in range(20):
        assert torch.equal(case.run().view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D", [(8, 1, 128), (8, 1, 64), (16, 2, 256), (24, 2, 80)])
@pytest.mark.parametrize("scale", [None, -0.3, 0.0, 1e-3])
def test_scales_of_both_signs_and_zero_under_many_rows(cuda_lib, Hq, H, D, scale, format):
    """The kernels of many rows: queries' signs turned over, every weight 1; whole tiles and an item's end."""
    case = Case([(200, members(*[5] * 40)), (300, members(*[2, 9] * 20)), (128, members(*[3] * 40))], Hq, H, D, 16, format=format, seed=D)
    case.check(case.run(scale=scale), scale=scale)


@pytest.mark.parametrize("Hq,H", [(8, 2), (16, 1)])
@pytest.mark.parametrize("starts", [[-5, 4, 4, 4, 4, 4], [0, 99, 99, 99, 99, 99], [9, 7, 5, 3, 1, 0], [3, 6, 0, 2, 2, 2], [5, 9, 0, 3, 3, 3],
                                    [-2 ** 31, 2 ** 31 - 1, 0, 0, 0, 0], [2 ** 31 - 1] * 6, [-1] * 6])
def test_group_starts_that_fall_or_pass_the_batch(cuda_lib, Hq, H, starts):
    """Requests of one prefix whose tables have its pages, too: whichever of them stand in a group, and in which, the rows
    are the same.  (No request stands in two groups here.)"""
    case = Case([(64, members(5, 1, 30, 9, 2, 70, 1, 1, 16))], Hq, H, 128, 16, seed=18)
    table = case.table.copy()
    table[:, :4] = case.prefix_table[0, :4]
    kw = dict(group_starts=gpu(starts), prefix_table=gpu(np.repeat(case.prefix_table, 5, 0)), prefix_lens=gpu([64] * 5), block_table=gpu(table))
    case.check(case.run(**kw))
    case.check(case.run(**kw, starts=None))


def test_a_negative_prefix_length_is_none(cuda_lib):
    case = Case(FEW, 8, 2, 128, 16, before=members(20), after=members(30), seed=12)
    lens = case.prefix_lens.copy()
    lens[0] = -3
    out = case.run(status=w4.W4_ERR_INVALID_ARG, prefix_lens=gpu(lens))
    case.check(out, rows=slice(0, 1))
    case.check(out, rows=slice(int(case.starts[case.group_starts[1]]), None))


@pytest.mark.parametrize("Hq,H", [(8, 2), (64, 1)])
def test_what_the_stream_did_before_is_seen_by_every_kernel(cuda_lib, Hq, H):
    """Tables, lengths, queries and pages that change right before each call."""
    cases = [Case([(m, members(*own)) for m, own in groups], Hq, H, 128, 16, after=members(9), seed=40 + i)
             for i, groups in enumerate([((100, (5, 30, 1)), (33, (2, 8))), ((130, (90, 2, 3)), (64, (1, 50)))])]
    width, prefix_width = max(c.table.shape[1] for c in cases), max(c.prefix_table.shape[1] for c in cases)
    for c in cases:
        c.table = np.pad(c.table, ((0, 0), (0, width - c.table.shape[1])), constant_values=-1)
        c.prefix_table = np.pad(c.prefix_table, ((0, 0), (0, prefix_width - c.prefix_table.shape[1])), constant_values=-1)
    pages = max(c.k.shape[0] for c in cases)
    kw = cases[0].args()
    kw["k_cache"], kw["v_cache"] = (torch.zeros((pages, 16, H, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    args = [c.args() for c in cases]
    torch.cuda.synchronize()
    outs = []
    for i in range(60):
        for name, x in args[i % 2].items():
            (kw[name][:x.shape[0]] if name.endswith("cache") else kw[name]).copy_(x)
        outs.append(w4.w4_attn_decode_shared(**kw))
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    for i, c in enumerate(cases):
        c.check(outs[i])
        assert all(torch.equal(x.view(torch.int16), outs[i].view(torch.int16)) for x in outs[i::2])
