"""w4_kv_append_norm against its restatement in 64 bits: head layouts, rotations, weights, formats, extreme rows."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from oracle import kv_oracle as KO
from oracle import kv_share_oracle as SO
from tests.kv_cases import DEV, bf16_tensor, gpu, paged, values

pytestmark = pytest.mark.gpu

ROWS = 500


class Case:
    def __init__(self, T, Hq, H, D, rotary, sections=None, cycled=False, paired=False, dtype=torch.bfloat16, offset=False,
                 eps=1e-6, format=16, order="token", page_size=16, seed=0, k=None, q=None, fused=True):
        self.eps, self.offset, self.format = eps, offset, format
        self.kw = dict(eps=eps, unit_offset=offset, sections=sections, cycled=cycled, paired=paired)
        self.sections = sections or (rotary // 2,)
        rng = np.random.default_rng(seed)
        base = bf16_tensor((T, Hq + 2 * H, D), seed, 2.0)
        if q is not None:
            base[:, :Hq] = q
        if k is not None:
            base[:, Hq:Hq + H] = k
        base = base.to(DEV)
        if not fused:  # heads before tokens
            base = base.transpose(0, 1).contiguous().transpose(0, 1)
        self.q, self.k, self.v = base[:, :Hq], base[:, Hq:Hq + H], base[:, Hq + H:]
        self.qw, self.kw_ = ((torch.tensor(rng.normal(0 if offset else 1, 0.3, D)).to(dtype)).to(DEV) for _ in range(2))
        pages = -(-T // page_size) + 3
        self.slots = rng.permutation(pages * page_size)[:T]
        if T > 4:
            self.slots[rng.integers(0, T, max(1, T // 9))] = -1
        self.positions = rng.integers(0, ROWS, (len(self.sections), T))
        angle = rng.uniform(-np.pi, np.pi, (ROWS, rotary // 2))
        self.cos, self.sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        self.rotary = rotary
        self.kc, self.vc = paged(pages, page_size, H, D, order, 0.0, 0)
        self.scales = {}
        if format == 8:
            self.kc, self.vc = (torch.empty_strided(x.shape, x.stride(), dtype=torch.int8, device=DEV).fill_(77) for x in (self.kc, self.vc))
            self.scales = {n: torch.full((pages, H, page_size), 9.0, dtype=torch.bfloat16, device=DEV) for n in ("k_scales", "v_scales")}
        else:
            self.kc.fill_(77.0)
            self.vc.fill_(77.0)

    def run(self, q_out=None, no_q=False):
        rope = (gpu(self.positions), torch.tensor(self.cos, device=DEV), torch.tensor(self.sin, device=DEV)) if self.rotary else (None, None, None)
        kw = dict(self.kw) if self.rotary else dict(eps=self.eps, unit_offset=self.offset)
        out = w4.w4_kv_append_norm(None if no_q else self.q, self.k, self.v, None if no_q else self.qw, self.kw_, *rope, self.kc, self.vc,
                                   gpu(self.slots, torch.int64), q_out=q_out, **kw, **self.scales)
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0
        return out

    def turned(self, x, weight):
        """(values, bound) of rows x."""
        y = SO.norm(values(x), values(weight), np.float64(np.float32(self.eps)), self.offset)
        if not self.rotary:
            return y, SO.norm_bound(y, np.abs(y))
        args = (self.positions, self.cos, self.sin, self.sections, self.kw["cycled"], self.kw["paired"])
        t = KO.rotate(y, *args)
        return t, SO.norm_bound(t, SO.turned_size(y, *args))

    def check(self, out):
        P = self.kc.shape[1]
        kept = np.nonzero(self.slots >= 0)[0]
        at = (self.slots[kept] // P, self.slots[kept] % P)
        if out is not None:
            want, bound = self.turned(self.q, self.qw)
            assert (np.abs(values(out) - want) <= bound).all()
        want, bound = self.turned(self.k, self.kw_)
        untouched = np.ones(self.kc.shape[:2], bool)
        untouched[at] = False
        assert (values(self.kc)[untouched] == 77).all() and (values(self.vc)[untouched] == 77).all()
        if self.format == 16:
            assert (np.abs(values(self.kc)[at] - want[kept]) <= bound[kept]).all()
            assert torch.equal(self.vc[at].view(torch.int16), self.v[torch.tensor(kept, device=DEV)].contiguous().view(torch.int16))
        else:
            ks, vs = (values(self.scales[n]).transpose(0, 2, 1) for n in ("k_scales", "v_scales"))
            codes, d = KO.rtn8(values(self.v)[kept])
            assert np.array_equal(values(self.vc)[at], codes) and np.array_equal(vs[at], d)
            # d: one rounding to bf16 of the row's largest value / 127; a code is off by at most half a step, a quarter of a
            # step more where 127.25 or 127.5 is clamped to 127.
            error = (bound - 2.0 ** -8 * np.abs(want))[kept]
            most = np.abs(want[kept]).max(-1)
            d = ks[at]
            assert (np.abs(d - most / 127) <= 2.0 ** -8 * most / 127 + error.max(-1) / 127).all()
            assert (np.abs(values(self.kc)[at] * d[..., None] - want[kept]) <= 0.501 * d[..., None] + error).all()


def check(case, **kw):
    case.check(case.run(**kw))


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D,rotary", [(16, 4, 256, 64), (40, 8, 128, 128), (64, 8, 128, 128), (7, 1, 64, 64), (6, 3, 80, 80),
                                           (4, 4, 112, 48), (8, 2, 192, 192), (5, 1, 16, 16), (36, 2, 96, 32), (2, 2, 256, 256), (3, 3, 176, 16)])
@pytest.mark.parametrize("paired", [False, True])
def test_layouts(cuda_lib, Hq, H, D, rotary, paired, format):
    for T in (1, 3, 78):
        check(Case(T, Hq, H, D, rotary, paired=paired, format=format, seed=D + T))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [False, True])
@pytest.mark.parametrize("format", [16, 8])
def test_weights(cuda_lib, dtype, offset, format):
    check(Case(33, 8, 2, 128, 64, dtype=dtype, offset=offset, format=format, seed=5))
    check(Case(20, 8, 2, 128, 64, dtype=dtype, offset=offset, format=format, eps=0.5, seed=6))


@pytest.mark.parametrize("sections,cycled", [((16, 24, 24), False), ((11, 11, 10), True), ((1, 7, 0, 24), True), ((32,), False)])
@pytest.mark.parametrize("order,page_size", [("token", 1), ("head", 16), ("pair", 24)])
def test_axes_and_pages(cuda_lib, sections, cycled, order, page_size):
    check(Case(50, 4, 2, 128, 2 * sum(sections), sections, cycled, order=order, page_size=page_size, seed=7))


@pytest.mark.parametrize("T", [75, 76, 77, 1215, 1216, 3001])
@pytest.mark.parametrize("format", [16, 8])
def test_many_tokens(cuda_lib, T, format):
    check(Case(T, 6, 2, 128, 128, format=format, seed=T))
    check(Case(T, 2, 1, 256, 64, paired=True, format=format, seed=T))


def test_without_rotation_and_without_queries(cuda_lib):
    check(Case(9, 4, 2, 128, 0, seed=1))
    check(Case(9, 4, 2, 64, 0, format=8, offset=True, seed=2))
    case = Case(9, 4, 2, 128, 64, seed=3)
    assert case.run(no_q=True) is None
    case.check(None)


def test_in_place_and_strided(cuda_lib):
    case = Case(70, 8, 2, 128, 128, seed=8)
    kept = case.q.clone()
    out = case.run(q_out=case.q)
    assert out.data_ptr() == case.q.data_ptr()
    case.q = kept
    case.check(out)
    check(Case(70, 8, 2, 128, 128, fused=False, seed=9))


def test_rows_of_zeros_and_of_large_and_small_values(cuda_lib):
    """Squares past fp32's range, sums past it, and rows far below eps; a row of zeros stays one."""
    sizes = torch.tensor([0.0, 1e-38, 1e-30, 1e-20, 1e-10, 1e-3, 1.0, 1e10, 3e18, 1e19, 1e25, 1e37, 3e38], dtype=torch.float64)
    for format in (16, 8):
        for rotary, D in ((64, 128), (0, 256)):
            shape = torch.rand((13, 4, D), generator=torch.Generator().manual_seed(1), dtype=torch.float64) * 2 - 1
            rows = (shape * sizes[:, None, None]).to(torch.bfloat16)
            case = Case(13, 4, 4, D, rotary, format=format, q=rows, k=rows, seed=2)
            out = case.run()
            case.check(out)
            assert (values(out)[0] == 0).all()


def test_rows_that_are_not_finite(cuda_lib):
    """By the formula: a NaN spoils its row, an infinity becomes NaN and all else of its row zero; other rows are as ever."""
    D = 128
    for format in (16, 8):
        clean = Case(6, 4, 2, D, 64, format=format, seed=4)
        out = clean.run()
        case = Case(6, 4, 2, D, 64, format=format, seed=4)
        case.q[2, 1, 100], case.q[3, 0, 100] = float("nan"), float("inf")
        case.k[2, 1, 5], case.k[4, 0, 120] = float("nan"), float("-inf")
        got = case.run()
        spoilt = torch.zeros((6, 4), dtype=torch.bool)
        spoilt[2, 1] = spoilt[3, 0] = True
        assert torch.equal(got[~spoilt.to(DEV)].view(torch.int16), out[~spoilt.to(DEV)].view(torch.int16))
        assert torch.isnan(got[2, 1]).all()
        row = got[3, 0].cpu()
        assert torch.isnan(row[100]) and (row[torch.arange(D) != 100] == 0).all()
        at = [(int(s) // 16, int(s) % 16) for s in case.slots]
        for t, h in ((2, 1), (4, 0)):
            if case.slots[t] < 0:
                continue
            if format == 8:
                assert torch.isnan(case.scales["k_scales"][at[t][0], h, at[t][1]]) and (case.kc[at[t]][h] == 0).all()
            else:
                assert torch.isnan(case.kc[at[t]][h]).any()


def test_numbers_out_of_range(cuda_lib):
    case = Case(5, 4, 2, 128, 64, seed=4)
    case.slots[:] = [3, -1, -2, 10 ** 12, 4]
    case.positions[0, 4] = ROWS
    rope = (gpu(case.positions), torch.tensor(case.cos, device=DEV), torch.tensor(case.sin, device=DEV))
    out = w4.w4_kv_append_norm(case.q, case.k, case.v, case.qw, case.kw_, *rope, case.kc, case.vc, gpu(case.slots, torch.int64))
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == w4.W4_ERR_INVALID_ARG
    case.slots[2:4] = -1
    case.positions[0, 4] = 0
    case.check(out)


def test_the_same_bits_again_and_in_a_graph(cuda_lib):
    case = Case(300, 8, 2, 128, 128, seed=11)
    out = torch.empty_like(case.q)
    first = case.run(q_out=out).clone()
    rope = (gpu(case.positions), torch.tensor(case.cos, device=DEV), torch.tensor(case.sin, device=DEV))
    slots = gpu(case.slots, torch.int64)
    keys = case.kc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4_kv_append_norm(case.q, case.k, case.v, case.qw, case.kw_, *rope, case.kc, case.vc, slots, q_out=out, **case.kw)
    out.zero_(), case.kc.fill_(77.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16)) and torch.equal(case.kc.view(torch.int16), keys.view(torch.int16))


def test_checks_of_the_binding(cuda_lib):
    case = Case(5, 4, 2, 128, 64, seed=4)
    slots = gpu(case.slots, torch.int64)
    rope = (gpu(case.positions), torch.tensor(case.cos, device=DEV), torch.tensor(case.sin, device=DEV))
    for qw, kw, error in ((case.qw.float(), case.kw_, TypeError), (case.qw[:64], case.kw_, ValueError), (case.qw, case.kw_.half(), TypeError),
                          (None, case.kw_, TypeError), (case.qw, None, TypeError), (case.qw.cpu(), case.kw_, TypeError)):
        with pytest.raises(error):
            w4.w4_kv_append_norm(case.q, case.k, case.v, qw, kw, *rope, case.kc, case.vc, slots)
    with pytest.raises(w4.W4Error):
        w4.w4_kv_append_norm(case.q, case.k, case.v, case.qw, case.kw_, *rope, case.kc, case.vc, slots, eps=0.0)


def test_no_tokens_and_two_streams_at_once(cuda_lib):
    case = Case(0, 4, 2, 128, 64, seed=12)
    case.check(case.run())
    cases = [Case(n, 8, 2, 128, 128, seed=13 + n) for n in (40, 1300)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    args = [(c.q, c.k, c.v, c.qw, c.kw_, gpu(c.positions), torch.tensor(c.cos, device=DEV), torch.tensor(c.sin, device=DEV), c.kc, c.vc,
             gpu(c.slots, torch.int64)) for c in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for s, c, a, out in zip(streams, cases, args, outs):
            with torch.cuda.stream(s):
                out.append(w4.w4_kv_append_norm(*a, **c.kw))
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    for c, out in zip(cases, outs):
        c.check(out[0])
        assert all(torch.equal(x.view(torch.int16), out[0].view(torch.int16)) for x in out)


@pytest.mark.parametrize("Hq,H,D", [(64, 8, 128), (40, 8, 128), (16, 4, 256), (9, 1, 64)])
@pytest.mark.parametrize("format", [16, 8])
def test_both_sides_of_the_shares_of_a_token(cuda_lib, Hq, H, D, format):
    """A CTA for some of a token's rows, or for all of them."""
    for T in (76, 101, 102, 121, 122, 151, 152, 153):
        check(Case(T, Hq, H, D, 64, format=format, seed=T))
