"""w4_kv_pages and w4_kv_append against their restatements: page rings that wrap, run short and take pages back, axes,
layouts and formats of the rotation and the cache write, and numbers out of range."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from oracle import kv_oracle as KO
from tests.kv_cases import DEV, bf16_tensor, gpu, paged, values

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- pages
def pool(lens, target, page_size, free, seed, width=None):
    """(table, ring, free_range): requests with `lens` tokens and `free` pages in a ring that wraps."""
    rng = np.random.default_rng(seed)
    have = [-(-n // page_size) for n in lens]
    want = [-(-n // page_size) for n in target]
    width = max(have + want + [1]) + 1 if width is None else width
    pages = max(1, sum(have) + free)
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = free
    for b, h in enumerate(have):
        table[b, :h] = ids[at:at + h]
        at += h
    head = int(rng.integers(0, 1 << 50))
    ring = rng.integers(0, pages, pages).astype(np.int32)
    ring[[(head + i) % pages for i in range(free)]] = ids[:free]
    return table, ring, [head, head + free]


def check_pages(lens, target, page_size, table, ring, free, T, status=0):
    ref = KO.pages(lens, target, table, ring, free, page_size, T)
    t, r = gpu(table), gpu(ring)
    new_lens, starts, slots, positions, left = w4.w4_kv_pages(gpu(lens), gpu(target), t, r, gpu(free, torch.int64),
                                                              page_size, T)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == status
    got = {"new_lens": new_lens, "starts": starts, "slots": slots, "positions": positions, "free_range": left,
           "table": t, "ring": r}
    for name, x in got.items():
        assert np.array_equal(x.cpu().numpy(), ref[name]), name
    return ref


def mixed(B, longest, seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, B).tolist()
    target = [max(0, n + int(rng.integers(-20, 30))) if rng.random() < 0.8 else 0 for n in lens]
    return lens, target


@pytest.mark.parametrize("page_size", [1, 3, 16, 64, 1000])
@pytest.mark.parametrize("B", [1, 2, 31, 33, 1023, 1024, 1025, 2500])
def test_pages(cuda_lib, B, page_size):
    lens, target = mixed(B, 300, B + page_size)
    grown = sum(max(0, m - n) for n, m in zip(lens, target))
    need = sum(max(0, -(-m // page_size) - -(-n // page_size)) for n, m in zip(lens, target))
    check_pages(lens, target, page_size, *pool(lens, target, page_size, need + 2, 1), grown)


@pytest.mark.parametrize("free", [0, 1, 40, 41])
@pytest.mark.parametrize("B", [50, 1500])
def test_a_pool_that_runs_short(cuda_lib, B, free):
    """Requests in order get pages until one asks for more than are left; those after it that need none still grow."""
    lens, target = mixed(B, 300, B)
    grown = sum(max(0, m - n) for n, m in zip(lens, target))
    ref = check_pages(lens, target, 16, *pool(lens, target, 16, free, 2), grown)
    need = sum(max(0, -(-m // 16) - -(-n // 16)) for n, m in zip(lens, target))
    assert (ref["slots"] == -1).any() == (need > free)


def test_prompts(cuda_lib):
    lens, target = [0, 5, 0, 64, 0], [20000, 37, 1, 30000, 0]
    check_pages(lens, target, 16, *pool(lens, target, 16, 4000, 3), sum(target) - sum(lens))


def test_a_target_past_the_table(cuda_lib):
    lens, target = [10, 20, 30], [11, 200, 31]
    check_pages(lens, target, 16, *pool(lens, target, 16, 20, 4, width=3), 182)


@pytest.mark.parametrize("T", [0, 5, 12, 60])
def test_rows_fewer_or_more_than_the_tokens(cuda_lib, T):
    lens, target = [10, 20, 30], [17, 40, 31]  # 28 new tokens
    table, ring, free = pool(lens, target, 16, 20, 5)
    check_pages(lens, target, 16, table, ring, free, T, status=w4.W4_ERR_INVALID_ARG if T < 28 else 0)


def test_lengths_out_of_range(cuda_lib):
    lens, target = [10, 20, 30, 7], [12, 22, 33, 9]
    table, ring, free = pool(lens, target, 16, 20, 6)
    for bad_lens, bad_target in (([10, -1, 30, 7], target), (lens, [12, -22, 33, 9]), ([10, 2 ** 31 - 1, 30, 7], target)):
        check_pages(bad_lens, bad_target, 16, table, ring, free, 9, status=w4.W4_ERR_INVALID_ARG)


def test_page_ids_out_of_range(cuda_lib):
    lens, target = [10, 30], [12, 40]
    table, ring, free = pool(lens, target, 16, 20, 7)
    table[0, 0] = 10 ** 6
    check_pages(lens, target, 16, table, ring, free, 12, status=w4.W4_ERR_INVALID_ARG)


def test_no_requests(cuda_lib):
    t = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    _, starts, _, _, left = w4.w4_kv_pages(gpu([]), gpu([]), t, gpu([0, 1]), gpu([4, 6], torch.int64), 16, 0)
    assert starts.tolist() == [0] and left.tolist() == [4, 6] and w4.w4_last_device_status() == 0


def test_a_pool_over_many_steps_loses_no_page(cuda_lib):
    """Growing, rejected drafts and finished requests: every page is in one table or in the ring, once."""
    rng = np.random.default_rng(8)
    B, P, pages, width = 40, 4, 300, 40
    table, ring = gpu(np.full((B, width), -1)), gpu(rng.permutation(pages))
    lens, free = gpu(np.zeros(B)), gpu([0, pages], torch.int64)
    for step in range(30):
        now = lens.cpu().numpy()
        target = np.where(rng.random(B) < 0.1, 0, np.maximum(0, now + rng.integers(-5, 14, B)))
        T = int(np.maximum(target - now, 0).sum())
        lens, starts, slots, positions, free = w4.w4_kv_pages(lens, gpu(target), table, ring, free, P, T)
        held = [int(table[b, i]) for b, n in enumerate(lens.tolist()) for i in range(-(-n // P))]
        head, tail = free.tolist()
        held += [int(ring[i % pages]) for i in range(head, tail)]
        assert sorted(held) == list(range(pages)), f"step {step}"
    assert w4.w4_last_device_status() == 0


# ------------------------------------------------------------------ append
class AppendCase:
    def __init__(self, T, Hq, H, D, rotary, sections, page_size=16, order="token", format=16, seed=0, std=1.0):
        self.T, self.sections, self.page_size, self.format, self.D = T, sections, page_size, format, D
        rng = np.random.default_rng(seed)
        self.q, self.k, self.v = (bf16_tensor((T, h, D), seed + i, std) for i, h in enumerate((Hq, H, H)))
        self.pages = -(-T // page_size) + 3
        self.slots = rng.permutation(self.pages * page_size)[:T].astype(np.int64)
        self.slots[rng.random(T) < 0.1] = -1
        rows = 500
        angle = rng.uniform(-3, 3, (rows, rotary // 2))
        self.cos, self.sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        self.positions = rng.integers(0, rows, (len(sections), T)).astype(np.int32)
        self.k_cache, self.v_cache = paged(self.pages, page_size, H, D, order, None, seed + 5)
        self.k_scales = self.v_scales = None
        if format == 8:
            strides = self.k_cache.stride()
            self.k_cache, self.v_cache = (torch.empty_strided(x.shape, strides, dtype=torch.int8, device=DEV).fill_(77)
                                          for x in (self.k_cache, self.v_cache))
            self.k_scales, self.v_scales = (torch.full((self.pages, H, page_size), 5.0, dtype=torch.bfloat16, device=DEV)
                                            for _ in range(2))
        self.before = [values(x) for x in (self.k_cache, self.v_cache)]

    def run(self, q=None, k=None, v=None, cycled=False, paired=False, slots=None, positions=None, **more):
        return w4.w4_kv_append(self.q.to(DEV) if q is None else q, self.k.to(DEV) if k is None else k,
                               self.v.to(DEV) if v is None else v,
                               gpu(self.positions if positions is None else positions), gpu(self.cos, torch.float32),
                               gpu(self.sin, torch.float32), self.k_cache, self.v_cache,
                               gpu(self.slots if slots is None else slots, torch.int64), sections=self.sections,
                               cycled=cycled, paired=paired, k_scales=self.k_scales, v_scales=self.v_scales, **more)

    def turned(self, x, cycled=False, paired=False):
        """fp32, operation by operation as documented, then bf16."""
        y = values(x).astype(np.float32)
        z = y.copy()
        F = self.cos.shape[1]
        for i, a in enumerate(KO.axis_of(self.sections, cycled)):
            c, s = self.cos[self.positions[a], i][:, None], self.sin[self.positions[a], i][:, None]
            j, k = (2 * i, 2 * i + 1) if paired else (i, i + F)
            z[..., j] = y[..., j] * c - y[..., k] * s
            z[..., k] = y[..., k] * c + y[..., j] * s
        return KO.bf16(z).astype(np.float64)

    def check(self, q_out, slots=None, **kw):
        """Bit for bit: every operation's rounding is specified."""
        torch.cuda.synchronize()
        slots = self.slots if slots is None else slots
        if q_out is not None:
            assert np.array_equal(values(q_out), self.turned(self.q, **kw))
        kept = slots >= 0
        place = (slots[kept] // self.page_size, slots[kept] % self.page_size)
        for x, rows, cache, scales in ((self.turned(self.k, **kw), self.before[0], self.k_cache, self.k_scales),
                                       (values(self.v), self.before[1], self.v_cache, self.v_scales)):
            want = rows.copy()
            if self.format == 16:
                want[place] = x[kept]
            else:
                codes, d = KO.rtn8(x[kept])
                want[place] = codes
                want_scales = np.full(scales.shape, 5.0).transpose(0, 2, 1)
                want_scales[place] = d
                assert np.array_equal(values(scales).transpose(0, 2, 1), want_scales, equal_nan=True)
            assert np.array_equal(values(cache), want)


SHAPES = [  # Hq, H, D, rotary, sections
    (16, 4, 256, 64, (11, 11, 10)), (40, 8, 128, 128, (16, 24, 24)), (7, 1, 64, 64, (32,)), (6, 3, 80, 80, (13, 27)),
    (4, 4, 112, 96, (1, 0, 40, 7)), (8, 2, 192, 16, (3, 5)), (5, 1, 16, 16, (8,)), (3, 2, 256, 256, (50, 40, 38)),
    (2, 2, 48, 32, (16,)),
]


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("cycled,paired", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("shape", SHAPES)
def test_append(cuda_lib, shape, cycled, paired, format):
    Hq, H, D, rotary, sections = shape
    case = AppendCase(37, Hq, H, D, rotary, sections, format=format, seed=D)
    case.check(case.run(cycled=cycled, paired=paired), cycled=cycled, paired=paired)
    assert w4.w4_last_device_status() == 0


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("order,page_size", [("head", 16), ("pair", 24), ("token", 1), ("head", 3)])
@pytest.mark.parametrize("T", [1, 2, 300])
def test_append_lengths_pages_and_orders(cuda_lib, T, order, page_size, format):
    case = AppendCase(T, 10, 2, 128, 64, (10, 11, 11), page_size, order, format, seed=T)
    case.check(case.run(cycled=True), cycled=True)


def test_rotation_against_64_bits(cuda_lib):
    """The rotation itself, not its rounding: each value's fp32 products and sum err by at most 2⁻²² of the products,
    the rounding to bf16 by 2⁻⁸ of the value at most."""
    case = AppendCase(64, 8, 2, 128, 128, (20, 22, 22), seed=1)
    out = values(case.run())
    ref = KO.rotate(values(case.q), case.positions, case.cos, case.sin, case.sections)
    size = np.abs(values(case.q)) + np.abs(np.roll(values(case.q), 64, -1))
    assert (np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * size).all()


def test_turning_back_returns_the_rows(cuda_lib):
    """The rotation is its own inverse with the sines negated (its gradient is that rotation)."""
    case = AppendCase(50, 8, 2, 128, 96, (20, 14, 14), seed=2)
    q = case.run()
    case.sin = -case.sin
    back = values(case.run(q=q))
    size = np.abs(values(case.q)).max()
    assert np.abs(back - values(case.q)).max() <= 2.0 ** -6 * size


def test_slices_of_a_fused_projection_in_place(cuda_lib):
    case = AppendCase(33, 8, 2, 128, 128, (64,), seed=3)
    fused = torch.empty((33, 12 * 128 + 64), dtype=torch.bfloat16, device=DEV).fill_(9.0)
    q, k, v = (fused[:, a * 128:b * 128].view(33, -1, 128) for a, b in ((0, 8), (8, 10), (10, 12)))
    for x, y in ((q, case.q), (k, case.k), (v, case.v)):
        x.copy_(y)
    before = fused.clone()
    assert case.run(q=q, k=k, v=v, q_out=q) is q
    case.check(q)
    assert torch.equal(fused[:, 1024:], before[:, 1024:])


def test_one_position_for_every_axis_and_no_rotation(cuda_lib):
    case = AppendCase(20, 8, 2, 128, 64, (10, 11, 11), seed=4)
    one = case.positions[0]
    case.positions = np.stack([one] * 3)
    case.check(case.run(positions=one))
    plain = AppendCase(20, 8, 2, 128, 64, (32,), seed=5)
    out = w4.w4_kv_append(None, plain.k.to(DEV), plain.v.to(DEV), None, None, None, plain.k_cache, plain.v_cache,
                          gpu(plain.slots, torch.int64))
    plain.cos[:], plain.sin[:] = 1, 0
    assert out is None
    plain.check(None)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_are_not_finite_in_8_bits(cuda_lib, bad):
    case = AppendCase(20, 8, 2, 128, 32, (16,), format=8, seed=6)
    case.k[3, 1, 100] = case.v[4, 0, 2] = bad
    case.check(case.run())


@pytest.mark.parametrize("std", [0.0, 1e-39, 1e-30, 1e37])
def test_small_and_large_rows_in_8_bits(cuda_lib, std):
    case = AppendCase(20, 8, 2, 128, 32, (16,), format=8, seed=7, std=std)
    case.check(case.run())


def test_slots_and_positions_out_of_range(cuda_lib):
    case = AppendCase(20, 8, 2, 128, 32, (16,), seed=8)
    bad = case.slots.copy()
    bad[3], bad[5], bad[6] = case.pages * 16, -2, 1 << 62
    out = case.run(slots=bad)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == w4.W4_ERR_INVALID_ARG
    case.check(out, slots=np.where((bad < 0) | (bad >= case.pages * 16), -1, bad))
    case = AppendCase(20, 8, 2, 128, 32, (16,), seed=9)
    bad = case.positions.copy()
    bad[0, 4], bad[0, 7] = -1, 500
    out = case.run(positions=bad)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == w4.W4_ERR_INVALID_ARG
    case.positions[0, [4, 7]] = 0
    case.check(out)


def test_cache_past_32_bit_offsets(cuda_lib):
    H, D, P, far = 2, 128, 16, (1 << 32) // (16 * 2 * 128 * 2) + 5
    both = torch.empty((far + 8, 2, P, H, D), dtype=torch.bfloat16, device=DEV)
    case = AppendCase(3, 4, H, D, 32, (16,), seed=10)
    slots = np.array([(far + 7) * P + 3, 5, (far + 1) * P], np.int64)
    case.k_cache, case.v_cache = both[:, 0], both[:, 1]
    case.run(slots=slots)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    for t, s in enumerate(slots):
        assert np.array_equal(values(both[s // P, 0, s % P]), case.turned(case.k)[t])
        assert np.array_equal(values(both[s // P, 1, s % P]), values(case.v)[t])


def test_empty(cuda_lib):
    case = AppendCase(0, 8, 2, 128, 32, (16,), seed=11)
    case.check(case.run())


def test_binding_refusals(cuda_lib):
    case = AppendCase(4, 8, 2, 128, 32, (16,), seed=12)
    with pytest.raises(TypeError):
        case.run(k=case.k.to(DEV).float())
    with pytest.raises(ValueError):
        case.run(v=case.v.to(DEV)[:3])
    with pytest.raises(ValueError):
        case.run(positions=case.positions[:, :3])
    with pytest.raises(ValueError):
        case.run(q=case.q.to(DEV).transpose(1, 2))
    case.sections = (15,)
    with pytest.raises(w4.W4Error):
        case.run()
    with pytest.raises(ValueError):
        w4.w4_kv_pages(gpu([1, 2]), gpu([3]), gpu([[0], [1]]), gpu([2, 3]), gpu([0, 2], torch.int64), 16, 3)
    with pytest.raises(w4.W4Error):
        w4.w4_kv_pages(gpu([1]), gpu([3]), gpu([[0]]), gpu([2, 3]), gpu([0, 2], torch.int64), 0, 2)
    same = gpu([1])
    with pytest.raises(w4.W4Error):
        w4.w4_kv_pages(same, gpu([3]), gpu([[0]]), gpu([2, 3]), gpu([0, 2], torch.int64), 16, 2, new_lens=same)


@pytest.mark.parametrize("where", ["token", "head", "page of heads"])
@pytest.mark.parametrize("format", [16, 8])
def test_append_and_attend_with_keys_and_values_side_by_side(cuda_lib, where, format):
    """One pool whose keys and values interleave below the page: in each token, in each row, or by head in each page."""
    case = AppendCase(33, 8, 2, 128, 64, (10, 11, 11), format=format, seed=3)
    shape = {"token": (case.pages, 16, 2, 2, 128), "head": (case.pages, 16, 2, 256),
             "page of heads": (case.pages, 2, 2, 16, 128)}[where]
    both = torch.zeros(shape, dtype=case.k_cache.dtype, device=DEV)
    if where == "token":
        case.k_cache, case.v_cache = both[:, :, 0], both[:, :, 1]
    elif where == "head":
        case.k_cache, case.v_cache = both[..., :128], both[..., 128:]
    else:
        case.k_cache, case.v_cache = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    case.before = [values(case.k_cache), values(case.v_cache)]
    case.check(case.run())
    lens, table = gpu([20, 13]), gpu([[0, 1], [2, 3]])
    q, scales = case.q[:2].to(DEV), dict(k_scales=case.k_scales, v_scales=case.v_scales)
    apart = w4.w4_attn_decode(q, case.k_cache.contiguous(), case.v_cache.contiguous(), table, lens, **scales)
    out = w4.w4_attn_decode(q, case.k_cache, case.v_cache, table, lens, **scales)
    assert torch.equal(out.view(torch.int16), apart.view(torch.int16)) and w4.w4_last_device_status() == 0


def test_targets_whose_tokens_pass_2_to_the_31(cuda_lib):
    """Targets far out of range: the requests behind them start past every row, not at rows that others have."""
    lens, target = [0, 0, 0, 0], [4, 2 ** 31 - 1, 2 ** 31 - 1, 5]
    new_lens, starts, slots, positions, left = w4.w4_kv_pages(gpu(lens), gpu(target), gpu(np.full((4, 3), -1)),
                                                              gpu(np.arange(9)), gpu([0, 9], torch.int64), 16, 9)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == w4.W4_ERR_INVALID_ARG
    assert starts.tolist() == [0, 4] + [2 ** 31 - 1] * 3
    assert new_lens.tolist() == [4, 0, 0, 0] and left.tolist() == [1, 9]
    assert slots.tolist() == [0, 1, 2, 3] + [-1] * 5 and positions.tolist() == [0, 1, 2, 3, 0, 1, 2, 3, 4]
