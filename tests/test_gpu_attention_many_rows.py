"""The tensor-core kernel of w4_attn_decode (many rows to a key-value head): CTAs that take several items in a row,
requests without tokens among them.  Each case says that it reaches that kernel."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from tests.kv_cases import DEV, AttentionCase, gpu, values
from tests.test_gpu_attention_8bit import check

pytestmark = pytest.mark.gpu


def reaches_tensor_kernel(case):
    """Whether the call runs the tensor-core kernel: the other one's workspace has 2 · 512 arrival words and as many
    parts of 16 or 32 rows, with two more numbers for each row."""
    D = next(d for d in (64, 128, 256) if case.q.shape[2] <= d)
    size = w4.w4_attn_decode_workspace_bytes(case.q, case.k, len(case.lens))
    return size not in [1024 * (8 + 4 * rows * (2 + D)) for rows in (16, 32)]


def empty_then_full(case, sms):
    """CTAs whose piece of the work has an item without tokens right before one with tokens.  An item (request, head,
    128 rows) counts two units and one for each of its tiles; the units are cut into equal runs, one for each CTA, and
    an item belongs to those whose runs hold a part of its tiles."""
    H, G, D = case.k.shape[2], case.q.shape[1] // case.k.shape[2], case.q.shape[2]
    tile = 128 if D <= 128 else 64
    items = []  # (first unit of its tiles, past its last, whether it has tokens)
    unit = 0
    for n, new in zip(case.lens, case.fresh):
        for _ in range(H * -(-new * G // 128)):
            tiles = max(1, -(-n // tile))
            items.append((unit + 2, unit + 2 + tiles, n > 0))
            unit += 2 + tiles
    size, longer = divmod(unit, sms)
    found = 0
    for p in range(sms):
        a, b = (x * size + min(x, longer) for x in (p, p + 1))
        mine = [full for lo, hi, full in items if lo < b and hi > a]
        found += any(not x and y for x, y in zip(mine, mine[1:]))
    return found


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D", [(64, 8, 128), (104, 8, 64), (40, 4, 256), (64, 8, 96)])
def test_requests_without_tokens_before_others(cuda_lib, Hq, H, D, format):
    """Requests that got no pages keep their rows (which are zeros) at length 0; the request behind one must be answered
    with its own queries.  The same bits in every run."""
    lens = [0 if b % 2 == 0 else 1 + 37 * b % 300 for b in range(64)]
    case = AttentionCase(lens, [13] * 64, Hq, H, D, 16, format=format, seed=31)
    assert reaches_tensor_kernel(case)
    assert empty_then_full(case, torch.cuda.get_device_properties(0).multi_processor_count) >= 10
    first = case.run(w4, uniform=True)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    case.check(first)
    q, table, n = case.q.to(DEV), gpu(case.table), gpu(case.lens)
    for _ in range(20):
        out = torch.full_like(first, 7.0)
        w4.w4_attn_decode(q, case.k, case.v, table, n, k_scales=case.k_scales, v_scales=case.v_scales, out=out)
        assert torch.equal(first.view(torch.int16), out.view(torch.int16))


# ---- the same, over caches in 8 bits (and in bf16): what the other kernel's tests try, at shapes that reach this one
RAGGED = ([0, 7, 1, 13, 200, 300, 64, 0, 129, 20, 257], [5, 7, 1, 13, 5, 13, 0, 0, 1, 20, 9])


@pytest.mark.parametrize("Hq,H,D", [(40, 2, 64), (32, 2, 128), (16, 1, 256), (48, 3, 80), (16, 1, 192), (20, 1, 16)])
@pytest.mark.parametrize("order,page_size", [("token", 16), ("head", 24), ("token", 1)])
@pytest.mark.parametrize("format", [16, 8])
def test_ragged(cuda_lib, Hq, H, D, order, page_size, format):
    case = AttentionCase(*RAGGED, Hq, H, D, page_size, order, format=format, seed=Hq + D)
    assert reaches_tensor_kernel(case)
    out = case.run(w4)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    case.check(out)


@pytest.mark.parametrize("window", [1, 9, 100, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("format", [16, 8])
def test_windows(cuda_lib, window, D, format):
    case = AttentionCase([1, 40, 500, 333, 13, 130], [1, 13, 9, 13, 13, 6], 32, 2, D, 16, format=format, seed=window)
    assert reaches_tensor_kernel(case)
    out = case.run(w4, window=window)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    case.check(out, window=window)


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (-0.1, 1.0), (1.0, 8.0), (-0.3, 30.0)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_and_sharp_scores_in_8_bits(cuda_lib, D, scale, std):
    """Codes of zero among them: what a dominant token leaves to others that weigh next to nothing."""
    case = AttentionCase([50, 300, 777], [13, 9, 13], 16, 1, D, 16, format=8, seed=21, std=std)
    assert reaches_tensor_kernel(case)
    check(case, case.run(w4, scale=scale), scale)


@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_hidden_token(cuda_lib, D, window, bad, format):
    """One that some rows of a pass see and others do not, in an item's first tile and in a later one."""
    for L in (45, 300):
        case = AttentionCase([L, 200], [13, 13], 32, 2, D, 16, format=format, seed=22)
        assert reaches_tensor_kernel(case)
        token = L - 8
        page, place = int(case.table[0, token // 16]), token % 16
        for x, s in ((case.k, case.k_scales), (case.v, case.v_scales)):
            if format == 16:
                x[page, place, :, 5] = bad
            else:
                s[page, :, place] = bad
        out = case.run(w4, window=window)
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0
        position = np.arange(L - 13, L)
        sees = np.concatenate([(token <= position) & ((window == 0) | (token > position - window)), [False] * 13])
        case.check(out, window=window, rows=~sees)
        assert not np.isfinite(values(out)[sees]).all(axis=(1, 2)).any()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("format", [16, 8])
def test_many_requests(cuda_lib, D, format):
    """Requests × heads for half of the SMs and more, five rows of sixteen query heads each."""
    rng = np.random.default_rng(D)
    lens = rng.integers(0, 200, 60).tolist()
    case = AttentionCase(lens, [int(x) for x in rng.integers(4, 7, 60)], 32, 2, D, 16, format=format, seed=D)
    assert reaches_tensor_kernel(case)
    out = case.run(w4)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    case.check(out)


@pytest.mark.parametrize("n", [1, 13])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("zeros", [3, 900])
def test_values_of_zero_in_8_bits(cuda_lib, D, n, zeros):
    """Tokens whose values are all zero have a value scale of zero; their weights count all the same."""
    case = AttentionCase([1000, zeros + n], [n, n], 160 if n == 1 else 16, 1, D, 16, format=8, seed=zeros + D)
    assert reaches_tensor_kernel(case)
    for b in range(2):
        for token in range(zeros):
            page, place = case.table[b, token // 16], token % 16
            case.v[page, place] = 0
            case.v_scales[page, :, place] = 0
            case.vv[page, place] = 0.0
    check(case, case.run(w4), D ** -0.5)
