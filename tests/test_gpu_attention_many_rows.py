"""The tensor-core kernel of w4_attn_decode (many rows to a key-value head): CTAs that take several items in a row,
requests without tokens among them.  Each case says that it reaches that kernel."""
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from tests.kv_cases import DEV, AttentionCase, gpu

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
