"""The calls on shared pages at the far end of caches whose offsets, in elements, pass 2^32: keys and values side by side in
one tensor, so that a page's stride is that of both."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from tests.kv_cases import DEV, gpu
from tests.test_gpu_attention_shared import Case, members
from tests.test_gpu_kv_norm import Case as Norm

pytestmark = pytest.mark.gpu


def far_cache(k, v):
    """(keys, values, number of pages before theirs): pages [2, page_size, heads, dim] of one tensor, the given ones last."""
    pages, P, H, D = k.shape
    before = 2 ** 32 // (2 * P * H * D) + 7
    both = torch.zeros((before + pages, 2, P, H, D), dtype=k.dtype, device=DEV)
    both[before:, 0], both[before:, 1] = k, v
    assert both[before, 0].data_ptr() - both.data_ptr() > 2 ** 32 * k.element_size()
    return both[:, 0], both[:, 1], before


def far_scales(scales, before):
    return {n: torch.cat([torch.zeros((before, *x.shape[1:]), dtype=x.dtype, device=DEV), x]) for n, x in scales.items()}


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D,P,groups", [(8, 2, 128, 16, [(200, members(5, 60, 33))]), (16, 2, 128, 16, [(300, members(*range(3, 43)))]),
                                             (16, 2, 128, 24, [(300, members(*range(3, 43)))]), (16, 2, 64, 64, [(300, members(*[4] * 40))]),
                                             (16, 2, 256, 16, [(150, members(*[4] * 40))]), (16, 2, 128, 16, [(140, [(30, 13)] * 6)])])
def test_attention(cuda_lib, Hq, H, D, P, groups, format):
    case = Case(groups, Hq, H, D, P, format=format, seed=P + D)
    k, v, before = far_cache(case.k, case.v)
    shift = lambda t: gpu(np.where(t >= 0, t + before, -1))  # noqa: E731
    case.check(case.run(k_cache=k, v_cache=v, block_table=shift(case.table), prefix_table=shift(case.prefix_table), **far_scales(case.scales, before)))


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("T", [3, 100, 1300])
def test_append_with_norms(cuda_lib, T, format):
    case = Norm(T, 4, 2, 128, 64, format=format, seed=T)
    near = case.kc, case.vc, case.scales, case.slots
    case.kc, case.vc, before = far_cache(case.kc, case.vc)
    case.scales = far_scales(case.scales, before)
    case.slots = np.where(case.slots >= 0, case.slots + before * 16, -1)
    out = case.run()
    assert not case.kc[:before:1000].any() and not case.kc[before - 1].any()
    # (the checks are those of the pages that the case began with)
    case.kc, case.vc = case.kc[before:], case.vc[before:]
    case.scales = {n: x[before:] for n, x in case.scales.items()}
    case.slots = near[3]
    case.check(out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_copies(cuda_lib, dtype):
    """From the far end to the start, and back, by whole pages and in part."""
    shape = (9, 16, 2, 128)
    one, two = ((torch.arange(9 * 16 * 2 * 128, device=DEV).reshape(shape) * m % 101 - 50).to(dtype) for m in (7, 11))
    k, v, before = far_cache(one, two)
    pages = k.shape[0]
    scales = {}
    if dtype is torch.int8:
        scales = {n: torch.zeros((pages, 2, 16), dtype=torch.bfloat16, device=DEV) for n in ("k_scales", "v_scales")}
        scales["k_scales"][before + 2], scales["v_scales"][before + 2] = 2.0, 3.0
    w4.w4_kv_copy(k, v, gpu([[before + 2, before + 3, before + 4], [0, before - 1, 5], [16, 16, 7]]), **scales)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    for x, want in ((k, one), (v, two)):
        assert torch.equal(x[before:], want)
        assert torch.equal(x[0], want[2]) and torch.equal(x[before - 1], want[3]) and torch.equal(x[5, :7], want[4, :7])
        assert not x[5, 7:].any() and not x[1:5].any() and not x[6].any() and not x[before - 2].any()
    if scales:
        assert (scales["k_scales"][0] == 2).all() and (scales["v_scales"][0] == 3).all()
    w4.w4_kv_copy(k, v, gpu([[0], [before + 8], [9]]), **scales)
    torch.cuda.synchronize()
    assert torch.equal(k[before + 8, :9], one[2, :9]) and torch.equal(k[before + 8, 9:], one[8, 9:])
    assert torch.equal(v[before + 8, :9], two[2, :9]) and torch.equal(v[before + 8, 9:], two[8, 9:])
