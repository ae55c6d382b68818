"""w4_attn_decode over a cache in 8 bits, where its fp16 operands are short of range: weights and query values far below
the largest."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from oracle import kv_oracle as KO
from tests.kv_cases import AttentionCase, gpu, values

pytestmark = pytest.mark.gpu


def check(case, out, scale, window=0):
    """Against 64 bits, within the bound of any format and what format 8's weights may add."""
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    scale = float(np.float32(scale))
    args = (values(case.q), case.kv, case.vv, case.table, case.lens, case.starts, scale, window)
    ref, spread, largest = KO.attention(*args)
    d = values(case.v_scales.transpose(1, 2))
    codes = case.v.cpu().numpy().astype(np.float64)
    floor = KO.attention8_floor(*args[:2], codes, np.where(np.isfinite(d), d, 0.0), *args[3:])
    # a query value errs by 2⁻³⁹ of its row's largest, which moves weights by twice that times the keys' sum
    keys = np.where(np.isfinite(case.kv), np.abs(case.kv), 0.0).sum(-1).max()
    moved = 2 * abs(scale) * 2.0 ** -39 * np.abs(args[0]).max(-1, keepdims=True) * keys
    bound = KO.attention_bound(ref, spread, largest, case.q.shape[2], max(case.lens), 8) + floor + moved * spread
    got = values(out)
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) / np.maximum(bound, 1e-300)).max()
    assert worst <= 1.0, f"largest error is {worst:.3g} of the bound"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("below", [10, 14, 18, 21, 24, 28, 40, 60])
def test_columns_of_small_weights(cuda_lib, D, below):
    """Every sixteenth token weighs most and has a value of zero in the column that the fifteen around it have: the
    column is made of weights about 2^-below of the largest alone."""
    N = 16 * D
    case = AttentionCase([N], [1], 4, 1, D, 16, format=8, seed=below)
    case.q[:] = 0
    case.q[..., 0] = 1  # scores, to base 2: the keys' first values
    rng = np.random.default_rng(below)
    t = np.arange(N)
    heavy = t % 16 == 5
    keys, vals = np.zeros((N, D)), np.zeros((N, D))
    keys[:, 0] = np.where(heavy, 0, -128)
    vals[t, t // 16] = np.where(heavy, 0, rng.integers(1, 128, N))
    key_scales = KO.bf16((below + rng.uniform(-1, 1, N)) / 128).astype(np.float64)
    page, place = case.table[0, t // 16], t % 16
    at = (gpu(page, torch.int64), gpu(place, torch.int64))
    for name, codes, d in (("k", keys, key_scales), ("v", vals, np.ones(N))):
        getattr(case, name)[at[0], at[1], 0] = gpu(codes, torch.int8)
        getattr(case, name + "_scales")[at[0], 0, at[1]] = gpu(d, torch.bfloat16)
        getattr(case, name + "v")[page, place, 0] = codes * d[:, None]
    check(case, case.run(w4, scale=np.log(2)), np.log(2))


@pytest.mark.parametrize("n", [1, 13])
@pytest.mark.parametrize("scale,std", [(1.0, 8.0), (-0.3, 30.0)])
def test_sharp_scores_with_any_codes(cuda_lib, scale, std, n):
    """One token outweighs the others by far; columns where its code is zero are left to weights that may underflow."""
    case = AttentionCase([50, 300, 777], [n] * 3, 8, 2, 128, 16, format=8, seed=21, std=std)
    check(case, case.run(w4, scale=scale), scale)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("exponent", [10, 20, 24])
def test_queries_with_one_large_value(cuda_lib, D, exponent):
    """A query value that meets keys of zero, next to others 2^exponent times smaller that make the scores."""
    case = AttentionCase([300, 17], [1, 2], 8, 2, D, 16, format=8, seed=exponent)
    case.q[..., 3] = 2.0 ** exponent
    case.k[..., 3] = 0
    case.kv[..., 3] = 0
    check(case, case.run(w4), D ** -0.5)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("exponent", [100, -100, -118])
def test_large_and_small_queries(cuda_lib, D, exponent):
    """Queries times 2^exponent on keys times 2^-exponent: the same scores."""
    case = AttentionCase([300, 17], [1, 2], 8, 2, D, 16, format=8, seed=-exponent if exponent < 0 else exponent)
    case.q *= 2.0 ** exponent
    case.k_scales *= 2.0 ** -exponent
    case.kv *= 2.0 ** -exponent
    check(case, case.run(w4), D ** -0.5)
