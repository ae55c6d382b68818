"""w4_attn_decode against attention in 64 bits: head layouts, lengths, pages, windows, both cache formats, and what
masked and unused places hold."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from oracle import kv_oracle as KO
from tests.kv_cases import DEV, AttentionCase, bf16_tensor, gpu, values

pytestmark = pytest.mark.gpu

HEADS = [(16, 4, 256), (40, 8, 128), (64, 8, 128), (7, 1, 64), (6, 3, 80), (4, 4, 112), (8, 2, 192), (5, 1, 16), (36, 2, 96)]
LENGTHS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 257, 500]


def finish(case, out, **kw):
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    case.check(out, **kw)


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D", HEADS)
def test_one_new_token(cuda_lib, Hq, H, D, format):
    case = AttentionCase(LENGTHS, [1] * len(LENGTHS), Hq, H, D, 16, format=format, seed=Hq + D)
    finish(case, case.run(w4, uniform=True))


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("order,page_size", [("token", 1), ("token", 3), ("head", 16), ("pair", 24), ("head", 64), ("token", 700)])
def test_page_sizes_and_orders(cuda_lib, order, page_size, format):
    case = AttentionCase(LENGTHS, [1] * len(LENGTHS), 10, 2, 128, page_size, order, format, seed=page_size)
    finish(case, case.run(w4))


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("Hq,H,D", HEADS)
def test_rows_of_a_verify_pass(cuda_lib, Hq, H, D, format):
    """Ragged numbers of new tokens: none, more than the request's length (its
    first rows then see nothing and are zeros), up to 13."""
    lens = [0, 1, 5, 13, 14, 64, 70, 200, 333, 12, 3]
    fresh = [0, 1, 5, 13, 13, 7, 0, 5, 13, 2, 6]
    case = AttentionCase(lens, fresh, Hq, H, D, 16, format=format, seed=D)
    finish(case, case.run(w4))


@pytest.mark.parametrize("fresh", [2, 13, 40])
def test_many_rows(cuda_lib, fresh):
    case = AttentionCase([fresh, fresh + 1, 300, 1000], [fresh] * 4, 16, 2, 128, 16, seed=fresh)
    finish(case, case.run(w4, uniform=True))


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("window", [1, 7, 16, 64, 100, 5000])
def test_windows(cuda_lib, window, format):
    lens = [1, 7, 8, 64, 65, 200, 333, 500, 13]
    fresh = [1, 1, 5, 1, 13, 5, 13, 1, 13]
    case = AttentionCase(lens, fresh, 8, 2, 128, 16, format=format, seed=window)
    finish(case, case.run(w4, window=window), window=window)


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("lens", [[5000], [20000, 3, 9000], [1, 1, 1, 33333]])
def test_long(cuda_lib, lens, format):
    case = AttentionCase(lens, [1] * len(lens), 8, 2, 128, 16, format=format, seed=len(lens))
    finish(case, case.run(w4))


def test_many_requests(cuda_lib):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 1500).tolist()
    fresh = [int(rng.integers(0, 3)) for _ in lens]
    case = AttentionCase(lens, fresh, 4, 1, 64, 8, seed=9)
    finish(case, case.run(w4))


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (-0.1, 1.0), (1.0, 8.0), (0.3, 30.0)])
def test_scales_and_sharp_scores(cuda_lib, scale, std):
    """Scores of thousands: the maximum's bookkeeping carries everything."""
    case = AttentionCase([1, 50, 300, 777], [1, 3, 1, 2], 8, 2, 128, 16, seed=3, std=std)
    finish(case, case.run(w4, scale=scale), scale=scale)


@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), float("-inf"), torch.finfo(torch.bfloat16).max])
@pytest.mark.parametrize("format", [16, 8])
def test_unused_places_change_nothing(cuda_lib, garbage, format):
    lens = [1, 15, 33, 100, 260]
    case = AttentionCase(lens, [1, 5, 13, 2, 7], 8, 2, 128, 16, format=format, seed=4, garbage=garbage)
    finish(case, case.run(w4))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_hidden_token_changes_nothing(cuda_lib, D, format, window, bad):
    """A key and value that are not finite reach the rows that see them, and no
    other: later rows of the pass where a window has left them behind, earlier
    rows where they are still to come."""
    n, L = 13, 45
    case = AttentionCase([L, 20], [n, 1], 8, 2, D, 16, format=format, seed=6)
    token = 37  # the row of position 37 and those after it see it
    page, place = int(case.table[0, token // 16]), token % 16
    for x, s in ((case.k, case.k_scales), (case.v, case.v_scales)):
        if format == 16:
            x[page, place, :, 5] = bad
        else:
            s[page, :, place] = bad
    out = case.run(w4, window=window)
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0
    position = np.arange(L - n, L)
    sees = np.concatenate([(token <= position) & ((window == 0) | (token > position - window)), [False]])
    case.check(out, window=window, rows=~sees)
    assert not np.isfinite(values(out)[sees]).all(axis=(1, 2)).any()


@pytest.mark.parametrize("token", [3, 30])
def test_values_that_are_not_finite_reach_their_rows(cuda_lib, token):
    """An infinite value leaves the rows that see it without a finite number in
    its column, and their other columns as they are."""
    case = AttentionCase([40], [13], 4, 1, 128, 16, seed=8)
    page, place = int(case.table[0, token // 16]), token % 16
    case.v[page, place, 0, 77] = float("inf")
    out = case.run(w4)
    torch.cuda.synchronize()
    sees = np.arange(27, 40) >= token
    assert not np.isfinite(values(out)[sees][..., 77]).any()
    case.check(out, columns=np.arange(128) != 77)
    if not sees.all():
        case.check(out, rows=~sees)


def test_strided_queries_and_outputs(cuda_lib):
    case = AttentionCase([33, 100, 7], [2, 1, 5], 8, 2, 128, 16, seed=10)
    T = case.q.shape[0]
    fused = torch.zeros((T, 12 * 128 + 16), dtype=torch.bfloat16, device=DEV)
    q = fused[:, 16:16 + 8 * 128].view(T, 8, 128)
    q.copy_(case.q)
    before = fused.clone()
    out = torch.zeros((8, T, 128), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    w4.w4_attn_decode(q, case.k, case.v, gpu(case.table), gpu(case.lens), starts=gpu(case.starts), out=out)
    finish(case, out)
    assert torch.equal(fused, before)
    w4.w4_attn_decode(q, case.k, case.v, gpu(case.table), gpu(case.lens), starts=gpu(case.starts), out=q)
    finish(case, q)
    assert torch.equal(fused[:, :16], before[:, :16]) and torch.equal(fused[:, 16 + 8 * 128:], before[:, 16 + 8 * 128:])


def test_table_with_a_row_stride(cuda_lib):
    case = AttentionCase([40, 90, 200], [1, 1, 1], 8, 2, 128, 16, seed=11)
    wide = torch.full((3, 64), -7, dtype=torch.int32, device=DEV)
    table = wide[:, 5:5 + case.table.shape[1]]
    table.copy_(gpu(case.table))
    out = w4.w4_attn_decode(case.q.to(DEV), case.k, case.v, table, gpu(case.lens))
    finish(case, out)


def test_rows_past_the_last_start_are_left_alone(cuda_lib):
    case = AttentionCase([40, 90], [2, 3], 8, 2, 128, 16, seed=12)
    q = torch.cat([case.q, case.q]).to(DEV)
    out = torch.full_like(q, 3.0)
    w4.w4_attn_decode(q, case.k, case.v, gpu(case.table), gpu(case.lens), starts=gpu(case.starts), out=out)
    finish(case, out[:5])
    assert (out[5:] == 3.0).all()


@pytest.mark.parametrize("format", [16, 8])
def test_same_bits_again_on_another_stream_and_in_a_graph(cuda_lib, format):
    case = AttentionCase([3000, 17, 900, 1], [1, 13, 1, 1], 16, 2, 128, 16, format=format, seed=13)
    q, table, lens, starts = case.q.to(DEV), gpu(case.table), gpu(case.lens), gpu(case.starts)
    scales = dict(k_scales=case.k_scales, v_scales=case.v_scales)
    first = w4.w4_attn_decode(q, case.k, case.v, table, lens, starts=starts, **scales)
    finish(case, first)
    dirty = torch.full((w4.w4_attn_decode_workspace_bytes(q, case.k, 4),), 255, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = w4.w4_attn_decode(q, case.k, case.v, table, lens, starts=starts, workspace=dirty, **scales)
    side.synchronize()
    assert torch.equal(first.view(torch.int16), second.view(torch.int16))
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4_attn_decode(q, case.k, case.v, table, lens, starts=starts, workspace=dirty, out=out, **scales)
    for _ in range(2):
        out.zero_()
        dirty.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), out.view(torch.int16))


def test_cache_past_32_bit_offsets(cuda_lib):
    """Pages whose elements start beyond 2³² of them from the cache's address."""
    H, D, P, far = 2, 128, 16, (1 << 32) // (16 * 2 * 128 * 2) + 5
    both = torch.empty((far + 8, 2, P, H, D), dtype=torch.bfloat16, device=DEV)
    k, v = both[:, 0], both[:, 1]
    used = torch.tensor([far + 3, 1, far + 7, far], device=DEV)
    k[used] = bf16_tensor((4, P, H, D), 1).to(DEV)
    v[used] = bf16_tensor((4, P, H, D), 2).to(DEV)
    q = bf16_tensor((1, 8, D), 3)
    out = w4.w4_attn_decode(q.to(DEV), k, v, used.to(torch.int32)[None], gpu([61]))
    torch.cuda.synchronize()
    ref, spread, largest = KO.attention(values(q), values(k[used]), values(v[used]), np.arange(4)[None], [61], [0, 1], D ** -0.5)
    assert (np.abs(values(out) - ref) <= KO.attention_bound(ref, spread, largest, D, 61)).all()
    assert w4.w4_last_device_status() == 0


@pytest.mark.parametrize("what", ["page", "length", "negative", "starts"])
def test_numbers_out_of_range_are_reported(cuda_lib, what):
    case = AttentionCase([40, 90, 64], [1, 2, 1], 8, 2, 128, 16, seed=14, garbage=0.0)
    table, lens, starts = case.table.copy(), list(case.lens), case.starts.copy()
    if what == "page":
        table[1, 2] = 10 ** 6
    elif what == "length":
        lens[1] = 10 ** 8
    elif what == "negative":
        lens[1] = -5
    else:
        starts[1:] = [1, 5, 4]   # past T, then falling: request 1 is cut to rows 1 to 3, request 2 has none
    assert w4.w4_last_device_status() == 0
    out = case.run(w4, table=table, lens=lens, starts=starts)
    torch.cuda.synchronize()
    if what != "starts":
        assert w4.w4_last_device_status() == w4.W4_ERR_INVALID_ARG
    case.check(out, rows=np.array([True, False, False, what != "starts"]))
    if what == "negative":
        assert (out[1:3] == 0).all()


def test_nothing_to_do(cuda_lib):
    case = AttentionCase([40], [1], 8, 2, 128, 16, seed=15)
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16, device=DEV)
    assert w4.w4_attn_decode(q, case.k, case.v, gpu(case.table), gpu([40])).shape == (0, 8, 128)
    out = w4.w4_attn_decode(q, case.k, case.v, gpu(case.table), gpu([40]), starts=gpu([0, 0]))
    torch.cuda.synchronize()
    assert out.shape == (0, 8, 128) and w4.w4_last_device_status() == 0


def test_binding_refusals(cuda_lib):
    case = AttentionCase([40], [1], 8, 2, 128, 16, seed=16)
    q, table, lens = case.q.to(DEV), gpu(case.table), gpu(case.lens)
    with pytest.raises(TypeError):
        w4.w4_attn_decode(q.float(), case.k, case.v, table, lens)
    with pytest.raises(TypeError):
        w4.w4_attn_decode(q, case.k.float(), case.v, table, lens)
    with pytest.raises(TypeError):
        w4.w4_attn_decode(q, case.k.to(torch.int8), case.v.to(torch.int8), table, lens)  # no scales
    with pytest.raises(ValueError):
        w4.w4_attn_decode(q, case.k, case.v.transpose(0, 1), table, lens)
    with pytest.raises(ValueError):
        w4.w4_attn_decode(q, case.k, case.v, table, gpu([40, 40]))
    with pytest.raises(ValueError):
        w4.w4_attn_decode(q[..., :64], case.k, case.v, table, lens)
    with pytest.raises(w4.W4Error):
        w4.w4_attn_decode(q[:, :7].contiguous(), case.k, case.v, table, lens)  # 7 query heads on 2
    with pytest.raises(w4.W4Error):
        w4.w4_attn_decode(q, case.k, case.v, table, lens, window=-1)
    with pytest.raises(w4.W4Error):
        w4.w4_attn_decode(q, case.k, case.v, table, lens, scale=float("nan"))
    with pytest.raises(w4.W4Error):
        w4.w4_attn_decode(q, case.k, case.v, table, lens, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


# ---- many rows to a key-value head (the tensor-core kernel), and enough tokens for each CTA's ring to go round
MANY = [(32, 2, 64), (16, 1, 128), (24, 2, 128), (16, 1, 256), (18, 1, 80), (64, 4, 192), (9, 1, 16)]


@pytest.mark.parametrize("Hq,H,D", MANY)
@pytest.mark.parametrize("order,page_size", [("token", 16), ("head", 24), ("pair", 1)])
def test_many_rows_ragged(cuda_lib, Hq, H, D, order, page_size):
    """Rows in all amounts on one call: none, a few, more than 128; requests without tokens among them."""
    lens = [0, 7, 1, 13, 200, 300, 64, 0, 129, 20, 257]
    fresh = [5, 7, 1, 13, 5, 13, 0, 0, 1, 20, 9]
    case = AttentionCase(lens, fresh, Hq, H, D, page_size, order, seed=Hq + D)
    finish(case, case.run(w4))


@pytest.mark.parametrize("window", [1, 9, 100, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_windows(cuda_lib, window, D):
    lens, fresh = [1, 40, 500, 333, 13, 130], [1, 13, 9, 13, 13, 6]
    case = AttentionCase(lens, fresh, 16, 2, D, 16, seed=window)
    finish(case, case.run(w4, window=window), window=window)


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (-0.1, 1.0), (0.3, 30.0)])
def test_many_rows_scales(cuda_lib, scale, std):
    case = AttentionCase([50, 300, 777], [13, 9, 13], 16, 2, 128, 16, seed=21, std=std)
    finish(case, case.run(w4, scale=scale), scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_many_rows_hidden_tokens(cuda_lib, D, window, bad):
    """As test_a_hidden_token_changes_nothing, in the first tile of an item and in a later one."""
    for L in (45, 300):
        n = 13
        case = AttentionCase([L, 200], [n, 13], 16, 2, D, 16, seed=22)
        token = L - 8
        page, place = int(case.table[0, token // 16]), token % 16
        case.k[page, place, :, 5] = bad
        case.v[page, place, :, 5] = bad
        out = case.run(w4, window=window)
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0
        position = np.arange(L - n, L)
        sees = np.concatenate([(token <= position) & ((window == 0) | (token > position - window)), [False] * 13])
        case.check(out, window=window, rows=~sees)
        assert not np.isfinite(values(out)[sees]).all(axis=(1, 2)).any()


def test_many_rows_values_that_are_not_finite(cuda_lib):
    """Of the values alone: the column of the rows that see the token, and nothing else."""
    case = AttentionCase([300], [13], 16, 1, 128, 16, seed=23)
    page, place = int(case.table[0, 290 // 16]), 290 % 16
    case.v[page, place, 0, 77] = float("inf")
    out = case.run(w4)
    torch.cuda.synchronize()
    sees = np.arange(287, 300) >= 290
    assert not np.isfinite(values(out)[sees][..., 77]).any()
    case.check(out, columns=np.arange(128) != 77)
    case.check(out, rows=~sees)


@pytest.mark.parametrize("Hq,H,D,n,format", [(40, 8, 128, 1, 16), (40, 8, 128, 1, 8), (64, 8, 64, 5, 16), (64, 8, 128, 5, 16),
                                             (32, 4, 256, 5, 16), (16, 4, 256, 2, 16), (16, 4, 256, 2, 8), (64, 8, 128, 5, 8)])
def test_long_runs(cuda_lib, Hq, H, D, n, format):
    """Many tiles for every CTA, and items that two, three and more of them share."""
    rng = np.random.default_rng(D + n)
    lens = [int(x) for x in rng.integers(500, 4500, 20)] + [9000, n]
    case = AttentionCase(lens, [n] * len(lens), Hq, H, D, 16, format=format, seed=24)
    finish(case, case.run(w4, uniform=True))


@pytest.mark.parametrize("Hq,H", [(8, 1), (64, 1)])
def test_one_item_shared_by_every_cta(cuda_lib, Hq, H):
    """More parts than are joined at once: groups of them, then the groups."""
    case = AttentionCase([60000], [1], Hq, H, 128, 16, seed=25)
    finish(case, case.run(w4))


def test_many_rows_same_bits_again(cuda_lib):
    case = AttentionCase([3000, 170, 900, 13], [13] * 4, 16, 2, 128, 16, seed=26)
    q, table, lens, starts = case.q.to(DEV), gpu(case.table), gpu(case.lens), gpu(case.starts)
    first = w4.w4_attn_decode(q, case.k, case.v, table, lens, starts=starts)
    finish(case, first)
    dirty = torch.full((w4.w4_attn_decode_workspace_bytes(q, case.k, 4),), 255, dtype=torch.uint8, device=DEV)
    out = q.clone()
    for i in range(20):
        if i % 5 == 0:
            dirty.fill_(i)
        out.copy_(q)
        w4.w4_attn_decode(out, case.k, case.v, table, lens, starts=starts, workspace=dirty, out=out)  # in place
        assert torch.equal(first.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("zeros", [3, 60, 900])
@pytest.mark.parametrize("n", [1, 13])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_of_zero_in_8_bits(cuda_lib, zeros, n, D):
    """Tokens whose values are all zero have a value scale of zero; their weights count all the same."""
    case = AttentionCase([1000, zeros + n], [n, n], 8, 1, D, 16, format=8, seed=zeros + D)
    for b in range(2):
        for token in range(zeros):
            page, place = case.table[b, token // 16], token % 16
            case.v[page, place] = 0
            case.v_scales[page, :, place] = 0
            case.vv[page, place] = 0.0
    finish(case, case.run(w4))


# ---- many rows over a cache in 8 bits
@pytest.mark.parametrize("Hq,H,D", MANY)
@pytest.mark.parametrize("order,page_size", [("token", 16), ("head", 24), ("token", 1)])
def test_many_rows_in_8_bits(cuda_lib, Hq, H, D, order, page_size):
    lens = [0, 7, 1, 13, 200, 300, 64, 0, 129, 20, 257]
    fresh = [5, 7, 1, 13, 5, 13, 0, 0, 1, 20, 9]
    case = AttentionCase(lens, fresh, Hq, H, D, page_size, order, format=8, seed=Hq + D)
    finish(case, case.run(w4))


@pytest.mark.parametrize("window", [1, 9, 100, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_windows_in_8_bits(cuda_lib, window, D):
    lens, fresh = [1, 40, 500, 333, 13, 130], [1, 13, 9, 13, 13, 6]
    case = AttentionCase(lens, fresh, 16, 2, D, 16, format=8, seed=window)
    finish(case, case.run(w4, window=window), window=window)


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_many_rows_scales_in_8_bits(cuda_lib, scale):
    case = AttentionCase([50, 300, 777], [13, 9, 13], 16, 2, 128, 16, format=8, seed=21)
    finish(case, case.run(w4, scale=scale), scale=scale)


@pytest.mark.parametrize("n", [1, 13])
@pytest.mark.parametrize("scale,std", [(1.0, 8.0), (-0.3, 30.0)])
def test_sharp_scores_in_8_bits(cuda_lib, scale, std, n):
    """One token outweighs the others by far.  Its values have no codes of zero, under which a column would hold nothing
    but weights that underflow."""
    case = AttentionCase([50, 300, 777], [n] * 3, 16, 2, 128, 16, format=8, seed=21, std=std)
    step = np.where(case.vv == 0, values(case.v_scales.transpose(1, 2))[..., None], 0.0)
    case.vv = case.vv + np.where(np.isfinite(step), step, 0.0)
    case.v[case.v == 0] = 1
    finish(case, case.run(w4, scale=scale), scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_many_rows_hidden_tokens_in_8_bits(cuda_lib, D, window, bad):
    for L in (45, 300):
        n = 13
        case = AttentionCase([L, 200], [n, 13], 16, 2, D, 16, format=8, seed=22)
        token = L - 8
        page, place = int(case.table[0, token // 16]), token % 16
        case.k_scales[page, :, place] = bad
        case.v_scales[page, :, place] = bad
        out = case.run(w4, window=window)
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0
        position = np.arange(L - n, L)
        sees = np.concatenate([(token <= position) & ((window == 0) | (token > position - window)), [False] * 13])
        case.check(out, window=window, rows=~sees)
        assert not np.isfinite(values(out)[sees]).all(axis=(1, 2)).any()


@pytest.mark.parametrize("Hq,H,D,n", [(64, 8, 64, 13), (64, 8, 128, 13), (40, 8, 128, 13), (32, 4, 256, 5), (16, 1, 192, 20)])
def test_long_runs_of_many_rows_in_8_bits(cuda_lib, Hq, H, D, n):
    """Many tiles for every CTA: each ring goes round, and a cache page may end inside a tile."""
    rng = np.random.default_rng(D + n)
    lens = [int(x) for x in rng.integers(300, 2500, 8)] + [6000, n]
    case = AttentionCase(lens, [n] * len(lens), Hq, H, D, 24, format=8, seed=24)
    out = case.run(w4, uniform=True)
    finish(case, out)
    for _ in range(3):
        assert torch.equal(out.view(torch.int16), case.run(w4, uniform=True).view(torch.int16))


def test_calls_without_a_workspace_in_a_graph_and_among_other_allocations(cuda_lib):
    """The workspace of a call goes back to the allocator with it: what is allocated next on the stream may lie there."""
    case = AttentionCase([3000, 170, 900, 13], [1] * 4, 16, 2, 128, 16, seed=27)
    q, table, lens = case.q.to(DEV), gpu(case.table), gpu(case.lens)
    first = w4.w4_attn_decode(q, case.k, case.v, table, lens)
    finish(case, first)
    size = w4.w4_attn_decode_workspace_bytes(q, case.k, 4)
    outs = []
    for i in range(10):
        outs.append(w4.w4_attn_decode(q, case.k, case.v, table, lens))
        torch.empty(size, dtype=torch.uint8, device=DEV).fill_(i)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(3):
            outs.append(w4.w4_attn_decode(q, case.k, case.v, table, lens))
            torch.empty(size, dtype=torch.uint8, device=DEV).fill_(i)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first.view(torch.int16), x.view(torch.int16)) for x in outs)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 9, 100])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_more_than_128_rows_in_8_bits(cuda_lib, D, window, bad):
    """208 rows to a key-value head: two row tiles of the tensor-core kernel, whatever the head_dim, with a hidden token."""
    for L in (45, 300):
        n = 13
        case = AttentionCase([L, 200, 13], [n, 13, 13], 32, 2, D, 16, format=8, seed=28)
        token = L - 8
        page, place = int(case.table[0, token // 16]), token % 16
        case.k_scales[page, :, place] = bad
        case.v_scales[page, :, place] = bad
        out = case.run(w4, window=window)
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0
        position = np.arange(L - n, L)
        sees = np.concatenate([(token <= position) & ((window == 0) | (token > position - window)), [False] * 26])
        case.check(out, window=window, rows=~sees)
        assert not np.isfinite(values(out)[sees]).all(axis=(1, 2)).any()
