"""Refusals of the paged key-value cache's entry points: each is made on the host, before any launch (the addresses are
never read)."""
import os
import random

import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from gemm_rtn_sym_gb300 import build as b

A = 0x10000  # fake addresses, 64 KB apart


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.library_path()):
        b.build()
    return w4.load()


def cache(**kw):
    # 4 pages of 16 tokens, 2 heads of 128: 4096 elements a page
    base = dict(k=A, v=2 * A, k_scales=None, v_scales=None, pages=4, page_stride=4096, token_stride=256, head_stride=128,
                page_size=16, kv_heads=2, head_dim=128, format=16)
    return w4._KvCache(**{**base, **kw})


def rows(at, token_stride=1024, head_stride=128):
    return w4._Rows(at, token_stride, head_stride)


def pages(lib, **kw):
    a = dict(lens=A, target=2 * A, B=4, page_size=16, ring=3 * A, pages=8, free=4 * A, table=5 * A, stride=6, width=6, T=10,
             new=6 * A, starts=7 * A, slots=8 * A, positions=9 * A, left=10 * A)
    a.update(kw)
    return lib.w4_kv_pages(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(page_size=0), "INVALID_ARG"),
    (dict(pages=0), "INVALID_ARG"), (dict(width=0), "INVALID_ARG"), (dict(stride=5), "INVALID_ARG"),
    (dict(T=1 << 31), "UNSUPPORTED"), (dict(pages=1 << 31), "UNSUPPORTED"),
    (dict(lens=None), "INVALID_ARG"), (dict(ring=None), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"),
    (dict(starts=None), "INVALID_ARG"), (dict(left=None), "INVALID_ARG"),
    (dict(slots=8 * A + 4), "MISALIGNED"), (dict(lens=A + 2), "MISALIGNED"), (dict(free=4 * A + 4), "MISALIGNED"),
    (dict(new=A), "INVALID_ARG"),                 # in place
    (dict(left=4 * A), "INVALID_ARG"),            # counters in place
    (dict(positions=8 * A + 40), "INVALID_ARG"),  # positions inside slots
    (dict(starts=5 * A + 92), "INVALID_ARG"),     # starts on the table's last entry
])
def test_pages_refusals(lib, kw, expect):
    assert pages(lib, **kw) == getattr(w4, "W4_ERR_" + expect)


def append(lib, c=None, rope=None, T=3, q_heads=8, q=None, out=None, k=None, v=None, slots=20 * A, no_rope=False):
    c = cache() if c is None else c
    r = dict(positions=11 * A, axis_stride=3, cos=12 * A, sin=13 * A, rows=100, rotary=64, axes=2,
             sections=(w4._i32 * 4)(10, 22, 0, 0), cycled=0, paired=0)
    r.update(rope or {})
    return lib.w4_kv_append(c, None if no_rope else w4._Rope(**r), T, q_heads, q or rows(14 * A), out or rows(15 * A),
                            k or rows(16 * A), v or rows(17 * A), slots, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), "INVALID_ARG"), (dict(q_heads=-1), "INVALID_ARG"), (dict(no_rope=True), "INVALID_ARG"),
    (dict(c=cache(pages=0)), "INVALID_ARG"), (dict(c=cache(page_size=0)), "INVALID_ARG"),
    (dict(c=cache(head_dim=120)), "UNSUPPORTED"), (dict(c=cache(head_dim=272)), "UNSUPPORTED"),
    (dict(c=cache(format=4)), "UNSUPPORTED"), (dict(c=cache(format=8)), "INVALID_ARG"),      # no scales
    (dict(c=cache(k=None)), "INVALID_ARG"), (dict(c=cache(k=A + 8)), "MISALIGNED"),
    (dict(c=cache(token_stride=255)), "INVALID_ARG"),                                        # tokens overlap
    (dict(c=cache(page_stride=0)), "INVALID_ARG"),
    (dict(c=cache(page_stride=4100)), "MISALIGNED"),
    (dict(c=cache(page_stride=1 << 60)), "INVALID_ARG"),                                     # sizes overflow
    (dict(c=cache(v=A + 16384)), "INVALID_ARG"),                                             # values inside the keys
    (dict(rope=dict(rotary=24)), "UNSUPPORTED"), (dict(rope=dict(rotary=144)), "INVALID_ARG"),
    (dict(rope=dict(rotary=-16)), "INVALID_ARG"),
    (dict(rope=dict(axes=0)), "UNSUPPORTED"), (dict(rope=dict(axes=5)), "UNSUPPORTED"),
    (dict(rope=dict(sections=(w4._i32 * 4)(10, 21, 0, 0))), "INVALID_ARG"),
    (dict(rope=dict(sections=(w4._i32 * 4)(-10, 42, 0, 0))), "INVALID_ARG"),
    (dict(rope=dict(rows=0)), "INVALID_ARG"), (dict(rope=dict(axis_stride=2)), "INVALID_ARG"),
    (dict(rope=dict(cos=None)), "INVALID_ARG"), (dict(rope=dict(cos=12 * A + 4)), "MISALIGNED"),
    (dict(slots=None), "INVALID_ARG"), (dict(slots=20 * A + 4), "MISALIGNED"),
    (dict(k=rows(16 * A, head_stride=120)), "INVALID_ARG"), (dict(k=rows(16 * A, head_stride=132)), "MISALIGNED"),
    (dict(q=rows(14 * A, token_stride=512)), "INVALID_ARG"), (dict(out=rows(0)), "INVALID_ARG"),
    (dict(out=rows(14 * A, token_stride=2048)), "INVALID_ARG"),  # over q, not q itself
    (dict(out=rows(16 * A)), "INVALID_ARG"),                     # over k
    (dict(k=rows(A)), "INVALID_ARG"),                            # k inside the cache
])
def test_append_refusals(lib, kw, expect):
    assert append(lib, **kw) == getattr(w4, "W4_ERR_" + expect)


def test_append_of_nothing(lib):
    assert append(lib, T=0) == w4.W4_OK


def attend(lib, c=None, B=3, T=6, q_heads=8, q=None, out=None, table=18 * A, stride=5, width=5, lens=19 * A, starts=21 * A,
           scale=0.1, window=0, workspace=64 * A, size=1 << 40):
    return lib.w4_attn_decode(cache() if c is None else c, B, T, q_heads, q or rows(14 * A), out or rows(15 * A), table,
                              stride, width, lens, starts, scale, window, workspace, size, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(q_heads=0), "INVALID_ARG"),
    (dict(q_heads=7), "INVALID_ARG"), (dict(width=0), "INVALID_ARG"), (dict(stride=4), "INVALID_ARG"),
    (dict(window=-1), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(T=7, starts=None), "INVALID_ARG"), (dict(T=1 << 30), "UNSUPPORTED"),
    (dict(c=cache(head_dim=100)), "UNSUPPORTED"), (dict(c=cache(format=8)), "INVALID_ARG"),
    (dict(table=None), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"), (dict(workspace=None), "INVALID_ARG"),
    (dict(table=18 * A + 1), "MISALIGNED"), (dict(starts=21 * A + 2), "MISALIGNED"), (dict(workspace=64 * A + 16), "MISALIGNED"),
    (dict(size=0), "INVALID_ARG"), (dict(q=rows(14 * A + 2)), "MISALIGNED"), (dict(out=rows(A)), "INVALID_ARG"),
    (dict(out=rows(18 * A)), "INVALID_ARG"), (dict(out=rows(14 * A + 256)), "INVALID_ARG"),
    (dict(workspace=0x100, size=16 * A), "INVALID_ARG"),  # workspace over q
])
def test_attention_refusals(lib, kw, expect):
    assert attend(lib, **kw) == getattr(w4, "W4_ERR_" + expect)


def test_attention_of_nothing(lib):
    assert attend(lib, T=0) == w4.W4_OK
    assert attend(lib, B=0, T=0) == w4.W4_OK


def test_workspace_bytes(lib):
    c = cache()
    assert lib.w4_attn_decode_workspace_bytes(c, 3, 6, 8) > 0
    assert lib.w4_attn_decode_workspace_bytes(c, 3, 6, 7) == 0
    assert lib.w4_attn_decode_workspace_bytes(c, -1, 6, 8) == 0
    assert lib.w4_attn_decode_workspace_bytes(cache(head_dim=300), 3, 6, 8) == 0


@pytest.mark.parametrize("size", [2 ** 31 - 1, 2 ** 31 - 2 ** 16 + 1])
def test_sizes_whose_loops_would_pass_2_to_the_31(lib, size):
    """Kernels count requests, tokens and rows in 32 bits and step past the last by less than 2¹⁶."""
    assert pages(lib, B=size) == w4.W4_ERR_UNSUPPORTED
    assert append(lib, T=size, rope=dict(rotary=0)) == w4.W4_ERR_UNSUPPORTED
    assert attend(lib, B=size, T=0) == w4.W4_ERR_UNSUPPORTED
    assert attend(lib, c=cache(kv_heads=1), B=1, T=size, q_heads=1) == w4.W4_ERR_UNSUPPORTED
    assert attend(lib, B=1, T=size // 8 + 1, q_heads=8) == w4.W4_ERR_UNSUPPORTED


# ---- keys and values (and the rows of a projection) side by side in one piece of memory: places that share no byte
#      pass, and those that do are refused.  Units: elements of bf16, 2 heads of 128.
SIDE_BY_SIDE = {  # strides of page, token, head; where the values start
    "page": (8192, 256, 128, 4096),         # [pages, 2, 16, heads, dim]
    "token": (8192, 512, 128, 256),         # [pages, 16, 2, heads, dim]
    "head": (8192, 512, 256, 128),          # [pages, 16, heads, 2, dim]
    "head, page of heads": (8192, 256, 4096, 128),  # [pages, heads, 16, 2, dim]
    "page of heads": (8192, 128, 4096, 2048),       # [pages, heads, 2, 16, dim]
    "pool": (4096, 256, 128, 4 * 4096),     # [2, pages, 16, heads, dim]
}


def side_by_side(where, shift=0):
    page, token, head, v = SIDE_BY_SIDE[where]
    return cache(k=A, v=A + 2 * (v + shift), page_stride=page, token_stride=token, head_stride=head)


def far_rows(i, token_stride=1024, head_stride=128):
    return rows(0x1000000 + i * 0x10000, token_stride, head_stride)


def append_far(lib, c, **kw):
    a = dict(q=far_rows(0), out=far_rows(1), k=far_rows(2), v=far_rows(3), slots=0x1000000 + 20 * A,
             rope=dict(positions=0x1000000 + 11 * A, cos=0x1000000 + 12 * A, sin=0x1000000 + 13 * A))
    return append(lib, c=c, **{**a, **kw})


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory: only without a device")


@needs_no_gpu
@pytest.mark.parametrize("where", SIDE_BY_SIDE)
def test_keys_and_values_side_by_side_pass(lib, where):
    assert append_far(lib, side_by_side(where)) == w4.W4_ERR_CUDA  # (no device here)


@pytest.mark.parametrize("shift", [-120, -8, 8, 120])
@pytest.mark.parametrize("where", [w for w in SIDE_BY_SIDE if w != "pool"])
def test_keys_and_values_that_share_bytes_are_refused(lib, where, shift):
    assert append_far(lib, side_by_side(where, shift)) == w4.W4_ERR_INVALID_ARG


@needs_no_gpu
def test_rows_of_a_projection_with_the_heads_side_by_side_pass(lib):
    """[T, heads, 3, dim]: query, key and value of each head in turn, the queries turned in place."""
    q, k, v = (rows(0x1000000 + 2 * 128 * i, 2 * 384, 384) for i in range(3))
    assert append_far(lib, cache(), q_heads=2, q=q, out=q, k=k, v=v) == w4.W4_ERR_CUDA


def test_rows_of_a_projection_that_share_bytes_are_refused(lib):
    q, k, v = (rows(0x1000000 + 2 * 128 * i, 2 * 384, 384) for i in range(3))
    assert append_far(lib, cache(), q_heads=2, q=q, out=k, k=k, v=v) == w4.W4_ERR_INVALID_ARG
    k = rows(0x1000000 + 2 * 120, 2 * 384, 384)
    assert append_far(lib, cache(), q_heads=2, q=q, out=q, k=k, v=v) == w4.W4_ERR_INVALID_ARG


@pytest.mark.parametrize("seed", range(40))
def test_rows_meet_where_they_share_a_byte(lib, seed):
    """Against a count of the bytes: queries out over keys, at any offset and with any nested strides."""
    r = random.Random(seed)
    for _ in range(50):
        T, Hq = r.randint(1, 4), 2 * r.randint(1, 3)
        dim, kind = 16, r.random()
        inner = r.choice([16, 32, 48, 64])
        def strides(heads):
            if r.random() < 0.5:
                return (inner * heads + 16 * r.randint(0, 4), inner)
            return (inner, inner * T + 16 * r.randint(0, 4))
        so, sk = strides(Hq), strides(2)
        if kind < 0.5:
            sk = so
        at = 8 * r.randint(-60, 60)
        c = cache(head_dim=dim, page_stride=4096, token_stride=256, head_stride=128)
        out, k = rows(0x4000000, *so), rows(0x4000000 + 2 * at, *sk)

        def taken(base, s, heads):
            return {base + t * s[0] + h * s[1] + i for t in range(T) for h in range(heads) for i in range(dim)}
        nested = all(s[0] >= (heads - 1) * s[1] + dim if s[0] >= s[1] else s[1] >= (T - 1) * s[0] + dim or heads == 1
                     for s, heads in ((so, Hq), (sk, 2)))
        share = bool(taken(0, so, Hq) & taken(at, sk, 2))
        if not nested or (not share and torch.cuda.is_available()):
            continue
        rope = dict(rotary=0)
        got = append(lib, c=c, rope=rope, T=T, q_heads=Hq, q=rows(0x6000000, 4096, 64), out=out, k=k, v=far_rows(3),
                     slots=0x1000000 + 20 * A)
        if share:
            assert got == w4.W4_ERR_INVALID_ARG
        elif so == sk:
            assert got == w4.W4_ERR_CUDA
        else:  # strides that differ may be refused without need
            assert got in (w4.W4_ERR_CUDA, w4.W4_ERR_INVALID_ARG)


@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("head_dim,D", [(64, 64), (128, 128), (256, 256), (16, 64), (80, 128), (192, 256)])
def test_workspace_of_many_rows(lib, head_dim, D, format):
    """208 rows to each of 8 heads: parts of 128 rows, two for each CTA of a grid of one on an SM (152 of them)."""
    size = lib.w4_attn_decode_workspace_bytes(cache(kv_heads=8, head_dim=head_dim, format=format), 16, 208, 128)
    parts = 2 * 152 * 128 * (2 + D) * 4
    assert parts <= size <= 1.1 * parts
