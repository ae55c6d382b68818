"""Refusals of the entry points for shared pages, normalised appends and shared prefixes: on the host, before any launch (the
addresses are never read)."""
import os

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
    base = dict(k=A, v=2 * A, k_scales=None, v_scales=None, pages=4, page_stride=4096, token_stride=256, head_stride=128,
                page_size=16, kv_heads=2, head_dim=128, format=16)
    return w4._KvCache(**{**base, **kw})


def rows(at, token_stride=1024, head_stride=128):
    return w4._Rows(at, token_stride, head_stride)


def held(lib, **kw):
    a = dict(lens=A, target=2 * A, B=4, page_size=16, ring=3 * A, pages=8, free=4 * A, table=5 * A, stride=6, width=6, T=10,
             holders=11 * A, new=6 * A, starts=7 * A, slots=8 * A, positions=9 * A, left=10 * A, workspace=None, size=0)
    a.update(kw)
    return lib.w4_kv_pages_held(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), "INVALID_ARG"), (dict(pages=1 << 31), "UNSUPPORTED"), (dict(holders=None), "INVALID_ARG"),
    (dict(holders=11 * A + 2), "MISALIGNED"), (dict(holders=A), "INVALID_ARG"), (dict(holders=3 * A + 16), "INVALID_ARG"),
    (dict(holders=5 * A + 92), "INVALID_ARG"), (dict(stride=5), "INVALID_ARG"), (dict(left=4 * A), "INVALID_ARG"),
])
def test_held_pages_refusals(lib, kw, expect):
    assert held(lib, **kw) == getattr(w4, "W4_ERR_" + expect)


def test_workspace_of_held_pages(lib):
    """None for few entries; then a word for each page and a bit for each entry."""
    assert lib.w4_kv_pages_held_workspace_bytes(64, 256, 5000) == 0
    assert lib.w4_kv_pages_held_workspace_bytes(1000, 300, 5000) >= 4 * 5000 + 1000 * 300 // 8
    for bad in ((-1, 4, 8), (4, 0, 8), (4, 4, 0), (4, 4, 1 << 31), (1 << 16, 1 << 16, 8)):
        assert lib.w4_kv_pages_held_workspace_bytes(*bad) == 0
    far = dict(lens=1 << 32, target=2 << 32, new=3 << 32, starts=4 << 32, table=5 << 32, B=1000, width=300, stride=300, pages=8)
    need = lib.w4_kv_pages_held_workspace_bytes(1000, 300, 8)
    assert held(lib, **far) == w4.W4_ERR_INVALID_ARG
    assert held(lib, **far, workspace=20 * A, size=need - 1) == w4.W4_ERR_INVALID_ARG
    assert held(lib, **far, workspace=20 * A + 64, size=need) == w4.W4_ERR_MISALIGNED
    assert held(lib, **far, workspace=3 << 32, size=need) == w4.W4_ERR_INVALID_ARG  # over the new lengths
    assert held(lib, **{**far, "B": 1 << 16, "width": 1 << 16, "stride": 1 << 16}) == w4.W4_ERR_UNSUPPORTED


def fork(lib, **kw):
    a = dict(lens=A, source=2 * A, keep=3 * A, B=4, page_size=16, table=4 * A, stride=6, width=6, holders=5 * A, ring=6 * A,
             pages=8, free=7 * A, new=8 * A, copies=9 * A, left=10 * A)
    a.update(kw)
    return lib.w4_kv_fork(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), "INVALID_ARG"), (dict(B=2 ** 31 - 1), "UNSUPPORTED"), (dict(page_size=0), "INVALID_ARG"),
    (dict(width=0), "INVALID_ARG"), (dict(pages=0), "INVALID_ARG"), (dict(pages=1 << 31), "UNSUPPORTED"),
    (dict(stride=5), "INVALID_ARG"), (dict(stride=1 << 60), "INVALID_ARG"),
    *((dict([(n, None)]), "INVALID_ARG") for n in ("lens", "source", "keep", "table", "holders", "ring", "free", "new", "copies", "left")),
    (dict(lens=A + 2), "MISALIGNED"), (dict(free=7 * A + 4), "MISALIGNED"), (dict(copies=9 * A + 1), "MISALIGNED"),
    (dict(new=A), "INVALID_ARG"), (dict(left=7 * A), "INVALID_ARG"), (dict(holders=6 * A), "INVALID_ARG"),
    (dict(copies=8 * A + 8), "INVALID_ARG"), (dict(source=9 * A + 44), "INVALID_ARG"), (dict(keep=4 * A + 92), "INVALID_ARG"),
])
def test_fork_refusals(lib, kw, expect):
    assert fork(lib, **kw) == getattr(w4, "W4_ERR_" + expect)


def compact(lib, **kw):
    a = dict(lens=A, B=4, page_size=16, table=2 * A, stride=6, width=6, holders=3 * A, pages=8, free=4 * A, new=5 * A,
             new_stride=6, new_holders=6 * A, ring=7 * A, left=8 * A, copies=9 * A)
    a.update(kw)
    return lib.w4_kv_compact(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), "INVALID_ARG"), (dict(page_size=0), "INVALID_ARG"), (dict(pages=0), "INVALID_ARG"),
    (dict(pages=(1 << 20) + 1), "UNSUPPORTED"), (dict(width=0), "INVALID_ARG"), (dict(stride=5), "INVALID_ARG"),
    (dict(new_stride=5), "INVALID_ARG"),
    *((dict([(n, None)]), "INVALID_ARG") for n in ("lens", "table", "holders", "free", "new", "new_holders", "ring", "left", "copies")),
    (dict(table=2 * A + 1), "MISALIGNED"), (dict(left=8 * A + 4), "MISALIGNED"),
    (dict(new=2 * A), "INVALID_ARG"), (dict(new_holders=3 * A), "INVALID_ARG"), (dict(left=4 * A), "INVALID_ARG"),
    (dict(ring=6 * A + 28), "INVALID_ARG"), (dict(copies=9 * A, ring=9 * A + 44), "INVALID_ARG"),
])
def test_compact_refusals(lib, kw, expect):
    assert compact(lib, **kw) == getattr(w4, "W4_ERR_" + expect)


@pytest.mark.parametrize("c,copies,n,expect", [
    (cache(), 20 * A, -1, "INVALID_ARG"), (cache(), None, 3, "INVALID_ARG"), (cache(), 20 * A + 2, 3, "MISALIGNED"),
    (cache(), A + 64, 3, "INVALID_ARG"), (cache(), 20 * A, 2 ** 31 - 1, "UNSUPPORTED"),
    (cache(format=8), 20 * A, 3, "INVALID_ARG"), (cache(head_dim=120), 20 * A, 3, "UNSUPPORTED"),
    (cache(page_size=1 << 24, page_stride=1 << 32, v=A + (1 << 36)), 20 * A, 3, "UNSUPPORTED"),  # 4 GB of keys in a page and more
    (cache(v=A + 16), 20 * A, 3, "INVALID_ARG"),
])
def test_copy_refusals(lib, c, copies, n, expect):
    assert lib.w4_kv_copy(c, copies, n, None) == getattr(w4, "W4_ERR_" + expect)


def test_copy_of_nothing(lib):
    assert lib.w4_kv_copy(cache(), None, 0, None) == w4.W4_OK


def append(lib, norm=None, T=3, q_heads=8, no_norm=False, c=None):
    r = dict(positions=11 * A, axis_stride=3, cos=12 * A, sin=13 * A, rows=100, rotary=64, axes=2,
             sections=(w4._i32 * 4)(10, 22, 0, 0), cycled=0, paired=0)
    n = dict(q_weight=30 * A, k_weight=31 * A, format=16, eps=1e-6, unit_offset=0)
    n.update(norm or {})
    return lib.w4_kv_append_norm(c or cache(), w4._Rope(**r), None if no_norm else w4._Norm(**n), T, q_heads, rows(14 * A), rows(15 * A),
                                 rows(16 * A), rows(17 * A), 20 * A, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(no_norm=True), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(c=cache(head_dim=272)), "UNSUPPORTED"),
    *((dict(norm=n), e) for n, e in [
        (dict(format=8), "UNSUPPORTED"), (dict(eps=0.0), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"),
        (dict(eps=float("nan")), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"), (dict(eps=1e-21), "INVALID_ARG"),
        (dict(q_weight=None), "INVALID_ARG"), (dict(k_weight=None), "INVALID_ARG"), (dict(q_weight=30 * A + 1), "MISALIGNED"),
        (dict(k_weight=31 * A + 2, format=32), "MISALIGNED"),
        (dict(k_weight=15 * A + 128), "INVALID_ARG"),      # inside the queries that are written
        (dict(q_weight=A + 256), "INVALID_ARG"),           # inside the cache
    ]),
])
def test_append_refusals(lib, kw, expect):
    assert append(lib, **kw) == getattr(w4, "W4_ERR_" + expect)


def test_append_of_nothing(lib):
    assert append(lib, T=0) == w4.W4_OK


def attend(lib, c=None, B=3, T=6, q_heads=8, q=None, out=None, table=18 * A, stride=5, width=5, lens=19 * A, starts=21 * A,
           groups=2, group_starts=22 * A, prefix=23 * A, prefix_stride=7, prefix_width=7, prefix_lens=24 * A, scale=0.1,
           workspace=64 * A, size=1 << 40):
    return lib.w4_attn_decode_shared(c or cache(), B, T, q_heads, q or rows(14 * A), out or rows(15 * A), table, stride, width,
                                     lens, starts, groups, group_starts, prefix, prefix_stride, prefix_width, prefix_lens,
                                     scale, workspace, size, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), "INVALID_ARG"), (dict(q_heads=7), "INVALID_ARG"), (dict(groups=-1), "INVALID_ARG"),
    (dict(groups=2 ** 31 - 1), "UNSUPPORTED"), (dict(prefix_width=0), "INVALID_ARG"), (dict(prefix_stride=6), "INVALID_ARG"),
    (dict(T=7, starts=None), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
    (dict(q_heads=1, c=cache(kv_heads=1), T=(1 << 30) + 1), "UNSUPPORTED"),
    (dict(group_starts=None), "INVALID_ARG"), (dict(prefix=None), "INVALID_ARG"), (dict(prefix_lens=None), "INVALID_ARG"),
    (dict(group_starts=22 * A + 2), "MISALIGNED"), (dict(prefix=23 * A + 1), "MISALIGNED"), (dict(prefix_lens=24 * A + 3), "MISALIGNED"),
    (dict(workspace=None), "INVALID_ARG"), (dict(size=0), "INVALID_ARG"), (dict(workspace=64 * A + 16), "MISALIGNED"),
    (dict(out=rows(23 * A)), "INVALID_ARG"), (dict(out=rows(24 * A)), "INVALID_ARG"), (dict(out=rows(22 * A)), "INVALID_ARG"),
    (dict(out=rows(14 * A + 256)), "INVALID_ARG"), (dict(workspace=0x100, size=16 * A), "INVALID_ARG"),
])
def test_attention_refusals(lib, kw, expect):
    assert attend(lib, **kw) == getattr(w4, "W4_ERR_" + expect)


def test_attention_of_nothing(lib):
    assert attend(lib, T=0) == w4.W4_OK
    assert attend(lib, B=0, T=0) == w4.W4_OK


def test_workspace_bytes(lib):
    c = cache()
    plain = lib.w4_attn_decode_workspace_bytes(c, 3, 6, 8)
    assert lib.w4_attn_decode_shared_workspace_bytes(c, 3, 6, 8, 0) == plain
    # at least the rows' sums besides
    assert lib.w4_attn_decode_shared_workspace_bytes(c, 3, 6, 8, 2) >= plain + 6 * 8 * (128 + 2) * 4
    for bad in ((c, 3, 6, 7, 2), (c, -1, 6, 8, 2), (c, 3, 6, 8, -1), (cache(head_dim=300), 3, 6, 8, 2)):
        assert lib.w4_attn_decode_shared_workspace_bytes(*bad) == 0
    need = lib.w4_attn_decode_shared_workspace_bytes(c, 3, 6, 8, 2)
    assert attend(lib, size=need - 1) == w4.W4_ERR_INVALID_ARG


def test_binding_checks_before_a_call():
    t = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        w4.w4_kv_fork(t, t, t, torch.zeros(3, 2, dtype=torch.int32), t, t, torch.zeros(2, dtype=torch.int64), 16)
    with pytest.raises(TypeError):
        w4.w4_kv_copy(torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16), t)


def test_the_compiled_module_leaves_unusual_calls_alone():
    """Tensors on the host, of other types or numbers of dimensions, no tensors at all, a wrong number of arguments."""
    w4.load()
    fast = w4._fast
    t, table, r = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    k = torch.zeros((2, 16, 2, 128), dtype=torch.bfloat16)
    q = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    calls = {"kv_fork": [t, t, t, table, t, t, r, 16, None, None, None], "kv_copy": [k, k, table, None, None],
             "kv_compact": [t, table, t, r, 16, None, None, None, None, None],
             "kv_pages_held": [t, t, table, t, r, 16, 4, t, None, None, None, None, None],
             "kv_append_norm": [q, q, q, q, q, t, k, k, k, k, r, 1e-6, False, None, False, False, None, None, None],
             "attn_decode_shared": [q, k, k, table, t, t, table, t, None, None, None, None, None]}
    for name, args in calls.items():
        fn = getattr(fast, name)
        assert fn(*args) is NotImplemented
        assert fn(*args[:-1]) is NotImplemented and fn(*args, None) is NotImplemented and fn() is NotImplemented
        for i in range(len(args)):
            for other in (None, 3, "x", torch.zeros(0), object()):
                assert fn(*args[:i], other, *args[i + 1:]) is NotImplemented
