"""Pages that several requests hold: forks, releases, compaction and copies against their restatement, call by call and in
runs as a server makes them."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from oracle import kv_share_oracle as SO
from tests.kv_cases import DEV, bf16_tensor, gpu, paged, values

pytestmark = pytest.mark.gpu


def finish(status=0):
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == status


def same(got, want, name=""):
    assert np.array_equal(got.cpu().numpy(), want), name


class Pool:
    """Bookkeeping on the GPU and beside it in numpy."""

    def __init__(self, B, width, pages, page_size, head=0, seed=0):
        self.page_size, self.pages = page_size, pages
        self.table = np.full((B, width), -1, np.int32)
        self.holders = np.zeros(pages, np.int32)
        self.ring = np.random.default_rng(seed).permutation(pages).astype(np.int32)
        self.ring = np.roll(self.ring, head % pages)
        self.free = np.array([head, head + pages])
        self.lens = np.zeros(B, np.int32)
        self.upload()

    def upload(self):
        self.t, self.h, self.r = gpu(self.table), gpu(self.holders), gpu(self.ring)
        self.f, self.l = gpu(self.free, torch.int64), gpu(self.lens)

    def step(self, target, tokens=None, status=0):
        T = int(np.maximum(np.asarray(target) - self.lens, 0).sum()) if tokens is None else tokens
        want = SO.pages_held(self.lens, target, self.table, self.ring, self.free, self.page_size, T, self.holders)
        got = w4.w4_kv_pages(self.l, gpu(target), self.t, self.r, self.f, self.page_size, T, holders=self.h)
        finish(status)
        self.l, starts, slots, positions, self.f = got
        for x, name in ((self.l, "new_lens"), (starts, "starts"), (slots, "slots"), (positions, "positions"),
                        (self.f, "free_range"), (self.t, "table"), (self.r, "ring"), (self.h, "holders")):
            same(x, want[name], name)
        self.lens, self.free, self.table, self.ring, self.holders = (want[n] for n in ("new_lens", "free_range", "table", "ring", "holders"))
        return starts, slots, positions

    def fork(self, source, keep, status=0):
        want = SO.fork(self.lens, source, keep, self.table, self.holders, self.ring, self.free, self.page_size)
        self.l, copies, self.f = w4.w4_kv_fork(self.l, gpu(source), gpu(keep), self.t, self.h, self.r, self.f, self.page_size)
        finish(status)
        for x, name in ((self.l, "new_lens"), (copies, "copies"), (self.f, "free_range"), (self.t, "table"), (self.h, "holders")):
            same(x, want[name], name)
        self.lens, self.free, self.table, self.holders = (want[n] for n in ("new_lens", "free_range", "table", "holders"))
        return copies

    def compact(self, status=0):
        want = SO.compact(self.lens, self.table, self.holders, self.free, self.page_size)
        self.t, self.h, self.r, self.f, copies = w4.w4_kv_compact(self.l, self.t, self.h, self.f, self.page_size)
        finish(status)
        for x, name in ((self.t, "table"), (self.h, "holders"), (self.r, "ring"), (self.f, "free_range"), (copies, "copies")):
            same(x, want[name], name)
        self.table, self.holders, self.ring, self.free = (want[n] for n in ("table", "holders", "ring", "free_range"))
        return copies

    def consistent(self):
        count = np.zeros(self.pages, np.int64)
        for b, n in enumerate(self.lens):
            np.add.at(count, self.table[b, :-(-int(n) // self.page_size)], 1)
        assert np.array_equal(count, self.holders)
        free = {int(self.ring[i % self.pages]) for i in range(self.free[0], self.free[1])}
        assert len(free) == self.free[1] - self.free[0] and free == set(np.nonzero(count == 0)[0].tolist())


# ---------------------------------------------------------------- call by call
@pytest.mark.parametrize("page_size", [1, 3, 16, 64])
def test_forks_and_ends(cuda_lib, page_size):
    B = 9
    pool = Pool(B, 40, 300, page_size, head=12345678901, seed=page_size)
    n = min(30 * page_size, 39 * page_size)
    pool.step([n, n - 1, 0, 0, 0, 0, 0, 0, page_size])
    pool.fork([-1, -1, 0, 0, 1, 1, 8, 8, -1], [0, 0, n, n // 2, n - 1, 0, page_size, 1, 0])
    pool.step(pool.lens + 1)
    pool.step([0, n // 3, *pool.lens[2:]])
    pool.consistent()
    pool.step(np.zeros(B, np.int32))
    pool.consistent()
    assert pool.free[1] - pool.free[0] == 300


def test_growth_into_a_page_with_other_holders_is_refused(cuda_lib):
    pool = Pool(4, 8, 20, 16)
    pool.step([40, 0, 0, 7])
    pool.fork([-1, 0, -1, -1], [0, 32, 0, 0])
    pool.step([40, 20, 0, 9])       # request 1 shrinks into the second shared page
    pool.step([41, 21, 0, 9])
    assert pool.lens.tolist() == [41, 20, 0, 9]
    pool.step([0, 20, 0, 9])        # its other holder lets go
    pool.step([0, 21, 0, 9])
    assert pool.lens.tolist() == [0, 21, 0, 9]
    pool.consistent()


def test_a_ring_that_runs_out(cuda_lib):
    pool = Pool(8, 8, 6, 16)
    pool.step([33, 0, 0, 0, 0, 0, 0, 0])
    pool.fork([-1] + [0] * 7, [0, 33, 32, 20, 1, 33, 16, 5])
    assert pool.lens.tolist() == [33, 33, 32, 20, 1, 0, 16, 0]
    pool.step([0] * 8)
    assert pool.free[1] - pool.free[0] == 6


@pytest.mark.parametrize("B", [1, 37, 1024, 1025, 2600])
def test_many_requests(cuda_lib, B):
    rng = np.random.default_rng(B)
    pool = Pool(B, 12, 9 * B + 50, 16, seed=B)
    parents = max(1, B // 5)
    pool.step(np.concatenate([rng.integers(1, 190, parents), np.zeros(B - parents, np.int64)]).astype(np.int32))
    source = np.where(np.arange(B) < parents, -1, rng.integers(0, parents, B))
    keep = np.where(source >= 0, (pool.lens[source] * rng.choice([1.0, 1.0, 0.5, 0.1, 0.0], B)).astype(int), 0)
    pool.fork(source, keep)
    pool.step(pool.lens + rng.integers(0, 3, B).astype(np.int32))
    pool.consistent()
    pool.step(np.where(rng.random(B) < 0.7, 0, pool.lens + 1))
    pool.consistent()
    pool.compact()
    pool.consistent()
    pool.step(np.zeros(B, np.int32))
    pool.consistent()


@pytest.mark.parametrize("width", [2300, 3000, 40000])
def test_many_pages_let_go_at_once(cuda_lib, width):
    """More entries than a CTA takes at a time, each page let go of several times: by one CTA and by many."""
    n = 4 * width - 10
    pool = Pool(7, width, width + 300, 4, seed=2)
    pool.step([n, 0, 0, 0, 0, 0, 100])
    pool.fork([-1, 0, 0, 0, 0, 0, -1], [0, n, n - 2, n // 2, n - 2, 3, 0])
    pool.step([0, 0, n - 2, 17, 0, 0, 99])
    pool.consistent()
    pool.step([0, 0, 0, 0, 0, 0, 0])
    pool.consistent()


@pytest.mark.parametrize("pages", [1, 2, 31, 32, 33, 127, 128, 129, 1000, 4096, 70001, 300000])
def test_compaction(cuda_lib, pages):
    rng = np.random.default_rng(pages)
    for fill in (0.0, 0.3, 0.9, 1.0):
        pool = Pool(3, max(pages, 2), pages, 4, head=977)
        used = np.nonzero(rng.random(pages) < fill)[0]
        a, b = used[:len(used) // 2], used[len(used) // 2:]
        pool.table[:] = rng.integers(-5, pages + 5, pool.table.shape)
        for row, ids in ((0, a), (1, b), (2, a[:5])):
            pool.table[row, :len(ids)] = rng.permutation(ids) if row < 2 else ids
            np.add.at(pool.holders, pool.table[row, :len(ids)], 1)
        pool.lens[:] = [len(a) * 4, max(0, len(b) * 4 - 3), 4 * len(a[:5])]
        free = np.nonzero(pool.holders == 0)[0]
        pool.free[:] = [977, 977 + len(free)]
        pool.ring[:] = -7
        pool.ring[(977 + np.arange(len(free))) % pages] = free
        pool.upload()
        pool.compact()
        pool.consistent()
        pool.compact()  # nothing moves any more
        pool.consistent()


def test_compaction_into_given_outputs(cuda_lib):
    pool = Pool(3, 5, 20, 16, seed=4)
    pool.step([50, 0, 70])
    pool.step([0, 20, 70])
    outs = dict(new_table=torch.full((3, 5), 9, dtype=torch.int32, device=DEV), new_holders=gpu(np.full(20, 9)),
                free_pages=gpu(np.full(20, 9)), free_range_out=gpu([9, 9], torch.int64), copies=gpu(np.full((3, 10), 9)))
    wide = torch.full((3, 8), 77, dtype=torch.int32, device=DEV)
    wide[:, :5] = pool.t
    got = w4.w4_kv_compact(pool.l, wide[:, :5], pool.h, pool.f, 16, **outs)
    want = SO.compact(pool.lens, pool.table, pool.holders, pool.free, 16)
    finish()
    for x, o, name in zip(got, outs.values(), ("table", "holders", "ring", "free_range", "copies")):
        assert x is o
        same(x, want[name], name)
    with pytest.raises(ValueError):
        w4.w4_kv_compact(pool.l, pool.t, pool.h, pool.f, 16, copies=gpu(np.zeros((3, 9))))


# ---------------------------------------------------------------- out of range
def test_numbers_out_of_range(cuda_lib):
    pool = Pool(6, 4, 12, 16)
    pool.step([30, 20, 0, 0, 0, 0])
    pool.fork([-1, -1, 7, -2, 0, 0], [0, 0, 5, 5, 31, -1], status=w4.W4_ERR_INVALID_ARG)
    assert pool.lens.tolist() == [30, 20, 0, 0, 0, 0]
    pool.fork([1, -1, -1, -1, 3, -1], [5, 0, 0, 0, 0, 0], status=w4.W4_ERR_INVALID_ARG)  # request 0 has tokens
    assert pool.lens.tolist() == [30, 20, 0, 0, 0, 0]
    pool.step([30, 20, 0, 0, 0, 70])       # past the table: not granted
    pool.step([-1, 20, 0, 0, 0, 0], status=w4.W4_ERR_INVALID_ARG)
    # pages that the pool does not have, in a table
    pool.table[0, :2] = [99, -3]
    pool.upload()
    pool.fork([-1, -1, 0, -1, -1, -1], [0, 0, 30, 0, 0, 0], status=w4.W4_ERR_INVALID_ARG)
    pool.compact(status=w4.W4_ERR_INVALID_ARG)
    pool.step([0, 0, 30, 0, 0, 0], status=w4.W4_ERR_INVALID_ARG)


def test_a_length_past_the_table_is_left_alone(cuda_lib):
    pool = Pool(3, 4, 12, 16)
    pool.step([30, 20, 0])
    pool.lens[1] = 1000
    pool.upload()
    pool.step([31, 0, 0], status=w4.W4_ERR_INVALID_ARG)
    pool.fork([-1, -1, 1], [0, 0, 500], status=w4.W4_ERR_INVALID_ARG)
    pool.compact(status=w4.W4_ERR_INVALID_ARG)


@pytest.mark.parametrize("width", [4, 6000])
def test_pages_that_nobody_holds_are_not_given_back(cuda_lib, width):
    pool = Pool(3, width, 12, 16)
    pool.step([30, 20, 0])
    pool.holders[pool.table[0, 0]] = 0
    pool.holders[pool.table[1, 1]] = -5
    pool.upload()
    pool.step([0, 0, 0], status=w4.W4_ERR_INVALID_ARG)


# ------------------------------------------------------------------- copies
@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("order", ["token", "head", "pair"])
@pytest.mark.parametrize("heads,dim,page_size", [(2, 128, 16), (8, 128, 64), (3, 80, 7), (1, 16, 1), (4, 256, 16), (5, 192, 33), (1, 64, 300)])
def test_copies(cuda_lib, heads, dim, page_size, order, format):
    pages = 23
    k, v = paged(pages, page_size, heads, dim, order, None, seed=dim)
    scales = {}
    if format == 8:
        g = torch.Generator().manual_seed(dim)
        k, v = (torch.empty_strided(x.shape, x.stride(), dtype=torch.int8, device=DEV).copy_(
            torch.randint(-128, 128, x.shape, generator=g, dtype=torch.int8)) for x in (k, v))
        scales = {n: bf16_tensor((pages, heads, page_size), i).to(DEV) for i, n in enumerate(("k_scales", "v_scales"))}
    rng = np.random.default_rng(page_size)
    ids = rng.permutation(pages)
    copies = np.full((3, 30), -1, np.int32)
    copies[2] = 0
    at = rng.permutation(30)[:11]
    copies[0, at], copies[1, at] = ids[:11], ids[11:22]
    copies[0, at[1]] = copies[0, at[0]]                  # one page to two
    copies[2, at] = rng.integers(0, page_size + 1, 11)
    copies[2, at[:3]] = page_size
    want = {n: SO.copy(x.float().cpu().numpy(), copies) for n, x in (("k", k), ("v", v))}
    want.update({n: SO.copy(values(x).transpose(0, 2, 1), copies) for n, x in scales.items()})
    w4.w4_kv_copy(k, v, gpu(copies), **scales)
    finish()
    same(k.float(), want["k"])
    same(v.float(), want["v"])
    for n, x in scales.items():
        same(x.double().transpose(1, 2), want[n])


def test_many_copies_and_bad_ones(cuda_lib):
    """More entries than a CTA lists at a time; entries out of range copy nothing."""
    pages = 6001
    k, v = paged(pages, 2, 1, 32, "token", None, seed=1)
    copies = np.stack([np.arange(3000), 3000 + np.random.default_rng(2).permutation(3000), np.full(3000, 2)]).astype(np.int32)
    copies[:, 100:2500:7] = np.array([[-1], [-1], [0]])
    bad = copies.copy()
    bad[:, 5], bad[:, 6], bad[:, 7], bad[:, 8] = [pages, 3001, 2], [3, -1, 2], [3, 3002, 3], [-1, 5000, 1]
    bad[:, 9], bad[:, 10] = [7, 3003, -1], [2 ** 31 - 1, -2 ** 31, 1]
    done = bad.copy()
    done[:, 5:11] = np.array([[-1], [-1], [0]])
    want = SO.copy(k.float().cpu().numpy(), done)
    w4.w4_kv_copy(k, v, gpu(bad))
    finish(w4.W4_ERR_INVALID_ARG)
    same(k.float(), want)
    w4.w4_kv_copy(k, v, torch.empty((3, 0), dtype=torch.int32, device=DEV))
    w4.w4_kv_copy(k, v, gpu([[4, 4], [4, 4], [2, 1]]))  # a page to itself
    finish()
    same(k.float(), want)


def test_copies_past_2_to_the_32_bytes(cuda_lib):
    """A cache of 6 GB: a page near its end to one near its start and back."""
    k = torch.zeros((45000, 16, 8, 256), dtype=torch.int8, device=DEV)
    v = torch.zeros_like(k)
    scales = {n: torch.zeros((45000, 8, 16), dtype=torch.bfloat16, device=DEV) for n in ("k_scales", "v_scales")}
    both = torch.zeros((45000, 2, 16, 8, 256), dtype=torch.int8, device=DEV)  # 2.9 GB
    k, v = both[:, 0], both[:, 1]
    k[44999], v[44999], k[1], v[1] = 7, 8, 3, 4
    scales["k_scales"][44999], scales["v_scales"][1] = 2.0, 5.0
    w4.w4_kv_copy(k, v, gpu([[44999, 1], [0, 44998], [16, 9]]), **scales)
    finish()
    assert (k[0] == 7).all() and (v[0] == 8).all() and (scales["k_scales"][0] == 2).all()
    assert (k[44998, :9] == 3).all() and (v[44998, :9] == 4).all() and (k[44998, 9:] == 0).all()
    assert (scales["v_scales"][44998, :, :9] == 5).all() and (scales["v_scales"][44998, :, 9:] == 0).all()


# ---------------------------------------------------------------- a server's run
@pytest.mark.parametrize("format", [16, 8])
@pytest.mark.parametrize("seed", range(3))
def test_a_run_keeps_every_requests_tokens(cuda_lib, seed, format):
    """Requests begin, grow, drop tokens, are forked and end, the pool is compacted; after each step the cache has, for
    every request, the tokens that were written for it or for the one it was forked from."""
    rng = np.random.default_rng(seed)
    B, P, pages, H, D = 12, [16, 5, 1][seed], [90, 250, 700][seed], 2, 64
    pool = Pool(B, -(-400 // P), pages, P, head=int(rng.integers(0, 10 ** 12)), seed=seed)
    k, v = paged(pages, P, H, D, ["token", "head", "pair"][seed], 0.0, 0)
    scales = {}
    if format == 8:
        k, v = (torch.empty_strided(x.shape, x.stride(), dtype=torch.int8, device=DEV).zero_() for x in (k, v))
        scales = {n: torch.zeros((pages, H, P), dtype=torch.bfloat16, device=DEV) for n in ("k_scales", "v_scales")}
    history, stamp = [[] for _ in range(B)], 1

    def check():
        got = {"k": values(k), "v": values(v)}
        for n, x in scales.items():
            got[n[0]] = got[n[0]] * values(x).transpose(0, 2, 1)[..., None]
        for b in range(B):
            n = int(pool.lens[b])
            assert n == len(history[b])
            at = np.arange(n)
            rows = pool.table[b, at // P] if n else np.zeros(0, int)
            assert (got["k"][rows, at % P] == np.array(history[b]).reshape(-1, 1, 1)).all()
            assert (got["v"][rows, at % P] == -np.array(history[b]).reshape(-1, 1, 1)).all()

    for turn in range(25):
        what = rng.random(B)
        target = pool.lens.copy()
        for b in range(B):
            n = int(pool.lens[b])
            if n == 0 and what[b] < 0.5:
                target[b] = rng.integers(1, 60)
            elif what[b] < 0.15:
                target[b] = 0
            elif what[b] < 0.3:
                target[b] = rng.integers(0, n + 1)
            elif n:
                target[b] = min(n + int(rng.integers(0, 20)), 390)
        before = pool.lens
        starts, slots, _ = pool.step(target)
        T = slots.numel()
        # each token's rows hold its stamp (a power of two times at most 127: exact in both formats)
        marks = (stamp + np.arange(T)) % 100 + 1
        stamp += T
        x = torch.tensor(marks, dtype=torch.bfloat16, device=DEV)[:, None, None].expand(T, H, D).contiguous()
        if T:
            w4.w4_kv_append(None, x, -x, None, None, None, k, v, slots, **scales)
        for b in range(B):
            new = marks[int(starts[b]):int(starts[b + 1])].tolist()
            if pool.lens[b] == target[b]:
                history[b] = history[b][:int(target[b])] + new
            else:
                assert pool.lens[b] == before[b]
        if format == 8:  # (a stamp comes back as scale times code: check what is exact there)
            for b in range(B):
                history[b] = [float(torch.tensor(m / 127, dtype=torch.bfloat16)) * 127 if isinstance(m, (int, np.integer)) else m for m in history[b]]
        check()
        live = np.nonzero(pool.lens > 0)[0]
        if len(live):
            source = np.where((pool.lens == 0) & (rng.random(B) < 0.6), rng.choice(live, B), -1)
            keep = np.where(source >= 0, np.minimum(pool.lens[source], rng.integers(0, 400, B)), 0)
            copies = pool.fork(source, keep)
            w4.w4_kv_copy(k, v, copies, **scales)
            for b in range(B):
                if source[b] >= 0 and pool.lens[b] == keep[b]:
                    history[b] = list(history[source[b]][:keep[b]])
            check()
        if turn % 5 == 4:
            w4.w4_kv_copy(k, v, pool.compact(), **scales)
            check()
        pool.consistent()


def test_captured_steps_run_again(cuda_lib):
    """A fork, its copies and a step in one graph, replayed on other numbers in the same tensors."""
    P, pages, H, D = 16, 64, 2, 64
    pool = Pool(4, 12, pages, P, seed=9)
    k, v = paged(pages, P, H, D, "token", None, seed=3)
    lens, source, keep, target = gpu([0] * 4), gpu([-1] * 4), gpu([0] * 4), gpu([0] * 4)
    free = pool.f.clone()
    side = torch.cuda.Stream()

    def steps():
        new, copies, left = w4.w4_kv_fork(lens, source, keep, pool.t, pool.h, pool.r, free, P)
        w4.w4_kv_copy(k, v, copies)
        return new, copies, left, w4.w4_kv_pages(new, target, pool.t, pool.r, left, P, 40, holders=pool.h)

    with torch.cuda.stream(side):
        steps()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new, copies, left, (end, _, slots, _, after) = steps()
    cache, state = values(k), None
    for turn, (l, s, n, m) in enumerate([([0] * 4, [-1] * 4, [0] * 4, [20, 0, 0, 0]), (None, [-1, 0, 0, -1], [0, 20, 7, 0], [21, 21, 8, 0]),
                                         (None, [-1, -1, -1, 2], [0, 0, 0, 8], [0, 25, 8, 9])]):
        lens.copy_(gpu(l) if l else end)
        free.copy_(free if turn == 0 else after)
        source.copy_(gpu(s)), keep.copy_(gpu(n)), target.copy_(gpu(m))
        a = SO.fork(lens.tolist(), s, n, pool.t.cpu().numpy(), pool.h.cpu().numpy(), pool.r.cpu().numpy(), free.tolist(), P)
        b = SO.pages_held(a["new_lens"], m, a["table"], pool.r.cpu().numpy(), a["free_range"], P, 40, a["holders"])
        cache = SO.copy(cache, a["copies"])
        graph.replay()
        finish()
        for x, want in ((copies, a["copies"]), (end, b["new_lens"]), (pool.t, b["table"]), (pool.h, b["holders"]),
                        (pool.r, b["ring"]), (after, b["free_range"]), (slots, b["slots"])):
            same(x, want)
        assert np.array_equal(values(k), cache)
        assert end.tolist() == m
        state = m
    assert state == [0, 25, 8, 9]


def test_calls_on_another_stream(cuda_lib):
    pool = Pool(3, 10, 40, 16, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pool.step([100, 0, 33])
        pool.fork([-1, 0, -1], [0, 90, 0])
        pool.step([0, 91, 33])
        pool.compact()
    pool.consistent()


def test_captured_release_of_many_pages(cuda_lib):
    """The kernels with a workspace: two captured calls, replayed in turn and again, and an eager call in between."""
    width, n = 6000, 23900
    pools = [Pool(4, width, width + 200, 4, seed=s) for s in (21, 22)]
    for pool in pools:
        pool.step([n, 0, 0, 70])
        pool.fork([-1, 0, 0, -1], [0, n - 1, n // 2, 0])
    target = gpu([0, n // 3, 0, 71])
    graphs, start, outs = [], [], []
    for pool in pools:
        start.append([x.clone() for x in (pool.t, pool.h, pool.r)])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(w4.w4_kv_pages(pool.l, target, pool.t, pool.r, pool.f, 4, 1, holders=pool.h))
        graphs.append(graph)
    want = [SO.pages_held(p.lens, target.tolist(), p.table, p.ring, p.free, 4, 1, p.holders) for p in pools]
    for turn in range(3):
        for i in (0, 1):
            for x, before in zip((pools[i].t, pools[i].h, pools[i].r), start[i]):
                x.copy_(before)
            graphs[i].replay()
            if turn == 1:
                t, h, r = (x.clone() for x in start[1 - i])
                w4.w4_kv_pages(pools[1 - i].l, target, t, r, pools[1 - i].f, 4, 1, holders=h)
                same(h, want[1 - i]["holders"])
        finish()
        for pool, out, w in zip(pools, outs, want):
            for x, name in ((out[0], "new_lens"), (out[4], "free_range"), (pool.t, "table"), (pool.r, "ring"), (pool.h, "holders")):
                same(x, w[name], name)


def test_releases_on_two_streams_at_once(cuda_lib):
    width, n = 6000, 23900
    pools = [Pool(4, width, width + 200, 4, seed=s) for s in (31, 32)]
    for pool in pools:
        pool.step([n, 0, 0, 0])
        pool.fork([-1, 0, 0, -1], [0, n - 1, n // 2, 0])
    target = [0, 5, 0, 0]
    want = [SO.pages_held(p.lens, target, p.table, p.ring, p.free, 4, 0, p.holders) for p in pools]
    target = gpu(target)
    streams, calls = [torch.cuda.Stream() for _ in pools], [[], []]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, pool, got in zip(streams, pools, calls):
            with torch.cuda.stream(s):
                state = [x.clone() for x in (pool.t, pool.r, pool.h)]
                got.append((*state, w4.w4_kv_pages(pool.l, target, *state[:2], pool.f, 4, 0, holders=state[2])[4]))
    finish()
    for got, w in zip(calls, want):
        for t, r, h, left in got:
            same(t, w["table"]), same(r, w["ring"]), same(h, w["holders"]), same(left, w["free_range"])


def test_calls_of_nothing(cuda_lib):
    """No requests, no tokens, no copies."""
    pool = Pool(0, 4, 10, 16, head=3)
    pool.step([])
    pool.fork([], [])
    pool.compact()
    pool.step([], tokens=5)
    pool = Pool(3, 4, 1, 16)
    pool.step([0, 0, 0])
    pool.fork([-1, 0, 1], [0, 0, 0])
    copies = pool.compact()
    assert copies.shape == (3, 0)
    k, v = paged(1, 16, 2, 64, "token", 1.0, 0)
    w4.w4_kv_copy(k, v, copies)
    finish()


def test_the_same_source_and_the_same_page_many_times(cuda_lib):
    """Every request forks the first one; the entries of one page let go together."""
    B = 1500
    pool = Pool(B, 3, 2 * B, 16, seed=5)
    pool.step([40] + [0] * (B - 1))
    pool.fork([-1] + [0] * (B - 1), [0] + [40 - i % 41 for i in range(B - 1)])
    pool.consistent()
    pool.step([40 if b in (7, 900) else 0 for b in range(B)], tokens=80)
    pool.consistent()
    pool.step([0] * B)
    assert pool.free[1] - pool.free[0] == 2 * B


@pytest.mark.parametrize("B,width", [(5, 130000), (2600, 300)])
def test_more_entries_let_go_than_the_grid_has_blocks(cuda_lib, B, width):
    """400000 entries in one call: every CTA has several blocks of them; then a few, and none, of the same table."""
    pages, n = 2 * width + 400000, 4 * (width - 10)
    pool = Pool(B, width, pages, 4, seed=B)
    parents = max(1, B // 8)
    lens = np.where(np.arange(B) < parents, n, 0)
    pool.step(lens)
    child = np.arange(B) >= parents
    keep = np.where(child, n - np.arange(B) % 7 * 10, 0)
    pool.fork(np.where(child, np.arange(B) % parents, -1), keep)
    pool.consistent()
    back = pool.free[1] - pool.free[0]
    pool.step(np.where(np.arange(B) % 11 == 3, 50, np.where(np.arange(B) % 13 == 5, pool.lens, 0)))
    pool.consistent()
    assert pool.free[1] - pool.free[0] > back
    pool.step(pool.lens - np.minimum(pool.lens, 9))
    pool.consistent()
    pool.step(pool.lens)
    pool.step(np.zeros(B, np.int32))
    assert pool.free[1] - pool.free[0] == pages


@pytest.mark.parametrize("ends", [0, 3])
def test_the_time_of_a_step_follows_what_is_let_go_of(cuda_lib, ends):
    """1000 requests of a few hundred tokens whose tables have room for two million: a step that lets go of nothing, or of
    three requests' pages, takes microseconds (a walk over the table's 131 million entries would take a hundred times the limit)."""
    B, width, P, pages = 1000, 131072, 16, 40000
    lens = gpu(np.arange(B) % 500 + 17)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    free, ring = gpu([0, pages], torch.int64), gpu(np.arange(pages))
    holders = gpu(np.zeros(pages))
    total = int(lens.sum())
    lens, *_, free = w4.w4_kv_pages(gpu(np.zeros(B)), lens, table, ring, free, P, total, holders=holders)
    target = (lens + 1) * gpu(np.arange(B) >= ends)
    want = SO.pages_held(lens.tolist(), target.tolist(), table[:, :40].cpu().numpy(), ring.cpu().numpy(), free.tolist(), P, B, holders.cpu().numpy())
    state = [x.clone() for x in (ring, holders)]
    got = w4.w4_kv_pages(lens, target, table, state[0], free, P, B, holders=state[1])
    finish()
    for x, name in ((got[0], "new_lens"), (got[4], "free_range"), (state[0], "ring"), (state[1], "holders"), (table[:, :40], "table")):
        same(x, want[name], name)
    times = []
    for _ in range(10):
        for x, old in zip(state, (ring, holders)):
            x.copy_(old)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        w4.w4_kv_pages(lens, target, table, state[0], free, P, B, holders=state[1])
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end) * 1e3)
    assert min(times) < 500, f"{min(times):.0f} us"
