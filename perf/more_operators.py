"""Operators around the paged key-value cache: cases to measure, their plain forms and their 64-bit values.

Five operators, which a server runs next to the cache's pages, append and attention:

* ``norm``: queries and keys of new tokens normalised head by head (root mean square, with weights), turned by their
  rotary positions in the same pass, keys and values written to the cache.
* ``fork``: requests that begin as others' first tokens: full pages are shared and counted, the page that a request
  will go on writing is its own, a copy.
* ``release``: a step of block tables whose pages have several holders: pages go back to the ring when the last of
  them lets go.
* ``compact``: pages in use move to the pool's lowest ids, so that the rest of the pool lies in one piece.
* ``shared``: attention of the newest tokens of requests that share a long prefix, whose keys and values are read
  once for all of them.

Head layouts and verify rows are those of the repository's layer classes: 16 query and 4 key-value heads of 256, 40 and
8 of 128, 64 and 8 of 128; 16 requests of 13 rows are the 208 rows of the benchmark's largest case.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
HIDDEN = float("-inf")


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One decode token of the smallest layer: latency.  A quarter of the head turns; weights count from 1.
        {"name": "norm-decode-1", "kind": "norm", "tokens": 1, "q_heads": 16, "kv_heads": 4, "dim": 256, "rotary": 64,
         "sections": "11,11,10", "cycled": True, "paired": False, "page": 16, "order": "token", "weights": "bf16",
         "offset": True},
        # The 208 rows of 16 verify passes.
        {"name": "norm-verify-208", "kind": "norm", "tokens": 208, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "rotary": 128, "sections": "64", "cycled": False, "paired": False, "page": 32, "order": "head",
         "weights": "fp32", "offset": False},
        # A prompt of text and images.
        {"name": "norm-prompt-16001", "kind": "norm", "tokens": 16001, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "rotary": 128, "sections": "16,24,24", "cycled": False, "paired": False, "page": 16, "order": "token",
         "weights": "bf16", "offset": False},
        # Four samples for each of two prompts: latency.
        {"name": "fork-2x4", "kind": "fork", "parents": 2, "samples": 4, "shortest": 200, "longest": 1400, "q_heads": 16,
         "kv_heads": 4, "dim": 256, "page": 16, "bits": 16, "order": "token", "mix": 41},
        # Seven samples for each of 64 prompts, in large pages, with a pool that runs out before the last of them.
        {"name": "fork-64x7", "kind": "fork", "parents": 64, "samples": 7, "shortest": 100, "longest": 4097, "q_heads": 40,
         "kv_heads": 8, "dim": 128, "page": 64, "bits": 16, "order": "token", "mix": 42},
        # A decode step of a small server whose requests share prompts: most grow, a few end.
        {"name": "release-step-64", "kind": "release", "parents": 8, "samples": 7, "shortest": 50, "longest": 2000,
         "page": 16, "ends": 0.06, "mix": 43},
        # Samples of many prompts end together, others go on.
        {"name": "release-ends-1000", "kind": "release", "parents": 125, "samples": 7, "shortest": 1, "longest": 4097,
         "page": 16, "ends": 0.6, "mix": 44},
        # A small pool, half of it in use.
        {"name": "compact-300", "kind": "compact", "pages": 300, "requests": 8, "fill": 0.5, "kv_heads": 4, "dim": 256,
         "page": 16, "bits": 16, "order": "token", "mix": 45},
        # The pool of a server that has run for long.
        {"name": "compact-8000", "kind": "compact", "pages": 8001, "requests": 200, "fill": 0.55, "kv_heads": 8, "dim": 128,
         "page": 16, "bits": 16, "order": "token", "mix": 46},
        # Four samples of one short prompt: latency.
        {"name": "shared-4-short", "kind": "shared", "groups": 1, "members": 4, "alone": 0, "prefix_low": 517,
         "prefix_high": 517, "own_low": 1, "own_high": 40, "fresh": 1, "q_heads": 16, "kv_heads": 4, "dim": 256,
         "page": 16, "bits": 16, "order": "token", "mix": 47},
        # Sixty-four questions about one long document.
        {"name": "shared-64-document", "kind": "shared", "groups": 1, "members": 64, "alone": 0, "prefix_low": 16385,
         "prefix_high": 16385, "own_low": 1, "own_high": 512, "fresh": 1, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "page": 16, "bits": 16, "order": "token", "mix": 48},
        # Verify passes of several prompts' samples, some requests on their own, over a cache in 8 bits.
        {"name": "shared-verify-8bit", "kind": "shared", "groups": 12, "members": 8, "alone": 5, "prefix_low": 300,
         "prefix_high": 8192, "own_low": 5, "own_high": 900, "fresh": 5, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "page": 32, "bits": 8, "order": "token", "mix": 49},
    ]


#: What a drawn attention case may cost: bytes, operations and scores of the plain form.
MOST_BYTES, MOST_FLOPS, MOST_SCORES = 4e8, 3.2e10, 3e8
#: Bytes of keys and values that a drawn cache may have.
MOST_CACHE = 6e8


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 3, 4, 8])
    return kv * rng.choice([1, 2, 4, 5, 7, 8]), kv, rng.choice([64, 80, 112, 128, 128, 192, 256])


def draw(rng):
    kind = rng.choice(["norm", "norm", "fork", "release", "compact", "shared", "shared", "shared"])
    q, kv, dim = _heads(rng)
    page, order = rng.choice([8, 16, 24, 32, 64]), rng.choice(["token", "head"])
    if kind == "norm":
        half = rng.choice([dim, dim, dim // 2, dim // 4]) // 16 * 8
        axes = rng.choice([1, 2, 3])
        cuts = sorted(rng.sample(range(1, half), axes - 1)) if axes > 1 else []
        sections = [b - a for a, b in zip([0] + cuts, cuts + [half])]
        most = 16001 * (40 + 2 * 8) * 128 // ((q + 2 * kv) * dim)
        return {"kind": kind, "tokens": _log_int(rng, 1, min(most, 30000)), "q_heads": q, "kv_heads": kv, "dim": dim,
                "rotary": 2 * half, "sections": ",".join(map(str, sections)), "cycled": rng.random() < 0.5,
                "paired": rng.random() < 0.3, "page": page, "order": order, "weights": rng.choice(["bf16", "fp32"]),
                "offset": rng.random() < 0.5}
    if kind == "fork":
        while True:
            case = {"kind": kind, "parents": _log_int(rng, 1, 64), "samples": rng.randint(1, 7), "shortest": 1,
                    "longest": _log_int(rng, 20, 4097), "q_heads": q, "kv_heads": kv, "dim": dim, "page": page,
                    "bits": rng.choice([16, 16, 8]), "order": order, "mix": rng.randrange(1 << 30)}
            pages = sum(-(-n // page) for n in _parent_lengths(case)) + case["parents"] * case["samples"]
            if 4 * pages * page * kv * dim < MOST_CACHE and work(case)["bytes"] <= work(listed()[4])["bytes"]:
                return case
    if kind == "release":
        return {"kind": kind, "parents": _log_int(rng, 1, 125), "samples": rng.randint(1, 7), "shortest": 1,
                "longest": _log_int(rng, 20, 4097), "page": page, "ends": rng.choice([0.05, 0.3, 0.6]),
                "mix": rng.randrange(1 << 30)}
    if kind == "compact":
        most = int(min(8000, 8001 * 16 * 8 * 128 // (page * kv * dim)))
        pages = _log_int(rng, 2, most)
        return {"kind": kind, "pages": pages, "requests": _log_int(rng, 1, min(pages, 200)), "fill": rng.uniform(0.05, 0.55),
                "kv_heads": kv, "dim": dim, "page": page, "bits": rng.choice([16, 16, 8]), "order": order,
                "mix": rng.randrange(1 << 30)}
    while True:
        low, high = sorted([_log_int(rng, 1, 32768), _log_int(rng, 1, 32768)])
        fresh = rng.choice([1, 1, 1, 5, 7, 13])
        case = {"kind": kind, "groups": _log_int(rng, 1, 16), "members": _log_int(rng, 2, 128),
                "alone": rng.choice([0, 0, 1, 5]), "prefix_low": low, "prefix_high": high, "own_low": fresh,
                "own_high": fresh + _log_int(rng, 1, 1000), "fresh": fresh, "q_heads": q, "kv_heads": kv, "dim": dim,
                "page": page, "bits": rng.choice([16, 16, 8]), "order": order, "mix": rng.randrange(1 << 30)}
        prefix, group, own_lens = _shared_lengths(case)
        B = len(group)
        scores = max(case["members"] * max(prefix), B * case["own_high"]) * fresh * q
        padded = B * (case["own_high"] + 2 * page) * kv * dim
        cache = 4 * (sum(prefix) + sum(own_lens) + page * (B + len(prefix))) * kv * dim
        cost = work(case)
        if scores <= MOST_SCORES and padded <= 3e8 and cache <= MOST_CACHE and cost["bytes"] <= MOST_BYTES and \
                cost["flops"] <= MOST_FLOPS:
            return case


# ---------------------------------------------------------------- lengths
def _parent_lengths(case):
    r = random.Random(case["mix"])
    return [_log_int(r, case["shortest"], case["longest"]) for _ in range(case["parents"])]


def _kept(case):
    """Tokens that each sample takes over from its parent: most of them all, the others a part."""
    r = random.Random(case["mix"] + 1)
    return [n if r.random() < 0.8 else r.randint(0, n) for n in _parent_lengths(case) for _ in range(case["samples"])]


def _release_lengths(case):
    """(length of each parent, of each sample, what a sample kept, targets): parents first, then samples."""
    r = random.Random(case["mix"] + 2)
    parents, kept = _parent_lengths(case), _kept(case)
    lens = parents + [k + r.randrange(300) for k in kept]
    target = []
    for n in lens:
        what = r.random()
        if what < case["ends"]:
            target.append(0)
        elif what < 0.8:
            target.append(n + 1)
        elif what < 0.9:
            target.append(n + r.choice([5, 7, 13]))
        else:
            target.append(max(0, n - r.randrange(13)))
    return parents, lens, kept, target


def _compact_lengths(case):
    """Pages of each request; about `fill` of the pool in all."""
    r = random.Random(case["mix"])
    left = max(1, int(case["pages"] * case["fill"]))
    weights = [r.random() ** 2 + 0.01 for _ in range(case["requests"])]
    return [int(left * w / sum(weights)) for w in weights]


def _shared_lengths(case):
    """(prefix of each group, group of each request, −1 for those alone, own tokens of each request)."""
    r = random.Random(case["mix"])
    prefix = [_log_int(r, case["prefix_low"], case["prefix_high"]) for _ in range(case["groups"])]
    group = [g for g in range(case["groups"]) for _ in range(r.randint(max(1, case["members"] // 2), case["members"]))]
    if case["groups"] == 1:
        group = [0] * case["members"]
    group += [-1] * case["alone"]
    return prefix, group, [_log_int(r, case["own_low"], case["own_high"]) for _ in group]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"norm": _prepare_norm, "fork": _prepare_fork, "release": _prepare_release, "compact": _prepare_compact,
            "shared": _prepare_shared}[case["kind"]](case, seed, g)


def _ints(values, dtype=torch.int32):
    return torch.tensor(np.asarray(values), dtype=dtype, device=DEV)


def _cache(case, pages, g):
    """Key or value pages [pages, page, heads, dim] as a view of memory in the case's order."""
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    shape = (pages, P, H, D) if case["order"] == "token" else (pages, H, P, D)
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    return x if case["order"] == "token" else x.transpose(1, 2)


def _codes(x):
    """Codes and scales in 8 bits of the rows of x [pages, page, heads, dim]; scales [pages, heads, page]."""
    scale = (x.float().abs().amax(-1) / 127).to(torch.bfloat16)
    codes = torch.round(x.float() / scale.float()[..., None]).clamp(-128, 127).to(torch.int8)
    return codes, scale.transpose(1, 2).contiguous()


def _caches(case, pages, g):
    k, v = _cache(case, pages, g), _cache(case, pages, g)
    if case["bits"] == 16:
        return {"k_cache": k, "v_cache": v, "k_scales": None, "v_scales": None}
    (k, ks), (v, vs) = _codes(k), _codes(v)
    return {"k_cache": k, "v_cache": v, "k_scales": ks, "v_scales": vs}


def _prepare_norm(case, seed, g):
    T, Hq, H, D, rot = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["rotary"]
    sections = tuple(int(s) for s in case["sections"].split(","))
    rows = 32768
    # Heads of different sizes, as a projection leaves them.
    size = torch.empty((1, Hq + 2 * H, 1), device=DEV).normal_(generator=g).exp()
    qkv = (torch.empty((T, Hq + 2 * H, D), device=DEV).normal_(generator=g) * size).to(torch.bfloat16).view(T, -1)
    P = case["page"]
    pages = -(-T // P) + 9
    ids = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(T, device=DEV) + 3
    slots = ids[t // P] * P + t % P
    drop = torch.rand(T, generator=g, device=DEV) < 0.01
    drop[0] = False
    slots = torch.where(drop, -1, slots)
    start = random.Random(seed).randrange(rows - 20000)
    span = t // 256
    grid = [span, span + t % 256 // 16, span + t % 16]
    positions = torch.stack([torch.where(span % 2 == 1, grid[a], t // 2) + start for a in range(len(sections))]).to(torch.int32)
    frequency = 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / rot)
    angle = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * frequency
    weights = torch.empty((2, D), device=DEV).normal_(std=0.25, generator=g) + (0.0 if case["offset"] else 1.0)
    weights = weights.to(torch.bfloat16 if case["weights"] == "bf16" else torch.float32)
    return {"kind": "norm", "q": qkv[:, :Hq * D].view(T, Hq, D), "k": qkv[:, Hq * D:(Hq + H) * D].view(T, H, D),
            "v": qkv[:, (Hq + H) * D:].view(T, H, D), "q_weight": weights[0], "k_weight": weights[1], "eps": 1e-6,
            "offset": case["offset"], "positions": positions, "cos": angle.cos().float(), "sin": angle.sin().float(),
            "sections": sections, "cycled": case["cycled"], "paired": case["paired"], "k_cache": _cache(case, pages, g),
            "v_cache": _cache(case, pages, g), "slots": slots,
            "q_out": torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)}


def _pool(pages, free, rng):
    """(ring, head): `free` are the free pages in the ring's order."""
    head = int(rng.integers(0, 1 << 40))
    ring = rng.integers(0, pages, pages).astype(np.int32)
    ring[(head + np.arange(len(free))) % pages] = free
    return ring, head


def _prepare_fork(case, seed, g):
    P, S = case["page"], case["samples"]
    lens, kept = _parent_lengths(case), _kept(case)
    n, B = len(lens), len(lens) * (1 + S)
    rng = np.random.default_rng(seed)
    at = rng.permutation(B)                                       # rows of the parents, then of the samples
    have = np.array([-(-x // P) for x in lens])
    need = sum(1 for k in kept if k % P)
    short = need // 20 if n > 32 else 0
    free = need - short + (0 if short else 3)
    pages = int(have.sum()) + free
    ids = rng.permutation(pages).astype(np.int32)
    width = int(have.max()) + 2
    table = np.full((B, width), -1, dtype=np.int32)
    holders = np.zeros(pages, dtype=np.int32)
    begin = np.concatenate([[0], np.cumsum(have)])
    for i in range(n):
        table[at[i], :have[i]] = ids[begin[i]:begin[i + 1]]
        holders[ids[begin[i]:begin[i + 1]]] = 1
    length, source, keep = np.zeros(B, np.int32), np.full(B, -1, np.int32), np.zeros(B, np.int32)
    length[at[:n]] = lens
    source[at[n:]] = np.repeat(at[:n], S)
    keep[at[n:]] = kept
    ring, head = _pool(pages, ids[int(have.sum()):], rng)
    return {"kind": "fork", "page": P, "lens": _ints(length), "source": _ints(source), "keep": _ints(keep),
            "table": _ints(table), "holders": _ints(holders), "ring": _ints(ring),
            "range": _ints([head, head + free], torch.int64), **_caches(case, pages, g)}


def _prepare_release(case, seed, g):
    P, S = case["page"], case["samples"]
    parents, lens, kept, target = _release_lengths(case)
    n, B = len(parents), len(lens)
    rng = np.random.default_rng(seed)
    at = rng.permutation(B)
    have = np.array([-(-x // P) for x in lens])
    want = np.array([-(-x // P) for x in target])
    full = np.array([0] * n + [k // P for k in kept])             # pages that a sample shares
    mine = have - full
    # Samples that have not grown out of their parent's pages keep those to themselves.
    need = int(np.maximum(want - have, 0).sum())
    pages = int(mine.sum()) + need + 11
    ids = rng.permutation(pages).astype(np.int32)
    width = int(max(have.max(), want.max())) + 2
    table = np.full((B, width), -1, dtype=np.int32)
    holders = np.zeros(pages, dtype=np.int32)
    begin = np.concatenate([[0], np.cumsum(mine)])
    for i in range(B):
        row = table[at[i]]
        if i >= n:
            row[:full[i]] = table[at[(i - n) // S], :full[i]]
        row[full[i]:have[i]] = ids[begin[i]:begin[i + 1]]
        np.add.at(holders, row[:have[i]], 1)
    length, goal = np.zeros(B, np.int32), np.zeros(B, np.int32)
    length[at], goal[at] = lens, target
    free = ids[int(mine.sum()):]
    ring, head = _pool(pages, free, rng)
    return {"kind": "release", "page": P, "tokens": int(np.maximum(goal - length, 0).sum()), "lens": _ints(length),
            "target": _ints(goal), "table": _ints(table), "holders": _ints(holders), "ring": _ints(ring),
            "range": _ints([head, head + len(free)], torch.int64)}


def _prepare_compact(case, seed, g):
    P, pages = case["page"], case["pages"]
    mine = _compact_lengths(case)
    B, live = len(mine), sum(mine)
    rng = np.random.default_rng(seed)
    ids = rng.permutation(pages).astype(np.int32)
    shared = [int(rng.integers(0, max(mine[0], 1))) if b and rng.random() < 0.3 else 0 for b in range(B)]
    width = max(mine) + mine[0] + 2
    table = rng.integers(-1, pages, (B, width)).astype(np.int32)  # what lies behind a request's pages is of no meaning
    holders = np.zeros(pages, dtype=np.int32)
    lens, begin = np.zeros(B, np.int32), np.concatenate([[0], np.cumsum(mine)])
    for b in range(B):
        row = np.concatenate([table[0, :shared[b]], ids[begin[b]:begin[b + 1]]])  # some begin with request 0's pages
        table[b, :len(row)] = row
        np.add.at(holders, row, 1)
        lens[b] = max(0, len(row) * P - int(rng.integers(0, P)))
    head = int(rng.integers(0, 1 << 40))
    return {"kind": "compact", "page": P, "lens": _ints(lens), "table": _ints(table), "holders": _ints(holders),
            "range": _ints([head, head + pages - live], torch.int64), **_caches(case, pages, g)}


def _prepare_shared(case, seed, g):
    P, N = case["page"], case["fresh"]
    prefix, group, own_lens = _shared_lengths(case)
    rng = np.random.default_rng(seed)
    G, B = len(prefix), len(group)
    counts = [group.count(i) for i in range(G)]
    order = rng.permutation(G)                                    # of the groups in the batch
    group = [int(i) for i in order for _ in range(counts[i])] + [-1] * (B - sum(counts))
    own_lens = rng.permutation(own_lens)
    before = np.array([prefix[i] if i >= 0 else 0 for i in group])
    lens = before + own_lens
    have_p = np.array([-(-p // P) for p in prefix])
    have, full = -(-lens // P), before // P
    mine = have - full
    pages = int(have_p.sum() + mine.sum()) + 5
    ids = rng.permutation(pages).astype(np.int32)
    prefix_table = np.full((G, int(have_p.max()) + 1), -1, dtype=np.int32)
    begin = np.concatenate([[0], np.cumsum(have_p)])
    for i in range(G):
        prefix_table[i, :have_p[i]] = ids[begin[i]:begin[i + 1]]
    table = np.full((B, int(have.max()) + 2), -1, dtype=np.int32)
    at = int(have_p.sum())
    for b in range(B):
        if group[b] >= 0:
            table[b, :full[b]] = prefix_table[group[b], :full[b]]
        table[b, full[b]:have[b]] = ids[at:at + mine[b]]
        at += int(mine[b])
    starts = np.concatenate([[0], np.cumsum([counts[i] for i in order])])
    q = torch.empty((B * N, case["q_heads"], case["dim"]), dtype=torch.bfloat16, device=DEV).normal_(std=1.5, generator=g)
    return {"kind": "shared", "q": q, "table": _ints(table), "lens": _ints(lens), "group_starts": _ints(starts),
            "prefix_table": _ints(prefix_table[order]), "prefix_lens": _ints(np.array(prefix)[order]), "fresh": N,
            "out": torch.empty_like(q), **_caches(case, pages, g),
            "host": (starts.tolist(), np.array(prefix)[order].tolist(), before.tolist(), lens.tolist())}


# ---------------------------------------------------------------- one pass
def run(state):
    kind = state["kind"]
    if own:
        return {"norm": _own_norm, "fork": _own_fork, "release": _own_release, "compact": _own_compact,
                "shared": _own_shared}[kind](state)
    return {"norm": _plain_norm, "fork": _plain_fork, "release": _plain_release, "compact": _plain_compact,
            "shared": _plain_shared}[kind](state)


def _caches_of(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales") if s[n] is not None}


def _own_norm(s):
    import gemm_rtn_sym_gb300 as w4

    w4.w4_kv_append_norm(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"], s["cos"], s["sin"],
                         s["k_cache"], s["v_cache"], s["slots"], eps=s["eps"], unit_offset=s["offset"],
                         sections=s["sections"], cycled=s["cycled"], paired=s["paired"], q_out=s["q_out"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_fork(s):
    import gemm_rtn_sym_gb300 as w4

    holders = s["holders"].clone()  # (counted up in place: a second pass begins where the first did)
    lens, copies, left = w4.w4_kv_fork(s["lens"], s["source"], s["keep"], s["table"], holders, s["ring"], s["range"],
                                       s["page"])
    w4.w4_kv_copy(s["k_cache"], s["v_cache"], copies, k_scales=s["k_scales"], v_scales=s["v_scales"])
    return {"lens": lens, "table": s["table"], "holders": holders, "copies": copies, "range": left, **_caches_of(s)}


def _own_release(s):
    import gemm_rtn_sym_gb300 as w4

    holders = s["holders"].clone()
    lens, starts, slots, positions, left = w4.w4_kv_pages(s["lens"], s["target"], s["table"], s["ring"], s["range"],
                                                          s["page"], s["tokens"], holders=holders)
    return {"table": s["table"], "ring": s["ring"], "holders": holders, "range": left, "lens": lens, "starts": starts,
            "slots": slots, "positions": positions}


def _own_compact(s):
    import gemm_rtn_sym_gb300 as w4

    table, holders, ring, left, copies = w4.w4_kv_compact(s["lens"], s["table"], s["holders"], s["range"], s["page"])
    w4.w4_kv_copy(s["k_cache"], s["v_cache"], copies, k_scales=s["k_scales"], v_scales=s["v_scales"])
    return {"table": table, "holders": holders, "ring": ring, "range": left, "copies": copies, **_caches_of(s)}


def _own_shared(s):
    import gemm_rtn_sym_gb300 as w4

    return w4.w4_attn_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["group_starts"],
                                    s["prefix_table"], s["prefix_lens"], k_scales=s["k_scales"],
                                    v_scales=s["v_scales"], out=s["out"])


def _axes(sections, cycled):
    """The axis of each frequency: blocks one after another, or the axes in turn while they have frequencies left."""
    if not cycled:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    turns = sorted((i, a) for a, n in enumerate(sections) for i in range(n))
    return [a for _, a in turns]


def _normed(x, weight, eps, offset):
    x, w = x.float(), weight.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps) * (1 + w if offset else w)


def _turned(x, cos, sin, paired):
    """x [T, heads, dim] in 32 bits, its first 2·F values rotated by cos, sin [T, F]."""
    F = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    a, b = (x[..., 0:2 * F:2], x[..., 1:2 * F:2]) if paired else (x[..., :F], x[..., F:2 * F])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if paired else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., 2 * F:]], -1)


def _plain_norm(s):
    axis = torch.tensor(_axes(s["sections"], s["cycled"]), device=DEV)
    rows = s["positions"].long()[axis].t()                        # [T, F]
    cos, sin = s["cos"].gather(0, rows), s["sin"].gather(0, rows)
    q = _turned(_normed(s["q"], s["q_weight"], s["eps"], s["offset"]), cos, sin, s["paired"]).to(torch.bfloat16)
    k = _turned(_normed(s["k"], s["k_weight"], s["eps"], s["offset"]), cos, sin, s["paired"]).to(torch.bfloat16)
    stored = s["slots"] >= 0
    # A token without a slot stands for the first one that has a slot, which is then written twice alike.
    source = torch.where(stored, torch.arange(stored.numel(), device=DEV), stored.to(torch.uint8).argmax())
    slots, P = s["slots"][source], s["k_cache"].shape[1]
    s["k_cache"][slots // P, slots % P] = k[source]
    s["v_cache"][slots // P, slots % P] = s["v"][source]
    s["q_out"].copy_(q)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_copy(s, copies):
    """The first copies[2] tokens of pages copies[0] to pages copies[1]; −1 for none."""
    if copies.shape[1] == 0:
        return
    there = copies[0] >= 0
    # An entry without a copy stands for the first one that has one.
    i = torch.where(there, torch.arange(there.numel(), device=DEV), there.to(torch.uint8).argmax())
    source, to, n = copies[:, i].long().clamp(min=0)
    P = s["k_cache"].shape[1]
    first = torch.arange(P, device=DEV) < n[:, None]
    for name in ("k_cache", "v_cache"):
        s[name][to] = torch.where(first[..., None, None], s[name][source], s[name][to])
    for name in ("k_scales", "v_scales"):
        if s[name] is not None:
            s[name][to] = torch.where(first[:, None, :], s[name][source], s[name][to])


def _plain_fork(s):
    P, table, ring, holders = s["page"], s["table"], s["ring"], s["holders"].clone()
    lens, keep = s["lens"].long(), s["keep"].long()
    B, W = table.shape
    head, tail = s["range"][0], s["range"][1]
    parent = s["source"].long().clamp(min=0)
    valid = (s["source"] >= 0) & (lens == 0) & (keep <= lens[parent])
    need = (valid & (keep % P > 0)).long()
    cum = need.cumsum(0)
    granted = valid & ((need == 0) | (cum <= tail - head))
    full = keep // P
    fresh = ring[(head + cum - 1) % ring.numel()]
    c = torch.arange(W, device=DEV)[None, :]
    takes = granted[:, None] & (c < full[:, None])
    own_page = (granted & (need > 0))[:, None] & (c == full[:, None])
    source_page = table[parent, full.clamp(max=W - 1)]
    rows = torch.where(takes, table[parent], torch.where(own_page, fresh[:, None], table))
    table.copy_(rows)
    longer = torch.cat([holders, holders[:1]])
    longer.scatter_add_(0, torch.where(takes | own_page, rows, ring.numel()).flatten().long(),
                        torch.ones(B * W, dtype=torch.int32, device=DEV))
    copies_there = granted & (need > 0)
    copies = torch.stack([torch.where(copies_there, source_page, -1), torch.where(copies_there, fresh, -1),
                          torch.where(copies_there, keep % P, 0).to(torch.int32)])
    _plain_copy(s, copies)
    used = torch.where(copies_there, cum, 0).max()
    return {"lens": torch.where(granted, keep, lens).to(torch.int32), "table": table, "holders": longer[:-1],
            "copies": copies, "range": torch.stack([head + used, tail]), **_caches_of(s)}


def _plain_release(s):
    P, table, ring, holders = s["page"], s["table"], s["ring"], s["holders"]
    lens, target = s["lens"].long(), s["target"].long()
    B, W = table.shape
    R = ring.numel()
    head, tail = s["range"][0], s["range"][1]
    have, want = (lens + P - 1) // P, (target + P - 1) // P
    grow = (target - lens).clamp(min=0)
    last = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long().clamp(min=0)
    fits = (target <= W * P) & ~((grow > 0) & (lens % P > 0) & (holders[last] > 1))
    need = torch.where(fits, (want - have).clamp(min=0), 0)
    cum = need.cumsum(0)
    granted = fits & ((need == 0) | (cum <= tail - head))
    first = head + cum - need
    starts = torch.cat([torch.zeros_like(grow[:1]), grow.cumsum(0)])
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(starts[1:], t, right=True).clamp(max=B - 1)
    position = lens[b] + t - starts[b]
    index = position // P
    fresh = index - have[b]
    page = torch.where(fresh >= 0, ring[(first[b] + fresh) % R], table[b, index.clamp(max=W - 1)]).long()
    slots = torch.where(granted[b], page * P + position % P, -1)
    c = torch.arange(W, device=DEV)[None, :]
    back = (c >= want[:, None]) & (c < have[:, None])             # entries that let go of their page
    entry = torch.where(back, table, R).long().flatten()
    count = torch.zeros(R + 1, dtype=torch.int64, device=DEV).scatter_add_(0, entry, torch.ones_like(entry))
    order = torch.arange(B * W, device=DEV)
    latest = torch.full((R + 1,), -1, device=DEV).scatter_reduce_(0, entry, order, "amax")
    after = holders - count[:R]
    gone = back.flatten() & (latest[entry] == order) & (torch.cat([after, after[:1]])[entry] == 0)
    given = gone.cumsum(0)
    longer = torch.cat([ring, ring[:1]])
    longer[torch.where(gone, (tail + given - 1) % R, R)] = table.flatten()
    new = granted[:, None] & (c >= have[:, None]) & (c < want[:, None])
    pages = ring[(first[:, None] + c - have[:, None]) % R]
    after = torch.cat([after, after[:1]]).to(torch.int32)
    after[torch.where(new, pages, R).flatten().long()] = 1
    table.copy_(torch.where(new, pages, table))
    ring.copy_(longer[:R])
    used = torch.where(granted & (need > 0), cum, 0).max()
    return {"table": table, "ring": ring, "holders": after[:R], "range": torch.stack([head + used, tail + given[-1]]),
            "lens": torch.where(granted, target, lens).to(torch.int32), "starts": starts.to(torch.int32), "slots": slots,
            "positions": position.to(torch.int32)}


def _plain_compact(s):
    P, table, holders = s["page"], s["table"], s["holders"]
    pages, head = holders.numel(), s["range"][0]
    M = pages // 2
    ids = torch.arange(pages, device=DEV)
    live = holders > 0
    count = live.sum()
    hole, mover = ~live & (ids < count), live & (ids >= count)
    hole_at, mover_at = torch.where(hole, hole.cumsum(0) - 1, M), torch.where(mover, mover.cumsum(0) - 1, M)
    copies = torch.full((3, M + 1), -1, device=DEV)
    copies[1].scatter_(0, hole_at, torch.where(hole, ids, -1))
    copies[0].scatter_(0, mover_at, torch.where(mover, ids, -1))
    moved = torch.arange(M + 1, device=DEV) < mover.sum()
    copies = torch.where(moved, copies, -1)
    copies[2] = torch.where(moved, P, 0)
    to = torch.where(mover, copies[1][mover_at], ids)
    have = (s["lens"].long() + P - 1) // P
    c = torch.arange(table.shape[1], device=DEV)[None, :]
    new_table = torch.where(c < have[:, None], to[table.long().clamp(min=0)], table).to(torch.int32)
    new_holders = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)
    new_holders[torch.where(live, to, pages)] = holders
    ring = torch.full((pages + 1,), -1, dtype=torch.int32, device=DEV)
    ring[torch.where(ids >= count, (head + ids - count) % pages, pages)] = ids.to(torch.int32)
    copies = copies[:, :M].to(torch.int32)
    _plain_copy(s, copies)
    return {"table": new_table, "holders": new_holders[:pages], "ring": ring[:pages],
            "range": torch.stack([head, head + pages - count]), "copies": copies, **_caches_of(s)}


def _rows32(cache, scales, pages):
    """Rows of pages [..., n] in 32 bits: [..., heads, n · page, dim]."""
    x = cache[pages].float()                                      # [..., n, P, H, D]
    if scales is not None:
        x = x * scales[pages].float().transpose(-2, -1)[..., None]
    return x.flatten(-4, -3).transpose(-3, -2)


def _plain_shared(s):
    q, N = s["q"], s["fresh"]
    T, Hq, D = q.shape
    P, H = s["k_cache"].shape[1], s["k_cache"].shape[2]
    G, B = Hq // H, T // N
    starts, prefix, before, lens = s["host"]
    factor = 1.0 / math.sqrt(D)
    rows = q.float().view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    # Each request's own tokens, from the page on that the prefix ends in.
    first = [p // P for p in before]
    wide = max(-(-n // P) - f for n, f in zip(lens, first))
    low, length = torch.tensor(before, device=DEV), s["lens"].long()
    column = (low // P)[:, None] + torch.arange(wide, device=DEV)
    pages = s["table"].long().gather(1, column.clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k, v = _rows32(s["k_cache"], s["k_scales"], pages), _rows32(s["v_cache"], s["v_scales"], pages)
    token = (low // P * P)[:, None] + torch.arange(wide * P, device=DEV)          # [B, tokens]
    last = (length - N)[:, None] + torch.arange(N, device=DEV)                    # [B, N]
    seen = (token[:, None] <= last[..., None]) & (token >= low[:, None])[:, None]
    scores = torch.matmul(rows, k.transpose(2, 3)).view(B, H, N, G, -1) * factor
    scores = torch.where(seen[:, None, :, None], scores, HIDDEN).view(B, H, N * G, -1)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    total, out = p.sum(-1, keepdim=True), torch.matmul(p, v)
    for i, n in enumerate(prefix):                                # the prefix of each group, for all of its rows
        a, b = starts[i], starts[i + 1]
        pages = s["prefix_table"][i, :-(-n // P)].long()
        k = _rows32(s["k_cache"], s["k_scales"], pages)[:, :n]
        v = _rows32(s["v_cache"], s["v_scales"], pages)[:, :n]
        x = rows[a:b].transpose(0, 1).reshape(H, -1, D)           # [H, requests · N · G, D]
        scores = torch.matmul(x, k.transpose(1, 2)) * factor
        pm = scores.amax(-1, keepdim=True)
        w = torch.exp(scores - pm)
        shape = (H, b - a, N * G, -1)
        pm, pl, po = (y.view(shape).transpose(0, 1) for y in (pm, w.sum(-1, keepdim=True), torch.matmul(w, v)))
        top = torch.maximum(pm, m[a:b])
        fp, fo = torch.exp(pm - top), torch.exp(m[a:b] - top)
        total[a:b] = total[a:b] * fo + pl * fp
        out[a:b] = out[a:b] * fo + po * fp
    out = (out / total).view(B, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(T, Hq, D)
    s["out"].copy_(out)
    return s["out"]


# ---------------------------------------------------------------- values in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "fork": _exact_fork, "release": _exact_release, "compact": _exact_compact,
            "shared": _exact_shared}[case["kind"]](s)


def _exact_norm(s):
    """Rows over their lengths in 64 bits, turned as complex numbers."""
    axes = _axes(s["sections"], s["cycled"])
    F = len(axes)
    at = torch.stack([s["positions"][a] for a in axes], 1).long()
    column = torch.arange(F, device=DEV)[None, :]
    turn = torch.complex(s["cos"].double()[at, column], s["sin"].double()[at, column])[:, None, :]
    one = slice(0, 2 * F, 2) if s["paired"] else slice(0, F)
    two = slice(1, 2 * F, 2) if s["paired"] else slice(F, 2 * F)

    def row(x, weight):
        x = x.double()
        x = x / (x.pow(2).mean(-1, keepdim=True) + s["eps"]).sqrt() * (weight.double() + (1 if s["offset"] else 0))
        z = torch.complex(x[..., one].contiguous(), x[..., two].contiguous()) * turn
        x[..., one], x[..., two] = z.real, z.imag
        return x

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    P = k_cache.shape[1]
    kept = torch.nonzero(s["slots"] >= 0).flatten()
    slot = s["slots"][kept]
    k_cache[slot // P, slot % P] = row(s["k"], s["k_weight"])[kept]
    v_cache[slot // P, slot % P] = s["v"].double()[kept]
    return {"q": row(s["q"], s["q_weight"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_caches(s, moves):
    """Page by page."""
    for source, to, n in moves:
        s["k_cache"][to, :n], s["v_cache"][to, :n] = s["k_cache"][source, :n], s["v_cache"][source, :n]
        if s["k_scales"] is not None:
            s["k_scales"][to, :, :n], s["v_scales"][to, :, :n] = s["k_scales"][source, :, :n], s["v_scales"][source, :, :n]
    return {n: x.double() if x.is_floating_point() else x for n, x in _caches_of(s).items()}


def _numbers(s, *names):
    return (s[n].cpu().numpy().astype(np.int64) for n in names)


def _exact_fork(s):
    """Request by request, as a server's host code would do it."""
    P = s["page"]
    lens, source, keep, table, holders, ring = _numbers(s, "lens", "source", "keep", "table", "holders", "ring")
    head, tail = s["range"].tolist()
    free = tail - head
    asked = used = 0
    after, old, copies, moves = lens.copy(), table.copy(), np.zeros((3, len(lens)), np.int64), []
    copies[:2] = -1
    for b, (p, n) in enumerate(zip(source.tolist(), keep.tolist())):
        if p < 0 or lens[b] != 0 or n > lens[p]:
            continue
        full, rest = divmod(n, P)
        if rest:
            asked += 1
            if asked > free:
                continue
            used = asked
            page = int(ring[(head + asked - 1) % len(ring)])
            table[b, full] = page
            holders[page] += 1
            copies[:, b] = old[p, full], page, rest
            moves.append((int(old[p, full]), page, rest))
        for i in range(full):
            table[b, i] = old[p, i]
            holders[old[p, i]] += 1
        after[b] = n
    return {"lens": after, "table": table, "holders": holders, "copies": copies, "range": np.array([head + used, tail]),
            **_exact_caches(s, moves)}


def _exact_release(s):
    """Request by request; counts go down at the end, in the same order."""
    P = s["page"]
    lens, target, table, ring, holders = _numbers(s, "lens", "target", "table", "ring", "holders")
    head, tail = s["range"].tolist()
    R, width, asked, used = len(ring), table.shape[1] * P, 0, 0
    starts, slots, positions, after = [0], [], [], []
    before, old, count = ring.copy(), table.copy(), holders.copy()
    for b, (n, m) in enumerate(zip(lens.tolist(), target.tolist())):
        have, want = math.ceil(n / P), math.ceil(m / P)
        ok = m <= width and not (m > n and n % P and holders[old[b, have - 1]] > 1)
        if ok and want > have:
            asked += want - have
            ok = asked <= tail - head
            if ok:
                used = asked
                for i in range(want - have):
                    table[b, have + i] = before[(head + asked - (want - have) + i) % R]
                    count[table[b, have + i]] = 1
        at = np.arange(n, max(n, m))
        starts.append(starts[-1] + len(at))
        positions.append(at)
        slots.append(table[b, at // P] * P + at % P if ok else np.full(len(at), -1))
        after.append(m if ok else n)
    given = tail
    for b, (n, m) in enumerate(zip(lens.tolist(), target.tolist())):
        for i in range(math.ceil(m / P), math.ceil(n / P)):
            page = old[b, i]
            count[page] -= 1
            if count[page] == 0:
                ring[given % R] = page
                given += 1
    return {"table": table, "ring": ring, "holders": count, "range": np.array([head + used, given]),
            "lens": np.array(after), "starts": np.array(starts), "slots": np.concatenate(slots),
            "positions": np.concatenate(positions)}


def _exact_compact(s):
    P = s["page"]
    lens, table, holders = _numbers(s, "lens", "table", "holders")
    head, pages = s["range"][0].item(), len(holders)
    used = [p for p in range(pages) if holders[p] > 0]
    holes = [p for p in range(len(used)) if holders[p] == 0]
    to = {p: p for p in used}
    copies = np.zeros((3, pages // 2), np.int64)
    copies[:2] = -1
    for i, p in enumerate(p for p in used if p >= len(used)):
        to[p] = holes[i]
        copies[:, i] = p, holes[i], P
    after = np.zeros(pages, np.int64)
    for p in used:
        after[to[p]] = holders[p]
    for b, n in enumerate(lens.tolist()):
        for i in range(math.ceil(n / P)):
            table[b, i] = to[int(table[b, i])]
    ring = np.full(pages, -1, np.int64)
    for p in range(len(used), pages):
        ring[(head + p - len(used)) % pages] = p
    moves = [tuple(int(x) for x in c) for c in copies.T if c[0] >= 0]
    return {"table": table, "holders": after, "ring": ring, "range": np.array([head, head + pages - len(used)]),
            "copies": copies, **_exact_caches(s, moves)}


def _exact_shared(s):
    """Request by request and head by head, over the prefix's and the request's own tokens in one row."""
    starts, prefix, before, lens = s["host"]
    N, (T, Hq, D) = s["fresh"], s["q"].shape
    P, H = s["k_cache"].shape[1], s["k_cache"].shape[2]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)

    def tokens(name, pages, low, high):                           # [H, tokens, D]
        x = s[name + "_cache"][pages].double()
        if s[name + "_scales"] is not None:
            x = x * s[name + "_scales"][pages].double().transpose(1, 2)[..., None]
        return x.flatten(0, 1)[low:high].transpose(0, 1)

    group = {b: g for g in range(len(prefix)) for b in range(starts[g], starts[g + 1])}
    held = {}
    for b, n in enumerate(lens):
        low = before[b]
        g = group.get(b)
        if g is not None and g not in held:
            pages = s["prefix_table"][g, :-(-low // P)].long()
            held = {g: [tokens(x, pages, 0, low) for x in ("k", "v")]}
        pages = s["table"][b, low // P:-(-n // P)].long()
        k, v = (tokens(x, pages, low % P, n - low // P * P) for x in ("k", "v"))
        if g is not None:
            k, v = torch.cat([held[g][0], k], 1), torch.cat([held[g][1], v], 1)
        x = s["q"][b * N:(b + 1) * N].double().view(N, H, G, D)
        logits = torch.einsum("nhgd,htd->hgnt", x, k) / D ** 0.5
        hidden = torch.arange(n, device=DEV)[None, :] > torch.arange(n - N, n, device=DEV)[:, None]
        weights = torch.softmax(logits.masked_fill(hidden, HIDDEN), -1)
        out[b * N:(b + 1) * N] = torch.einsum("hgnt,htd->nhgd", weights, v).reshape(N, Hq, D)
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    kind = case["kind"]
    if kind == "norm":
        T, Hq, H, D = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        axes = len(case["sections"].split(","))
        # every row read and written, the tokens' rows of the two tables, slots and positions.
        return {"bytes": T * (4 * (Hq + 2 * H) * D + 4 * case["rotary"] + 8 + 4 * axes),
                "flops": T * (Hq + H) * (3 * D + 3 * case["rotary"])}
    P = case["page"]
    if kind == "fork":
        kept, B = _kept(case), case["parents"] * (1 + case["samples"])
        row = 2 * case["kv_heads"] * (2 * case["dim"] if case["bits"] == 16 else case["dim"] + 2)
        # lengths, sources, tokens kept; new lengths and copies; shared pages: id read and written, count up; rows copied.
        return {"bytes": 28 * B + sum(16 * (n // P) + 2 * (n % P) * row for n in kept), "flops": B}
    if kind == "release":
        _, lens, kept, target = _release_lengths(case)
        grown = sum(max(0, m - n) for n, m in zip(lens, target))
        moved = sum(abs(-(-m // P) - -(-n // P)) for n, m in zip(lens, target))
        # lengths, targets, new lengths and starts; slots and positions; each page's id and count read and written.
        return {"bytes": 16 * len(lens) + 12 * grown + 16 * moved, "flops": 2 * grown + 8 * len(lens)}
    if kind == "compact":
        mine = _compact_lengths(case)
        live, pages = sum(mine), case["pages"]
        row = 2 * case["kv_heads"] * (2 * case["dim"] if case["bits"] == 16 else case["dim"] + 2)
        # counts and ring; table entries; of pages that lie anyhow, a share of (1 − fill) of those in use moves.
        moves = live * (pages - live) // pages
        return {"bytes": 12 * pages + 8 * live + 2 * moves * P * row, "flops": pages}
    prefix, group, own_lens = _shared_lengths(case)
    N, Hq, H, D = case["fresh"], case["q_heads"], case["kv_heads"], case["dim"]
    tokens = sum(prefix) + sum(own_lens)
    pairs = sum(N * (prefix[g] if g >= 0 else 0) + sum(max(0, n - N) + j + 1 for j in range(N))
                for g, n in zip(group, own_lens))
    row = 2 * D if case["bits"] == 16 else D + 2
    return {"bytes": 2 * tokens * H * row + 4 * len(group) * N * Hq * D + 4 * tokens // P, "flops": 4 * pairs * Hq * D}
