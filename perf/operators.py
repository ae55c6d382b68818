"""The paged key-value cache's operators: cases to measure, their plain forms and their 64-bit values.

Three operators, which a decode or a speculative-verify step of an attention layer runs between the
4-bit projections:

* ``pages``: block tables and slot maps built on the GPU from request lengths.  Every request goes from
  its present length to a target; the pages it needs come from a ring of free pages, the pages it no
  longer needs go back to it, and every new token gets its slot in the cache and its position.
* ``append``: rotary positions with several axes (time, height, width) applied to the queries and keys of
  new tokens, the keys and values written to the cache at the tokens' slots.
* ``attention``: attention of the newest tokens of each request (one, or the rows of a verify pass) over
  its pages of the cache, split over the cache's length and joined.

Head layouts are those of the three layer classes the repository's workloads have: 16 query and 4
key-value heads of 256 (2560-wide model, 4096-wide projections), 40 and 8 of 128 (the 7168×5120 fused
projection), 64 and 8 of 128 (the 10240×8192 one); verify passes have 5, 7 or 13 rows, and 16 requests
of 13 rows are the 208 rows of the benchmark's largest case.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
MASKED = float("-inf")


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of a small batch: every request grows by one token, few of them need a page.
        {"name": "pages-step-64", "kind": "pages", "requests": 64, "page": 16, "shortest": 1, "longest": 8192,
         "mode": "step", "mix": 11},
        # A full server between verify passes: requests that drop rejected drafts, finish, start or grow,
        # with a pool that runs out before the last of them.
        {"name": "pages-mixed-1000", "kind": "pages", "requests": 1000, "page": 16, "shortest": 1, "longest": 4097,
         "mode": "mixed", "mix": 12},
        # Prompts of a batch entering the cache at once.
        {"name": "pages-prompts-37", "kind": "pages", "requests": 37, "page": 64, "shortest": 100, "longest": 32768,
         "mode": "prompts", "mix": 13},
        # One decode token of the smallest layer: latency.  A quarter of the head rotates, axes interleaved.
        {"name": "append-decode-1", "kind": "append", "tokens": 1, "q_heads": 16, "kv_heads": 4, "dim": 256,
         "rotary": 64, "sections": "11,11,10", "cycled": True, "paired": False, "page": 16, "order": "token"},
        # The 208 rows of 16 verify passes.
        {"name": "append-verify-208", "kind": "append", "tokens": 208, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "rotary": 128, "sections": "16,24,24", "cycled": False, "paired": False, "page": 32, "order": "head"},
        # A prompt of text and images.
        {"name": "append-prompt-16001", "kind": "append", "tokens": 16001, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "rotary": 128, "sections": "16,24,24", "cycled": False, "paired": False, "page": 16, "order": "token"},
        # One request, short: latency.
        {"name": "attention-1-short", "kind": "attention", "requests": 1, "fresh_low": 1, "fresh_high": 1, "q_heads": 16,
         "kv_heads": 4, "dim": 256, "page": 16, "shortest": 517, "longest": 517, "window": 0, "bits": 16,
         "order": "token", "mix": 21},
        # One request with a long document: all of the GPU on one sequence.
        {"name": "attention-1-long", "kind": "attention", "requests": 1, "fresh_low": 1, "fresh_high": 1, "q_heads": 64,
         "kv_heads": 8, "dim": 128, "page": 16, "shortest": 131071, "longest": 131071, "window": 0, "bits": 16,
         "order": "token", "mix": 22},
        # A batch of decoding requests of very different lengths.
        {"name": "attention-64-ragged", "kind": "attention", "requests": 64, "fresh_low": 1, "fresh_high": 1, "q_heads": 40,
         "kv_heads": 8, "dim": 128, "page": 16, "shortest": 1, "longest": 16384, "window": 0, "bits": 16,
         "order": "token", "mix": 23},
        # The same batch over a cache in 8 bits.
        {"name": "attention-64-ragged-8bit", "kind": "attention", "requests": 64, "fresh_low": 1, "fresh_high": 1,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 16, "shortest": 1, "longest": 16384, "window": 0, "bits": 8,
         "order": "token", "mix": 23},
        # 16 verify passes of 12 drafts each: 104 query rows for each key-value head.
        {"name": "attention-16-verify-13", "kind": "attention", "requests": 16, "fresh_low": 13, "fresh_high": 13,
         "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 32, "shortest": 1024, "longest": 8192, "window": 0, "bits": 16,
         "order": "head", "mix": 24},
        # Decoding and verifying requests of a layer that sees a window of the cache only.
        {"name": "attention-96-window", "kind": "attention", "requests": 96, "fresh_low": 1, "fresh_high": 5, "q_heads": 16,
         "kv_heads": 4, "dim": 256, "page": 16, "shortest": 1, "longest": 9000, "window": 1024, "bits": 16,
         "order": "token", "mix": 25},
    ]


#: What a drawn attention case may cost: bytes and operations, and the values and scores of the plain form's padded batch.
MOST_BYTES, MOST_FLOPS = 6.4e8, 2.6e10
MOST_PADDED, MOST_SCORES = 64 * 16384 * 8 * 128, 3e8


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng):
    while True:
        kv = rng.choice([1, 2, 3, 4, 8])
        q = kv * rng.choice([1, 2, 4, 5, 7, 8])
        dim = rng.choice([64, 80, 112, 128, 128, 192, 256])
        if 3072 not in (q * dim, kv * dim, (q + kv) * dim, (q + 2 * kv) * dim):
            return q, kv, dim


def draw(rng):
    kind = rng.choice(["pages", "append", "attention", "attention"])
    if kind == "pages":
        mode = rng.choice(["step", "mixed", "prompts"])
        requests = _log_int(rng, 1, 1000 if mode != "prompts" else 37)
        return {"kind": kind, "requests": requests, "page": rng.choice([8, 16, 24, 32, 64]), "shortest": 1,
                "longest": _log_int(rng, 50, {"step": 8192, "mixed": 4097, "prompts": 32768}[mode]), "mode": mode,
                "mix": rng.randrange(1 << 30)}
    if kind == "append":
        q, kv, dim = _heads(rng)
        half = rng.choice([dim, dim, dim // 2, dim // 4]) // 16 * 8
        axes = rng.choice([1, 2, 3, 3])
        cuts = sorted(rng.sample(range(1, half), axes - 1)) if axes > 1 else []
        sections = [b - a for a, b in zip([0] + cuts, cuts + [half])]
        most = 16001 * (40 + 2 * 8) * 128 // ((q + 2 * kv) * dim)
        return {"kind": kind, "tokens": _log_int(rng, 1, min(most, 30000)), "q_heads": q, "kv_heads": kv, "dim": dim,
                "rotary": 2 * half, "sections": ",".join(map(str, sections)), "cycled": rng.random() < 0.5,
                "paired": rng.random() < 0.3, "page": rng.choice([8, 16, 24, 32, 64]),
                "order": rng.choice(["token", "head"])}
    while True:
        q, kv, dim = _heads(rng)
        requests = _log_int(rng, 1, 256)
        longest = _log_int(rng, 1, 131071)
        fresh = rng.choice([1, 1, 1, 5, 7, 13])
        padded = requests * (longest + 64)
        if padded * kv * dim > MOST_PADDED or padded * q * fresh > MOST_SCORES or 3072 in (longest, requests):
            continue
        case = {"kind": kind, "requests": requests, "fresh_low": rng.choice([1, fresh]), "fresh_high": fresh, "q_heads": q,
                "kv_heads": kv, "dim": dim, "page": rng.choice([8, 16, 24, 32, 64]),
                "shortest": min(longest, _log_int(rng, 1, max(1, longest))), "longest": longest,
                "window": rng.choice([0, 0, 0, _log_int(rng, 16, 8192)]), "bits": rng.choice([16, 16, 8]),
                "order": rng.choice(["token", "head"]), "mix": rng.randrange(1 << 30)}
        cost = work(case)
        if cost["bytes"] <= MOST_BYTES and cost["flops"] <= MOST_FLOPS:
            return case


# ---------------------------------------------------------------- lengths
def _page_lengths(case):
    """(lengths, targets, whether the pool is short): from the case alone."""
    r = random.Random(case["mix"])
    lens, target = [], []
    for _ in range(case["requests"]):
        n = _log_int(r, case["shortest"], case["longest"])
        if case["mode"] == "step":
            lens.append(n)
            target.append(n + 1)
        elif case["mode"] == "prompts":  # one in four has a part of its prompt in the cache already
            lens.append(r.randrange(n) if r.random() < 0.25 else 0)
            target.append(n)
        else:
            what = r.random()
            lens.append(0 if what < 0.05 else n)
            if what < 0.05:      # starts
                target.append(n)
            elif what < 0.10:    # finished
                target.append(0)
            elif what < 0.55:    # drops rejected drafts
                target.append(max(0, n - r.randrange(13)))
            else:                # appends a verify pass
                target.append(n + r.choice([1, 5, 7, 13]))
    return lens, target, case["mode"] == "mixed"


def _attention_lengths(case):
    """(lengths, new tokens of each request): from the case alone; a length counts its new tokens."""
    r = random.Random(case["mix"])
    fresh = [r.randint(case["fresh_low"], case["fresh_high"]) for _ in range(case["requests"])]
    return [max(n, _log_int(r, case["shortest"], case["longest"])) for n in fresh], fresh


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"pages": _prepare_pages, "append": _prepare_append, "attention": _prepare_attention}[case["kind"]](case, seed, g)


def _ints(values, dtype=torch.int32):
    return torch.tensor(np.asarray(values), dtype=dtype, device=DEV)


def _prepare_pages(case, seed, g):
    lens, target, short = _page_lengths(case)
    order = np.random.default_rng(seed).permutation(len(lens))
    lens, target = np.array(lens)[order], np.array(target)[order]
    P = case["page"]
    have, want = -(-lens // P), -(-target // P)
    need = int(np.maximum(want - have, 0).sum())
    free = need - need // 20 if short else need + 7
    width = int(max(have.max(), want.max())) + 3
    pages = int(have.sum()) + free
    rng = np.random.default_rng(seed + 1)
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    column = np.arange(width)[None, :]
    table[column < have[:, None]] = ids[free:]
    head = int(rng.integers(0, 1 << 40))
    ring = rng.integers(0, pages, pages).astype(np.int32)
    ring[(head + np.arange(free)) % pages] = ids[:free]
    return {"kind": "pages", "page": P, "tokens": int(np.maximum(target - lens, 0).sum()), "lens": _ints(lens),
            "target": _ints(target), "table": _ints(table), "ring": _ints(ring),
            "range": _ints([head, head + free], torch.int64)}


def _cache(case, pages, g):
    """Key or value pages [pages, page, heads, dim] as a view of memory in the case's order."""
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    shape = (pages, P, H, D) if case["order"] == "token" else (pages, H, P, D)
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    return x if case["order"] == "token" else x.transpose(1, 2)


def _prepare_append(case, seed, g):
    T, Hq, H, D, rot = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["rotary"]
    sections = tuple(int(s) for s in case["sections"].split(","))
    rows = 32768
    qkv = torch.empty((T, (Hq + 2 * H) * D), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    P = case["page"]
    pages = -(-T // P) + 9
    ids = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(T, device=DEV) + 3
    slots = ids[t // P] * P + t % P
    drop = torch.rand(T, generator=g, device=DEV) < 0.01
    drop[0] = False
    slots = torch.where(drop, -1, slots)
    # Spans of text, where the axes agree, and of images, where height and width run over a grid.
    start = random.Random(seed).randrange(rows - 20000) if rows > 20000 else 0
    span = t // 256
    grid = [span, span + t % 256 // 16, span + t % 16]
    image = span % 2 == 1
    positions = torch.stack([torch.where(image, grid[a], t // 2) + start for a in range(len(sections))]).to(torch.int32)
    frequency = 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / rot)
    angle = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * frequency
    return {"kind": "append", "q": qkv[:, :Hq * D].view(T, Hq, D), "k": qkv[:, Hq * D:(Hq + H) * D].view(T, H, D),
            "v": qkv[:, (Hq + H) * D:].view(T, H, D), "positions": positions, "cos": angle.cos().float(),
            "sin": angle.sin().float(), "sections": sections, "cycled": case["cycled"], "paired": case["paired"],
            "k_cache": _cache(case, pages, g), "v_cache": _cache(case, pages, g), "slots": slots,
            "q_out": torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)}


def _codes(x):
    """Codes and scales in 8 bits of the rows of x [pages, page, heads, dim]; scales [pages, heads, page]."""
    scale = (x.float().abs().amax(-1) / 127).to(torch.bfloat16)
    codes = torch.round(x.float() / scale.float()[..., None]).clamp(-128, 127).to(torch.int8)
    return codes, scale.transpose(1, 2).contiguous()


def _prepare_attention(case, seed, g):
    lens, fresh = _attention_lengths(case)
    order = np.random.default_rng(seed).permutation(len(lens))
    lens, fresh = np.array(lens)[order], np.array(fresh)[order]
    P, B = case["page"], len(lens)
    have = -(-lens // P)
    width = int(have.max()) + 2
    pages = int(have.sum()) + 5
    table = np.full((B, width), -1, dtype=np.int32)
    table[np.arange(width)[None, :] < have[:, None]] = np.random.default_rng(seed + 1).permutation(pages)[:int(have.sum())]
    starts = np.concatenate([[0], np.cumsum(fresh)])
    T = int(starts[-1])
    q = torch.empty((T, case["q_heads"], case["dim"]), dtype=torch.bfloat16, device=DEV).normal_(std=1.5, generator=g)
    k, v = _cache(case, pages, g), _cache(case, pages, g)
    state = {"kind": "attention", "q": q, "k_cache": k, "v_cache": v, "k_scales": None, "v_scales": None,
             "table": _ints(table), "lens": _ints(lens), "starts": _ints(starts), "longest": int(lens.max()),
             "fresh": int(fresh.max()), "uniform": bool((fresh == fresh[0]).all()), "window": case["window"],
             "out": torch.empty_like(q), "host": (lens.tolist(), starts.tolist())}
    if case["bits"] == 8:
        state["k_cache"], state["k_scales"] = _codes(k)
        state["v_cache"], state["v_scales"] = _codes(v)
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    kind = state["kind"]
    if own:
        return {"pages": _own_pages, "append": _own_append, "attention": _own_attention}[kind](state)
    return {"pages": _plain_pages, "append": _plain_append, "attention": _plain_attention}[kind](state)


def _own_pages(s):
    import gemm_rtn_sym_gb300 as w4

    lens, starts, slots, positions, left = w4.w4_kv_pages(s["lens"], s["target"], s["table"], s["ring"], s["range"],
                                                          s["page"], s["tokens"])
    return {"table": s["table"], "ring": s["ring"], "range": left, "lens": lens, "starts": starts, "slots": slots,
            "positions": positions}


def _own_append(s):
    import gemm_rtn_sym_gb300 as w4

    w4.w4_kv_append(s["q"], s["k"], s["v"], s["positions"], s["cos"], s["sin"], s["k_cache"], s["v_cache"], s["slots"],
                    sections=s["sections"], cycled=s["cycled"], paired=s["paired"], q_out=s["q_out"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import gemm_rtn_sym_gb300 as w4

    return w4.w4_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                             starts=None if s["uniform"] else s["starts"], k_scales=s["k_scales"],
                             v_scales=s["v_scales"], window=s["window"], out=s["out"])


def _plain_pages(s):
    P, table, ring = s["page"], s["table"], s["ring"]
    lens, target = s["lens"].long(), s["target"].long()
    B, W = table.shape
    R = ring.numel()
    head, tail = s["range"][0], s["range"][1]
    have, want = (lens + P - 1) // P, (target + P - 1) // P
    grow = (target - lens).clamp(min=0)
    fits = target <= W * P
    need = torch.where(fits, (want - have).clamp(min=0), 0)
    cum = need.cumsum(0)
    granted = fits & ((need == 0) | (cum <= tail - head))
    first = head + cum - need                                    # ring position of a request's first new page
    starts = torch.cat([torch.zeros_like(grow[:1]), grow.cumsum(0)])
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(starts[1:], t, right=True).clamp(max=B - 1)
    position = lens[b] + t - starts[b]
    index = position // P
    fresh = index - have[b]
    page = torch.where(fresh >= 0, ring[(first[b] + fresh) % R], table[b, index.clamp(max=W - 1)]).long()
    slots = torch.where(granted[b], page * P + position % P, -1)
    c = torch.arange(W, device=DEV)[None, :]
    gives = (have - want).clamp(min=0)
    given = gives.cumsum(0)
    back = (c >= want[:, None]) & (c < have[:, None])
    at = torch.where(back, (tail + given[:, None] - gives[:, None] + c - want[:, None]) % R, R)
    longer = torch.cat([ring, ring[:1]])
    longer[at.flatten()] = table.flatten()                        # the entry after the last takes what is not given back
    new = granted[:, None] & (c >= have[:, None]) & (c < want[:, None])
    table.copy_(torch.where(new, ring[(first[:, None] + c - have[:, None]) % R], table))
    ring.copy_(longer[:R])
    used = torch.where(granted & (need > 0), cum, 0).max()
    return {"table": table, "ring": ring, "range": torch.stack([head + used, tail + given[-1]]),
            "lens": torch.where(granted, target, lens).to(torch.int32), "starts": starts.to(torch.int32), "slots": slots,
            "positions": position.to(torch.int32)}


def _axes(sections, cycled):
    """The axis of each frequency: blocks one after another, or the axes in turn while they have frequencies left."""
    if not cycled:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    turns = sorted((i, a) for a, n in enumerate(sections) for i in range(n))
    return [a for _, a in turns]


def _rotate(x, cos, sin, paired):
    """x [T, heads, dim] in 32 bits, its first 2·F values rotated by cos, sin [T, F]."""
    F = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    x = x.float()
    a, b = (x[..., 0:2 * F:2], x[..., 1:2 * F:2]) if paired else (x[..., :F], x[..., F:2 * F])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if paired else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., 2 * F:]], -1)


def _plain_append(s):
    axis = torch.tensor(_axes(s["sections"], s["cycled"]), device=DEV)
    rows = s["positions"].long()[axis].t()                        # [T, F]
    cos, sin = s["cos"].gather(0, rows), s["sin"].gather(0, rows)
    q = _rotate(s["q"], cos, sin, s["paired"]).to(torch.bfloat16)
    k = _rotate(s["k"], cos, sin, s["paired"]).to(torch.bfloat16)
    stored = s["slots"] >= 0
    # A token without a slot stands for the first one that has a slot, which is then written twice alike.
    source = torch.where(stored, torch.arange(stored.numel(), device=DEV), stored.to(torch.uint8).argmax())
    slots, P = s["slots"][source], s["k_cache"].shape[1]
    s["k_cache"][slots // P, slots % P] = k[source]
    s["v_cache"][slots // P, slots % P] = s["v"][source]
    s["q_out"].copy_(q)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, scales, table):
    """The requests' rows of the cache in 32 bits: [requests, heads, tokens, dim]."""
    x = cache[table].float()                                      # [B, W, P, H, D]
    if scales is not None:
        x = x * scales[table].float().transpose(2, 3)[..., None]
    return x.flatten(1, 2).transpose(1, 2)


def _plain_attention(s):
    q, starts = s["q"], s["starts"].long()
    T, Hq, D = q.shape
    P, H = s["k_cache"].shape[1], s["k_cache"].shape[2]
    pages = -(-s["longest"] // P)
    table = s["table"][:, :pages].long().clamp(min=0)
    k = _gathered(s["k_cache"], s["k_scales"], table)
    v = _gathered(s["v_cache"], s["v_scales"], table)
    B, G, N = table.shape[0], Hq // H, s["fresh"]
    lens, fresh = s["lens"].long(), starts[1:] - starts[:-1]
    row = (starts[:-1, None] + torch.arange(N, device=DEV)).clamp(max=T - 1)   # [B, N]
    rows = q.float()[row].view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    scores = torch.matmul(rows, k.transpose(2, 3)).view(B, H, N, G, -1) * (1.0 / math.sqrt(D))
    last = (lens - fresh)[:, None] + torch.arange(N, device=DEV)              # the position of each new token
    token = torch.arange(pages * P, device=DEV)
    seen = token <= last[..., None]
    if s["window"]:
        seen &= token > last[..., None] - s["window"]
    scores = torch.where(seen[:, None, :, None, :], scores, MASKED)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    out = torch.matmul((p / p.sum(-1, keepdim=True)).view(B, H, N * G, -1), v)
    out = out.view(B, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(starts[1:], t, right=True)
    s["out"].copy_(out[b, t - starts[b]])
    return s["out"]


# ---------------------------------------------------------------- values in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "append": _exact_append, "attention": _exact_attention}[case["kind"]](s)


def _exact_pages(s):
    """Request by request, as a server's host code would do it."""
    P = s["page"]
    lens, target, table, ring = (s[n].cpu().numpy().astype(np.int64) for n in ("lens", "target", "table", "ring"))
    head, tail = s["range"].tolist()
    R, width, asked, given = len(ring), table.shape[1] * P, 0, tail
    used, starts, slots, positions, after = 0, [0], [], [], []
    before, old = ring.copy(), table.copy()
    for b, (n, m) in enumerate(zip(lens.tolist(), target.tolist())):
        have, want = math.ceil(n / P), math.ceil(m / P)
        ok = m <= width
        if ok and want > have:
            asked += want - have
            ok = asked <= tail - head
            if ok:
                used = asked
                for i in range(want - have):
                    table[b, have + i] = before[(head + asked - (want - have) + i) % R]
        for i in range(want, have):
            ring[given % R] = old[b, i]
            given += 1
        at = np.arange(n, max(n, m))
        starts.append(starts[-1] + len(at))
        positions.append(at)
        slots.append(table[b, at // P] * P + at % P if ok else np.full(len(at), -1))
        after.append(m if ok else n)
    return {"table": table, "ring": ring, "range": np.array([head + used, given]), "lens": np.array(after),
            "starts": np.array(starts), "slots": np.concatenate(slots), "positions": np.concatenate(positions)}


def _exact_append(s):
    """The rotation as a product of complex numbers in 64 bits."""
    axes = _axes(s["sections"], s["cycled"])
    F = len(axes)
    at = torch.stack([s["positions"][a] for a in axes], 1).long()
    column = torch.arange(F, device=DEV)[None, :]
    turn = torch.complex(s["cos"].double()[at, column], s["sin"].double()[at, column])[:, None, :]
    one = slice(0, 2 * F, 2) if s["paired"] else slice(0, F)
    two = slice(1, 2 * F, 2) if s["paired"] else slice(F, 2 * F)

    def turned(x):
        x = x.double().clone()
        z = torch.complex(x[..., one], x[..., two]) * turn
        x[..., one], x[..., two] = z.real, z.imag
        return x

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    P = k_cache.shape[1]
    kept = torch.nonzero(s["slots"] >= 0).flatten()
    slot = s["slots"][kept]
    k_cache[slot // P, slot % P] = turned(s["k"])[kept]
    v_cache[slot // P, slot % P] = s["v"].double()[kept]
    return {"q": turned(s["q"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_attention(s):
    """Request by request and head by head, over the visible tokens alone, in 64 bits."""
    lens, starts = s["host"]
    T, Hq, D = s["q"].shape
    P, H = s["k_cache"].shape[1], s["k_cache"].shape[2]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        pages = s["table"][b, :-(-n // P)].long()
        fresh = starts[b + 1] - starts[b]
        low = max(0, n - fresh - s["window"] + 1) if s["window"] else 0
        query = torch.arange(n - fresh, n, device=DEV)[:, None]
        token = torch.arange(low, n, device=DEV)[None, :]
        hidden = token > query
        if s["window"]:
            hidden = hidden | (query - token >= s["window"])
        for h in range(H):
            k, v = s["k_cache"][pages, :, h].double().flatten(0, 1), s["v_cache"][pages, :, h].double().flatten(0, 1)
            if s["k_scales"] is not None:
                k = k * s["k_scales"][pages, h].double().flatten()[:, None]
                v = v * s["v_scales"][pages, h].double().flatten()[:, None]
            x = s["q"][starts[b]:starts[b + 1], h * G:(h + 1) * G].double()
            logits = torch.einsum("ngd,td->gnt", x, k[low:n]) / D ** 0.5
            weights = torch.softmax(logits.masked_fill(hidden, MASKED), -1)
            out[starts[b]:starts[b + 1], h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", weights, v[low:n])
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["kind"] == "pages":
        lens, target, _ = _page_lengths(case)
        P, B = case["page"], case["requests"]
        grown = sum(max(0, m - n) for n, m in zip(lens, target))
        moved = sum(abs(-(-m // P) - -(-n // P)) for n, m in zip(lens, target))
        # lengths, targets, new lengths and starts; a slot (8) and a position (4) for each new token, each page once
        # read from the ring or the table and once written.
        return {"bytes": 16 * B + 12 * grown + 8 * moved, "flops": 2 * grown + 8 * B}
    if case["kind"] == "append":
        T, Hq, H, D = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        axes = len(case["sections"].split(","))
        # every row read and written, the tokens' rows of the two tables, slots and positions.
        return {"bytes": T * (4 * (Hq + 2 * H) * D + 4 * case["rotary"] + 8 + 4 * axes),
                "flops": 3 * T * (Hq + H) * case["rotary"]}
    lens, fresh = _attention_lengths(case)
    rows = tokens = pairs = 0
    for n, f in zip(lens, fresh):
        rows += f
        tokens += n - (max(0, n - f - case["window"] + 1) if case["window"] else 0)
        pairs += sum(min(n - f + j + 1, case["window"] or n) for j in range(f))
    H, D = case["kv_heads"], case["dim"]
    row = 2 * D if case["bits"] == 16 else D + 2
    return {"bytes": 2 * tokens * H * row + 4 * rows * case["q_heads"] * D + 4 * tokens // case["page"],
            "flops": 4 * pairs * case["q_heads"] * D}
