"""Plain numpy restatement of the operators on shared pages of the key-value cache, request by request and in 64 bits.

bf16 tensors come in as float64 arrays of their values; nothing here uses the library.
"""
from __future__ import annotations

import numpy as np

from oracle import kv_oracle as KO


def pages_held(lens, target, table, ring, free, page_size, T, holders):
    """One call of w4_kv_pages with holders.  Returns a dict of the outputs; table, ring and holders are copies."""
    lens, target = [int(x) for x in lens], [int(x) for x in target]
    R, width = len(ring), table.shape[1]
    # A request that may not go on in its last page is one whose target does not fit.
    asked = list(target)
    for b, (n, m) in enumerate(zip(lens, target)):
        if 0 <= n <= width * page_size and m > n and n % page_size:
            page = int(table[b, n // page_size])
            if 0 <= page < R and holders[page] > 1:
                asked[b] = None
    got = _pages(lens, target, asked, table, ring, free, page_size, T)
    after, out, back = holders.copy(), ring.copy(), 0
    for b, (n, m) in enumerate(zip(lens, target)):
        if n < 0 or m < 0 or n > width * page_size:
            continue
        for i in range(-(-m // page_size), -(-n // page_size)):
            page = int(table[b, i])
            if not 0 <= page < R or after[page] <= 0:
                continue
            after[page] -= 1
            if after[page] == 0:
                out[(int(free[1]) + back) % R] = page
                back += 1
    for b, (n, m) in enumerate(zip(lens, got["new_lens"])):
        for i in range(-(-n // page_size), -(-int(m) // page_size)):
            after[got["table"][b, i]] = 1
    got.update(ring=out, holders=after, free_range=np.array([got["free_range"][0], int(free[1]) + back]))
    return got


def _pages(lens, target, asked, table, ring, free, page_size, T):
    """KO.pages without the ring's side, where a request with asked[b] None takes no pages and is not granted."""
    width, R = table.shape[1], len(ring)
    head, tail = int(free[0]), int(free[1])
    out, slots, positions = table.copy(), np.full(T, -1, np.int64), np.zeros(T, np.int32)
    starts, new_lens, row, needs, used = [], [], 0, 0, 0
    for b, (n, m) in enumerate(zip(lens, target)):
        starts.append(row)
        if n < 0 or m < 0 or n > width * page_size:
            new_lens.append(n)
            continue
        have, want = -(-n // page_size), -(-m // page_size)
        ok = m <= width * page_size and asked[b] is not None
        if ok and want > have:
            needs += want - have
        if m > n and row + m - n > T:
            ok = False
        if ok and want > have:
            ok = needs <= tail - head
        if ok and want > have:
            used = needs
            for i in range(have, want):
                out[b, i] = ring[(head + needs - (want - i)) % R]
        for p in range(n, m):
            if row < T:
                positions[row] = p
                page = int(out[b, p // page_size]) if ok else -1
                if 0 <= page < R:
                    slots[row] = page * page_size + p % page_size
            row += 1
        new_lens.append(m if ok else n)
    starts.append(row)
    return {"new_lens": np.array(new_lens, np.int32), "starts": np.array(starts, np.int32), "slots": slots,
            "positions": positions, "free_range": np.array([head + used, tail]), "table": out}


def fork(lens, source, keep, table, holders, ring, free, page_size):
    """One call of w4_kv_fork; table and holders are copies."""
    lens, source, keep = ([int(x) for x in v] for v in (lens, source, keep))
    B, (R, width) = len(lens), (len(ring), table.shape[1])
    out, held, old = table.copy(), holders.copy(), table.copy()
    head, tail = int(free[0]), int(free[1])
    copies = np.zeros((3, B), np.int32)
    copies[:2] = -1
    new_lens, asked, used = list(lens), 0, 0
    for b in range(B):
        p, n = source[b], keep[b]
        if p == -1 or not 0 <= p < B or lens[b] != 0 or n < 0 or n > min(lens[p], width * page_size):
            continue
        full, rest = divmod(n, page_size)
        if rest:
            asked += 1
            if asked > min(tail - head, R):
                continue
            used = asked
            page = int(ring[(head + asked - 1) % R])
            out[b, full] = page
            if 0 <= page < R:
                held[page] = 1
                if 0 <= old[p, full] < R:
                    copies[:, b] = old[p, full], page, rest
        for i in range(full):
            out[b, i] = old[p, i]
            if 0 <= old[p, i] < R:
                held[old[p, i]] += 1
        new_lens[b] = n
    return {"new_lens": np.array(new_lens, np.int32), "table": out, "holders": held, "copies": copies,
            "free_range": np.array([head + used, tail])}


def compact(lens, table, holders, free, page_size):
    """One call of w4_kv_compact."""
    pages, width, head = len(holders), table.shape[1], int(free[0])
    live = [p for p in range(pages) if holders[p] > 0]
    U = len(live)
    movers, holes = [p for p in live if p >= U], [p for p in range(U) if holders[p] <= 0]
    to = {p: p for p in live}
    to.update(zip(movers, holes))
    copies = np.zeros((3, pages // 2), np.int32)
    copies[:2] = -1
    for i, (p, h) in enumerate(zip(movers, holes)):
        copies[:, i] = p, h, page_size
    held = np.zeros(pages, np.int32)
    for p in live:
        held[to[p]] = holders[p]
    out = table.copy()
    for b, n in enumerate(int(x) for x in lens):
        if 0 <= n <= width * page_size:
            for i in range(-(-n // page_size)):
                out[b, i] = to.get(int(table[b, i]), int(table[b, i]))
    ring = np.full(pages, -1, np.int32)
    for p in range(U, pages):
        ring[(head + p - U) % pages] = p
    return {"table": out, "holders": held, "ring": ring, "free_range": np.array([head, head + pages - U]), "copies": copies}


def copy(x, copies):
    """Pages x [pages, page_size, ...] with the copies done."""
    y = x.copy()
    for source, to, n in copies.T:
        if source >= 0:
            y[to, :n] = x[source, :n]
    return y


def norm(x, weight, eps, unit_offset):
    """x [T, heads, dim] over its rows' root mean squares, times the weights."""
    with np.errstate(all="ignore"):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (weight + (1.0 if unit_offset else 0.0))


def turned_size(y, positions, cos, sin, sections, cycled=False, paired=False):
    """The sums of absolute values whose differences and sums the turn of y gives."""
    args = (np.abs(y), positions, np.abs(cos), np.abs(sin), sections, cycled, paired)
    return np.maximum(KO.rotate(*args), KO.rotate(*args[:3], -np.abs(sin), *args[4:]))


def norm_bound(turned, size):
    """Largest |error| of values that are normalised and turned in fp32 and rounded once to bf16.

    u = 2⁻²⁴.  A sum of at most 256 squares: eight products in a row and five additions, 13·u, half of it in the root;
    the reciprocal root 2·u, mean and eps 3·u, the two products and the weight 3·u: less than 16·u of a normalised
    value.  A turned one is a sum of two products of such values, `size` with all signs alike: 19·u of that.  The result's
    rounding is 2⁻⁸ of it (2⁻¹³⁴ where it is subnormal).
    """
    return 2.0 ** -8 * np.abs(turned) + 2.0 ** -24 * 20 * size + 2.0 ** -133


def token_rows(table, lens, page_size, prefix_of=None, prefix_table=None):
    """Token numbers (page · page_size + place) of every request, int [B, longest], −1 behind its last.  prefix_of[b]:
    (group, tokens) of the prefix that request b reads from prefix_table, or None."""
    longest = max((int(n) for n in lens), default=0)
    out = np.full((len(lens), max(longest, 1)), -1, np.int64)
    for b, n in enumerate(int(x) for x in lens):
        p = np.arange(n)
        page = table[b, p // page_size].astype(np.int64) if n else np.zeros(0, np.int64)
        if prefix_of is not None and prefix_of[b] is not None:
            g, m = prefix_of[b]
            page[:m] = prefix_table[g, p[:m] // page_size]
        out[b, :n] = page * page_size + p % page_size
    return out
