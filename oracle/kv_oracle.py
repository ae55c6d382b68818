"""Plain numpy restatement of the paged key-value cache's operators, in 64 bits.

bf16 tensors come in as float64 arrays of their values; nothing here uses the
library.  The cache comes as keys and values [pages, page_size, heads, dim]
(already multiplied by the scales for the 8-bit format).
"""
from __future__ import annotations

import numpy as np


def pages(lens, target, table, ring, free, page_size, T):
    """One call of w4_kv_pages, request by request.  Returns a dict of the
    outputs; table and ring are copies."""
    lens, target = [int(x) for x in lens], [int(x) for x in target]
    table, ring, taken_from = table.copy(), ring.copy(), ring.copy()
    R, width = len(ring), table.shape[1]
    head, tail = int(free[0]), int(free[1])
    asked = used = back = row = 0
    starts, new_lens = [], []
    slots, positions = np.full(T, -1, np.int64), np.zeros(T, np.int32)
    for b, (n, m) in enumerate(zip(lens, target)):
        starts.append(row)
        if n < 0 or m < 0 or n > width * page_size:
            new_lens.append(n)
            continue
        have, want = -(-n // page_size), -(-m // page_size)
        ok = m <= width * page_size
        if ok and want > have:
            asked += want - have
        if m > n and row + m - n > T:
            ok = False
        if ok and want > have:
            ok = asked <= tail - head
        if ok and want > have:
            used = asked
            for i in range(have, want):
                table[b, i] = taken_from[(head + asked - (want - i)) % R]
        for i in range(want, have):
            ring[(tail + back) % R] = table[b, i]
            back += 1
        for p in range(n, m):
            if row < T:
                positions[row] = p
                page = int(table[b, p // page_size]) if ok else -1
                if 0 <= page < R:
                    slots[row] = page * page_size + p % page_size
            row += 1
        new_lens.append(m if ok else n)
    starts.append(row)
    return {"new_lens": np.array(new_lens, np.int32), "starts": np.array(starts, np.int32), "slots": slots,
            "positions": positions, "free_range": np.array([head + used, tail + back]), "table": table, "ring": ring}


def axis_of(sections, cycled):
    """Axis of each frequency."""
    if not cycled:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out, a = list(sections), [], 0
    while any(left):
        if left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % len(left)
    return out


def rotate(x, positions, cos, sin, sections, cycled=False, paired=False):
    """x [T, heads, dim], positions [axes, T], cos and sin [rows, F]."""
    y = np.array(x, np.float64)
    F = cos.shape[1]
    for i, a in enumerate(axis_of(sections, cycled)):
        c, s = (np.float64(t[positions[a], i])[:, None] for t in (cos, sin))
        j, k = (2 * i, 2 * i + 1) if paired else (i, i + F)
        y[..., j] = x[..., j] * c - x[..., k] * s
        y[..., k] = x[..., k] * c + x[..., j] * s
    return y


def rtn8(rows):
    """(codes int8, scale bits as float64) of rows [..., dim] of bf16 values:
    d = bf16(fp32(max|x| / 127)), c = clamp(rint(fp32(x / d)), −128, 127)."""
    rows = rows.astype(np.float32)
    most = np.abs(rows).max(-1)
    with np.errstate(all="ignore"):
        d = bf16(most / np.float32(127)).astype(np.float32)
        c = np.clip(np.rint(rows / d[..., None]), -128, 127)
    c = np.where(d[..., None] > 0, c, 0)
    bad = ~np.isfinite(rows).all(-1)
    return np.where(bad[..., None], 0, c).astype(np.int8), np.where(bad, np.nan, d).astype(np.float64)


def bf16(x):
    """fp32 values rounded to bf16 (round half to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    u = u + 0x7FFF + ((u >> 16) & 1)
    return (u & np.uint32(0xFFFF0000)).view(np.float32)


def attention(q, k, v, table, lens, starts, scale, window=0):
    """(out, spread, scores) for queries q [T, heads, dim]: spread = Σ p|v| of
    each output, scores = the largest Σ_i |scale · q_i k_i| of each row."""
    T, Hq, D = q.shape
    P, H = k.shape[1], k.shape[2]
    G = Hq // H
    out, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    largest = np.zeros((T, Hq, 1))
    for b, L in enumerate(lens):
        n = int(starts[b + 1] - starts[b])
        used = table[b, :-(-int(L) // P)]
        kb, vb = k[used].reshape(-1, H, D), v[used].reshape(-1, H, D)
        for j in range(n):
            p = int(L) - n + j
            if p < 0:
                continue
            low = max(0, p - window + 1) if window else 0
            for h in range(H):
                row = (starts[b] + j, slice(h * G, (h + 1) * G))
                x, kk, vv = q[row], kb[low:p + 1, h], vb[low:p + 1, h]
                s = scale * (x @ kk.T)
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                out[row], spread[row] = w @ vv, w @ np.abs(vv)
                largest[row] = abs(scale) * (np.abs(x) @ np.abs(kk).T).max(-1, keepdims=True)
    return out, spread, largest


def attention_bound(out, spread, largest, dim, longest, format=16):
    """Largest |error| a correct fp32 attention with a bf16 result may have.

    u = 2⁻²⁴.  A score's fp32 dot product errs by at most (dim + 2)·u·Σ|q_i k_i|,
    which moves its weight by that much relative, in numerator and denominator:
    twice.  Sums over at most `longest` tokens err by longest·u·Σ p|v|.  The
    exponential and the weights as two bf16 (16 bits) err by less than 2⁻¹⁵; in
    format 8 the weights are fp16, 2⁻¹¹.  The result's rounding: 2⁻⁹, and one
    more for a rounding of the 64-bit value the other way.
    """
    u = 2.0 ** -24
    return 2.0 ** -8 * np.abs(out) + (2 * (dim + 2) * u * largest + longest * u + (2.0 ** -15 if format == 16 else 2.0 ** -11)) * spread


def attention8_floor(q, k, codes, d, table, lens, starts, scale, window=0):
    """What format 8's weights may add to attention_bound, for codes [pages, page_size, heads, dim] and value scales d
    [pages, page_size, heads].

    A token's weight times its value scale is one fp16 number in units of (at least 2⁻⁷ of) the largest such product M
    that its row has met: 11 bits down to 2⁻¹⁴ of the unit, and an error of at most 2⁻²⁵ of it below, 2⁻³² of M.  Each
    token's codes take that much: 2⁻³² · M · Σ|c|.
    """
    T, Hq, D = q.shape
    P, H = k.shape[1], k.shape[2]
    G = Hq // H
    out = np.zeros((T, Hq, D))
    for b, L in enumerate(lens):
        n = int(starts[b + 1] - starts[b])
        used = table[b, :-(-int(L) // P)]
        kb, db, cb = k[used].reshape(-1, H, D), d[used].reshape(-1, H), np.abs(codes[used]).reshape(-1, H, D)
        for j in range(n):
            p = int(L) - n + j
            if p < 0:
                continue
            low = max(0, p - window + 1) if window else 0
            for h in range(H):
                row = (starts[b] + j, slice(h * G, (h + 1) * G))
                s = scale * (q[row] @ kb[low:p + 1, h].T)
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                out[row] = 2.0 ** -32 * (w * db[low:p + 1, h]).max(-1, keepdims=True) * cb[low:p + 1, h].sum(0)
    return out
