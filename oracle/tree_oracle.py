"""Statements of the page plan, of trees' ancestors and of candidates from logits (numpy, CPU).

Shares no code with the GPU path. Whole numbers are exact; the adjusted logits are defined with each step rounded to fp32, so
numpy's fp32 arithmetic states them to the last bit.
"""
from __future__ import annotations

import numpy as np


def plan(ctx, change, table, queue, state, page, num_pages, rows=None, place=None):
    """One sequence after the other. Returns dict(ctx, state, offsets, slots, positions, table, queue, bad): bad holds the
    kinds of what a call records (-1: lengths, state or ring, -6: pages)."""
    table, queue, out = table.copy(), list(queue), list(ctx)
    B, width = table.shape
    Q = len(queue)
    head, count = state
    ok_state = 0 <= head < Q and 0 <= count <= Q
    bad = set() if ok_state else {-1}
    shape = (rows,) if place is None else place.shape
    slots, positions = np.full(shape, -1, np.int64), np.full(shape, -1, np.int32)
    offsets = [0]
    asked = returned = filled = 0
    rows_full = False
    taken, back = 0, []
    for b in range(B):
        offsets.append(offsets[-1])
        L, end = int(ctx[b]), int(ctx[b]) + int(change[b])
        if not (ok_state and 0 <= L <= width * page and 0 <= end <= width * page):
            bad.add(-1)
            continue
        have, want = -(-L // page), -(-end // page)
        if want > have:
            asked += want - have
            if asked > count:
                continue
        if want < have:
            returned += have - want
            if returned > Q - count:
                bad.add(-1)
                continue
        gain = max(0, end - L)
        if place is None and gain:
            filled += gain
            rows_full = rows_full or filled > rows
            if rows_full:
                continue
        for i in range(have, want):
            table[b, i] = queue[(head + taken) % Q]
            taken += 1
            if not 0 <= table[b, i] < num_pages:
                bad.add(-6)
        for i in range(want, have):
            back.append(int(table[b, i]))
            if not 0 <= table[b, i] < num_pages:
                bad.add(-6)
        out[b] = end
        offsets[-1] += gain
        for r in range(shape[-1]) if place is not None else range(gain):
            j = int(place[b, r]) if place is not None else r
            if not 0 <= j < gain:
                continue
            at = (b, r) if place is not None else offsets[-2] + r
            p = int(table[b, (L + j) // page])
            positions[at] = L + j
            if 0 <= p < num_pages:
                slots[at] = p * page + (L + j) % page
            else:
                bad.add(-6)
    for i, p in enumerate(back):
        queue[(head + count + i) % Q] = p
    new_state = ((head + taken) % Q, count - taken + len(back)) if ok_state else (head, count)
    return dict(ctx=np.array(out), state=np.array(new_state), offsets=np.array(offsets), slots=slots, positions=positions,
                table=table, queue=np.array(queue), bad=bad)


def lines(parents):
    """Each row's rows from its root down to itself; empty for a row that is not there."""
    got = []
    for t, p in enumerate(parents):
        if p >= t or p < -1 or (p >= 0 and not got[p]):
            got.append([])
        else:
            got.append((got[p] if p >= 0 else []) + [t])
    return got


def tree_seen(parents, L, window=0):
    """[G, L + G] which keys each row of a tree over L cached tokens sees."""
    G = len(parents)
    see = np.zeros((G, L + G), bool)
    for t, line in enumerate(lines(parents)):
        if line:
            pos = L + len(line) - 1
            see[t, max(0, pos - window + 1) if window else 0:L] = True
            for d, j in enumerate(line):
                see[t, L + j] = not window or len(line) - 1 - d < window
    return see


def adjust(x, counts, in_prompt, rep=1.0, freq=0.0, pres=0.0, bias=None, allowed=None):
    """One row of logits (fp32 values) as fp32: counts and in_prompt [V], bias dict, allowed [V] or None."""
    f = np.float32
    rep, freq, pres = f(rep), f(freq), f(pres)
    y = x.astype(f).copy()
    hit = in_prompt | (counts > 0)
    with np.errstate(all="ignore"):
        y[hit] = np.where(y[hit] > 0, y[hit] / rep, y[hit] * rep)
        some = counts > 0
        y[some] = y[some] - (freq * counts[some].astype(f) + pres)
        for v, w in (bias or {}).items():
            y[v] = y[v] + f(w)
    if allowed is not None:
        y[~allowed] = -np.inf
    return y


def best(y, K):
    """The K best places of y: by value, NaN first, the lower place among equals."""
    rank = np.where(np.isnan(y), np.inf, y.astype(np.float64))
    order = sorted(range(len(y)), key=lambda v: (not np.isnan(y[v]), -rank[v], v)) if len(y) < 4000 else \
        np.lexsort((np.arange(len(y)), -rank, ~np.isnan(y)))
    return np.asarray(order[:K], dtype=int)
