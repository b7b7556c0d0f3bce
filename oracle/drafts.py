"""Drafted-token trees over a paged cache, and the reservation of its pages, on the CPU.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Draft t of a sequence of n slots, c of them drafts, sits in slot n - c + t; it
sees itself, its ancestors and the slots before the drafts, with a window the
nearest so many of them in that order.
"""
from __future__ import annotations

import numpy as np

from . import prompt


def line(parents, t: int):
    """Draft t and its ancestors, nearest first."""
    out = []
    while t >= 0:
        out.append(t)
        p = int(parents[t])
        t = p if -1 <= p < t else -1
    return out


def seen(n: int, c: int, parents, window=0):
    """[c, n] of bool: the slots that each draft sees."""
    m = np.zeros((c, n), bool)
    for t in range(c):
        slots = [n - c + a for a in line(parents, t)] + list(range(n - c - 1, -1, -1))
        m[t, slots[:window] if window else slots] = True
    return m


def attend(q, k, v, table, lengths, counts, parents, scale, window=0):
    """(out, lse, magnitudes, reaches, [seqs, drafts] of bool: there is one); pools [page, head, row, dim]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n_seqs, drafts, heads, d = q.shape
    group, page = heads // k.shape[1], k.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach, real = np.zeros(q.shape[:3]), np.zeros(q.shape[:3]), np.zeros(q.shape[:2], bool)
    for b in range(n_seqs):
        n = min(max(int(lengths[b]), 0), table.shape[1] * page)
        c = min(drafts, n) if counts is None else min(max(int(counts[b]), 0), drafts, n)
        if not c:
            continue
        real[b, :c] = True
        pages = np.array([int(table[b, j // page]) for j in range(n)])
        there = (pages >= 0) & (pages < k.shape[0])  # slots of pages outside the pool are unseen
        pages, row = np.where(there, pages, 0), np.arange(n) % page
        m = seen(n, c, parents[b], window) & there
        for h in range(heads):
            out[b, :c, h], lse[b, :c, h], mag[b, :c, h], reach[b, :c, h] = prompt.rows(
                q[b, :c, h], k[pages, h // group, row], v[pages, h // group, row], m, scale)
    return out, lse, mag, reach, real


def accept(lengths, counts, path, capacity: int):
    """([(sequence, slot from, slot to)], new lengths)."""
    moves, new = [], []
    for b, row in enumerate(path):
        n = min(max(int(lengths[b]), 0), capacity)
        c = min(len(row), n) if counts is None else min(max(int(counts[b]), 0), 64, n)
        last, kept = -1, 0
        for p in row:
            if not last < p < c:
                break
            moves.append((b, n - c + int(p), n - c + kept))
            last, kept = p, kept + 1
        new.append(n - c + kept)
    return moves, new


def reserve(table, lengths, counts, free, page: int, max_tokens: int):
    """(table, lengths, starts, [(slot, position, sequence)], stack) as lists; ``free``: the stack, its top last."""
    table, stack, per = [list(map(int, r)) for r in table], list(map(int, free)), len(table[0]) if len(table) else 0
    held = [sum(p >= 0 for p in r) for r in table]
    n = [min(max(int(x), 0), per * page) for x in lengths]
    c = [max(int(x), 0) for x in counts]
    ok = [x + y <= per * page for x, y in zip(n, c)]
    want = [-(-(x + y) // page) if o else h for x, y, o, h in zip(n, c, ok, held)]
    for b, r in enumerate(table):               # given back first
        for j in range(want[b], held[b]):
            stack.append(r[j])
            r[j] = -1
    need = [max(w - h, 0) if o else 0 for w, h, o in zip(want, held, ok)]
    asked = 0
    for b in range(len(table)):                 # in order, as long as the pages last
        asked += need[b]
        if need[b] and asked > len(stack):
            ok[b] = False
    asked = 0
    for b in range(len(table)):                 # and the packed lists
        asked += c[b] if ok[b] else 0
        if ok[b] and c[b] and asked > max_tokens:
            ok[b] = False
    starts, packed = [0], []
    for b, r in enumerate(table):
        if ok[b]:
            for j in range(held[b], want[b]):
                r[j] = stack.pop()
            packed += [(r[i // page] * page + i % page, i, b) for i in range(n[b], n[b] + c[b])]
        starts.append(len(packed))
    return table, [x + (y if o else 0) for x, y, o in zip(n, c, ok)], starts, packed, stack
