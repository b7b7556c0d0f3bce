"""Paged key-value cache operators on the CPU, in 64 bits.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A pool is an array [page, head, row, ...]; slot j of sequence b is row j %
page_size of page table[b, j // page_size].  Written one sequence and head at
a time from the operators' definitions:

  attend  x_j = scale * q . k_j over the seen slots, w = softmax(x),
          out = sum_j w_j v_j, lse = log sum_j exp x_j; nothing seen gives
          out = 0, lse = -inf, no weights
  append  row t of sequence b goes to slot n_b + t; E4M3 rows are x / scale
          with scale = max(max|x| / 448, 2^-126)
  evict   the `recent` newest slots and, of the others, the budget - recent
          of largest score (equal: the lowest slot), in slot order
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def seen_slots(n: int, window: int = 0, mask=None):
    """Slots of a sequence of n that its query sees."""
    return [j for j in range(max(0, n - window) if window else 0, n) if mask is None or mask[j]]


def attend(q, k, v, table, lengths, scale, window=0, mask=None):
    """(out, lse, weights [seq, kv_head, capacity]) and, for error bounds, the
    magnitudes sum_j w_j |v_j| (as out) and the largest scale * sum |q||k_j| (as lse)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n_seq, n_q, d = q.shape
    heads, page = k.shape[1], k.shape[2]
    group = n_q // heads
    out, mag = np.zeros((n_seq, n_q, d)), np.zeros((n_seq, n_q, d))
    lse, reach = np.full((n_seq, n_q), -math.inf), np.zeros((n_seq, n_q))
    weights = np.zeros((n_seq, heads, table.shape[1] * page))
    for b in range(n_seq):
        slots = seen_slots(int(lengths[b]), window, None if mask is None else mask[b])
        if not slots:
            continue
        at = np.array([(table[b, j // page], j % page) for j in slots])
        for i in range(n_q):
            h = i // group
            kk, vv = k[at[:, 0], h, at[:, 1]], v[at[:, 0], h, at[:, 1]]
            x = scale * (kk @ q[b, i])
            top = x.max()
            e = np.exp(x - top)
            w = e / e.sum()
            out[b, i] = w @ vv
            mag[b, i] = w @ np.abs(vv)
            lse[b, i] = top + math.log(e.sum())
            reach[b, i] = abs(scale) * (np.abs(kk) @ np.abs(q[b, i])).max()
            weights[b, h, slots] += w
    return out, lse, weights, mag, reach


def e4m3_round(x: float) -> float:
    """The nearest E4M3 value (ties to the even code), saturating at 448."""
    if x == 0 or math.isnan(x):
        return x
    e = max(math.frexp(abs(x))[1] - 1, -6)       # |x| in [2^e, 2^(e+1)), or below 2^-6
    step = math.ldexp(1.0, e - 3)
    return math.copysign(min(round(abs(x) / step) * step, E4M3_MAX), x)  # round() is to even


def e4m3_value(code: int) -> float:
    """The value of a code other than 0x7f and 0xff."""
    e, m = code >> 3 & 15, code & 7
    x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
    return -x if code >> 7 else x


def quantise(row):
    """(values as multiples of the scale, scale) of one row; the scale and the quotients are float32's."""
    row = np.asarray(row, np.float32)
    if not np.all(np.isfinite(row)):
        return np.full(row.shape, np.nan), np.float32(np.nan)
    scale = np.float32(max(np.float32(np.abs(row).max() / np.float32(E4M3_MAX)), np.float32(2.0 ** -126)))
    return np.array([e4m3_round(float(np.float32(x / scale))) for x in row]), scale


def append_slots(lengths, counts, capacity):
    """[(sequence, token, slot)] of the tokens that find room, and the new lengths."""
    to, new = [], []
    for b, (n, m) in enumerate(zip(lengths, counts)):
        fits = min(int(m), capacity - int(n))
        to += [(b, t, int(n) + t) for t in range(fits)]
        new.append(int(n) + fits)
    return to, new


def evict_kept(scores, n: int, budget: int, recent: int):
    """The slots of one sequence and head that stay, ascending."""
    if n <= budget:
        return list(range(n))
    key = [-math.inf if math.isnan(s) else float(s) for s in scores[:n - recent]]
    best = sorted(range(n - recent), key=lambda j: (-key[j], j))[:budget - recent]
    return sorted(best) + list(range(n - recent, n))
