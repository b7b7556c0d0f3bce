"""Attention over whole prompts on the CPU, in 64 bits.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Query i of a sequence of nq queries and nk keys has the place p = i + nk - nq
and sees the keys j <= p (all, where not causal) with j > p - window (all,
without a window); x_j = scale * q . k_j, w = softmax(x), out = sum_j w_j v_j,
lse = log sum_j exp x_j; nothing seen gives out = 0 and lse = -inf.
"""
from __future__ import annotations

import math

import numpy as np


def seen(nq: int, nk: int, causal=True, window=0):
    """[nq, nk] of bool."""
    p, j = np.arange(nq)[:, None] + nk - nq, np.arange(nk)[None, :]
    m = np.ones((nq, nk), bool)
    if causal:
        m &= j <= p
    if window:
        m &= j > p - window
    return m


def rows(q, k, v, m, scale):
    """(out, lse, sum_j w_j |v_j|, largest |scale| sum |q||k_j|) of one head: q [n, d], k and v [nk, d], m [n, nk].

    What is not seen by a row does not reach it, NaN included."""
    n, d = q.shape
    out, mag, lse, reach = np.zeros((n, d)), np.zeros((n, d)), np.full(n, -math.inf), np.zeros(n)
    if not k.shape[0]:
        return out, lse, mag, reach
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.where(m, scale * (q @ k.T), -math.inf)
        top = x.max(1)
        none = np.isneginf(top)
        e = np.where(m, np.exp(x - np.where(none, 0.0, top)[:, None]), 0.0)
        total = e.sum(1)
        w = e / np.where(none, 1.0, total)[:, None]
        odd = ~np.isfinite(v)
        plain = np.where(odd, 0.0, v)
        out, mag = w @ plain, w @ np.abs(plain)
        lse = np.where(none, -math.inf, top + np.log(np.where(none, 1.0, total)))
        reach = np.where(m, abs(scale) * (np.abs(q) @ np.abs(np.where(np.isfinite(k), k, 0.0)).T), 0.0).max(1)
        out = np.where((m.astype(float) @ odd) > 0, math.nan, out)  # a value seen that is no number
    return out, lse, mag, reach


def attend(q, k, v, starts, k_starts=None, scale=1.0, causal=True, window=0):
    """(out, lse, magnitudes, reaches, [tokens] of bool: some sequence's) of packed q, k, v."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    tokens, heads, d = q.shape
    group = heads // k.shape[1]
    k_starts = starts if k_starts is None else k_starts
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach, real = np.zeros((tokens, heads)), np.zeros((tokens, heads)), np.zeros(tokens, bool)
    for b in range(len(starts) - 1):
        qs, ks = slice(starts[b], starts[b + 1]), slice(k_starts[b], k_starts[b + 1])
        real[qs] = True
        m = seen(qs.stop - qs.start, ks.stop - ks.start, causal, window)
        for h in range(heads):
            out[qs, h], lse[qs, h], mag[qs, h], reach[qs, h] = rows(q[qs, h], k[ks, h // group], v[ks, h // group], m, scale)
    return out, lse, mag, reach, real
