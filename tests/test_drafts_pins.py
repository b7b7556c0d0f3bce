"""The 64-bit oracles of prompt attention, drafted trees and reservations against values worked out by hand
and against torch's own attention in 64 bits."""
import math

import numpy as np
import pytest

from oracle import drafts as od, prompt as op

torch = pytest.importorskip("torch")


def test_seen_by_hand():
    assert op.seen(2, 3).tolist() == [[True, True, False], [True, True, True]]
    assert op.seen(3, 1).tolist() == [[False], [False], [True]]
    assert op.seen(3, 3, window=2).tolist() == [[True, False, False], [True, True, False], [False, True, True]]
    assert op.seen(2, 2, causal=False, window=1).tolist() == [[True, True], [False, True]]


def test_tree_seen_by_hand():
    #   0 - 1 - 3
    #    \- 2        4 (a second root)
    parents = [-1, 0, 0, 1, -1]
    assert od.line(parents, 3) == [3, 1, 0]
    m = od.seen(7, 5, parents)
    assert m.astype(int).tolist() == [[1, 1, 1, 0, 0, 0, 0], [1, 1, 1, 1, 0, 0, 0], [1, 1, 1, 0, 1, 0, 0],
                                      [1, 1, 1, 1, 0, 1, 0], [1, 1, 0, 0, 0, 0, 1]]
    assert od.seen(7, 5, parents, window=2).astype(int).tolist() == [
        [0, 1, 1, 0, 0, 0, 0], [0, 0, 1, 1, 0, 0, 0], [0, 0, 1, 0, 1, 0, 0], [0, 0, 0, 1, 0, 1, 0], [0, 1, 0, 0, 0, 0, 1]]
    assert od.line([0, 5, -7], 1) == [1] and od.line([0, 5, -7], 2) == [2]  # no earlier draft: a root


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3)])
def test_prompt_oracle_is_torchs(causal, window):
    g = torch.Generator().manual_seed(1)
    starts, ks = [0, 4, 4, 9], [0, 6, 7, 12]
    q, k, v = (torch.randn((n, h, 8), generator=g, dtype=torch.float64) for n, h in ((9, 4), (12, 2), (12, 2)))
    out, lse, _, _, real = op.attend(q.numpy(), k.numpy(), v.numpy(), starts, ks, 0.3, causal, window)
    assert real.all()
    for b in range(3):
        a, c = slice(starts[b], starts[b + 1]), slice(ks[b], ks[b + 1])
        if a.start == a.stop:
            continue
        m = torch.from_numpy(op.seen(a.stop - a.start, c.stop - c.start, causal, window))
        kk, vv = (x[c].repeat_interleave(2, 1).transpose(0, 1) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(q[a].transpose(0, 1), kk, vv, m, scale=0.3)
        assert np.allclose(out[a], want.transpose(0, 1), atol=1e-13)
        x = (0.3 * q[a].transpose(0, 1) @ kk.transpose(1, 2)).masked_fill(~m, -math.inf)
        assert np.allclose(lse[a], x.logsumexp(2).t(), atol=1e-13)


def test_tree_oracle_of_a_chain_is_the_prompts():
    g = np.random.default_rng(2)
    k, v = g.standard_normal((2, 6, 2, 4, 8))
    table = np.array([[5, 1, 3], [0, 4, 2]])
    q = g.standard_normal((2, 3, 4, 8))
    out, lse, *_ , real = od.attend(q, k, v, table, [10, 2], [3, 2], [[-1, 0, 1]] * 2, 0.4, 5)
    assert real.tolist() == [[True] * 3, [True, True, False]]
    for b, (n, c) in enumerate([(10, 3), (2, 2)]):
        kk, vv = (x[table[b]].transpose(0, 2, 1, 3).reshape(12, 2, 8)[:n] for x in (k, v))
        want = op.attend(q[b, :c], kk, vv, [0, c], [0, n], 0.4, True, 5)
        assert np.allclose(out[b, :c], want[0], atol=1e-13) and np.allclose(lse[b, :c], want[1], atol=1e-13)
    # every page outside the pool: nothing to see
    out, lse, *_ = od.attend(q, k, v, table + 100, [10, 2], [3, 2], [[-1, 0, 1]] * 2, 0.4)
    assert not out.any() and np.isneginf(lse[0]).all()


def test_accept_by_hand():
    moves, new = od.accept([10, 5, 3, 9], [4, 4, 0, 2], [[0, 2, -1], [1, 3, 2], [0, -1, -1], [-1, 0, 1]], 100)
    assert new == [8, 3, 3, 7]
    assert moves == [(0, 6, 6), (0, 8, 7), (1, 2, 1), (1, 4, 2)]


def test_reserve_by_hand():
    t = [[7, 8, -1], [3, -1, -1], [4, 5, 6], [-1, -1, -1]]
    # page of 4: 8 + 1 tokens want a third page; 2 + 1 none; an ended sequence gives three back; 5 tokens want two
    table, n, starts, packed, stack = od.reserve(t, [8, 2, 0, 0], [1, 1, 0, 5], [1, 2], 4, 8)
    assert table == [[7, 8, 6], [3, -1, -1], [-1, -1, -1], [5, 4, -1]]
    assert n == [9, 3, 0, 5] and starts == [0, 1, 2, 2, 7] and stack == [1, 2]
    assert packed[:3] == [(24, 8, 0), (14, 2, 1), (20, 0, 3)]
    # too few pages: the last is not served; too short a list: the one it ends in is not
    table, n, starts, _, stack = od.reserve(t, [8, 2, 9, 0], [1, 1, 0, 5], [1, 2], 4, 8)
    assert table[3] == [-1] * 3 and n == [9, 3, 9, 0] and stack == [1]
    _, n, starts, _, stack = od.reserve(t, [8, 2, 0, 0], [1, 1, 0, 5], [1, 2], 4, 6)
    assert n == [9, 3, 0, 0] and stack == [1, 2, 4, 5]
    _, n, starts, _, _ = od.reserve(t, [8, 2, 0, 0], [5, 1, 0, 5], [1, 2], 4, 6)  # past the table's columns
    assert n == [8, 3, 0, 5]
