"""The drafting example against a replay of it: reservations, prompts, packed appends, trees and accepted
drafts, together as they are used."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

from conftest import ROOT
from oracle import drafts as od, prompt as op

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(ROOT, "examples", "draft_and_verify.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("draft_and_verify", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rows(s):
    """[seq, slot, head, dim] of keys and values in 64 bits (slots without a page: page 0's)."""
    table = s.table.cpu().clamp(min=0).long().numpy()
    out = []
    for p, sc in ((s.cache.k, s.cache.k_scale), (s.cache.v, s.cache.v_scale)):
        y = p.float().double().cpu()
        y = (y if sc is None else y * sc.double().cpu()[..., None]).numpy()
        out.append(y[table].transpose(0, 1, 3, 2, 4).reshape(table.shape[0], -1, s.kv_heads, s.head_dim))
    return out


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_steps_follow_the_replay(example, cache):
    """Tolerances: weights and the result are rounded to bfloat16 once each (prompts), or better (trees): twice 2^-8 of
    sum w|v|, with half as much again for float32 sums."""
    parents, ranks = example.tree(2, 3)
    assert parents[:7] == [-1, 0, 0, 1, 1, 2, 2] and len(parents) == 15
    s = example.Server(3, 200, q_heads=8, kv_heads=2, n_pages=30, cache=cache, seed=1)
    counts = torch.tensor([60, 1, 37], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    tokens = torch.randint(0, 8, (98,), generator=g, device="cuda")
    out = s.prompt(tokens, counts)
    q, k, v = s.heads(tokens, torch.cat([torch.arange(n, device="cuda") for n in (60, 1, 37)]))
    want, _, mag, _, _ = op.attend(*(x.double().cpu().numpy() for x in (q, k, v)), [0, 60, 61, 98], None, 0.125)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 1.5 * 2.0 ** -8 * (mag + np.abs(want)))
    kk, vv = rows(s)
    for b, (at, n) in enumerate(((0, 60), (60, 1), (61, 37))):
        for got, x in ((kk[b, :n], k), (vv[b, :n], v)):
            x = x[at:at + n].double().cpu().numpy()
            tol = 0 if cache == "bf16" else 2.0 ** -4 * np.abs(x) + np.abs(x).max(-1, keepdims=True) / 448 * 2.0 ** -9
            assert np.all(np.abs(got - x) <= tol)
    n = [60, 1, 37]
    for _ in range(12):
        before = [x.copy() for x in rows(s)]
        nxt = s.next.tolist()
        guesses = torch.randint(0, 8, (3, 15), generator=g, device="cuda")
        accept, seen = example.lc.cache_accept, {}

        def spy(c, lengths, *a, **kw):  # the cache as the tree's attention saw it
            seen["rows"], seen["lengths"] = rows(s), lengths.tolist()
            return accept(c, lengths, *a, **kw)
        example.lc.cache_accept = spy
        try:
            path, tokens, out = s.step(parents, ranks, guesses)
        finally:
            example.lc.cache_accept = accept
        assert seen["lengths"] == [x + 15 for x in n]
        kk, vv = seen["rows"]
        depth = np.array([len(od.line(parents, t)) - 1 for t in range(15)])
        q = s.heads(tokens, torch.tensor(n, device="cuda")[:, None] + torch.tensor(depth, device="cuda"))[0].double().cpu().numpy()
        choice = s.chosen(out).cpu().tolist()
        kk2, vv2 = rows(s)
        for b in range(3):
            for x, y in zip((kk, vv), before):
                assert np.array_equal(x[b, :n[b]], y[b, :n[b]])
            m = od.seen(n[b] + 15, 15, parents)
            for h in range(8):
                want, _, mag, _ = op.rows(q[b, :, h], kk[b, :n[b] + 15, h // 4], vv[b, :n[b] + 15, h // 4], m, 0.125)
                got = out[b, :, h].double().cpu().numpy()
                assert np.all(np.abs(got - want) <= 1.5 * 2.0 ** -8 * (mag + np.abs(want)))
            # the chain of guesses that were chosen
            t, line = 0, [0]
            assert int(tokens[b, 0]) == nxt[b]
            while True:
                child = [c for c in range(15) if parents[c] == t and int(tokens[b, c]) == choice[b][t]]
                if not child:
                    break
                t = child[0]
                line.append(t)
            assert path[b].tolist() == line + [-1] * (15 - len(line)) and int(s.next[b]) == choice[b][t]
            for x, y in ((kk, kk2), (vv, vv2)):
                assert np.array_equal(y[b, n[b]:n[b] + len(line)], x[b, [n[b] + i for i in line]])
            n[b] += len(line)
        assert s.lengths.tolist() == n
        used = s.table[s.table >= 0].tolist()
        assert sorted(used + s.free[:int(s.n_free)].tolist()) == list(range(30))
    st, detail = example.lc.last_device_error()
    assert st == 0, "device error word %#x" % detail


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_example_runs_as_a_program(example, cache):
    r = subprocess.run([sys.executable, PATH, "--cache", cache, "--steps", "6", "--prompt", "50"], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
    assert "6 steps of 8 sequences, %s cache" % cache in r.stdout
