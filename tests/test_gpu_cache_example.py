"""The decoding example against a dense replay of it in 64 bits: appending,
attention with collected weights and eviction, together as they are used."""
import importlib.util
import math
import os
import subprocess
import sys

import numpy as np
import pytest

from conftest import ROOT
from oracle import cache as oc

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(ROOT, "examples", "paged_decode.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("paged_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_decoding_steps_follow_the_dense_replay(example, cache):
    """Every step is replayed from the library's own state before it (so that
    rounding does not build up over steps): the new row, the attention over the
    rows so far, the weights collected, and the slots that stay."""
    budget, recent, steps = 40, 8, 12
    layer = example.Layer(3, 64, q_heads=8, kv_heads=2, head_dim=64, cache=cache, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((3, 60, 256), generator=g, device="cuda").bfloat16()
    counts = torch.tensor([60, 33, 38], dtype=torch.int32, device="cuda")
    layer.prompt(x, counts)
    assert layer.lengths.tolist() == [60, 33, 38]
    last = x[:, 0]
    table = layer.cache.page_table.cpu().numpy()

    def rows():  # [seq, head, slot, dim] of keys and values
        out = []
        for p, s in ((layer.cache.k, layer.cache.k_scale), (layer.cache.v, layer.cache.v_scale)):
            y = p.double().cpu() if cache == "bf16" else p.float().double().cpu() * s.double().cpu()[..., None]
            y = y.numpy()[table]
            out.append(y.transpose(0, 2, 1, 3, 4).reshape(3, 2, -1, 64))
        return out

    for _ in range(steps):
        n0, k0, scores0 = layer.lengths.tolist(), rows(), layer.scores.double().cpu().numpy()
        q, k, v = (t[:, 0].double().cpu().numpy() for t in layer.heads(last[:, None]))
        new = layer.step(last, budget, recent)
        kv = []
        for old, fresh in zip(k0, (k, v)):
            now = old.copy()
            for b in range(3):
                for h in range(2):
                    row = fresh[b, h]
                    if cache == "e4m3":
                        codes, scale = oc.quantise(row)
                        row = codes * float(scale)
                    now[b, h, n0[b]] = row
            kv.append(now)
        want_lengths = [min(n + 1, budget) for n in n0]
        assert layer.lengths.tolist() == want_lengths
        got_rows, got_scores = rows(), layer.scores.double().cpu().numpy()
        out = np.zeros((3, 8, 64))
        for b in range(3):
            n = n0[b] + 1
            for h in range(2):
                logits = q[b, 4 * h:4 * h + 4] @ kv[0][b, h, :n].T / math.sqrt(64)
                w = np.exp(logits - logits.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                out[b, 4 * h:4 * h + 4] = w @ kv[1][b, h, :n]
                score = scores0[b, h, :n] + w.sum(0)
                # the kept ones by the library's own scores' order: its float32 sums may swap near equals
                kept = oc.evict_kept(score, n, budget, recent)
                m = len(kept)
                same = np.allclose(got_scores[b, h, :m], score[kept], rtol=1e-5, atol=1e-6)
                assert same and np.all(got_scores[b, h, m:] == 0)
                for got, now in zip(got_rows, kv):
                    assert np.array_equal(got[b, h, :m], now[b, h, kept])
        want = torch.tensor(out.reshape(3, -1)).bfloat16().cuda() @ layer.back
        # the attention's output in bfloat16 (twice its rounding), through a product of 512 terms
        scale = np.abs(out).max() * 2.0 ** -7 * layer.back.float().abs().sum(0).max().item()
        assert (new.float() - want.float()).abs().max().item() <= scale
        last = new
    import movement_primitives_gb300 as lc
    assert lc.last_device_error()[0] == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_example_runs_as_a_program(example, cache):
    r = subprocess.run([sys.executable, PATH, "--cache", cache, "--steps", "5", "--prompt", "70", "--budget", "50",
                        "--seqs", "4"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "lengths [6, 29, 50, 50]" in r.stdout, r.stdout
