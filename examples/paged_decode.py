"""Serving one attention layer from a paged key-value cache.

Prompts of different lengths are appended, then every step appends one token a
sequence, attends to the cache with the slots' weights collected, and, once a
sequence outgrows its budget, lets go of the slots that were attended to the
least (the newest ones always stay).  The "model" is a set of random
projections; keys and values are kept in E4M3 or in bfloat16.

    python examples/paged_decode.py [--cache e4m3] [--steps 64] [--budget 256]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import movement_primitives_gb300 as lc  # noqa: E402


class Layer:
    """Projections, cache and state of one attention layer."""

    def __init__(self, n_seqs: int, capacity: int, q_heads=16, kv_heads=4, head_dim=64, width=256, page_size=16,
                 cache="bf16", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        w = torch.randn((width, (q_heads + 2 * kv_heads) * head_dim), generator=g, device="cuda") * width ** -0.5
        self.project = w.bfloat16()
        self.back = (torch.randn((q_heads * head_dim, width), generator=g, device="cuda") *
                     (q_heads * head_dim) ** -0.5).bfloat16()
        per = -(-capacity // page_size)
        pool = (n_seqs * per, kv_heads, page_size, head_dim)
        dtype, scales = torch.bfloat16, [None, None]
        if cache == "e4m3":
            dtype = torch.float8_e4m3fn
            scales = [torch.zeros(pool[:3], device="cuda") for _ in range(2)]
        k, v = (torch.zeros(pool, dtype=torch.bfloat16, device="cuda").to(dtype) for _ in range(2))
        table = torch.randperm(n_seqs * per, generator=g, device="cuda").reshape(n_seqs, per).to(torch.int32)
        self.cache = lc.PagedCache(k, v, table, *scales)
        self.lengths = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.scores = torch.zeros((n_seqs, kv_heads, self.cache.capacity), device="cuda")

    def heads(self, x):
        """(q, k, v) of tokens x [seqs, tokens, width]."""
        y = (x @ self.project).unflatten(-1, (-1, self.head_dim))
        return y.split([self.q_heads, self.kv_heads, self.kv_heads], dim=2)

    def prompt(self, x, counts):
        """Takes in prompts x [seqs, tokens, width], counts[b] tokens of each."""
        _q, k, v = self.heads(x)
        self.lengths = lc.cache_append(self.cache, k, v, self.lengths, counts)

    def step(self, x, budget: int, recent: int):
        """One token a sequence, x [seqs, width]: its attention's output, [seqs, width]."""
        q, k, v = self.heads(x[:, None])
        self.lengths = lc.cache_append(self.cache, k, v, self.lengths)
        out = lc.cache_attend(self.cache, q[:, 0], self.lengths, scores=self.scores)
        _kept, self.scores, self.lengths = lc.cache_evict(self.cache, self.lengths, self.scores, budget, recent)
        return out.flatten(1) @ self.back


def decode(layer: Layer, prompts, counts, steps: int, budget: int, recent: int):
    """The outputs of `steps` steps, each fed the one before."""
    layer.prompt(prompts, counts)
    last = prompts.gather(1, (counts.long() - 1)[:, None, None].expand(-1, 1, prompts.shape[2]))[:, 0]
    outs = []
    for _ in range(steps):
        last = layer.step(last, budget, recent)
        outs.append(last)
    return torch.stack(outs)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--budget", type=int, default=256)
    a = ap.parse_args()
    layer = Layer(a.seqs, max(a.prompt, a.budget) + 1, cache=a.cache)
    x = torch.randn((a.seqs, a.prompt, 256), device="cuda").bfloat16()
    counts = torch.linspace(1, a.prompt, a.seqs, device="cuda").to(torch.int32)
    y = decode(layer, x, counts, a.steps, a.budget, a.budget // 4)
    status, detail = lc.last_device_error()
    if status:
        raise SystemExit("device error word %#x" % detail)
    print("%d steps of %d sequences, %s cache: lengths %s, last output's norm %.4f"
          % (a.steps, a.seqs, a.cache, layer.lengths.tolist(), y[-1].float().norm().item()))


if __name__ == "__main__":
    main()
