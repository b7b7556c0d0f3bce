"""Serving one attention layer with drafted tokens, its pages handed out on the GPU.

Prompts of different lengths are taken in packed, one behind the other: their pages
are reserved, their keys and values written into them, and their own attention
computed.  Every step then guesses a tree of tokens behind the one that was
chosen last, attends for all of them at once, follows the guesses that the layer
itself would have chosen, and keeps those: their rows move together behind the
tokens before, and pages that are no longer needed go back on the stack at
the next reservation.  The "model" is a set of random projections over a few tokens.

    python examples/draft_and_verify.py [--cache e4m3] [--steps 32] [--width 2] [--depth 3]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import movement_primitives_gb300 as lc  # noqa: E402


def tree(width: int, depth: int):
    """(parents, rank among siblings) of a root and `width` guesses behind every token, `depth` deep."""
    parents, ranks, level = [-1], [0], [0]
    for _ in range(depth):
        nodes = [(p, r) for p in level for r in range(width)]
        level = list(range(len(parents), len(parents) + len(nodes)))
        parents += [p for p, _ in nodes]
        ranks += [r for _, r in nodes]
    return parents, ranks


class Server:
    """Projections, pages and state of one attention layer."""

    def __init__(self, n_seqs: int, capacity: int, q_heads=16, kv_heads=4, head_dim=64, width=256, vocab=8, page_size=16,
                 n_pages=None, cache="bf16", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.page_size = q_heads, kv_heads, head_dim, page_size

        def weights(n, m):
            return (torch.randn((n, m), generator=g, device="cuda") * n ** -0.5).bfloat16()
        per = -(-capacity // page_size)
        n_pages = n_pages if n_pages is not None else n_seqs * per
        self.embed, self.place = (torch.randn((n, width), generator=g, device="cuda").bfloat16() for n in (vocab, per * page_size))
        self.project = weights(width, (q_heads + 2 * kv_heads) * head_dim)
        self.back, self.choose = weights(q_heads * head_dim, width), weights(width, vocab)
        pool = (n_pages, kv_heads, page_size, head_dim)
        dtype, scales = torch.bfloat16, [None, None]
        if cache == "e4m3":
            dtype = torch.float8_e4m3fn
            scales = [torch.zeros(pool[:3], device="cuda") for _ in range(2)]
        k, v = (torch.zeros(pool, dtype=torch.bfloat16, device="cuda").to(dtype) for _ in range(2))
        self.table = torch.full((n_seqs, per), -1, dtype=torch.int32, device="cuda")
        self.cache = lc.PagedCache(k, v, self.table, *scales)
        self.lengths = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.n_free = torch.tensor([n_pages], dtype=torch.int32, device="cuda")
        self.next = torch.zeros(n_seqs, dtype=torch.int64, device="cuda")  # the token that follows each sequence

    def reserve(self, counts, max_tokens: int):
        """Pages for counts[b] more tokens of each sequence."""
        r = lc.cache_reserve(self.table, self.lengths, counts, self.free, self.n_free, self.page_size, max_tokens)
        self.n_free = r.n_free
        return r

    def heads(self, tokens, positions):
        """(q, k, v) of tokens at their places."""
        y = ((self.embed[tokens] + self.place[positions]) @ self.project).unflatten(-1, (-1, self.head_dim))
        return y.split([self.q_heads, self.kv_heads, self.kv_heads], dim=-2)

    def chosen(self, out):
        """The token that follows each row of attention's output."""
        return ((out.flatten(-2) @ self.back) @ self.choose).argmax(-1)

    def prompt(self, tokens, counts):
        """Takes in packed prompts, counts[b] tokens of sequence b, which has none yet (a later piece of a prompt would
        need the keys before it as packed rows, and here they are in pages)."""
        if torch.any((counts > 0) & (self.lengths > 0)):
            raise ValueError("prompts are whole: a sequence that has tokens gets no more of them here")
        r = self.reserve(counts, tokens.shape[0])
        q, k, v = self.heads(tokens, r.positions)
        lc.cache_append_packed(self.cache, k, v, r.slots)
        out = lc.prompt_attend(q, k, v, r.starts)
        self.lengths = r.lengths
        self.next = torch.where(counts > 0, self.chosen(out[(r.starts[1:].long() - 1).clamp(min=0)]), self.next)
        return out

    def step(self, parents, ranks, guesses):
        """One tree a sequence, `guesses` [seqs, nodes] the token that a node's first child has.

        Returns (path [seqs, nodes], tokens [seqs, nodes], attention's output)."""
        n, m = self.lengths.shape[0], len(parents)
        up = torch.tensor(parents, device="cuda")
        tokens = (guesses[:, up.clamp(min=0)] + torch.tensor(ranks, device="cuda")) % self.embed.shape[0]
        tokens[:, 0] = self.next
        depth = [0]
        for p in parents[1:]:
            depth.append(depth[p] + 1)
        before = self.lengths
        self.reserve(torch.full_like(before, m), n * m)
        positions = before[:, None] + torch.tensor(depth, device="cuda")
        q, k, v = self.heads(tokens, positions)
        self.lengths = lc.cache_append(self.cache, k, v, before)
        out = lc.cache_attend_tree(self.cache, q, self.lengths, up.to(torch.int32).expand(n, m).contiguous())
        choice = self.chosen(out)
        # a guess stands if its parent does and chose it
        stands = torch.ones((n, m), dtype=torch.bool, device="cuda")
        for t in range(1, m):
            stands[:, t] = stands[:, parents[t]] & (choice[:, parents[t]] == tokens[:, t])
        at = torch.arange(m, device="cuda")
        path = torch.where(stands, at, m).sort(1)[0]
        last = stands.sum(1) - 1
        self.next = choice.gather(1, path.gather(1, last[:, None]))[:, 0]
        path = torch.where(path == m, -1, path).to(torch.int32)
        self.lengths = lc.cache_accept(self.cache, self.lengths, None, path)
        return path, tokens, out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--width", type=int, default=2)
    ap.add_argument("--depth", type=int, default=3)
    a = ap.parse_args()
    parents, ranks = tree(a.width, a.depth)
    s = Server(a.seqs, a.prompt + a.steps * (a.depth + 1) + len(parents), cache=a.cache)
    counts = torch.linspace(1, a.prompt, a.seqs, device="cuda").to(torch.int32)
    s.prompt(torch.randint(0, 8, (int(counts.sum()),), device="cuda"), counts)
    for _ in range(a.steps):
        s.step(parents, ranks, torch.randint(0, 8, (a.seqs, len(parents)), device="cuda"))
    status, detail = lc.last_device_error()
    if status:
        raise SystemExit("device error word %#x" % detail)
    gained = int((s.lengths - counts).sum())
    print("%d steps of %d sequences, %s cache, trees of %d: %.2f tokens a step, lengths %s, %d pages free"
          % (a.steps, a.seqs, a.cache, len(parents), gained / (a.steps * a.seqs), s.lengths.tolist(), int(s.n_free)))


if __name__ == "__main__":
    main()
