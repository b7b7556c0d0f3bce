"""What is measured of the operators around the paged key-value cache: prompts, drafts and pages.

Four operators (see include/layout_copy_cache.h and include/layout_copy_prompt.h):

  prompt   attention over whole prompts, packed one behind the other, causal
           or not, with grouped heads, a window, and keys that may begin before
           the queries (a later piece of a prompt)
  tree     attention of a tree of drafted tokens a sequence over its cached
           slots: a draft sees what was there before the drafts, and its own
           ancestors among them
  accept   the accepted path of drafts moves together behind the tokens before
           them, in place
  reserve  page tables that hold the pages of the requests' lengths, from a
           stack of free pages, and the slot of every packed token

Every operator has a plain form in elementary torch operations, computed in 32
bits and rounded once at the end.  `own` chooses between it and the library.
"""
import math
import random

import torch

own = False  # set by the caller: False runs the plain forms, True the library's kernels

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


def _prompt(**kw):
    """seqs, q_heads, kv_heads, dim, tokens (longest sequence's queries), ragged (lengths spread over 1 .. tokens, one
    sequence empty where there are four or more), prior (most keys before a sequence's first query), causal, window
    (0: none), pad (rows of the packed tensors behind the last sequence), type"""
    c = dict(op="prompt", seqs=1, q_heads=8, kv_heads=8, dim=128, tokens=128, ragged=False, prior=0, causal=True,
             window=0, pad=0, type="bf16")
    c.update(kw)
    return c


def _tree(**kw):
    """seqs, q_heads, kv_heads, dim, page (slots of a page), tokens (longest sequence, its drafts counted in), ragged,
    drafts (most drafts a sequence; ragged ones have fewer), bushy (a draft's parent is any earlier one, else mostly the
    one before it), cache (element type of the pages), order ("head": a page holds [head, slot, dim]; "token": [slot, head,
    dim]), window (0: none)"""
    c = dict(op="tree", seqs=1, q_heads=8, kv_heads=8, dim=128, page=16, tokens=128, ragged=False, drafts=4, bushy=True,
             cache="bf16", order="head", window=0)
    c.update(kw)
    return c


def _reserve(**kw):
    """seqs, page, per (columns of the table), held (most tokens a sequence has), new (most tokens it gets; ragged),
    finished (a quarter of the sequences have ended and give their pages back)"""
    c = dict(op="reserve", seqs=8, page=16, per=128, held=1024, new=1, finished=False)
    c.update(kw)
    return c


def listed():
    return [
        # one short question: latency is everything
        _prompt(name="prompt_short", q_heads=8, kv_heads=2, dim=64, tokens=61),
        # a serving batch of prompts of every length, packed, grouped heads, a padded tail
        _prompt(name="prompt_batch", seqs=24, q_heads=32, tokens=2048, ragged=True, pad=96),
        # one long document
        _prompt(name="prompt_long", q_heads=32, tokens=11585, type="fp16"),
        # later pieces of prompts over the keys before them; one query head a key head, an odd head size, a window
        _prompt(name="prompt_piece_window", seqs=6, q_heads=12, kv_heads=12, dim=80, tokens=1999, ragged=True, prior=3001,
                window=1024),
        # a short chain of drafts for one conversation
        _tree(name="tree_one_short", q_heads=8, kv_heads=2, dim=64, tokens=301, drafts=5, bushy=False),
        # a serving batch whose drafts are verified
        _tree(name="tree_batch", seqs=16, q_heads=32, page=64, tokens=4096, ragged=True, drafts=16),
        # the same of wide trees on an 8-bit cache of long sequences
        _tree(name="tree_e4m3", seqs=12, q_heads=32, page=32, tokens=32767, ragged=True, drafts=32, cache="e4m3"),
        # all query heads on one key head, wide heads, pages that are no power of two, a sliding window
        _tree(name="tree_mqa_window", seqs=8, q_heads=16, kv_heads=1, dim=256, page=24, tokens=5000, order="token",
              window=1024, drafts=12, cache="fp16"),
        # a few sequences keep some of their drafts
        dict(_tree(name="accept_few", seqs=4, tokens=1500, drafts=8), op="accept"),
        # a large batch of wide trees
        dict(_tree(name="accept_batch", seqs=192, tokens=1024, page=64, ragged=True, drafts=64, bushy=False), op="accept"),
        # a decoding step's pages
        _reserve(name="reserve_step", seqs=64, per=256, held=4000),
        # prompts come in while other requests end
        _reserve(name="reserve_prompts", seqs=256, per=1024, held=8000, new=512, finished=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    """One more case over the ranges that the listed ones stand for."""
    op = rng.choice(["prompt", "prompt", "prompt", "tree", "tree", "tree", "accept", "reserve"])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 12, 16])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    dim = rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 192, 256])
    if op == "prompt":
        c = _prompt(seqs=_log_int(rng, 1, 48), kv_heads=kv_heads, q_heads=q_heads, dim=dim, tokens=_log_int(rng, 1, 11585),
                    ragged=rng.random() < 0.7, causal=rng.random() < 0.8, pad=rng.choice([0, 0, 1, 77]),
                    type=rng.choice(["bf16", "bf16", "fp16"]))
        c["prior"] = _log_int(rng, 1, 8192) if rng.random() < 0.3 else 0
        c["window"] = _log_int(rng, 1, c["tokens"] + c["prior"]) if rng.random() < 0.25 else 0
        # the work stays within the largest listed case's: fewer sequences first, then shorter ones
        while c["seqs"] * c["q_heads"] * c["tokens"] * (2 if not c["causal"] else 1) * (c["tokens"] + 2 * c["prior"]) * \
                max(c["dim"], 128) > 32 * 11585 ** 2 * 128 or c["seqs"] * c["q_heads"] * c["tokens"] * c["dim"] > 2e8:
            if c["seqs"] > 1:
                c["seqs"] = max(1, c["seqs"] * 2 // 3)
            else:
                c["tokens"], c["prior"] = max(1, c["tokens"] * 2 // 3), c["prior"] * 2 // 3
        return c
    if op == "reserve":
        page = rng.choice([8, 16, 16, 24, 32, 64, 128])
        held, new = _log_int(rng, 1, 16384), _log_int(rng, 1, 2048) if rng.random() < 0.5 else 1
        return _reserve(seqs=_log_int(rng, 1, 256), page=page, held=held, new=new, per=-(-(held + new) // page) + 3,
                        finished=rng.random() < 0.5)
    c = _tree(seqs=_log_int(rng, 1, 96), kv_heads=kv_heads, q_heads=q_heads, dim=dim,
              page=rng.choice([8, 16, 16, 24, 32, 48, 64, 64, 128]), tokens=_log_int(rng, 64, 131071),
              ragged=rng.random() < 0.7, drafts=_log_int(rng, 1, 64), bushy=rng.random() < 0.5,
              cache=rng.choice(["bf16", "bf16", "fp16", "e4m3"]), order=rng.choice(["head", "token"]))
    c["op"] = op
    if op == "tree" and rng.random() < 0.25:
        c["window"] = _log_int(rng, 1, c["tokens"])
    # the pool and the logits stay within the largest listed ones'
    while _pool_bytes(c) > 7e8 or c["seqs"] * c["q_heads"] * c["drafts"] * c["tokens"] * max(c["dim"], 128) > 5e10:
        if c["seqs"] > 1:
            c["seqs"] = max(1, c["seqs"] * 2 // 3)
        else:
            c["tokens"] = max(c["drafts"], c["tokens"] * 2 // 3)
            c["window"] = min(c["window"], c["tokens"])
    return c


# -- sizes ------------------------------------------------------------------------------------------------------------

def _spread(n, most, ragged):
    """Lengths of n sequences, the same for every seed up to their order; with four ragged ones or more, one is empty."""
    if not ragged or n == 1:
        return [most] * n
    got = [max(1, most * (i + 1) // n) for i in range(n)]
    if n >= 4:
        got[0] = 0
    return got


def _priors(c):
    """Keys before each sequence's first query: from none to `prior`."""
    return [c["prior"] * (i % 4) // 3 if c["seqs"] > 1 else c["prior"] for i in range(c["seqs"])]


def _drafts(c):
    return [min(n, c["drafts"] if not c["ragged"] else max(1, c["drafts"] - i % 3)) for i, n in enumerate(_cached(c))]


def _cached(c):
    return [n and max(n, 1) for n in _spread(c["seqs"], c["tokens"], c["ragged"])]


def _elem(c):
    return 1 if c["cache"] == "e4m3" else 2


def _row_bytes(c):
    """Bytes of one token's row of one head, its scale included."""
    return c["dim"] * _elem(c) + (4 if c["cache"] == "e4m3" else 0)


def _pages_per_seq(c):
    return -(-c["tokens"] // c["page"])


def _pool_bytes(c):
    return 2 * c["seqs"] * _pages_per_seq(c) * c["page"] * c["kv_heads"] * _row_bytes(c)


def _pairs(c, nq, nk):
    """Seen (query, key) pairs of a sequence."""
    w = c["window"] or nk
    last = [i + nk - nq for i in range(nq)]  # the newest key of a causal row
    return sum(min(x + 1, w) if c["causal"] else nk - max(0, x - w + 1) for x in last)


def work(case):
    c = case
    if c["op"] == "prompt":
        d, nq = c["dim"], _spread(c["seqs"], c["tokens"], c["ragged"])
        nk = [n + p for n, p in zip(nq, _priors(c))]
        return {"bytes": sum(nq) * c["q_heads"] * (4 * d + 4) + sum(nk) * c["kv_heads"] * 4 * d,
                "flops": sum(_pairs(c, a, b) for a, b in zip(nq, nk)) * c["q_heads"] * d * 4}
    if c["op"] == "reserve":
        n = c["seqs"]
        return {"bytes": 8 * n * c["per"] + 16 * n + 16 * sum(_new_tokens(c)), "flops": 0}
    lens, drafts, h, d, row = _cached(c), _drafts(c), c["kv_heads"], c["dim"], _row_bytes(c)
    if c["op"] == "accept":
        # a path takes every second draft or so, and its first rows are in their place already
        return {"bytes": sum(drafts) // 2 * h * 2 * 2 * row + 8 * sum(drafts), "flops": 0}
    seen = [min(n, c["window"] + t) if c["window"] else n for n, t in zip(lens, drafts)]
    rows = sum(drafts) * c["q_heads"]
    return {"bytes": sum(seen) * h * 2 * row + rows * (4 * d + 4) + 4 * sum(drafts),
            "flops": sum(n * t for n, t in zip(seen, drafts)) * c["q_heads"] * d * 4}


# -- inputs -----------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed, torch.Generator(device="cuda").manual_seed(seed), random.Random(seed))


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_prompt(c, seed, g, host):
    """Packed queries, keys and values with their sequences' starts, and the buffers that a program's layers share."""
    order = list(range(c["seqs"]))
    host.shuffle(order)
    nq = [_spread(c["seqs"], c["tokens"], c["ragged"])[i] for i in order]
    nk = [n + _priors(c)[i] for n, i in zip(nq, order)]
    ends = lambda n: [sum(n[:i]) for i in range(len(n) + 1)]  # noqa: E731
    t, d = DTYPE[c["type"]], c["dim"]

    def rows(n, heads, scale):
        x = (scale * torch.randn((n + c["pad"], heads, d), generator=g, device="cuda")).to(t)
        x[n:] = float("nan")  # what a padded tail holds is nobody's
        return x
    s = dict(case=c, q=rows(sum(nq), c["q_heads"], 1.5), k=rows(sum(nk), c["kv_heads"], 1.0),
             v=rows(sum(nk), c["kv_heads"], 1.0), starts=_ints(ends(nq)), k_starts=_ints(ends(nk)) if c["prior"] else None)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:2], device="cuda")
    return s


def _pool(c, n_pages, g):
    """A pool of pages, [page, head, slot, dim] whatever their order in memory, of unit normal values."""
    shape = (n_pages, c["kv_heads"], c["page"], c["dim"]) if c["order"] == "head" else \
            (n_pages, c["page"], c["kv_heads"], c["dim"])
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    scale = None
    if c["cache"] == "e4m3":
        # rows whose largest value is near E4M3's, as quantised rows are
        x = (x * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        scale = 0.008 + 0.004 * torch.rand(shape[:3], generator=g, device="cuda")
    else:
        x = x.to(DTYPE[c["cache"]])
    if c["order"] == "token":
        x = x.transpose(1, 2)
        scale = None if scale is None else scale.transpose(1, 2)
    return x, scale


def _prepare_cache(c, seed, g, host):
    """Pools and page table with the drafts in place behind their sequences' tokens (pages in any order, -1 where a
    sequence has none), the trees, and for `accept` a path of each from its root."""
    n_seq, per, page = c["seqs"], _pages_per_seq(c), c["page"]
    n_pages = n_seq * per + 1
    k, k_scale = _pool(c, n_pages, g)
    v, v_scale = _pool(c, n_pages, g)
    order = list(range(n_seq))
    host.shuffle(order)
    lengths, counts = ([x[i] for i in order] for x in (_cached(c), _drafts(c)))
    parents = [[-1 if t == 0 else host.randrange(-1, t) if c["bushy"] or host.random() < 0.2 else t - 1
                for t in range(c["drafts"])] for _ in range(n_seq)]
    paths = []
    for tree, n in zip(parents, counts):
        path, t = [], host.randrange(n // 2, n) if n else -1
        while t >= 0:
            path.insert(0, t)
            t = tree[t]
        paths.append(path + [-1] * (c["drafts"] - len(path)))
    table = torch.randperm(n_pages, generator=g, device="cuda")[:n_seq * per].reshape(n_seq, per).to(torch.int32)
    used = torch.arange(per, device="cuda")[None, :] * page < _ints(lengths)[:, None]
    s = dict(case=c, k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=torch.where(used, table, -1).contiguous(),
             lengths=_ints(lengths), counts=_ints(counts), parents=_ints(parents), path=_ints(paths))
    if c["op"] == "tree":
        io = torch.float16 if c["cache"] == "fp16" else torch.bfloat16
        shape = (n_seq, c["drafts"], c["q_heads"], c["dim"])
        s["q"] = (1.5 * torch.randn(shape, generator=g, device="cuda")).to(io)
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(shape[:3], device="cuda")
    if own:
        import movement_primitives_gb300 as lc
        s["cache"] = lc.PagedCache(k, v, s["table"], k_scale, v_scale)
    return s


def _new_tokens(c):
    return [max(1, c["new"] * (i + 1) // c["seqs"]) for i in range(c["seqs"])]


def _prepare_reserve(c, seed, g, host):
    """A table in which every sequence has the pages of its tokens, the stack of the other pages, and a step's requests.
    Sequences that have ended have no tokens any more, but still their pages."""
    n, page, per = c["seqs"], c["page"], c["per"]
    held, new = [c["held"] * (i + 1) // n for i in range(n)], _new_tokens(c)
    total = sum(-(-x // page) for x in held + new) + 8  # all pages there are, room for every one on the stack
    host.shuffle(held)
    host.shuffle(new)
    need = [-(-x // page) for x in held]
    pages = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(per, device="cuda")[None, :]
    first = _ints([sum(need[:i]) for i in range(n)])[:, None]
    table = torch.where(at < _ints(need)[:, None], pages[(first + at).clamp(max=total - 1)], -1)
    free = torch.cat([pages[sum(need):], torch.full((sum(need),), -1, dtype=torch.int32, device="cuda")])
    for i in range(n):
        if c["finished"] and i % 4 == 1:
            held[i] = new[i] = 0
    return dict(case=c, table=table, lengths=_ints(held), counts=_ints(new), free=free,
                n_free=_ints([total - sum(need)]), tokens=sum(_new_tokens(c)), new_table=torch.empty_like(table))


_PREPARE = {"prompt": _prepare_prompt, "tree": _prepare_cache, "accept": _prepare_cache, "reserve": _prepare_reserve}


# -- the operators ----------------------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _OWN[c["op"]](state, c)
    return _PLAIN[c["op"]](state, c)


def _own_prompt(s, c):
    import movement_primitives_gb300 as lc
    out = lc.prompt_attend(s["q"], s["k"], s["v"], s["starts"], k_starts=s["k_starts"], causal=c["causal"],
                           window=c["window"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]}


def _own_tree(s, c):
    import movement_primitives_gb300 as lc
    out = lc.cache_attend_tree(s["cache"], s["q"], s["lengths"], s["parents"], s["counts"], window=c["window"],
                               out=s["out"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]}


def _own_accept(s, c):
    import movement_primitives_gb300 as lc
    lengths = lc.cache_accept(s["cache"], s["lengths"], s["counts"], s["path"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "lengths": lengths}


def _own_reserve(s, c):
    import movement_primitives_gb300 as lc
    r = lc.cache_reserve(s["table"], s["lengths"], s["counts"], s["free"], s["n_free"], c["page"], s["tokens"],
                         new_table=s["new_table"])
    return {"table": r.table, "starts": r.starts, "slots": r.slots, "positions": r.positions, "seqs": r.seqs,
            "lengths": r.lengths, "n_free": r.n_free, "free": s["free"]}


def _attend(q, k, v, seen):
    """Softmax attention in 32 bits: q [.., rows, d], k and v [.., keys, d], seen [.., rows, keys]; a row that sees nothing
    gives zeros."""
    x = torch.matmul(q * (1.0 / math.sqrt(q.shape[-1])), k.transpose(-1, -2))
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp_(x.sub_(top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out, (top + torch.log(total))[..., 0]


def _plain_prompt(s, c):
    h, d, group = c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    starts, k_starts = s["starts"].long(), (s["starts"] if s["k_starts"] is None else s["k_starts"]).long()
    nq, nk = starts.diff(), k_starts.diff()
    rows = torch.arange(c["tokens"], device="cuda")
    keys = torch.arange(c["tokens"] + c["prior"], device="cuda")
    there_q, there_k = rows < nq[:, None], keys < nk[:, None]
    at_q = torch.where(there_q, starts[:-1, None] + rows, 0)
    at_k = torch.where(there_k, k_starts[:-1, None] + keys, 0)
    # sequences padded to the longest, [seq, head, token, dim]; what is padded is zero
    q, k, v = (torch.where(there[..., None, None], x[at], 0.0).float().transpose(1, 2)
               for x, at, there in ((s["q"], at_q, there_q), (s["k"], at_k, there_k), (s["v"], at_k, there_k)))
    last = (rows[None, :] + (nk - nq)[:, None])[:, :, None]
    seen = there_k[:, None, :].expand(-1, rows.numel(), -1)
    if c["causal"]:
        seen = seen & (keys <= last)
    if c["window"]:
        seen = seen & (keys > last - c["window"])
    k, v = k[:, :, None], v[:, :, None]
    out, lse = _attend(q.unflatten(1, (h, group)), k, v, seen[:, None, None])
    out, lse = out.flatten(1, 2).transpose(1, 2), lse.flatten(1, 2).transpose(1, 2)
    s["out"][at_q[there_q]] = out[there_q].to(s["q"].dtype)
    s["lse"][at_q[there_q]] = lse[there_q]
    return {"out": s["out"], "lse": s["lse"]}


def _gather(pool, scale, table):
    """[seq, head, slot, dim] in 32 bits of the pages of each sequence."""
    at = table.clamp(min=0).long()
    x = pool[at].transpose(1, 2).flatten(2, 3).float()
    return x if scale is None else x * scale[at].transpose(1, 2).flatten(2, 3)[..., None]


def _plain_tree(s, c):
    n_seq, h, n_t = c["seqs"], c["kv_heads"], c["drafts"]
    group = c["q_heads"] // h
    k, v = _gather(s["k"], s["k_scale"], s["table"]), _gather(s["v"], s["v_scale"], s["table"])
    slot, t = torch.arange(k.shape[2], device="cuda"), torch.arange(n_t, device="cuda")
    there = t < s["counts"][:, None]
    # whom a draft descends from: powers of "itself or its parent"
    step = (s["parents"][:, :, None] == t).float() + torch.eye(n_t, device="cuda")
    kin = torch.linalg.matrix_power(step, 64) > 0
    depth = kin.sum(-1)
    before = (s["lengths"] - s["counts"])[:, None, None]
    draft = (slot - before).clamp(0, n_t - 1).expand(-1, n_t, -1)
    position = torch.where(slot < before, slot, before + depth[:, None].expand(-1, n_t, -1).gather(2, draft) - 1)
    seen = (slot < before) | ((slot < s["lengths"][:, None, None]) & kin.gather(2, draft))
    if c["window"]:
        seen = seen & (position > before + depth[..., None] - 1 - c["window"])
    live = (slot < s["lengths"][:, None])[:, None, :, None]
    q = s["q"].float().unflatten(2, (h, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [seq, head, draft and group, dim]
    out, lse = _attend(q, torch.where(live, k, 0.0), torch.where(live, v, 0.0), seen.repeat_interleave(group, 1)[:, None])
    out = out.unflatten(2, (n_t, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.unflatten(2, (n_t, group)).permute(0, 2, 1, 3).flatten(2, 3)
    s["out"][there] = out[there].to(s["q"].dtype)
    s["lse"][there] = lse[there]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_accept(s, c):
    before = s["lengths"] - s["counts"]
    seq, i = torch.nonzero(s["path"] >= 0, as_tuple=True)
    src = before[seq].long() + s["path"][seq, i]
    dst = before[seq].long() + i
    page_from, page_to = (s["table"][seq, x // c["page"]].long() for x in (src, dst))
    for x in (s["k"], s["v"], s["k_scale"], s["v_scale"]):
        if x is not None:
            x = x.view(torch.uint8) if c["cache"] == "e4m3" and x.dim() == 4 else x
            x[page_to, :, dst % c["page"]] = x[page_from, :, src % c["page"]]
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"],
            "lengths": before + (s["path"] >= 0).sum(-1, dtype=torch.int32)}


def _plain_reserve(s, c):
    n, per, page = c["seqs"], c["per"], c["page"]
    lengths, counts = s["lengths"].long(), s["counts"].long()
    held = (s["table"] >= 0).sum(-1)
    want = (lengths + counts + page - 1) // page
    at = torch.arange(per, device="cuda")
    # pages past a sequence's go on the stack, in the sequences' order; then what is missing is taken from its top
    over = (at >= want[:, None]) & (at < held[:, None])
    back = s["table"][over]
    base = s["n_free"].long()
    s["free"][base + torch.arange(back.numel(), device="cuda")] = back
    top = base + back.numel()
    missing = (at >= held[:, None]) & (at < want[:, None])
    rank = torch.cumsum(missing.flatten(), 0).reshape(n, per) - 1
    s["new_table"].copy_(torch.where(over, -1, s["table"]))
    s["new_table"][missing] = s["free"][top - 1 - rank[missing]]
    starts = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    i = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(starts[1:], i, right=True).clamp(max=n - 1)
    there = i < starts[-1]
    position = lengths[seq] + i - starts[seq]
    slot = s["new_table"][seq, (position // page).clamp(max=per - 1)].long() * page + position % page
    one = lambda x: torch.where(there, x, -1)  # noqa: E731
    return {"table": s["new_table"], "starts": starts.int(), "slots": one(slot), "positions": one(position).int(),
            "seqs": one(seq).int(), "lengths": (lengths + counts).int(), "n_free": (top - missing.sum()).int(),
            "free": s["free"]}


_PLAIN = {"prompt": _plain_prompt, "tree": _plain_tree, "accept": _plain_accept, "reserve": _plain_reserve}
_OWN = {"prompt": _own_prompt, "tree": _own_tree, "accept": _own_accept, "reserve": _own_reserve}


# -- the definitions in 64 bits ---------------------------------------------------------------------------------------

def exact(case, seed):
    """What run() returns for these inputs, one sequence at a time in 64 bits."""
    global own
    before, own = own, False  # the inputs alone: no handle of the library
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return _EXACT[case["op"]](s, case)


def _exact_prompt(s, c):
    group = c["q_heads"] // c["kv_heads"]
    out, lse = s["out"].double(), s["lse"].double()
    starts = s["starts"].tolist()
    k_starts = starts if s["k_starts"] is None else s["k_starts"].tolist()
    for q0, q1, k0, k1 in zip(starts, starts[1:], k_starts, k_starts[1:]):
        if q0 == q1:
            continue
        for i in range(c["q_heads"]):
            k, v = (s[x][k0:k1, i // group].double() for x in "kv")
            for a in range(q0, q1, 4096):  # a piece of the rows at a time
                b = min(q1, a + 4096)
                last = torch.arange(a, b, device="cuda")[:, None] - q1 + (k1 - k0)
                j = torch.arange(k1 - k0, device="cuda")
                x = s["q"][a:b, i].double() @ k.T / math.sqrt(c["dim"])
                if c["causal"]:
                    x[j > last] = -math.inf
                if c["window"]:
                    x[j <= last - c["window"]] = -math.inf
                z = torch.logsumexp(x, dim=1)
                w = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None])
                out[a:b, i] = w @ v
                lse[a:b, i] = z
    return {"out": out, "lse": lse}


def _exact_tree(s, c):
    h, page, group = c["kv_heads"], c["page"], c["q_heads"] // c["kv_heads"]
    out, lse = s["out"].double(), s["lse"].double()
    trees = s["parents"].tolist()
    for b, (n, m) in enumerate(zip(s["lengths"].tolist(), s["counts"].tolist())):
        seen = torch.zeros((m, n), dtype=torch.bool)
        for t in range(m):
            chain, a = [], t
            while a >= 0:
                chain.append(n - m + a)
                a = trees[b][a]
            chain += range(n - m - 1, -1, -1) if not c["window"] else range(n - m - 1, max(-1, n - m - 1 - c["window"]), -1)
            seen[t, chain[:c["window"] or None]] = True
        if m == 0:
            continue
        seen = seen.cuda()
        at = torch.arange(n, device="cuda")
        pg, row = s["table"][b, at // page].long(), at % page
        for i in range(h):
            k, v = (s[x][pg, i, row].double() for x in "kv")
            if c["cache"] == "e4m3":
                k, v = k * s["k_scale"][pg, i, row, None].double(), v * s["v_scale"][pg, i, row, None].double()
            for j in range(i * group, (i + 1) * group):
                x = s["q"][b, :m, j].double() @ k.T / math.sqrt(c["dim"])
                x[~seen] = -math.inf
                z = torch.logsumexp(x, dim=1)
                out[b, :m, j] = torch.exp(x - z[:, None]) @ v
                lse[b, :m, j] = z
    return {"out": out, "lse": lse}


def _exact_accept(s, c):
    pools = {n: None if s[n] is None else s[n].double() for n in ("k", "v", "k_scale", "v_scale")}
    lengths = []
    for b, (n, m) in enumerate(zip(s["lengths"].tolist(), s["counts"].tolist())):
        path = [t for t in s["path"][b].tolist() if t >= 0]
        src = torch.tensor([n - m + t for t in path], dtype=torch.long, device="cuda")
        dst = torch.arange(n - m, n - m + len(path), device="cuda")
        a, z = (s["table"][b, x // c["page"]].long() for x in (src, dst))
        for x in pools.values():
            if x is not None:
                x[z, :, dst % c["page"]] = x[a, :, src % c["page"]].clone()
        lengths.append(n - m + len(path))
    return {**pools, "lengths": torch.tensor(lengths, dtype=torch.int32)}


def _exact_reserve(s, c):
    page, table = c["page"], s["table"].tolist()
    stack, top = s["free"].tolist(), s["n_free"].item()
    lengths, counts = s["lengths"].tolist(), s["counts"].tolist()
    want = [-(-(n + m) // page) for n, m in zip(lengths, counts)]
    for row, w in zip(table, want):
        for j in range(w, len(row)):
            if row[j] >= 0:
                stack[top], row[j] = row[j], -1
                top += 1
    for row, w in zip(table, want):
        for j in range(w):
            if row[j] < 0:
                top -= 1
                row[j] = stack[top]
    slots, positions, seqs = ([-1] * s["tokens"] for _ in range(3))
    i = 0
    for b, (n, m) in enumerate(zip(lengths, counts)):
        for p in range(n, n + m):
            slots[i], positions[i], seqs[i] = table[b][p // page] * page + p % page, p, b
            i += 1
    return {"table": _ints(table), "starts": _ints([sum(counts[:b]) for b in range(len(counts) + 1)]),
            "slots": torch.tensor(slots), "positions": _ints(positions), "seqs": _ints(seqs),
            "lengths": _ints([n + m for n, m in zip(lengths, counts)]), "n_free": _ints([top]), "free": _ints(stack)}


_EXACT = {"prompt": _exact_prompt, "tree": _exact_tree, "accept": _exact_accept, "reserve": _exact_reserve}
