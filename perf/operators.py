"""What is measured of the paged key-value cache operators.

Three operators over one cache, a pool of pages whose strides the caller gives
(see include/layout_copy_cache.h):

  append   writes new tokens' keys and values into their slots, as they are or
           in E4M3 with one scale a token and head
  attend   attention of one new token a sequence over the cached slots; may
           add every slot's weight to an accumulator
  evict    keeps the slots of the largest accumulated weight and the newest
           ones, and moves their rows together at the front of the pages

Every operator has a plain form in elementary torch operations, computed in 32
bits and rounded once at the end.  `own` chooses between it and the library.
"""
import math
import random

import torch

own = False  # set by the caller: False runs the plain forms, True the library's kernels

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
FLT_MIN = 2.0 ** -126


def _case(op, **kw):
    """A case with every field set: op, seqs, q_heads, kv_heads, dim, page (slots of a page), tokens (longest
    sequence), ragged (lengths spread over 0 .. tokens, else all `tokens`), cache (element type of the pages),
    order ("head": a page holds [head, slot, dim]; "token": [slot, head, dim]), and per operator
      attend: window (0: none), mask (a quarter of the slots masked out), scores (weights are accumulated)
      append: new (most new tokens a sequence; `tokens` counts them in)
      evict:  budget (slots kept), recent (how many of them are the newest)"""
    c = dict(op=op, seqs=1, q_heads=8, kv_heads=8, dim=128, page=16, tokens=128, ragged=False, cache="bf16",
             order="head", window=0, mask=False, scores=False, new=0, budget=0, recent=0)
    c.update(kw)
    return c


def listed():
    return [
        # the first tokens of one conversation: a few slots, latency is everything
        _case("attend", name="attend_one_short", dim=64, tokens=37),
        # a small serving batch, sequences of every age, grouped heads
        _case("attend", name="attend_batch", seqs=16, q_heads=32, tokens=2048, ragged=True),
        # a full serving batch, the bulk of decoding time
        _case("attend", name="attend_full", seqs=64, q_heads=32, page=64, tokens=8192, ragged=True),
        # one long document: a single sequence has to fill the GPU
        _case("attend", name="attend_long", q_heads=32, tokens=131071, cache="fp16"),
        # one query head a key head, an odd head size, pages that are no power of two, left-out slots
        _case("attend", name="attend_mha_masked", seqs=7, q_heads=12, kv_heads=12, dim=80, page=24, tokens=1999,
              ragged=True, cache="fp16", order="token", mask=True),
        # 8-bit cache whose slots' weights are collected for eviction
        _case("attend", name="attend_e4m3_scores", seqs=32, q_heads=64, tokens=4096, ragged=True, cache="e4m3",
              page=64, scores=True),
        # all query heads on one key head, wide heads, a sliding window
        _case("attend", name="attend_mqa_window", seqs=8, q_heads=16, kv_heads=1, dim=256, page=32, tokens=5000,
              order="token", window=1024, scores=True),
        # one decoding step's new keys and values
        _case("append", name="append_step", seqs=64, tokens=4096, page=64, ragged=True, new=1),
        # prompts of several lengths enter an 8-bit cache
        _case("append", name="append_prompts_e4m3", seqs=8, tokens=4100, page=64, ragged=True, cache="e4m3",
              new=2050),
        # a few sequences just over their budget
        _case("evict", name="evict_small", seqs=4, tokens=1500, budget=1024, recent=128, scores=True),
        # a batch of long sequences is cut to a quarter
        _case("evict", name="evict_batch", seqs=16, tokens=16384, page=64, ragged=True, budget=4096, recent=256,
              scores=True),
        # one long document in an 8-bit cache, most of it let go
        _case("evict", name="evict_long_e4m3", tokens=131071, page=32, cache="e4m3", order="token", budget=32768,
              recent=1000, scores=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    """One more case over the ranges that the listed ones stand for."""
    op = rng.choice(["attend", "attend", "attend", "append", "evict"])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 12, 16])
    cache = rng.choice(["bf16", "bf16", "fp16", "e4m3"])
    c = _case(op, seqs=_log_int(rng, 1, 96), kv_heads=kv_heads, q_heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]),
              dim=rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 192, 256]),
              page=rng.choice([8, 16, 16, 24, 32, 48, 64, 64, 128]), tokens=_log_int(rng, 1, 131071),
              ragged=rng.random() < 0.7, cache=cache, order=rng.choice(["head", "token"]))
    if op == "attend":
        c["window"] = _log_int(rng, 1, c["tokens"]) if rng.random() < 0.25 else 0
        c["mask"] = rng.random() < 0.25
        c["scores"] = rng.random() < 0.4
    elif op == "append":
        c["new"] = _log_int(rng, 1, c["tokens"]) if rng.random() < 0.5 else 1
    else:
        c["scores"] = True
        c["budget"] = _log_int(rng, 1, c["tokens"])
        c["recent"] = rng.choice([0, c["budget"] // 16, c["budget"] // 4, c["budget"]])
    # the pool stays within the largest listed one's: fewer sequences first, then shorter ones
    while _pool_bytes(c) > 2.2e9:
        if c["seqs"] > 1:
            c["seqs"] = max(1, c["seqs"] * 2 // 3)
        else:
            c["tokens"] = max(1, c["tokens"] * 2 // 3)
            for k in ("window", "new", "budget"):
                c[k] = min(c[k], c["tokens"])
            c["recent"] = min(c["recent"], c["budget"])
    return c


# -- sizes ------------------------------------------------------------------------------------------------------------

def _elem(c):
    return 1 if c["cache"] == "e4m3" else 2


def _row_bytes(c):
    """Bytes of one token's row of one head, its scale included."""
    return c["dim"] * _elem(c) + (4 if c["cache"] == "e4m3" else 0)


def _pages_per_seq(c):
    return -(-c["tokens"] // c["page"])


def _pool_bytes(c):
    return 2 * c["seqs"] * _pages_per_seq(c) * c["page"] * c["kv_heads"] * _row_bytes(c)


def _lengths(c):
    """The sequences' lengths, the same for every seed up to their order; with four ragged ones or more, one is empty."""
    n, t = c["seqs"], c["tokens"]
    if not c["ragged"] or n == 1:
        return [t] * n
    got = [max(1, t * (i + 1) // n) for i in range(n)]
    if n >= 4:
        got[0] = 0
    return got


def _counts(c):
    """New tokens of each sequence of an append: all `new` for a decoding step, spread for prompts."""
    return [min(n, c["new"]) if c["new"] == 1 else min(n, max(1, c["new"] * (i + 1) // c["seqs"]))
            for i, n in enumerate(_lengths(c))]


def work(case):
    c = case
    lens, h, d, row = _lengths(c), c["kv_heads"], c["dim"], _row_bytes(c)
    if c["op"] == "append":
        n = sum(_counts(c))
        return {"bytes": n * h * 2 * (2 * d + row) + 8 * c["seqs"], "flops": n * h * d * 4 if c["cache"] == "e4m3" else 0}
    if c["op"] == "evict":
        # rows that stay where they are need no move; of n slots of which m are kept, a row other than the `recent` newest
        # keeps its place only at the front: all but a few move
        kept = [min(n, c["budget"]) for n in lens]
        moved = sum(m for n, m in zip(lens, kept) if n > m)
        cap = _pages_per_seq(c) * c["page"]
        return {"bytes": moved * h * 2 * 2 * row + h * (4 * sum(lens) + 4 * cap * c["seqs"] + 4 * c["budget"] * c["seqs"]),
                "flops": 0}
    seen = sum(min(n, c["window"]) if c["window"] else n for n in lens) * (0.75 if c["mask"] else 1.0)
    io = c["seqs"] * c["q_heads"] * (2 * 2 * d + 4)
    slots = sum(min(n, c["window"]) if c["window"] else n for n in lens)
    return {"bytes": seen * h * 2 * row + io + (slots if c["mask"] else 0) + (seen * h * 8 if c["scores"] else 0),
            "flops": seen * c["q_heads"] * d * 4}


# -- inputs -----------------------------------------------------------------------------------------------------------

def _pool(c, n_pages, g, dev):
    """A pool of pages, [page, head, slot, dim] whatever their order in memory, of unit normal values."""
    shape = (n_pages, c["kv_heads"], c["page"], c["dim"]) if c["order"] == "head" else \
            (n_pages, c["page"], c["kv_heads"], c["dim"])
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
    scale = None
    if c["cache"] == "e4m3":
        # rows whose largest value is near E4M3's, as quantised rows are
        x = (x * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        scale = 0.008 + 0.004 * torch.rand(shape[:3], generator=g, device=dev)
    else:
        x = x.to(DTYPE[c["cache"]])
    if c["order"] == "token":
        x = x.transpose(1, 2)
        scale = None if scale is None else scale.transpose(1, 2)
    return x, scale


def prepare(case, seed):
    """Pool, page table (pages in any order, -1 where a sequence has none), lengths, the step's inputs, and the cache
    handle that a serving program makes once."""
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    host = random.Random(seed)
    n_seq, per, page, h, d = c["seqs"], _pages_per_seq(c), c["page"], c["kv_heads"], c["dim"]
    n_pages = n_seq * per + 1
    k, k_scale = _pool(c, n_pages, g, dev)
    v, v_scale = _pool(c, n_pages, g, dev)
    order = list(range(n_seq))
    host.shuffle(order)
    lens = torch.tensor([_lengths(c)[i] for i in order], dtype=torch.int32, device=dev)
    table = torch.randperm(n_pages, generator=g, device=dev)[:n_seq * per].reshape(n_seq, per).to(torch.int32)
    used = torch.arange(per, device=dev)[None, :] * page < lens[:, None]
    table = torch.where(used, table, -1).contiguous()
    s = dict(case=c, k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table, lengths=lens)
    io = torch.float16 if c["cache"] == "fp16" else torch.bfloat16
    cap = per * page
    if c["op"] == "attend":
        s["q"] = (1.5 * torch.randn((n_seq, c["q_heads"], d), generator=g, device=dev)).to(io)
        s["mask"] = torch.rand((n_seq, cap), generator=g, device=dev) < 0.75 if c["mask"] else None
        s["scores"] = torch.rand((n_seq, h, cap), generator=g, device=dev) if c["scores"] else None
        # what earlier owners left past a sequence's end has to be harmless
        last = torch.clamp(lens.long() - 1, min=0)
        tail = torch.arange(page, device=dev)[None, :] > (last % page)[:, None]
        at = table.gather(1, (last // page)[:, None])[:, 0].clamp(min=0).long()
        if c["cache"] != "e4m3":
            for x in (k, v):
                rows = x[at].transpose(1, 2)
                rows[tail & (lens > 0)[:, None]] = float("nan")
                x[at[lens > 0]] = rows.transpose(1, 2)[lens > 0]
    elif c["op"] == "append":
        n = [_counts(c)[i] for i in order]
        s["counts"] = torch.tensor(n, dtype=torch.int32, device=dev)
        s["lengths"] = lens - s["counts"]  # the table has room for the new tokens
        s["new_k"], s["new_v"] = (torch.randn((n_seq, c["new"], h, d), generator=g, device=dev).to(io) for _ in "kv")
    else:
        # weights gathered over many steps: a few slots have most of them, many have none at all
        x = torch.exp(2.0 * torch.randn((n_seq, h, cap), generator=g, device=dev) - 3.0)
        x = torch.where(torch.rand((n_seq, h, cap), generator=g, device=dev) < 0.2, torch.zeros_like(x), x)
        s["scores"] = torch.where(torch.arange(cap, device=dev) < lens[:, None, None], x, 0.0)
    if own:
        import movement_primitives_gb300 as lc
        s["cache"] = lc.PagedCache(k, v, table, k_scale, v_scale)
    return s


# -- the operators ----------------------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _OWN[c["op"]](state, c)
    return _PLAIN[c["op"]](state, c)


def _own_attend(s, c):
    import movement_primitives_gb300 as lc
    lse = torch.empty((c["seqs"], c["q_heads"]), dtype=torch.float32, device="cuda")
    out = lc.cache_attend(s["cache"], s["q"], s["lengths"], window=c["window"], mask=s["mask"], lse=lse,
                          scores=s["scores"])
    return {"out": out, "lse": lse, "scores": s["scores"]}


def _own_append(s, c):
    import movement_primitives_gb300 as lc
    lengths = lc.cache_append(s["cache"], s["new_k"], s["new_v"], s["lengths"], s["counts"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "lengths": lengths}


def _own_evict(s, c):
    import movement_primitives_gb300 as lc
    kept, scores, lengths = lc.cache_evict(s["cache"], s["lengths"], s["scores"], c["budget"], c["recent"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "kept": kept,
            "scores": scores, "lengths": lengths}


def _gather(pool, scale, table):
    """[seq, head, slot, dim] in 32 bits of the pages of each sequence."""
    at = table.clamp(min=0).long()
    x = pool[at].transpose(1, 2).flatten(2, 3).float()
    return x if scale is None else x * scale[at].transpose(1, 2).flatten(2, 3)[..., None]


def _plain_attend(s, c):
    n_seq, h, d = c["seqs"], c["kv_heads"], c["dim"]
    k, v = _gather(s["k"], s["k_scale"], s["table"]), _gather(s["v"], s["v_scale"], s["table"])
    slot = torch.arange(k.shape[2], device=k.device)[None, :]
    seen = slot < s["lengths"][:, None]
    if c["window"]:
        seen = seen & (slot >= s["lengths"][:, None] - c["window"])
    if s["mask"] is not None:
        seen = seen & s["mask"]
    q = s["q"].float().reshape(n_seq, h, c["q_heads"] // h, d)
    x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = torch.where(seen[:, None, None, :], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)  # a row with nothing to see: weights of zero
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    w = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(w, torch.where(seen[:, None, :, None], v, 0.0))
    if s["scores"] is not None:
        s["scores"] += w.sum(2)
    return {"out": out.reshape(n_seq, c["q_heads"], d).to(s["q"].dtype),
            "lse": (top + torch.log(total)).reshape(n_seq, c["q_heads"]), "scores": s["scores"]}


def _quantise(x):
    """E4M3 values and their scale a row: the largest magnitude goes to 448; a row with an infinity or NaN gets the scale NaN."""
    top = x.abs().amax(-1)
    scale = torch.where(torch.isfinite(top), torch.clamp(top / E4M3_MAX, min=FLT_MIN), math.nan)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _plain_append(s, c):
    t = torch.arange(c["new"], device="cuda")
    new = t[None, :] < s["counts"][:, None]
    slot = s["lengths"][:, None].long() + t
    seq, tok = torch.nonzero(new, as_tuple=True)
    at = slot[seq, tok]
    page, row = s["table"][seq, at // c["page"]].long(), at % c["page"]
    for name in "kv":
        x = s["new_" + name][seq, tok]  # [token, head, dim]
        if c["cache"] == "e4m3":
            x, scale = _quantise(x.float())
            s[name + "_scale"][page, :, row] = scale
            s[name].view(torch.uint8)[page, :, row] = x.view(torch.uint8)
        else:
            s[name][page, :, row] = x
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"],
            "lengths": s["lengths"] + s["counts"]}


def _plain_evict(s, c):
    n_seq, h, cap = s["scores"].shape
    budget, recent = c["budget"], c["recent"]
    n = s["lengths"][:, None, None]
    slot = torch.arange(cap, device="cuda")
    # what is certain to stay outranks every score, what is past the end comes last
    rank = torch.where(slot >= n, -math.inf, torch.where((slot >= n - recent) | (n <= budget), math.inf, s["scores"]))
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    new_n = torch.clamp(n, max=budget)
    r = torch.arange(first.shape[-1], device="cuda")
    kept = torch.sort(torch.where(r < new_n, first, cap), dim=-1).values  # in their old order
    seq, head, to = torch.nonzero(r < new_n.expand(n_seq, h, 1), as_tuple=True)
    src = kept[seq, head, to]
    page_from, page_to = (s["table"][seq, x // c["page"]].long() for x in (src, to))
    for x in (s["k"], s["v"], s["k_scale"], s["v_scale"]):
        if x is not None:
            x = x.view(torch.uint8) if c["cache"] == "e4m3" and x.dim() == 4 else x
            x[page_to, head, to % c["page"]] = x[page_from, head, src % c["page"]]
    scores = torch.zeros_like(s["scores"])
    scores[seq, head, to] = s["scores"][seq, head, src]
    out = torch.full((n_seq, h, budget), -1, dtype=torch.int32, device="cuda")
    out[seq, head, to] = src.to(torch.int32)
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "kept": out,
            "scores": scores, "lengths": new_n[:, 0, 0]}


_PLAIN = {"attend": _plain_attend, "append": _plain_append, "evict": _plain_evict}
_OWN = {"attend": _own_attend, "append": _own_append, "evict": _own_evict}


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


def _exact_attend(s, c):
    h, d, page = c["kv_heads"], c["dim"], c["page"]
    group = c["q_heads"] // h
    out = torch.zeros((c["seqs"], c["q_heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["seqs"], c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    scores = None if s["scores"] is None else s["scores"].double()
    for b, n in enumerate(s["lengths"].tolist()):
        at = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device="cuda")
        if s["mask"] is not None:
            at = at[s["mask"][b, at]]
        if at.numel() == 0:
            continue
        pg, row = s["table"][b, at // page].long(), at % page
        for i in range(h):
            k, v = (x[pg, i, row].double() for x in (s["k"], s["v"]))
            if c["cache"] == "e4m3":
                k, v = k * s["k_scale"][pg, i, row, None].double(), v * s["v_scale"][pg, i, row, None].double()
            x = s["q"][b, i * group:(i + 1) * group].double() @ k.T / math.sqrt(d)
            z = torch.logsumexp(x, dim=1)
            w = torch.exp(x - z[:, None])
            out[b, i * group:(i + 1) * group] = w @ v
            lse[b, i * group:(i + 1) * group] = z
            if scores is not None:
                scores[b, i, at] += w.sum(0)
    return {"out": out, "lse": lse, "scores": scores}


def _exact_append(s, c):
    pools = {n: None if s[n] is None else s[n].double() for n in ("k", "v", "k_scale", "v_scale")}
    for b, (n, m) in enumerate(zip(s["lengths"].tolist(), s["counts"].tolist())):
        at = torch.arange(n, n + m, device="cuda")
        pg, row = s["table"][b, at // c["page"]].long(), at % c["page"]
        for name in "kv":
            x = s["new_" + name][b, :m].double()
            if c["cache"] == "e4m3":
                scale = x.abs().amax(-1) / E4M3_MAX
                pools[name + "_scale"][pg, :, row] = scale
                x = x / scale[..., None]
                # three bits after the leading one, down to steps of 2^-9
                step = torch.exp2(torch.clamp(torch.floor(torch.log2(x.abs())), min=-6.0) - 3.0)
                x = torch.round(x / step) * step
            pools[name][pg, :, row] = x
    return {**pools, "lengths": s["lengths"] + s["counts"]}


def _exact_evict(s, c):
    pools = {n: None if s[n] is None else s[n].double() for n in ("k", "v", "k_scale", "v_scale")}
    lens = s["lengths"].tolist()
    kept_all = torch.full((c["seqs"], c["kv_heads"], c["budget"]), -1, dtype=torch.int32, device="cuda")
    scores = torch.zeros(s["scores"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        m = min(n, c["budget"])
        for i in range(c["kv_heads"]):
            old = s["scores"][b, i, :n].double()
            if n > m:
                head = n - c["recent"]
                best = torch.argsort(-old[:head], stable=True)[:m - c["recent"]]
                kept = torch.cat([torch.sort(best).values, torch.arange(head, n, device="cuda")])
            else:
                kept = torch.arange(n, device="cuda")
            to = torch.arange(m, device="cuda")
            kept_all[b, i, :m] = kept.to(torch.int32)
            scores[b, i, :m] = old[kept]
            src, dst = (s["table"][b, x // c["page"]].long() for x in (kept, to))
            for x in pools.values():
                if x is not None:
                    x[dst, i, to % c["page"]] = x[src, i, kept % c["page"]].clone()
    return {**pools, "kept": kept_all, "scores": scores,
            "lengths": torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32)}


_EXACT = {"attend": _exact_attend, "append": _exact_append, "evict": _exact_evict}
