"""Paged key-value cache operators on the GPU: what their results may not depend on, and how near they come.

Cases beside those of ``test_gpu_cache.py``, whose caches and checks they use.
"""
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

from test_gpu_cache import IO, Setup, attend, check_attend, check_evict, lc, no_device_error  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("group", [1, 7, 16])
def test_weights_of_a_unit_over_a_cluster_repeat(kind, group):
    """Few units of some hundred slots: a cluster of blocks each, every block forms every row's log sum
    once.  Outputs, log sums and weights are the same bits each time."""
    s = Setup([700, 333, 0, 40], heads=2, dim=128, kind=kind, page=16, seed=group)
    q, out, lse, _ = attend(s, 2 * group, scores=True)
    first = torch.zeros((4, 2, s.cap), device="cuda")
    lc().cache_attend(s.cache, q, s.lengths, scores=first)
    for _ in range(20):
        again, logs = torch.zeros_like(first), torch.zeros_like(lse)
        assert torch.equal(lc().cache_attend(s.cache, q, s.lengths, scores=again, lse=logs), out)
        assert torch.equal(again, first) and torch.equal(logs, lse)


# What a result may be off by (U_OUT: rounding to the output's type; U_WEIGHT: what a weight of the second product may
# be off by, relatively).  16-bit caches: a weight is the sum of two numbers of the cache's type, its rounding (off by at
# most u = 2^-8 in bfloat16, 2^-11 in float16) and the rounding of the rest, so u^2 (with the leading bits as the first
# one: a rest below 2^-7 of the weight's power of two, rounded by half a step of at most 2^-15 of that, the same);
# float16's smallest step, 2^-24 beside a largest weight of 2^14, adds half of it a slot.  E4M3 caches: one float16 number, 2^-11; the scale's logarithm
# adds 2^-18 (2^-22 of at most 8, times ln 2 and a rounding), and the queries' conversion to float16 2^-25 of the
# head's largest element an element.
U_OUT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "e4m3": 2.0 ** -8}
U_WEIGHT = {"bf16": 2.0 ** -16, "fp16": 2.0 ** -22, "e4m3": 2.0 ** -11 + 2.0 ** -18}


def check_close(s, q, out, window=0, mask=None):
    scale = 1 / math.sqrt(s.dim)
    k, v = s.values()
    qn, n = q.double().cpu().numpy(), s.lengths.cpu().numpy()
    want, _, _, mag, reach = oc.attend(qn, k, v, s.table.cpu().numpy(), n, scale, window,
                                       None if mask is None else mask.cpu().numpy())
    err = (s.dim + 8) * 2.0 ** -24 * reach
    if s.kind == "e4m3":
        err = err + 2.0 ** -25 * scale * np.abs(qn).max(2) * np.abs(k).sum(3).max()
    rel = 2 * err + (n.max() / 8 + 8) * 2.0 ** -23
    off = mag * (U_WEIGHT[s.kind] + rel[..., None])
    if s.kind == "fp16":
        off = off + 2.0 ** -39 * n.max() * np.abs(v).max()
    got = out.double().cpu().numpy()
    tiny = {"fp16": 2.0 ** -25}.get(s.kind, 2.0 ** -134)  # half of the output's smallest step
    worst = (np.abs(got - want) - (off + U_OUT[s.kind] * (np.abs(want) + off) + tiny)).max()
    assert worst <= 0, worst


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("dim,group", [(64, 1), (80, 5), (128, 4), (128, 16), (192, 12), (256, 8), (256, 16), (33, 3)])
def test_attend_is_as_near_as_its_output_type_allows(kind, dim, group):
    """Every form: a block, a cluster or a warp a unit, and runs that are joined; a few slots and many."""
    for lens, heads in (([2, 3, 5, 17, 40, 0, 300], 3), ([(5 * i) % 67 for i in range(211)], 3),
                        ([2100, 35, 0, 1051], 12)):
        s = Setup(lens, heads=heads, dim=dim, kind=kind, page=16, seed=dim + group)
        q = s.queries(heads * group)
        check_close(s, q, lc().cache_attend(s.cache, q, s.lengths))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
def test_log_sums_keep_their_digits(kind):
    """One slot's log sum is its logit, that of n equal ones log n more: within a few of float32's steps there."""
    for n in (1, 2, 33, 700, 20000):
        s = Setup([n], heads=1, dim=64, kind=kind, page=64, seed=n)
        q = s.queries(2)
        k = s.k.view(torch.uint8) if kind == "e4m3" else s.k
        k.copy_(k[int(s.table[0, 0]), 0, 0].clone().expand_as(k))
        if kind == "e4m3":
            s.scales[0].fill_(0.01)
        lse = torch.empty((1, 2), device="cuda")
        lc().cache_attend(s.cache, q, s.lengths, lse=lse)
        _, want, _, _, reach = oc.attend(q.double().cpu().numpy(), *s.values(), s.table.cpu().numpy(), [n], 0.125)
        # the logit's sum of 64 products, twice (as it is and base 2), the sum of n weights, three roundings of the result
        bound = 2.0 ** -24 * (72 * reach + 2 * (n / 128 + 8) + 3 * np.abs(want) + 3 * math.log(n + 1))
        if kind == "e4m3":
            bound = bound + 2.0 ** -25 * 0.125 * np.abs(q.double().cpu().numpy()).max(2) * 448 * 64 * 0.01
        assert np.all(np.abs(lse.double().cpu().numpy() - want) <= bound), (n, lse.tolist(), want, bound)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("lens,heads,dim", [([1, 2, 30], 2, 64), ([700, 90], 2, 128), ([(5 * i) % 67 for i in range(211)], 3, 64),
                                            ([4200, 35, 1], 12, 64), ([20, 90], 2, 33)])
def test_values_near_the_largest_number(kind, lens, heads, dim):
    """The average of many of the type's largest values is no larger than they are, their sum past float32."""
    s = Setup(lens, heads=heads, dim=dim, kind=kind, page=16, seed=dim)
    sign = torch.where(torch.arange(dim, device="cuda") % 3 == 0, -1.0, 1.0)
    if kind == "e4m3":
        s.v.view(torch.uint8).copy_((448 * sign).to(torch.float8_e4m3fn).view(torch.uint8).expand_as(s.v))
        s.scales[1].fill_(2.0 ** 119)  # 448 * 2^119 = 0.875 * 2^128
    else:
        s.v.copy_((torch.finfo(IO[kind]).max * sign).to(IO[kind]).expand_as(s.v))
    q = s.queries(2 * heads)
    out = lc().cache_attend(s.cache, q, s.lengths)
    assert torch.all(out.isfinite())
    check_close(s, q, out)
    no_device_error()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,heads,dim", [([1, 2, 30], 2, 64), ([700, 1], 2, 128), ([4200, 35, 1], 12, 64), ([20, 1], 2, 33)])
def test_an_infinite_value_in_a_seen_slot_stays_infinite(kind, lens, heads, dim):
    """Weights that are whole in the cache's type (one slot's is 1) and weights that are not."""
    s = Setup(lens, heads=heads, dim=dim, kind=kind, page=16, seed=dim)
    for b in range(s.n_seq):
        page = int(s.table[b, 0])
        s.v[page, :, 0, 3], s.v[page, :, 0, 7] = math.inf, -math.inf
    q = s.queries(2 * heads) * 0.25  # no weight below 2^-38 of the largest
    q = q.to(IO[kind])
    out = lc().cache_attend(s.cache, q, s.lengths).float()
    assert torch.all(out[..., 3] == math.inf) and torch.all(out[..., 7] == -math.inf)
    rest = [c for c in range(dim) if c not in (3, 7)]
    assert torch.all(out[..., rest].isfinite())
    no_device_error()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("lens,heads,group,dim", [([40, 25], 2, 4, 64),                        # a block or a warp a unit
                                                  ([700, 90], 2, 4, 128),                      # a cluster a unit
                                                  ([(5 * i) % 67 for i in range(211)], 3, 2, 64),  # a warp a unit
                                                  ([4200, 35, 0, 2101], 12, 3, 64),            # runs
                                                  ([150, 60], 2, 20, 64),                      # units that share scores
                                                  ([90, 60], 2, 2, 33)])                       # rows by elements
def test_a_nan_row_adds_nothing_to_slots_it_does_not_see(kind, lens, heads, group, dim):
    """A query that is NaN makes its row and its seen slots' weights NaN, and no other slot's."""
    s = Setup(lens, heads=heads, dim=dim, kind=kind, page=16, seed=dim)
    q = s.queries(heads * group)
    b = max(range(s.n_seq), key=lambda i: lens[i])
    q[b, group, 1] = math.nan  # the first query head of key head 1
    mask = (torch.rand((s.n_seq, s.cap), generator=s.g) < 0.5).cuda()
    before = torch.rand((s.n_seq, heads, s.cap), generator=s.g).cuda()
    scores = before.clone()
    out = lc().cache_attend(s.cache, q, s.lengths, mask=mask, scores=scores)
    seen = mask & (torch.arange(s.cap, device="cuda") < s.lengths[:, None])
    assert torch.all(torch.isnan(out[b, group])) and int(torch.isnan(out).any(2).sum()) == 1
    assert torch.equal(scores.isnan().any(2).nonzero(), torch.tensor([[b, 1]], device="cuda"))
    assert torch.all(scores[b, 1].isnan() == seen[b])
    unseen = ~seen[:, None].expand_as(scores)
    assert torch.equal(scores[unseen], before[unseen])
    no_device_error()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,heads,group,dim", [([40, 25], 2, 4, 64), ([700, 90], 2, 16, 128),
                                                  ([(5 * i) % 67 for i in range(211)], 3, 2, 64),
                                                  ([4200, 35, 0, 2101], 12, 3, 64), ([150, 60], 2, 20, 64), ([90, 60], 2, 2, 33)])
def test_attend_into_the_queries_own_buffer_or_beside_it(kind, lens, heads, group, dim):
    """Every form may write its rows where the queries were, or between them."""
    s = Setup(lens, heads=heads, dim=dim, kind=kind, page=16, seed=dim)
    q = s.queries(heads * group)
    want = lc().cache_attend(s.cache, q, s.lengths)
    both = torch.stack([q, torch.zeros_like(q)], 2)
    got = lc().cache_attend(s.cache, both[:, :, 0], s.lengths, out=both[:, :, 1])
    assert torch.equal(got, want) and torch.equal(both[:, :, 0], q)
    assert torch.equal(lc().cache_attend(s.cache, q, s.lengths, out=q), want)
    no_device_error()


ASCENDING = """
import sys
sys.path[:0] = [%r, %r]
import torch
from test_gpu_cache import Setup, check_evict
for dim in (130, 136, 192, 255, 256, 64):
    s = Setup([8300, 40, 4099], heads=2, dim=dim, kind=%r, page=64, seed=dim)
    check_evict(s, torch.rand((3, 2, s.cap), generator=s.g).cuda(), 150, 10)
"""


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_evict_head_sizes_one_after_the_other(kind):
    """Two-launch evictions of growing rows in a process of their own: a small one may not limit a later one."""
    code = ASCENDING % (os.path.join(ROOT, "tests"), ROOT, kind)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_evict_between_interleaved_halves_of_one_buffer():
    """Scores and new scores whose ranges meet, but not their rows."""
    for heads_first in (False, True):
        s = Setup([100, 60], heads=3, dim=64, seed=2)
        both = torch.rand((2, 2, 3, s.cap) if heads_first else (2, 3, 2, s.cap), generator=s.g).cuda()
        old, new = (both[:, i] if heads_first else both[:, :, i] for i in range(2))
        check_evict(s, old, 37, 6, new_scores=new)


# ---------------------------------------------------------------------------
# append: the forms that long prompts take
# ---------------------------------------------------------------------------

E4M3 = torch.tensor([oc.e4m3_value(c) if c & 127 != 127 else math.nan for c in range(256)], dtype=torch.float64)


def quantised(x):
    """(values as multiples of the scale, scale) of rows x [..., dim] in 16 bits: oracle.cache.quantise of many rows."""
    x = x.double()
    top = x.abs().amax(-1)
    scale = torch.where(top.isfinite(), (top / 448).float().clamp(min=2.0 ** -126), math.nan).double()
    y = (x / scale[..., None]).float().double()  # the float32 quotient: 53 bits are enough to round twice
    e = torch.frexp(y.abs())[1].clamp(min=-5) - 1
    step = (e.long() - 3 + 1023 << 52).view(torch.float64)  # 2^(e - 3)
    return torch.copysign(((y.abs() / step).round() * step).clamp(max=448.0), y), scale


@pytest.mark.parametrize("device", ["cpu", "cuda"])
def test_the_vectorised_quantiser_is_the_oracle(device):
    g = torch.Generator().manual_seed(0)
    x = torch.randn((40, 24), generator=g) * torch.exp(4 * torch.randn((40, 1), generator=g))
    x[3], x[4, 2], x[5, 7], x[6] = 0, math.inf, math.nan, x[6] * 1e-38
    x = x.bfloat16()
    values, scale = (y.cpu().numpy() for y in quantised(x.to(device)))
    for row, v, sc in zip(x.float().numpy(), values, scale):
        want, want_scale = oc.quantise(row)
        assert np.array_equal(np.float32(sc), want_scale, equal_nan=True)
        if not np.isnan(sc):
            assert np.array_equal(v, want)


FOUR = 4 * 152 * 48  # rows from which a warp takes several heads; from twice that of up to eight
PROMPTS = [(1, 64, FOUR + 40), (2, 128, FOUR + 40), (3, 256, FOUR), (3, 72, FOUR + 9), (4, 64, 2 * FOUR),
           (4, 128, 2 * FOUR + 8), (5, 72, 2 * FOUR + 35), (5, 64, 2 * FOUR + 5), (5, 128, FOUR - 5), (7, 136, FOUR + 49),
           (7, 128, 2 * FOUR + 21), (8, 192, FOUR), (8, 64, 2 * FOUR), (8, 128, FOUR), (12, 256, 2 * FOUR),
           (12, 72, 2 * FOUR + 48), (12, 64, FOUR + 24), (7, 8, FOUR + 49)]


@pytest.mark.parametrize("kind,io,every", [("e4m3", "bf16", 1), ("e4m3", "fp16", 3), ("bf16", "bf16", 4), ("fp16", "fp16", 5)])
def test_append_long_prompts(kind, io, every):
    """Rows enough that a warp takes several heads: odd numbers of heads, lanes past a row's end, ragged counts,
    rows that are not finite or whose magnitudes divide."""
    for i, (heads, dim, rows) in enumerate(PROMPTS[::every]):
        n_new = rows // heads // 2
        s = Setup([3, 0], heads=heads, dim=dim, per=-(-(n_new + 3) // 64), page=64, kind=kind, seed=rows,
                  order="token" if i % 2 else "head")
        g = torch.Generator(device="cuda").manual_seed(rows)
        new = [(3 * torch.randn((2, n_new, heads, dim), generator=g, device="cuda")).to(IO[io]) for _ in "kv"]
        h = heads - 1
        new[0][0, 1, h, dim - 1], new[1][0, 2, 0, 0], new[0][1, 3, h, 0] = math.inf, math.nan, -math.inf
        new[0][0, 4, h] = 0
        if io == "bf16":
            for t, power in ((5, 100), (6, -91), (7, -126), (8, -133), (9, 126), (10, -90), (11, 90)):
                new[t % 2][0, t, h] *= 2.0 ** power
            new[1][1, 12, 0] = 2.0 ** -90  # the division's side of the bounds, and the other
            new[1][1, 13, 0] = 2.0 ** 90
        counts = torch.tensor([n_new, n_new - 37], dtype=torch.int32, device="cuda")
        before = [x.clone() for x in (s.k.view(torch.uint8), s.v.view(torch.uint8))] if kind == "e4m3" else \
                 [s.k.clone(), s.v.clone()]
        old_scales = [None if x is None else x.clone() for x in s.scales]
        got_n = lc().cache_append(s.cache, new[0], new[1], s.lengths, counts)
        assert got_n.tolist() == [3 + n_new, n_new - 37]
        t = torch.arange(n_new, device="cuda")
        seq, tok = torch.nonzero(t[None] < counts[:, None], as_tuple=True)
        at = s.lengths.long()[seq] + tok
        page, row = s.table[seq, at // 64].long(), at % 64
        for x, pool, old, scales, old_scale in zip(new, (s.k, s.v), before, s.scales, old_scales):
            if kind != "e4m3":
                old[page, :, row] = x[seq, tok]
                assert torch.equal(pool.contiguous().view(torch.int16), old.contiguous().view(torch.int16)), (heads, dim, rows)
                continue
            values, scale = quantised(x[seq, tok])
            codes = pool.view(torch.uint8)
            got = E4M3.cuda()[codes[page, :, row].long()]
            bad = scale.isnan()[..., None]
            assert torch.equal(torch.where(bad, 0, got), torch.where(bad, 0, values)), (heads, dim, rows)
            assert torch.equal(scales[page, :, row].nan_to_num(-1.0), scale.float().nan_to_num(-1.0))
            # nothing else is written
            old[page, :, row], old_scale[page, :, row] = codes[page, :, row], scales[page, :, row]
            assert torch.equal(codes, old)
            assert torch.equal(scales.nan_to_num(-1.0), old_scale.nan_to_num(-1.0))
        no_device_error()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def calls(s):
    """Every operator on this cache, by name."""
    q = s.queries(2 * s.heads)
    new = torch.zeros((s.n_seq, 1, s.heads, s.dim), dtype=IO[s.kind], device="cuda")
    scores = torch.zeros((s.n_seq, s.heads, s.cap), device="cuda")
    zero = torch.zeros_like(s.lengths)
    return {"append": lambda **kw: lc().cache_append(s.cache, **{**dict(k=new, v=new, lengths=zero), **kw}),
            "attend": lambda **kw: lc().cache_attend(s.cache, **{**dict(q=q, lengths=s.lengths), **kw}),
            "evict": lambda **kw: lc().cache_evict(s.cache, **{**dict(lengths=s.lengths, scores=scores, budget=4), **kw})}


def test_another_current_device_is_refused(monkeypatch):
    """The library launches on the current device: a cache elsewhere is refused before anything is allocated."""
    s = Setup([10, 20], heads=2, dim=64)
    ops = calls(s)
    for op in ops.values():
        op()
    from movement_primitives_gb300 import cache as module
    monkeypatch.setattr(module, "_DEVICE", lambda: s.k.device.index + 1)
    for name, op in ops.items():
        with pytest.raises(ValueError, match="device"):
            op()


def test_inputs_that_want_a_gradient_are_refused():
    """No operator here has a backward pass: an output without a gradient would not say so."""
    s = Setup([10, 20], heads=2, dim=64)
    ops = calls(s)
    q = s.queries(4).requires_grad_()
    new = torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    for name, args in (("attend", dict(q=q)), ("append", dict(k=new)), ("append", dict(v=new))):
        with pytest.raises(ValueError, match="gradient"):
            ops[name](**args)
        with torch.no_grad():
            ops[name](**args)


def test_streams_without_the_raw_binding(monkeypatch):
    """Where torch has no raw stream handle, the stream object's is used."""
    from movement_primitives_gb300 import cache as module
    s = Setup([10, 20], heads=2, dim=64)
    q = s.queries(4)
    want = lc().cache_attend(s.cache, q, s.lengths)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    for name in ("_TYPES", "_CURRENT"):
        monkeypatch.setattr(module, name, None)
    module._types()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lc().cache_attend(s.cache, q, s.lengths)
        assert module._CURRENT(s.cache._index) == side.cuda_stream
    side.synchronize()
    assert torch.equal(got, want)


LATE = """
import os, sys
os.environ["LC_WAIT_TIMEOUT_NS"] = "1"
sys.path[:0] = [%r, %r]
import torch
from test_gpu_cache import Setup, lc, no_device_error
n, cut, heads, dim = 20000, 40, 8, 64
s = Setup([n] * 3, heads=heads, dim=dim, kind=%r, page=64, seed=1)
other = Setup([700, 90], heads=2, dim=64, seed=2)
q = other.queries(4)
want = lc().cache_attend(other.cache, q, other.lengths)
no_device_error()
scores = torch.rand((3, heads, s.cap), generator=s.g).cuda()

def rows(p):  # [sequence, head, slot, bytes]
    p = p[s.table.long()].transpose(1, 2).flatten(2, 3).contiguous()
    return (p[..., None] if p.dim() == 3 else p).view(torch.uint8)

pools = [s.k, s.v] + [x for x in s.scales if x is not None]
before = [rows(p) for p in pools]
kept, new_scores, lengths = lc().cache_evict(s.cache, s.lengths, scores, n - cut)
status, _ = lc().last_device_error()
assert status == lc().STATUS["LC_ERR_TIMEOUT"], status
assert lengths.tolist() == [n - cut] * 3
chosen = scores[:, :, :n].topk(n - cut).indices.sort(-1).values
assert torch.equal(kept.long(), chosen)
assert torch.equal(new_scores[:, :, :n - cut], scores.gather(2, chosen))
moved = stayed = None
for pool, old in zip(pools, before):
    now = rows(pool)
    to = old.gather(2, kept.long()[..., None].expand(-1, -1, -1, old.shape[3]))
    by32 = lambda x: x.flatten(2)[:, :, :(n - cut) // 32 * 32 * old.shape[3]].unflatten(2, (-1, 32 * old.shape[3])).all(3)
    m, t = by32(now[:, :, :n - cut] == to), by32(now[:, :, :n - cut] == old[:, :, :n - cut])
    assert torch.equal(now[:, :, n - cut:], old[:, :, n - cut:])
    moved, stayed = (m, t) if moved is None else (moved & m, stayed & t)
assert torch.all(moved | stayed)  # thirty-two slots as one, in every pool
assert not torch.all(moved) and torch.any(moved & ~stayed)
no_device_error()  # reading it cleared it
assert torch.equal(lc().cache_attend(other.cache, q, other.lengths), want)
lc().cache_evict(other.cache, other.lengths, torch.zeros((2, 2, other.cap), device="cuda"), 700)
no_device_error()
"""


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_evict_waits_that_run_out(kind):
    """A limit of a nanosecond, in a process of its own: an ordinary eviction gives up where a lower chunk has not been
    read yet (thousands of the 15 thousand chunks do here).  The error word says so, the slots of a chunk that gave up
    are as they were, and what comes after runs as ever."""
    code = LATE % (os.path.join(ROOT, "tests"), ROOT, kind)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
