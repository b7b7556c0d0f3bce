"""Attention of drafted trees over the paged cache on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic: a logit is a float32 sum of d exact products, off
by at most E = (d + 8) 2^-24 |scale| sum|q||k|; a weight is off by a factor of
exp(2E), by the exponential and by the sum of n of them, (n / 8 + 8) 2^-23.  Weights
of 16-bit caches are two numbers of the type: 2^-16 (bfloat16), 2^-22 (float16) of sum
w|v|; those of E4M3 caches one float16: 2^-11, and the queries' elements below 2^-17 of
their row's largest are off by 2^-25 of it.  float16 numbers below 2^-14 are off
by 2^-25, and the weights are lifted by 2^8: n 2^-32 max|v| more.  The result is rounded once.
"""
import math

import numpy as np
import pytest

from oracle import drafts as od
from test_gpu_cache import IO, Setup, device_error_is, lc, no_device_error

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp16", "e4m3"]
WEIGHT = {"bf16": 2.0 ** -16, "fp16": 2.0 ** -22, "e4m3": 2.0 ** -11}
OUT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "e4m3": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def ints(x):
    return torch.tensor(np.array(x), dtype=torch.int32, device="cuda")


def trees(n_seqs, drafts, g, kind="random"):
    if kind == "chain":
        one = torch.arange(-1, drafts - 1)
        return one.repeat(n_seqs, 1).to(torch.int32).cuda()
    rows = [[int(torch.randint(-1, t, (1,), generator=g)) if t else -1 for t in range(drafts)] for _ in range(n_seqs)]
    return torch.tensor(rows, dtype=torch.int32).reshape(n_seqs, drafts).cuda()


def check(s, q, lengths, parents, counts, out, lse, scale=None, window=0, table=None):
    """`out` and `lse` hold 7 where nothing was written."""
    scale = 1 / math.sqrt(s.dim) if scale is None else scale
    k, v = s.values()
    f = q.double().cpu().numpy()
    want, want_lse, mag, reach, real = od.attend(
        f, k, v, (s.table if table is None else table).cpu().numpy(), lengths.cpu().numpy(),
        None if counts is None else counts.cpu().numpy(), parents.cpu().numpy(), scale, window)
    n = min(int(lengths.max()) if lengths.numel() else 0, s.cap)
    err = (s.dim + 8) * 2.0 ** -24 * reach
    if s.kind == "e4m3":
        err = err + 2.0 ** -25 * abs(scale) * np.abs(f).max(3) * np.abs(np.nan_to_num(k, nan=0, posinf=0, neginf=0)).sum(3).max(initial=0)
    rel = 2 * err + (n / 8 + 8) * 2.0 ** -23
    top = np.abs(np.where(np.isfinite(v), v, 0)).max(initial=0)
    tiny = (0 if s.kind == "bf16" else n * 2.0 ** -32 * top) + (2.0 ** -24 if s.kind == "fp16" else 0)
    got = out.double().cpu().numpy()
    bad = np.isnan(want)
    assert np.all(~np.isfinite(got[real][bad[real]]))
    with np.errstate(invalid="ignore"):
        good = np.abs(got - want) <= mag * (1.01 * WEIGHT[s.kind] + rel[..., None]) + 1.01 * OUT[s.kind] * np.abs(want) + tiny
    assert np.all((good | bad)[real]), np.argwhere(~(good | bad) & real[..., None, None])[:5]
    assert np.all(got[~real] == 7)
    if lse is not None:
        got = lse.double().cpu().numpy()
        assert np.all(got[~real] == 7)
        got, want_lse, slack = got[real], want_lse[real], rel[real]
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(got))
        got, want_lse, slack = got[~none], want_lse[~none], slack[~none]
        assert np.all((np.abs(got - want_lse) <= slack + 2.0 ** -22 * (1 + np.abs(want_lse))) | np.isnan(want_lse))


def queries(s, drafts, n_q, spread=1.5):
    return (spread * torch.randn((s.n_seq, drafts, n_q, s.dim), generator=s.g)).to(IO[s.kind]).cuda()


def run(s, drafts, group, counts=None, tree="random", error=None, **kw):
    n_q = s.heads * group
    q, parents = queries(s, drafts, n_q), trees(s.n_seq, drafts, s.g, tree)
    counts = counts if counts is None else ints(counts)
    out = torch.full_like(q, 7.0)
    lse = torch.full((s.n_seq, drafts, n_q), 7.0, device="cuda")
    got = lc().cache_attend_tree(s.cache, q, s.lengths, parents, counts, out=out, lse=lse, **kw)
    assert got is out
    check(s, q, s.lengths, parents, counts, out, lse, **kw)
    if error is None:
        no_device_error()
    else:
        device_error_is(error)
    return q, parents, counts, out, lse


EDGES = [1, 2, 7, 8, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300]
COUNTS = [1, 2, 7, 0, 8, 5, 8, 1, 8, 3, 8, 8, 2, 8, 0, 6]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("dim", [64, 80, 96, 112, 128, 192, 256])
def test_dims(kind, order, dim):
    run(Setup(EDGES, dim=dim, kind=kind, order=order, seed=dim), 8, 4, COUNTS)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 16, 24, 33, 72, 100, 130, 136, 200, 255])
def test_odd_dims(kind, dim):
    run(Setup([3, 17, 64, 150], dim=dim, kind=kind, seed=dim), 3, 3, [3, 3, 0, 2])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,drafts", [(1, 1), (1, 64), (2, 33), (3, 5), (4, 64), (7, 19), (8, 16), (16, 9), (33, 4),
                                          (64, 2), (71, 3), (130, 1), (5, 26), (2, 64)])
def test_groups_and_drafts(kind, group, drafts):
    run(Setup([70, 200, drafts], heads=3, dim=64, kind=kind, seed=group), drafts, group, [drafts, max(drafts - 1, 0), drafts])
    run(Setup([270], heads=1, dim=160, kind=kind, seed=drafts), drafts, group, tree="chain")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 3, 8, 24, 40, 64, 100, 128, 256, 1000])
@pytest.mark.parametrize("dim", [128, 192])
def test_pages(kind, page, dim):
    """Pages that end inside a step, that hold many, and sizes that tensor copies do not take."""
    run(Setup([4, page, page + 1, 2 * page + 5, 170], dim=dim, page=page, kind=kind, seed=page), 4, 2,
        [4, min(4, page), min(4, page), 4, 3])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 5, 16, 63, 128, 200, 1 << 30, 1 << 40])
@pytest.mark.parametrize("tree", ["random", "chain"])
def test_windows(kind, window, tree):
    run(Setup(EDGES, dim=128, kind=kind, seed=window % 999), 8, 4, COUNTS, tree, window=window)
    run(Setup([1000, 700], dim=64, kind=kind, seed=window % 999, page=24), 40, 2, [40, 17], tree, window=window)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-30])
def test_scales(kind, scale):
    run(Setup([100, 500, 9], dim=64, kind=kind, seed=5), 6, 4, [6, 4, 6], scale=scale)


def spoil(s, at):
    """NaN and infinities into slots (sequence, slot)."""
    table = s.table.cpu()
    for i, (b, j) in enumerate(at):
        p, r = int(table[b, j // s.page]), j % s.page
        odd = (math.nan, math.inf, -math.inf)[i % 3]
        for x, sc in zip((s.k, s.v), s.scales):
            if s.kind == "e4m3":
                sc[p, :, r] = odd
            else:
                x[p, :, r] = odd


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,page", [(80, 16), (128, 64), (256, 16), (64, 3)])
@pytest.mark.parametrize("scale", [0.1, 0.0, -0.1])
def test_what_unseen_slots_hold_does_not_matter(kind, dim, page, scale):
    """Slots behind the sequence, before every window, and drafts that are no ancestors."""
    lens, drafts, window = [140, 40, 300, 9], 8, 30
    s = Setup(lens, dim=dim, kind=kind, page=page, seed=6)
    parents, counts = trees(4, drafts, s.g), [8, 5, 8, 8]
    spoil(s, [(b, j) for b, n in enumerate(lens)
              for j in list(range(n, s.cap)) + list(range(max(0, n - counts[b] - window)))])
    q = queries(s, drafts, 4)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    lc().cache_attend_tree(s.cache, q, s.lengths, parents, ints(counts), window=window, scale=scale, out=out, lse=lse)
    check(s, q, s.lengths, parents, ints(counts), out, lse, scale, window)
    assert torch.all(torch.isfinite(out[0])) and torch.all(torch.isfinite(lse[2]))
    # the last draft's own slot: nobody else sees it
    res = [torch.full_like(q, 7.0) for _ in range(2)]
    for r in res:
        lc().cache_attend_tree(s.cache, q, s.lengths, parents, ints(counts), window=window, scale=scale, out=r)
        spoil(s, [(b, n - 1) for b, n in enumerate(lens)])
    check(s, q, s.lengths, parents, ints(counts), res[1], None, scale, window)
    for b, c in enumerate(counts):
        if kind != "e4m3":  # (a slot's scale decides how the step's weights are rounded)
            assert torch.equal(res[0][b, :c - 1], res[1][b, :c - 1])
        assert torch.all(torch.isfinite(res[0][b])) and not torch.all(torch.isfinite(res[1][b, c - 1]))
    no_device_error()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16), (256, 16), (64, 3)])
def test_values_that_are_no_numbers_reach_the_rows_that_see_them(kind, dim, page):
    s = Setup([200, 130, 64], dim=dim, kind=kind, page=page, seed=7)
    t = s.table.cpu()
    for b, j, h, c, odd in ((0, 20, 0, 3, math.nan), (0, 197, 1, 7, math.inf), (1, 129, 0, 0, -math.inf), (2, 61, 1, 5, math.nan)):
        s.v[int(t[b, j // page]), h, j % page, c] = odd
    for tree in ("random", "chain"):
        run(s, 6, 3, [6, 4, 5], tree)


def test_nan_and_infinite_logits():
    """A NaN key, or a logit of +infinity, makes the rows that see it NaN; one of -infinity weighs nothing."""
    for page in (16, 5):
        s = Setup([30, 30, 30, 30], heads=1, dim=64, page=page, seed=8)
        at = [(int(s.table[b, 5 // page]), 5 % page) for b in range(4)]
        q, parents = queries(s, 3, 2), trees(4, 3, s.g, "chain")
        q[:, :, 0, 0], q[:, :, 1, 0] = 1.0, -1.0
        s.k[at[0][0], 0, at[0][1], 3] = math.nan
        s.k[at[1][0], 0, at[1][1], 0] = math.inf
        s.v[at[2][0], 0, at[2][1], 3] = math.nan
        lse = torch.empty((4, 3, 2), device="cuda")
        out = lc().cache_attend_tree(s.cache, q, s.lengths, parents, lse=lse)
        assert torch.all(torch.isnan(out[0])) and torch.all(torch.isnan(out[1, :, 0]))
        assert torch.all(torch.isfinite(out[1, :, 1])) and torch.all(torch.isfinite(lse[1, :, 1]))
        assert torch.all(torch.isnan(out[2, :, :, 3])) and torch.all(torch.isfinite(out[2, :, :, 4:]))
        assert torch.all(torch.isfinite(out[3]))
        t = Setup([3], heads=1, dim=64, page=page, seed=9)
        t.k[:, :, :, 0] = math.inf
        q = queries(t, 2, 1).abs()
        q[..., 0] = -1.0
        lse = torch.empty((1, 2, 1), device="cuda")
        out = lc().cache_attend_tree(t.cache, q, t.lengths, ints([[-1, 0]]), lse=lse)
        assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    no_device_error()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 3])
def test_rising_maximum(kind, page):
    """Logits that rise along the sequence by more than exp's range, and the same falling."""
    n = 400
    s = Setup([n], heads=1, dim=64, kind=kind, page=page, seed=10)
    j = torch.arange(n)
    pages, row = s.table[0].cpu()[j // page].long(), j % page
    if kind == "e4m3":
        k = torch.zeros(s.k.shape)
        k[:, :, :, 0] = 1.0
        s.k.view(torch.uint8).copy_(k.to(torch.float8_e4m3fn).view(torch.uint8).cuda())
        s.scales[0][pages.cuda(), 0, row.cuda()] = j.float().cuda()
    else:
        s.k.zero_()
        s.k[pages.cuda(), 0, row.cuda(), 0] = (j // 2).to(s.k.dtype).cuda()
    q = torch.zeros((1, 2, 2, 64), dtype=IO[kind], device="cuda")
    q[:, :, 0, 0], q[:, :, 1, 0] = 1.0, -1.0
    out, lse = torch.full_like(q, 7.0), torch.full((1, 2, 2), 7.0, device="cuda")
    parents = ints([[-1, 0]])
    lc().cache_attend_tree(s.cache, q, s.lengths, parents, out=out, lse=lse, scale=1.0)
    check(s, q, s.lengths, parents, None, out, lse, 1.0)
    no_device_error()


@pytest.mark.parametrize("case", ["far", "zero", "negative", "tiny", "huge", "mixed"])
@pytest.mark.parametrize("page", [16, 3])
def test_e4m3_scales(case, page):
    """Value scales far from one another, zero, negative, and of any size a float32 holds; NaN in one."""
    s = Setup([300, 40], heads=2, dim=64, kind="e4m3", page=page, seed=11)
    x = s.scales[1]
    g = torch.Generator().manual_seed(12)
    r = torch.rand(x.shape, generator=g).cuda()
    if case == "far":
        x.copy_(torch.exp2(80 * (r - 0.5)))
    elif case == "zero":
        x[r < 0.5] = 0
    elif case == "negative":
        x[r < 0.5] *= -1
    elif case == "tiny":
        x.mul_(2.0 ** -90)
    elif case == "huge":
        x.mul_(2.0 ** 90)
    else:
        x.copy_(torch.where(r < 0.3, 2.0 ** -100, torch.where(r < 0.6, -1.0, 2.0 ** 30 * r)))
    run(s, 5, 4, [5, 3])
    x.zero_()
    run(s, 5, 4, [5, 3])


@pytest.mark.parametrize("kind", KINDS)
def test_many_small_weights_under_one_large(kind):
    """One slot's logit 18 above all the others': each of those weighs 2^-26 of it, together half a
    thousandth, which no 16-bit weight may lose."""
    n = 40000
    s = Setup([n], heads=1, dim=64, page=64, kind=kind, seed=13)
    table = s.table[0].cpu()
    p, r = int(table[100 // 64]), 100 % 64
    if kind == "e4m3":
        s.k.view(torch.uint8).zero_()
        s.v.view(torch.uint8).copy_(torch.ones(s.v.shape).to(torch.float8_e4m3fn).view(torch.uint8).cuda())
        s.scales[0].fill_(1.0)
        s.scales[1].fill_(0.01)
        s.k.view(torch.uint8)[p, 0, r, 0] = int(torch.tensor(18.0).to(torch.float8_e4m3fn).view(torch.uint8))
        s.v.view(torch.uint8)[p] = 0
    else:
        s.k.zero_()
        s.v.fill_(0.01)
        s.k[p, 0, r, 0] = 18.0
        s.v[p, 0, r] = 0
    q = torch.zeros((1, 2, 3, 64), dtype=IO[kind], device="cuda")
    q[..., 0] = 1.0
    out, lse = torch.full_like(q, 7.0), torch.full((1, 2, 3), 7.0, device="cuda")
    lc().cache_attend_tree(s.cache, q, s.lengths, ints([[-1, 0]]), out=out, lse=lse, scale=1.0)
    check(s, q, s.lengths, ints([[-1, 0]]), None, out, lse, 1.0)
    assert torch.all(out > 0)
    no_device_error()


@pytest.mark.parametrize("kind,dim,n", [("bf16", 128, 20011), ("fp16", 64, 33000), ("e4m3", 128, 40001), ("bf16", 256, 9001),
                                        ("e4m3", 256, 9001)])
def test_long(kind, dim, n):
    """One sequence over the whole GPU, split and joined; logits large enough that a few slots dominate."""
    run(Setup([n], heads=1, dim=dim, kind=kind, seed=n % 997, page=64), 5, 3, scale=0.4)
    run(Setup([n // 2, 30, n // 3], heads=2, dim=dim, kind=kind, seed=n % 997), 20, 8, [20, 9, 1])
    run(Setup([n // 2, 30], heads=2, dim=dim, kind=kind, seed=n % 997, page=20), 6, 3)


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    n = [(7 * i) % 97 for i in range(500)]
    run(Setup(n, heads=1, dim=64, kind=kind, seed=14), 3, 2, [min(x, i % 4) for i, x in enumerate(n)])
    n = [(131 * i) % 900 + 4 for i in range(90)]
    run(Setup(n, heads=4, dim=128, kind=kind, seed=15), 4, 4, tree="chain")
    s = Setup([0] * 40, heads=2, dim=64, per=4, kind=kind, seed=16)
    run(s, 2, 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_unaligned_pools(kind, shift):
    run(Setup([3, 50, 200], dim=64, kind=kind, seed=shift, shift=shift), 3, 4)


@pytest.mark.parametrize("kind", KINDS)
def test_strided_arguments(kind):
    s = Setup([20, 333, 64], heads=2, dim=96, kind=kind, order="token", seed=17)
    drafts, counts = 5, ints([5, 2, 4])
    q, parents = queries(s, drafts, 4), trees(3, 9, s.g)[:, :drafts]
    wide = torch.zeros((3, drafts, 4, 3, 97), dtype=q.dtype, device="cuda")
    wide[:, :, :, 1, 1:] = q
    big = torch.full((3, 7, 5, 2, 97), 7.0, dtype=q.dtype, device="cuda")
    logs = torch.full((3, 7, 9), 7.0, device="cuda")
    out, lse = big[:, :drafts, :4, 1, 1:], logs[:, 1:6, 2:6]
    lc().cache_attend_tree(s.cache, wide[:, :, :, 1, 1:], s.lengths, parents, counts, out=out, lse=lse)
    check(s, q, s.lengths, parents, counts, out, lse)
    out[:], lse[:] = 7, 7
    assert torch.all(big == 7) and torch.all(logs == 7)
    no_device_error()


def test_offsets_past_32_bits():
    """Pages more than 2^32 elements apart."""
    gap = 2_500_000_000
    flat = torch.zeros(2 * gap + 4096, dtype=torch.bfloat16, device="cuda")
    s = Setup([40], heads=1, dim=64, page=16, seed=18)
    k = torch.as_strided(flat, (3, 1, 16, 64), (gap, 2048, 64, 1))
    v = torch.as_strided(flat, (3, 1, 16, 64), (gap, 2048, 64, 1), 1024)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    k.copy_(s.k[s.table[0].long()][[1, 2, 0]])
    v.copy_(s.v[s.table[0].long()][[1, 2, 0]])
    q, parents = queries(s, 4, 2), trees(1, 4, s.g)
    want = lc().cache_attend_tree(s.cache, q, s.lengths, parents)
    assert torch.equal(lc().cache_attend_tree(lc().PagedCache(k, v, table), q, s.lengths, parents), want)
    # rows on no 16-byte boundary: the other way of reading pages
    k2 = torch.as_strided(flat, (3, 1, 16, 64), (gap, 2048, 64, 1), 2047)
    v2 = torch.as_strided(flat, (3, 1, 16, 64), (gap, 2048, 64, 1), 3071)
    kk, vv = k.clone(), v.clone()
    k2.copy_(kk)
    v2.copy_(vv)
    got = lc().cache_attend_tree(lc().PagedCache(k2, v2, table), q, s.lengths, parents)
    assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -7, atol=1e-6)  # (each is rounded once)
    no_device_error()


@pytest.mark.parametrize("kind,dim,page", [("bf16", 64, 16), ("e4m3", 128, 16), ("fp16", 33, 16), ("e4m3", 64, 3)])
def test_bad_device_values_are_reported(kind, dim, page):
    """Lengths, counts and parents are clamped, pages outside the pool hold nothing to see; all are recorded."""
    s = Setup([40, 40, 40], dim=dim, per=48 // page, page=page, kind=kind, seed=19)
    q, parents = queries(s, 4, 4), trees(3, 4, s.g)

    def call(lengths, parents, counts, table=None, want_parents=None):
        cache = s.cache if table is None else lc().PagedCache(s.k, s.v, table, *s.scales)
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
        lc().cache_attend_tree(cache, q, lengths, parents, counts, out=out, lse=lse)
        device_error_is("LC_ERR_CACHE_INDEX")
        check(s, q, lengths, parents, counts, out, lse, table=table)
    call(ints([40, 1000, -5]), parents, None)
    call(s.lengths, parents, ints([4, 5, -1]))
    call(ints([40, 2, 40]), parents, ints([4, 4, 0]))
    for bad in (1, 3, 64, -2, 1 << 30, -(1 << 31)):
        p = parents.clone()
        p[1, 1] = bad
        call(s.lengths, p, None)
    for bad in (-1, s.k.shape[0], 1 << 30, -(1 << 31)):
        t = s.table.clone()
        t[1, 1] = bad
        call(s.lengths, parents, None, t)
        t[2, :] = bad
        call(s.lengths, parents, None, t)


def test_repeatable_on_any_stream_and_in_graphs():
    s = Setup([3000, 17, 1200, 5], heads=2, dim=128, seed=20)
    q, parents, counts, out, lse = run(s, 6, 4, [6, 6, 3, 5])
    call = lambda **kw: lc().cache_attend_tree(s.cache, q, s.lengths, parents, counts, **kw)  # noqa: E731
    for _ in range(5):
        assert torch.equal(call(out=torch.full_like(out, 7.0)), out)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for x in sides:
        x.wait_stream(torch.cuda.current_stream())
    got = [call(out=torch.full_like(out, 7.0), stream=x if i else x.cuda_stream) for i, x in enumerate(sides)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], out)
    # two graphs, each with a workspace of its own, replayed at once
    size = s.cache.tree_workspace_bytes(8, 6)
    res, graphs = [torch.full_like(out, 7.0) for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for r, g, w in zip(res, graphs, spaces):
        with torch.cuda.graph(g):
            call(out=r, workspace=w)
    for lengths in ([3000, 17, 1200, 5], [40, 2900, 7, 1100]):
        s.lengths.copy_(ints(lengths))
        for r in res:
            r.fill_(7)
        want = call(out=torch.full_like(out, 7.0))
        torch.cuda.synchronize()
        for g, x in zip(graphs, sides):
            with torch.cuda.stream(x):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], want) and torch.equal(res[1], want)
    # a workspace that holds anything at all
    spaces[0].fill_(255)
    assert torch.equal(call(out=torch.full_like(out, 7.0), workspace=spaces[0]), want)
    no_device_error()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("per", [8, 16, 32, 33, 64, 120])
def test_short_sequences_behind_long_tables(kind, per):
    """Whether units may be cut, and how many blocks join them, goes by the table's columns."""
    n = [(37 * i) % 120 + 3 for i in range(90)]
    n[7], n[80] = per * 16, per * 16 - 5
    run(Setup(n, heads=2, dim=64, per=per, kind=kind, seed=per), 3, 2, [i % 4 if i % 4 else 1 for i in range(90)])
    run(Setup([per * 16, 5, 70], heads=1, dim=192, per=per, kind=kind, seed=per), 3, 3)
    run(Setup([per * 16 - 3] * 10, heads=8, dim=128, per=per, kind=kind, seed=per), 3, 2, tree="chain")


def test_calls_at_once():
    """Prompts, trees and accepted drafts on streams of their own, at the same time, and one after another on each."""
    g = torch.Generator().manual_seed(22)
    calls = []
    for kind, dim in (("bf16", 64), ("e4m3", 128), ("fp16", 256)):
        s = Setup([700, 33, 1500], heads=2, dim=dim, kind=kind, seed=dim)
        q, parents = queries(s, 7, 6), trees(3, 7, s.g)
        calls.append(lambda s=s, q=q, p=parents: lc().cache_attend_tree(s.cache, q, s.lengths, p))
    for dim in (64, 192):
        x = torch.randn((500, 8, dim), generator=g).bfloat16().cuda()
        starts = ints([0, 200, 201, 500])
        calls.append(lambda x=x, t=starts: lc().prompt_attend(x[:, :4], x[:, 4:6], x[:, 6:], t))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(4)], [[] for _ in calls]
    for turn in range(12):
        for i, c in enumerate(calls):
            with torch.cuda.stream(streams[(i + turn) % 4]):
                got[i].append(c())
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(want[i], x) for x in outs)
    no_device_error()


def test_a_draft_alone_is_decoding():
    """One draft a sequence sees what the query of cache_attend does."""
    for kind in KINDS:
        s = Setup([1, 100, 3000], heads=2, dim=128, kind=kind, seed=21)
        q = queries(s, 1, 8)
        a = lc().cache_attend_tree(s.cache, q, s.lengths, ints([[-1]] * 3))
        b = lc().cache_attend(s.cache, q[:, 0], s.lengths)
        assert torch.allclose(a[:, 0].float(), b.float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    no_device_error()


def test_python_refusals_and_empty_calls():
    M = lc()
    s = Setup([10, 20], heads=2, dim=64)
    q, parents = queries(s, 3, 4), trees(2, 3, s.g)
    ok = dict(q=q, lengths=s.lengths, parents=parents)
    for bad in (dict(q=q.half()), dict(q=q[:1]), dict(q=q[:, 0]), dict(q=q.cpu()), dict(lengths=s.lengths.long()),
                dict(parents=parents.long()), dict(parents=parents[:, :2]), dict(parents=parents.t().contiguous().t()),
                dict(counts=s.lengths[:1]), dict(lse=torch.empty((2, 3, 3), device="cuda")), dict(out=torch.empty_like(q).half()),
                dict(q=q[..., :32]), dict(workspace=torch.empty(64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            M.cache_attend_tree(s.cache, **{**ok, **bad})
    for bad, status in ((dict(window=-1), "LC_ERR_SHAPE"), (dict(scale=math.nan), "LC_ERR_SHAPE"),
                        (dict(q=q[:, :, :3]), "LC_ERR_SHAPE"), (dict(out=q), "LC_ERR_OVERLAP"),
                        (dict(out=torch.empty_like(q[:1]).expand_as(q)), "LC_ERR_NOT_INJECTIVE"),
                        (dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), "LC_ERR_WORKSPACE")):
        with pytest.raises((M.LayoutCopyError, ValueError)) as e:
            M.cache_attend_tree(s.cache, **{**ok, **bad})
        if isinstance(e.value, M.LayoutCopyError):
            assert e.value.status == M.STATUS[status]
    many = torch.zeros((2, 65, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises((M.LayoutCopyError, ValueError)):
        M.cache_attend_tree(s.cache, many, s.lengths, torch.zeros((2, 65), dtype=torch.int32, device="cuda"))
    none = M.PagedCache(s.k, s.v, s.table[:, :0])
    out = torch.full_like(q, 7.0)
    M.cache_attend_tree(none, q, torch.zeros_like(s.lengths), parents, out=out)
    assert torch.all(out == 7)
    assert M.cache_attend_tree(s.cache, q[:, :0], s.lengths, parents[:, :0]).shape == (2, 0, 4, 64)
    nobody = M.PagedCache(s.k, s.v, s.table[:0])
    assert M.cache_attend_tree(nobody, q[:0], s.lengths[:0], parents[:0]).shape == (0, 3, 4, 64)
    no_device_error()
