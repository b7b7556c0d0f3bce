"""Reservations of pages, packed tokens and accepted drafts on the GPU: exact, against the oracle."""
import numpy as np
import pytest

from oracle import drafts as od
from test_gpu_cache import IO, Setup, device_error_is, lc, no_device_error

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp16", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def ints(x, shape=None):
    t = torch.tensor(np.array(x), dtype=torch.int32, device="cuda")
    return t if shape is None else t.reshape(shape)


def raw(x):
    """Elements as they are stored, NaN codes too."""
    return x.view(torch.uint8 if x.dtype is torch.float8_e4m3fn else torch.int32 if x.dtype is torch.float32 else torch.int16)


# ---- reserve ----

def reservation(table, lengths, counts, free, page, max_tokens, spare=3, new=False, error=False, stream=None, wide=0):
    """The call on device copies, against the oracle; `spare` entries above the stack, `wide` columns beside the tables."""
    n, per = len(table), len(table[0]) if len(table) else 0
    big = torch.full((n, per + wide), -9, dtype=torch.int32, device="cuda")
    big[:, :per] = ints(table, (n, per))
    other = torch.full((n, per + 2 * wide), -9, dtype=torch.int32, device="cuda")
    stack = ints(list(free) + [-8] * spare, (-1,))
    lens, cnts, height = ints(lengths, (-1,)), ints(counts, (-1,)), ints([len(free)])
    was = big.clone()
    r = lc().cache_reserve(big[:, :per], lens, cnts, stack, height, page, max_tokens,
                           new_table=other[:, :per] if new else None, stream=stream)
    torch.cuda.synchronize()
    want, want_n, starts, packed, left = od.reserve(table, lengths, counts, free, page, max_tokens)
    assert r.table.tolist() == want and r.lengths.tolist() == want_n and r.starts.tolist() == starts
    pad = max_tokens - len(packed)
    assert r.slots.tolist() == [x[0] for x in packed] + [-1] * pad
    assert r.positions.tolist() == [x[1] for x in packed] + [-1] * pad
    assert r.seqs.tolist() == [x[2] for x in packed] + [-1] * pad
    assert r.n_free.tolist() == [len(left)] and stack[:len(left)].tolist() == left
    assert lens.tolist() == list(lengths) and cnts.tolist() == list(counts) and height.tolist() == [len(free)]
    assert torch.all(big[:, per:] == -9) and torch.all(other[:, per:] == -9)
    if new:
        assert torch.equal(big, was)
        assert r.table.data_ptr() == other.data_ptr() or not n or not per
    if error:
        device_error_is("LC_ERR_CACHE_INDEX")
    elif error is False:
        no_device_error()
    return r


def state(rng, n, per, page, ended=0.2, over=0.2):
    """A table of n sequences with the pages of their lengths, some with more, and the pages that are left."""
    ids = rng.permutation(n * per + 5)
    table, lengths, at = [], [], 0
    for _ in range(n):
        held = int(rng.integers(0, per + 1))
        length = int(rng.integers(max(held - 1, 0) * page, held * page + 1)) if held else 0
        if rng.random() < over and held:
            length = int(rng.integers(0, held * page + 1))
        if rng.random() < ended:
            length = 0
        table.append([int(x) for x in ids[at:at + held]] + [-1] * (per - held))
        lengths.append(length)
        at += held
    return table, lengths, [int(x) for x in ids[at:]]


@pytest.mark.parametrize("n", [1, 2, 31, 33, 200, 1024, 1025, 4096])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("new", [False, True])
def test_reserve(n, page, new):
    rng = np.random.default_rng(n + page)
    for per in (1, 7, 40 if n > 1000 else 300):
        table, lengths, free = state(rng, n, per, page)
        counts = [int(min(rng.integers(0, 9) if rng.random() < 0.8 else rng.integers(0, 4 * page + 1), per * page - x))
                  for x in lengths]
        total = sum(counts)
        reservation(table, lengths, counts, free, page, total, spare=n * per, new=new, wide=per % 3)
        reservation(table, lengths, [0] * n, free, page, 0, spare=n * per, new=new)


@pytest.mark.parametrize("new", [False, True])
def test_reserve_when_things_run_out(new):
    """Too few pages, lists that end, tables that end, negative lengths and counts, and a surplus beside a refusal."""
    rng = np.random.default_rng(5)
    for turn in range(30):
        n, per, page = int(rng.integers(1, 80)), int(rng.integers(1, 9)), int(rng.integers(1, 20))
        table, lengths, free = state(rng, n, per, page, over=0.5)
        counts = [int(rng.integers(0, 2 * page + 1)) for _ in lengths]
        free = free[:int(rng.integers(0, len(free) + 1))]
        if turn % 3 == 0:
            counts[0] = -3
        if turn % 5 == 0:
            lengths[-1] = -7
        most = int(sum(max(x, 0) for x in counts) * rng.random())
        reservation(table, lengths, counts, free, page, most, spare=n * per, new=new, error=None)
        lc().last_device_error()
    reservation([[4, 5, 6, -1]], [3], [1], [9], 4, 0, spare=4, new=new, error=True)  # three go back, none is served
    reservation([[4, 5, 6, -1]], [12], [5], [], 4, 9, new=new, error=True)


def test_reserve_a_stack_that_is_full_or_lies():
    """More pages come back than the stack holds: it is filled, the rest is dropped; its height is clamped."""
    table, zero, h = ints([[4, 5, 6], [7, -1, -1]]), ints([0, 0]), ints([2])
    stack = ints([1, 2, -1, -1])
    r = lc().cache_reserve(table, zero, zero, stack, h, 16, 4)
    device_error_is("LC_ERR_CACHE_INDEX")
    assert stack.tolist() == [1, 2, 4, 5] and r.n_free.tolist() == [4] and torch.all(table == -1)
    for height in (-1, 5, (1 << 31) - 1, -(1 << 31)):
        t, stack = ints([[3, -1]]), ints([8, 9, 7, 6])
        r = lc().cache_reserve(t, ints([2]), ints([1]), stack, ints([height]), 2, 1)
        device_error_is("LC_ERR_CACHE_INDEX")
        assert r.n_free.tolist() == [0 if height < 0 else 3]
        assert t.tolist() == [[3, -1 if height < 0 else 6]]


def test_reserve_long_prompts_and_none():
    rng = np.random.default_rng(6)
    table, lengths, free = state(rng, 20, 500, 16, ended=0.5)
    lengths = [0] * 20
    counts = [int(rng.integers(0, 8000)) for _ in range(20)]
    for new in (False, True):
        reservation(table, lengths, counts, free, 16, sum(counts) + 33, spare=20 * 500, new=new)
    e = lc().cache_reserve(ints([], (0, 4)), ints([]), ints([]), ints([]), ints([0]), 16, 5)
    assert e.starts.tolist() == [0] and e.slots.tolist() == [-1] * 5 and e.n_free.tolist() == [0]
    e = lc().cache_reserve(ints([], (2, 0)), ints([0, 0]), ints([0, 0]), ints([3]), ints([1]), 16, 0)
    assert e.starts.tolist() == [0, 0, 0] and e.n_free.tolist() == [1]
    no_device_error()


def test_reserve_on_streams_and_in_graphs():
    rng = np.random.default_rng(7)
    table, lengths, free = state(rng, 50, 20, 16)
    counts = [min(3, 320 - x) for x in lengths]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    reservation(table, lengths, counts, free, 16, 150, spare=1000, stream=side)
    # a captured step: pages and lengths go on from where the last replay left them
    t, n, h, stack = ints(table), ints(lengths), ints([len(free)]), ints(free + [-1] * 1000)
    g = torch.cuda.CUDAGraph()
    c = ints([1] * 50)
    with torch.cuda.graph(g):
        r = lc().cache_reserve(t, n, c, stack, h, 16, 50)
        n.copy_(r.lengths)
        h.copy_(r.n_free)
    want_t, want_n, left = table, lengths, free
    for _ in range(20):
        if any(x + 1 > 320 for x in want_n):
            break
        g.replay()
        torch.cuda.synchronize()
        want_t, want_n, _, packed, left = od.reserve(want_t, want_n, [1] * 50, left, 16, 50)
        assert t.tolist() == want_t and n.tolist() == want_n and stack[:len(left)].tolist() == left
        assert r.slots.tolist() == [x[0] for x in packed] + [-1] * (50 - len(packed))
    lc().last_device_error()


def test_reserve_refusals():
    M = lc()
    t, n, c, f, h = ints([[1, -1], [2, -1]]), ints([3, 4]), ints([1, 1]), ints([5, 6, 7]), ints([3])
    ok = dict(page_table=t, lengths=n, counts=c, free=f, n_free=h, page_size=16, max_tokens=4)
    for bad in (dict(page_table=t.long()), dict(page_table=t.cpu()), dict(page_table=t[0]), dict(page_table=t.t()),
                dict(lengths=n[:1]), dict(lengths=n.long()), dict(counts=c.cpu()), dict(free=f[None]), dict(n_free=ints([3, 3])),
                dict(new_table=t[:, :1]), dict(free=f[::2])):
        with pytest.raises(ValueError):
            M.cache_reserve(**{**ok, **bad})
    for bad, status in ((dict(page_size=0), "LC_ERR_SHAPE"), (dict(max_tokens=-1), "LC_ERR_SHAPE"),
                        (dict(page_size=1 << 30), "LC_ERR_OVERFLOW"), (dict(free=t[0]), "LC_ERR_OVERLAP"),
                        (dict(lengths=f[:2]), "LC_ERR_OVERLAP"), (dict(n_free=t[0, :1]), "LC_ERR_OVERLAP"),
                        (dict(new_table=ints([[0, 0]]).expand(2, 2)), "LC_ERR_NOT_INJECTIVE")):
        with pytest.raises(M.LayoutCopyError) as e:
            M.cache_reserve(**{**ok, **bad})
        assert e.value.status == M.STATUS[status], bad
    big = torch.full((4097, 1), -1, dtype=torch.int32, device="cuda")
    z = torch.zeros(4097, dtype=torch.int32, device="cuda")
    with pytest.raises(M.LayoutCopyError):
        M.cache_reserve(big, z, z, f, h, 16, 4)
    assert t.tolist() == [[1, -1], [2, -1]] and f.tolist() == [5, 6, 7]
    no_device_error()


# ---- packed appends ----

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,shift,order", [(64, 0, "head"), (80, 0, "token"), (128, 0, "head"), (33, 0, "head"), (64, 1, "token"),
                                             (256, 0, "head")])
def test_append_packed_is_append(kind, dim, shift, order):
    """The same rows by slots and by the page table; dropped tokens and slots outside the pool are not written."""
    lengths, counts = [5, 0, 30, 47], [7, 20, 1, 1]
    s = Setup(lengths, dim=dim, per=3, page=16, kind=kind, order=order, seed=dim, shift=shift)
    other = Setup(lengths, dim=dim, per=3, page=16, kind=kind, order=order, seed=dim, shift=shift)
    new = [torch.randn((4, 20, 2, dim), generator=s.g).to(IO[kind]).cuda() for _ in range(2)]
    lc().cache_append(s.cache, *new, s.lengths, ints(counts))
    table = s.table.tolist()
    slots, rows = [], []
    for b, c in enumerate(counts):
        for t in range(c):
            j = lengths[b] + t
            slots.append(table[b][j // 16] * 16 + j % 16)
            rows.append((b, t))
    slots[3:3], rows[3:3] = [-1], [(0, 19)]
    k, v = (torch.stack([x[b, t] for b, t in rows]) for x in new)
    lc().cache_append_packed(other.cache, k, v, torch.tensor(slots, device="cuda"))
    no_device_error()
    for x, y in ((s.k, other.k), (s.v, other.v)):
        assert torch.equal(raw(x), raw(y))
    if kind == "e4m3":
        assert torch.equal(s.scales[0], other.scales[0]) and torch.equal(s.scales[1], other.scales[1])
    before = raw(other.k).clone()
    n_pages = s.k.shape[0]
    for bad in (n_pages * 16, -2, 1 << 40, -(1 << 62), (1 << 32) + 3):
        lc().cache_append_packed(other.cache, k[:1], v[:1], torch.tensor([bad], device="cuda"))
        device_error_is("LC_ERR_CACHE_INDEX")
    assert torch.equal(raw(other.k), before)
    lc().cache_append_packed(other.cache, k[:0], v[:0], torch.tensor([], dtype=torch.int64, device="cuda"))
    no_device_error()


def test_append_packed_refusals():
    M = lc()
    s = Setup([5, 9], heads=2, dim=64)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 1, 2], device="cuda")
    for bad in (dict(k=k.float(), v=k.float()), dict(v=k[:2]), dict(k=k[:, :1], v=k[:, :1]), dict(slots=slots.int()),
                dict(slots=slots[:2]), dict(slots=slots.cpu()), dict(k=k[0], v=k[0])):
        with pytest.raises(ValueError):
            M.cache_append_packed(s.cache, **{**dict(k=k, v=k, slots=slots), **bad})
    with pytest.raises(M.LayoutCopyError) as e:
        M.cache_append_packed(s.cache, k.half(), k.half(), slots)
    assert e.value.status == M.STATUS["LC_ERR_TYPE"]
    no_device_error()


# ---- accept ----

def check_accept(s, lengths, counts, path, error=False, **kw):
    pools = [(s.k, s.v)] + ([tuple(s.scales)] if s.kind == "e4m3" else [])
    before = [[raw(x).clone() for x in p] for p in pools]
    table = s.table.cpu()
    moves, want = od.accept(lengths, counts, path, s.cap)
    got = lc().cache_accept(s.cache, ints(lengths), None if counts is None else ints(counts), ints(path, (len(lengths), -1)), **kw)
    torch.cuda.synchronize()
    assert got.tolist() == want
    for old in before:
        for x in old:
            y = x.clone()
            for b, a, c in moves:
                pa, pc = int(table[b, a // s.page]), int(table[b, c // s.page])
                y[pc, :, c % s.page] = x[pa, :, a % s.page]
            x.copy_(y)
    for old, p in zip(before, pools):
        for x, y in zip(old, p):
            assert torch.equal(x, raw(y))
    if error:
        device_error_is("LC_ERR_CACHE_INDEX")
    else:
        no_device_error()
    return got


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,shift,order,page", [(64, 0, "head", 16), (80, 0, "token", 3), (128, 0, "head", 64), (33, 0, "head", 1),
                                                  (64, 1, "token", 16), (256, 0, "head", 5), (1, 0, "head", 16)])
def test_accept(kind, dim, shift, order, page):
    lengths = [70, 64, 3, 90, 20, 66, 64]
    counts = [64, 64, 3, 5, 0, 40, 64]
    rng = np.random.default_rng(dim)
    path = np.full((7, 64), -1)
    path[0] = np.arange(64)                                                   # everything stays
    for b in (1, 5):
        p = np.sort(rng.choice(counts[b], 17, replace=False))
        path[b, :17] = p
    path[2, :1], path[3, :2] = 2, (1, 4)
    path[6, :1] = 63
    check_accept(Setup(lengths, dim=dim, per=-(-90 // page), page=page, kind=kind, order=order, seed=dim, shift=shift), lengths,
                 counts, path.tolist())


def test_accept_paths_that_do_not_rise():
    s = Setup([40, 40, 40, 40, 40], dim=64, kind="bf16", seed=1)
    for path in ([[1, 3, 3, 5], [2, 1, -1, -1], [0, 2, 8, -1], [-2, 0, 1, 2], [1, -1, 2, 3]],):
        check_accept(s, [40] * 5, [8] * 5, path, error=True)
    check_accept(s, [40] * 5, [8] * 5, [[-1] * 4] * 5)
    check_accept(s, [40] * 5, [0, -1, 41, 9, 70], [[0, 1, -1, -1]] * 5, error=True)
    check_accept(s, [40, 1000, -4, 0, 48], None, [[1, 2, -1, -1]] * 5, error=True)
    check_accept(s, [40] * 5, [8] * 5, np.zeros((5, 0)).tolist())


def test_accept_bad_pages():
    """A page outside the pool: what moves from or to it does not, the rest does."""
    for bad in (-1, 20, 1 << 30, -(1 << 31)):
        s = Setup([40, 40], dim=64, per=3, page=16, seed=2)
        s.table[0, 2] = bad
        cache = lc().PagedCache(s.k, s.v, s.table)
        before = raw(s.k).clone()
        n = lc().cache_accept(cache, ints([40, 40]), ints([16, 16]), ints([[1, 3, 12], [1, 3, 12]]))
        device_error_is("LC_ERR_CACHE_INDEX")
        assert n.tolist() == [27, 27]
        p = s.table.tolist()
        assert torch.equal(raw(s.k)[p[0][1], :, 8], before[p[0][1], :, 9])
        assert torch.equal(raw(s.k)[p[0][1], :, 10], before[p[0][1], :, 10])
        assert torch.equal(raw(s.k)[p[1][1], :, 10], before[p[1][2], :, 4])


def test_accept_on_streams_and_refusals():
    M = lc()
    s = Setup([40, 30], dim=64, kind="e4m3", seed=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_accept(s, [40, 30], [5, 6], [[1, 4, -1], [0, 2, 5]], stream=side)
    wide = ints([[1, 4, 9, 9], [0, 2, 9, 9]])
    assert M.cache_accept(s.cache, ints([40, 30]), ints([5, 6]), wide[:, :2]).tolist() == [37, 26]
    n, c, p = ints([40, 30]), ints([5, 6]), ints([[1, 4], [0, 2]])
    for bad in (dict(lengths=n.long()), dict(counts=c[:1]), dict(path=p[:1]), dict(path=p[0]), dict(path=p.long()),
                dict(new_lengths=n.long()), dict(path=p.t())):
        with pytest.raises(ValueError):
            M.cache_accept(s.cache, **{**dict(lengths=n, counts=c, path=p), **bad})
    for bad in (dict(new_lengths=n), dict(new_lengths=c), dict(new_lengths=p.view(-1)[1:3])):
        with pytest.raises(M.LayoutCopyError) as e:
            M.cache_accept(s.cache, **{**dict(lengths=n, counts=c, path=p), **bad})
        assert e.value.status == M.STATUS["LC_ERR_OVERLAP"]
    with pytest.raises(M.LayoutCopyError):
        M.cache_accept(s.cache, n, c, torch.zeros((2, 65), dtype=torch.int32, device="cuda"))
    nobody = M.PagedCache(s.k, s.v, s.table[:0], *s.scales)
    assert M.cache_accept(nobody, n[:0], c[:0], p[:0]).shape == (0,)
    no_device_error()
