"""Attention over packed prompts on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic: a logit is a float32 sum of d exact products, off
by at most E = (d + 8) 2^-24 |scale| sum|q||k| (the last of it for the product
with the scale and the difference to the maximum); a weight is off by a factor of
exp(2E), by the exponential and by the sum of n of them, (n / 8 + 8) 2^-23; rounding the
weights to the 16-bit type adds u = 2^-8 (bfloat16) or 2^-11 (float16) of sum w|v|, and
the result is rounded to that type once.  float16 weights below 2^-25 of the largest are
off by up to 2^-36 of it: n 2^-36 max|v| more.
"""
import math

import numpy as np
import pytest

from oracle import prompt as op

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def lc():
    import movement_primitives_gb300
    return movement_primitives_gb300


def no_device_error():
    st, detail = lc().last_device_error()
    assert st == 0, "device error word %#x" % detail


def device_error_is(status):
    st, _ = lc().last_device_error()
    assert st == lc().STATUS[status]
    no_device_error()


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def sums(x, first=0):
    out = [first]
    for n in x:
        out.append(out[-1] + n)
    return out


def rows(n, heads, dim, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((n, heads, dim), generator=g)).to(dtype).cuda()


def check(q, k, v, starts, k_starts, out, lse, before=None, scale=None, **kw):
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    f = [x.double().cpu().numpy() for x in (q, k, v)]
    want, want_lse, mag, reach, real = op.attend(*f, starts, k_starts, scale, **kw)
    u, dim, n = U[q.dtype], q.shape[2], k.shape[0]
    half = q.dtype is torch.float16
    rel = 2 * (dim + 8) * 2.0 ** -24 * reach + (n / 8 + 8) * 2.0 ** -23
    top = np.abs(np.where(np.isfinite(f[2]), f[2], 0)).max(initial=0)
    tiny = (n * 2.0 ** -36 * top + 2.0 ** -24) if half else 0.0
    got = out.double().cpu().numpy()
    bad = np.isnan(want)
    assert np.all(~np.isfinite(got[real][bad[real]]))
    with np.errstate(invalid="ignore"):
        good = np.abs(got - want) <= mag * (1.01 * u + rel[..., None]) + u * np.abs(want) + tiny
    assert np.all((good | bad)[real]), np.argwhere(~(good | bad))[:5]
    if before is not None:
        assert torch.equal(out.cpu()[~real], before.cpu()[~real])
    if lse is not None:
        got, want_lse, slack = lse.double().cpu().numpy()[real], want_lse[real], rel[real]
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(got))
        got, want_lse, slack = got[~none], want_lse[~none], slack[~none]
        assert np.all((np.abs(got - want_lse) <= slack + 2.0 ** -22 * (1 + np.abs(want_lse))) | np.isnan(want_lse))
    no_device_error()


def run(nq, nk=None, heads=4, kv=2, dim=64, dtype=torch.bfloat16, seed=0, spread=1.5, tail=0, first=0, **kw):
    """Sequences of nq queries and nk keys (None: the queries'), `first` rows before them and `tail` behind them."""
    starts = sums(nq, first)
    ks = None if nk is None else sums(nk, first)
    q = rows(starts[-1] + tail, heads, dim, dtype, seed, spread)
    k, v = (rows((starts if ks is None else ks)[-1] + tail, kv, dim, dtype, seed + i) for i in (1, 2))
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    got = lc().prompt_attend(q, k, v, ints(starts), k_starts=None if ks is None else ints(ks), out=out, lse=lse, **kw)
    assert got is out
    check(q, k, v, starts, ks, out, lse, torch.full_like(q, 7.0), **kw)
    real = op.attend(*(x.double().cpu().numpy()[:, :, :1] for x in (q, k, v)), starts, ks)[4]
    assert torch.all(lse.cpu()[~real] == 7)
    return q, k, v, out, lse


EDGES = [0, 1, 2, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 255, 257, 1, 0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [8, 16, 24, 64, 72, 80, 96, 112, 128, 136, 160, 192, 200, 256])
def test_dims(dtype, dim):
    run(EDGES, dim=dim, dtype=dtype, seed=dim)
    run([300, 5], [431, 140], dim=dim, dtype=dtype, seed=dim, causal=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 16, 17, 33, 64, 71, 128, 130, 257])
def test_groups(dtype, group):
    run([5, 0, 40, 1, 131], heads=2 * group, kv=2, dtype=dtype, seed=group)
    run([3, 20], [90, 20], heads=group, kv=1, dim=192, dtype=dtype, seed=group)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 63, 127, 128, 129, 300, 1 << 30, 1 << 40])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(dim, window, causal):
    run([1, 300, 129, 0, 500], [1, 700, 129, 30, 500], dim=dim, seed=window % 1000, window=window, causal=causal)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 192])
@pytest.mark.parametrize("causal", [True, False])
def test_later_pieces_and_queries_without_keys(dtype, dim, causal):
    """More keys than queries, fewer (the first queries see nothing: zeros and -inf), and none."""
    run([7, 130, 3, 200, 5, 1, 0], [900, 131, 3, 70, 0, 128, 40], dim=dim, dtype=dtype, seed=1, causal=causal)
    q, _, _, out, lse = run([200], [70], dim=dim, dtype=dtype, seed=2, causal=True)
    assert torch.all(out[:130] == 0) and torch.all(torch.isneginf(lse[:130]))
    run([5], [0], dim=dim, dtype=dtype, seed=3, causal=causal)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 256])
def test_rows_of_no_sequence_stay(dtype, dim):
    run([30, 0, 129], dim=dim, dtype=dtype, first=5, tail=9, seed=4)
    run([129, 1], [200, 60], dim=dim, dtype=dtype, first=3, tail=150, seed=4, causal=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 192])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-30])
def test_scales(dtype, dim, scale):
    run([100, 140, 1], heads=6, dim=dim, dtype=dtype, seed=5, scale=scale)


def poison(x, keep):
    for i, odd in enumerate((math.nan, math.inf, -math.inf)):
        x[[r for r in range(x.shape[0]) if r not in keep and r % 3 == i]] = odd


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.1, 0.0, -0.1])
def test_what_unseen_keys_and_values_hold_does_not_matter(dtype, dim, scale):
    """Rows between sequences, keys behind the last query's place and in front of every window."""
    starts, ks, window = [2, 42, 42, 172], [10, 150, 150, 400], 50
    q, k, v = rows(180, 4, dim, dtype, 6), rows(420, 2, dim, dtype, 7), rows(420, 2, dim, dtype, 8)
    seen = set()
    for b in range(3):
        nq, nk = starts[b + 1] - starts[b], ks[b + 1] - ks[b]
        seen |= {ks[b] + int(j) for j in np.flatnonzero(op.seen(nq, nk, True, window).any(0))}
    poison(k, seen)
    poison(v, seen)
    poison(q, range(2, 172))
    out, lse = torch.full_like(q, 7.0), torch.zeros((180, 4), device="cuda")
    lc().prompt_attend(q, k, v, ints(starts), k_starts=ints(ks), window=window, scale=scale, out=out, lse=lse)
    assert torch.all(torch.isfinite(out[2:172]))
    clean = [torch.nan_to_num(x, nan=0, posinf=0, neginf=0) for x in (q, k, v)]
    check(*clean, starts, ks, out, lse, torch.full_like(q, 7.0), window=window, scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_are_no_numbers_reach_the_rows_that_see_them(dtype, dim):
    """... and no other: a value of a later place, or of the sequence behind, in the same tile of keys."""
    starts = [0, 200, 420, 423]
    q, k, v = rows(423, 4, dim, dtype, 9), rows(423, 2, dim, dtype, 10), rows(423, 2, dim, dtype, 11)
    v[150, 0, 3], v[300, 1, 7], v[199, 1, 0], v[422, 0, 5] = math.nan, math.inf, -math.inf, math.nan
    out, lse = torch.empty_like(q), torch.zeros((423, 4), device="cuda")
    lc().prompt_attend(q, k, v, ints(starts), out=out, lse=lse)
    check(q, k, v, starts, None, out, lse)
    assert torch.all(~torch.isfinite(out[150:200, :2, 3])) and torch.all(torch.isfinite(out[:150]))
    assert torch.all(~torch.isfinite(out[300:420, 2:, 7])) and torch.all(torch.isfinite(out[200:300]))


def test_nan_and_infinite_logits():
    """A NaN key, or a logit of +infinity, makes the rows that see it NaN; one of -infinity weighs nothing."""
    q, k, v = rows(60, 2, 64, torch.bfloat16, 12), rows(60, 1, 64, torch.bfloat16, 13), rows(60, 1, 64, torch.bfloat16, 14)
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    k[5, 0, 3], k[35, 0, 0] = math.nan, math.inf
    out, lse = torch.empty_like(q), torch.empty((60, 2), device="cuda")
    lc().prompt_attend(q, k, v, ints([0, 30, 60]), out=out, lse=lse)
    assert torch.all(torch.isfinite(out[:5])) and torch.all(torch.isnan(out[5:30]))
    assert torch.all(torch.isfinite(out[30:35])) and torch.all(torch.isnan(out[35:, 0]))
    assert torch.all(torch.isfinite(out[30:, 1])) and torch.all(torch.isfinite(lse[30:, 1]))
    kz = k.clone()
    kz[35, 0, 0] = 0
    q2, k2, v2 = (torch.cat([x[30:35], x[36:]]) for x in (q, kz, v))
    a = lc().prompt_attend(q2, k2, v2, ints([0, 29]))
    assert torch.allclose(a[5:, 1].float(), out[36:, 1].float(), atol=2e-2)
    # every logit -infinity: nothing is left
    q[:, :, 0], k[:, :, 0], k[5, 0, 3] = -1.0, math.inf, 0.0
    out = lc().prompt_attend(q, k, v, ints([0, 30, 60]), lse=lse)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 192])
def test_rising_maximum(dtype, dim):
    """Logits that rise along the keys by more than exp's range, and the same falling."""
    n = 500
    q, k, v = rows(n, 2, dim, dtype, 15), torch.zeros((n, 1, dim), dtype=dtype, device="cuda"), rows(n, 1, dim, dtype, 16)
    q[:] = 0
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    k[:, 0, 0] = torch.arange(n, device="cuda") // 2 * (2 if dtype is torch.bfloat16 else 1)
    out, lse = torch.empty_like(q), torch.empty((n, 2), device="cuda")
    lc().prompt_attend(q, k, v, ints([0, n]), out=out, lse=lse, scale=1.0)
    check(q, k, v, [0, n], None, out, lse, scale=1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long(dtype, dim):
    run([1900, 3, 1200], [4100, 3, 1200], heads=2, kv=1, dim=dim, dtype=dtype, seed=17, spread=4.0)


def test_many_sequences():
    run([(7 * i) % 23 for i in range(700)], heads=2, kv=1, seed=18)
    run([(131 * i) % 300 for i in range(40)], heads=8, kv=4, dim=128, seed=19)
    run([0] * 50, heads=2, kv=1, tail=3, seed=20)
    run([1] * 300, [(i * 5) % 40 for i in range(300)], heads=6, kv=3, dim=96, seed=20)


@pytest.mark.parametrize("n", [32, 33, 64, 65, 333])
@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=70), dict(causal=False, window=9), dict(tail=130, first=7)])
def test_many_sequences_in_order(n, kw):
    """Past 32 sequences items come in another order: long and empty ones at either end and between."""
    nq = [(17 * i) % 61 for i in range(n)]
    nq[0], nq[-1], nq[n // 2] = 300, 400, 0
    run(nq, [(13 * i) % 150 for i in range(n)], heads=4, kv=2, dim=64, seed=n, **kw)
    run(nq, heads=2, kv=1, dim=192, seed=n, **kw)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_arguments(dtype):
    """q, k and v in one buffer; out among other rows; lse among other heads."""
    n, dim = 300, 80
    qkv = rows(n, 8, dim, dtype, 21)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    wide = torch.full((n, 6, 3, dim + 1), 9.0, dtype=dtype, device="cuda")
    out, lse = wide[:, 1:5, 1, 1:], torch.zeros((n, 9), device="cuda")
    lc().prompt_attend(q, k, v, ints([0, 100, 300]), out=out, lse=lse[:, 2:6])
    check(q, k, v, [0, 100, 300], None, out, lse[:, 2:6])
    out[:] = 9
    assert torch.all(wide == 9) and torch.all(lse[:, :2] == 0) and torch.all(lse[:, 6:] == 0)
    # heads before tokens
    qt, kt, vt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    got = lc().prompt_attend(qt, kt, vt, ints([0, 100, 300]))
    check(q, k, v, [0, 100, 300], None, got, None)
    # over the queries' own rows, in the buffer that holds the keys
    want = got.clone()
    keep = qkv[:, 4:].clone()
    assert lc().prompt_attend(q, k, v, ints([0, 100, 300]), out=q) is q
    assert torch.equal(q, want) and torch.equal(qkv[:, 4:], keep)
    no_device_error()


def test_offsets_past_32_bits():
    """Rows more than 2^32 elements apart."""
    gap, n = 700_000_000, 10
    flat = torch.zeros(n * gap, dtype=torch.bfloat16, device="cuda")
    q, k, v = (rows(n, h, 64, torch.bfloat16, 22 + h) for h in (2, 1, 1))
    big = [torch.as_strided(flat, x.shape, (gap, 64, 1), at) for x, at in ((q, 0), (k, 1024), (v, 2048), (q, 4096))]
    for x, y in zip(big, (q, k, v)):
        x.copy_(y)
    starts = ints([0, 3, 10])
    want = lc().prompt_attend(q, k, v, starts)
    lc().prompt_attend(*big[:3], starts, out=big[3])
    assert torch.equal(big[3], want)
    no_device_error()


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("n_before", [0, 40])
def test_bad_starts_are_clamped_or_refused_and_reported(dim, n_before):
    """Starts outside the rows are moved to their ends; with ones that fall nothing is computed."""
    q, k, v = rows(100, 2, dim, torch.bfloat16, 23), rows(90, 1, dim, torch.bfloat16, 24), rows(90, 1, dim, torch.bfloat16, 25)
    fine_q, fine_k = [0, 60, 60, 100], [0, 60, 60, 90]
    big, low = (1 << 31) - 1, -(1 << 31)
    for a, b in (([-5, 60, 60, 100], fine_k), ([0, 60, 60, big], fine_k), (fine_q, [low, 60, 60, 1000]),
                 ([0, 60, 40, 100], fine_k), ([0, 60, 1000, 70], fine_k), (fine_q, [0, 60, 40, 90]),
                 (fine_q, [0, big, 60, 90]), (fine_q, [0, 60, 60, low]), ([100, 0, 0, 0], [0, 0, 0, 90])):
        ca, cb = ([min(max(x, 0), n) for x in y] for y, n in ((a, 100), (b, 90)))
        falls = ca != sorted(ca) or cb != sorted(cb)
        out, lse = torch.full_like(q, 7.0), torch.full((100, 2), 7.0, device="cuda")
        lead_q, lead_k = ([x[0] if 0 <= x[0] else 0] * n_before for x in (a, b))  # sequences of no rows before them
        lc().prompt_attend(q, k, v, ints(lead_q + a), k_starts=ints(lead_k + b), out=out, lse=lse)
        device_error_is("LC_ERR_CACHE_INDEX")
        if falls:
            assert torch.all(out == 7) and torch.all(lse == 7)
        else:
            check(q, k, v, ca, cb, out, lse, torch.full_like(q, 7.0))


def test_repeatable_on_any_stream_and_in_graphs():
    q, k, v, out, lse = run([300, 17, 900, 0, 64], heads=8, kv=2, dim=128, seed=26)
    starts = ints(sums([300, 17, 900, 0, 64]))
    for _ in range(5):
        assert torch.equal(lc().prompt_attend(q, k, v, starts), out)
    sides = [torch.cuda.Stream() for _ in range(3)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [lc().prompt_attend(q, k, v, starts, stream=s if i else s.cuda_stream) for i, s in enumerate(sides)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, out) for x in got)
    # two graphs, replayed at once, of starts that change between the replays
    res, graphs = [torch.zeros_like(out) for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    for r, g in zip(res, graphs):
        with torch.cuda.graph(g):
            lc().prompt_attend(q, k, v, starts, out=r)
    for turn in ([300, 17, 900, 0, 64], [0, 64, 900, 300, 17]):
        starts.copy_(ints(sums(turn)))
        want = lc().prompt_attend(q, k, v, starts)
        torch.cuda.synchronize()
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], want) and torch.equal(res[1], want)
    no_device_error()


def test_python_refusals():
    M = lc()
    q, k, v = rows(20, 4, 64, torch.bfloat16, 0), rows(20, 2, 64, torch.bfloat16, 1), rows(20, 2, 64, torch.bfloat16, 2)
    ok = dict(q=q, k=k, v=v, starts=ints([0, 20]))
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0]), dict(k=k.half()), dict(k=k[:, :, :32]), dict(v=v[:19]),
                dict(v=v[:, :1]), dict(k=k.cpu()), dict(starts=ints([0, 20]).long()), dict(starts=ints([])),
                dict(starts=torch.tensor([0, 20], dtype=torch.int32)), dict(k_starts=ints([0, 20, 20])),
                dict(k=k[:10], v=v[:10]), dict(out=q.half()), dict(out=torch.empty_like(q)[:10]),
                dict(lse=torch.empty((20, 3), device="cuda")), dict(lse=torch.empty((20, 4), dtype=torch.float64, device="cuda")),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(starts=ints([0, 0, 20, 20])[::2])):
        with pytest.raises(ValueError):
            M.prompt_attend(**{**ok, **bad})
    with pytest.raises((ValueError, NotImplementedError, RuntimeError)):
        M.prompt_attend(**{**ok, "q": q.clone().requires_grad_()})
    wide = torch.zeros((21, 4, 64), dtype=torch.bfloat16, device="cuda")
    wide[:20] = q
    odd = torch.zeros(20 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(20, 4, 64)
    for bad, status in ((dict(window=-1), "LC_ERR_SHAPE"), (dict(scale=math.inf), "LC_ERR_SHAPE"),
                        (dict(q=q[:, :3]), "LC_ERR_SHAPE"), (dict(q=wide[:20], out=wide[1:]), "LC_ERR_OVERLAP"),
                        (dict(out=q[:1].expand(20, -1, -1)), "LC_ERR_NOT_INJECTIVE"), (dict(q=odd), "LC_ERR_ALIGN"),
                        (dict(q=q[:, :, :60], k=k[:, :, :60], v=v[:, :, :60]), "LC_ERR_SHAPE"),
                        (dict(k=q[:, :2], out=q), "LC_ERR_OVERLAP")):
        with pytest.raises(M.LayoutCopyError) as e:
            M.prompt_attend(**{**ok, **bad})
        assert e.value.status == M.STATUS[status], (bad.keys(), e.value)
    assert M.prompt_attend(q[:0], k[:0], v[:0], ints([0, 0])).shape == (0, 4, 64)
    assert M.prompt_attend(q, k, v, ints([0]), out=q.clone()).equal(q)
    no_device_error()
