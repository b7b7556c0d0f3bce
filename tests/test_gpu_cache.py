"""Paged key-value cache operators on the GPU against the 64-bit oracle.

Tolerances of attention, from the arithmetic: a logit is a float32 sum of d
exact products, so it is off by at most E = (d + 4) 2^-24 scale sum|q||k|
(plus a rounding of the result); a weight is then off by a factor of at most
exp(2E), and by the float32 exponentials and the sum of n of them, about (n / 8 + 8)
2^-23 as they are summed; rounding the weights to the values' 16-bit type before the
product adds u = 2^-8 (bfloat16) or 2^-11 (float16) of sum w|v|, and the
result is rounded to that type once.  Copies, kept slots and E4M3 codes are
exact.
"""
import math

import numpy as np
import pytest

from oracle import cache as oc

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "e4m3": 2.0 ** -8}


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


IO = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.bfloat16}


class Setup:
    """A cache on the device and its values in 64 bits on the host."""

    def __init__(self, lengths, heads=2, dim=64, page=16, per=None, kind="bf16", order="head", seed=0, shift=0,
                 spread=1.0):
        g = torch.Generator().manual_seed(seed)
        n_seq = len(lengths)
        per = per if per is not None else max(1, -(-max(lengths, default=1) // page))
        n_pages = n_seq * per + 2
        shape = (n_pages, heads, page, dim) if order == "head" else (n_pages, page, heads, dim)
        self.scales = [None, None]
        pools = []
        for i in range(2):
            x = spread * torch.randn(shape, generator=g)
            if kind == "e4m3":
                x = (100 * x).clamp(-448, 448).to(torch.float8_e4m3fn)
                s = 0.005 + 0.01 * torch.rand(shape[:3], generator=g)
                self.scales[i] = s.cuda() if order == "head" else s.cuda().transpose(1, 2)
            else:
                x = x.to(IO[kind])
            # `shift` elements off the allocation's boundary: rows on no 16-byte boundary
            flat = torch.zeros(x.numel() + shift, dtype=torch.uint8 if kind == "e4m3" else x.dtype, device="cuda")
            flat[shift:] = (x.view(torch.uint8) if kind == "e4m3" else x).reshape(-1).cuda()
            y = flat[shift:].view(shape)
            y = y.view(torch.float8_e4m3fn) if kind == "e4m3" else y
            pools.append(y if order == "head" else y.transpose(1, 2))
        self.k, self.v = pools
        self.table = torch.randperm(n_pages, generator=g)[:n_seq * per].reshape(n_seq, per).to(torch.int32).cuda()
        self.lengths = torch.tensor(list(lengths), dtype=torch.int32, device="cuda")
        self.kind, self.g, self.n_seq, self.heads, self.dim, self.page = kind, g, n_seq, heads, dim, page
        self.cap = per * page
        self.cache = lc().PagedCache(self.k, self.v, self.table, *self.scales)

    def values(self):
        """(k, v) in 64 bits, [page, head, row, dim]."""
        out = []
        for x, s in zip((self.k, self.v), self.scales):
            y = x.float().double().cpu()
            out.append((y if s is None else y * s.double().cpu()[..., None]).numpy())
        return out

    def queries(self, n_q):
        return (1.5 * torch.randn((self.n_seq, n_q, self.dim), generator=self.g)).to(IO[self.kind]).cuda()


def check_attend(s, q, out, lse, scores=None, before=None, scale=None, window=0, mask=None, lengths=None):
    scale = 1 / math.sqrt(s.dim) if scale is None else scale
    n = s.lengths.cpu().numpy() if lengths is None else lengths
    k, v = s.values()
    k, v = np.nan_to_num(k, nan=0, posinf=0, neginf=0), np.nan_to_num(v, nan=0, posinf=0, neginf=0)
    want, want_lse, w, mag, reach = oc.attend(q.double().cpu().numpy(), k, v, s.table.cpu().numpy(), n, scale, window,
                                              None if mask is None else mask.cpu().numpy())
    u = U[s.kind]
    err = (s.dim + 8) * 2.0 ** -24 * reach
    rel = 2 * err + (max(n, default=0) / 8 + 8) * 2.0 ** -23
    got = out.double().cpu().numpy()
    tiny = 2.0 ** -24 if s.kind == "fp16" else 0.0  # float16's smallest step
    assert np.all(np.abs(got - want) <= mag * (1.01 * u + rel[..., None]) + u * np.abs(want) + tiny)
    if lse is not None:
        got = lse.double().cpu().numpy()
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(got))
        got, want_lse, slack = got[~none], want_lse[~none], rel[~none]
        assert np.all(np.abs(got - want_lse) <= slack + 2.0 ** -22 * (1 + np.abs(want_lse)))
    if scores is not None:
        got, old = scores.double().cpu().numpy(), before.double().cpu().numpy()
        b = rel.reshape(s.n_seq, s.heads, -1).max(2) + 2.0 ** -22
        assert np.all(np.abs(got - old - w) <= w * b[..., None] + 2.0 ** -23 * (np.abs(old) + w))
        assert np.array_equal(got[w == 0], old[w == 0])  # slots that are not seen keep theirs
    no_device_error()


def attend(s, n_q, scores=False, **kw):
    q = s.queries(n_q)
    lse = torch.full((s.n_seq, n_q), 7.0, device="cuda")
    sc = torch.rand((s.n_seq, s.heads, s.cap), generator=s.g).cuda() if scores else None
    before = None if sc is None else sc.clone()
    out = lc().cache_attend(s.cache, q, s.lengths, lse=lse, scores=sc, **kw)
    check_attend(s, q, out, lse, sc, before, **kw)
    return q, out, lse, sc


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("dim", [64, 80, 96, 112, 128, 192, 256])
def test_attend_dims(kind, order, dim):
    attend(Setup(EDGES, dim=dim, kind=kind, order=order, seed=dim), 8, scores=True)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 24, 33, 72, 100, 130, 255])
def test_attend_odd_dims(kind, dim):
    attend(Setup([0, 1, 17, 64, 150], dim=dim, kind=kind, seed=dim), 6, scores=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 71])
def test_attend_groups(kind, group):
    attend(Setup([5, 0, 200], heads=3, dim=64, kind=kind, seed=group), 3 * group, scores=True)
    attend(Setup([70], heads=1, dim=128, kind=kind, seed=group), group)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 1000])
def test_attend_pages(kind, page):
    attend(Setup([0, 1, page, page + 1, 2 * page + 5, 170], dim=128, page=page, kind=kind, seed=page), 4, scores=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 100, 1 << 30])
def test_attend_windows(kind, window):
    attend(Setup(EDGES, dim=128, kind=kind, seed=window), 4, scores=True, window=window)
    s = Setup([1000, 700], dim=64, kind=kind, seed=window)
    attend(s, 4, scores=True, window=window, mask=torch.rand((2, s.cap), generator=s.g).cuda() < 0.5)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
def test_attend_masks_and_poison(kind):
    """A mask that leaves nothing gives zeros, -inf and no weight; what unseen slots hold does not matter."""
    lens = [40, 40, 300, 1, 90]
    s = Setup(lens, dim=80, kind=kind, seed=3)
    mask = (torch.rand((5, s.cap), generator=s.g) < 0.5).to(torch.uint8)
    mask[0] = 0
    mask[1, :39] = 0
    mask[1, 39] = 255
    mask[2, 64:192] = 0
    table = s.table.cpu()
    for x, sc in zip((s.k, s.v), s.scales):
        for b, n in enumerate(lens):
            for j in range(s.cap):
                if j >= n or not mask[b, j]:
                    p, r = int(table[b, j // s.page]), j % s.page
                    if kind == "e4m3":
                        sc[p, :, r] = (math.nan, math.inf, -math.inf)[j % 3]
                    else:
                        x[p, :, r] = (math.nan, math.inf, -math.inf)[j % 3]
    q, out, lse, sc = attend(s, 4, scores=True, mask=mask.cuda())
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0]))
    mb = mask.bool().cuda()
    assert torch.equal(lc().cache_attend(s.cache, q, s.lengths, mask=mb), out)
    # a mask stretched over one row
    one = mask[2:3].cuda().expand(5, -1)
    assert one.stride(0) == 0
    check = torch.empty_like(lse)
    got = lc().cache_attend(s.cache, q, s.lengths, mask=one, lse=check)
    assert torch.equal(got[2], out[2]) and torch.equal(check[2], lse[2])


def test_attend_nan_and_infinity_in_seen_slots():
    """A NaN key, or a logit of +infinity, makes its row NaN; a logit of -infinity is a weight of zero."""
    s = Setup([30, 30, 30, 30], heads=1, dim=64, kind="bf16", seed=4)
    at = [(int(s.table[b, 0]), 5) for b in range(4)]
    q = s.queries(2)
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    s.k[at[0][0], 0, 5, 3] = math.nan
    s.k[at[1][0], 0, 5, 0] = math.inf
    s.v[at[2][0], 0, 5, 3] = math.nan
    out = lc().cache_attend(s.cache, q, s.lengths)
    assert torch.all(torch.isnan(out[0])) and torch.all(torch.isnan(out[1, 0]))
    assert torch.all(torch.isfinite(out[1, 1]))
    assert torch.all(torch.isnan(out[2, :, 3])) and torch.all(torch.isfinite(out[2, :, 4:]))
    assert torch.all(torch.isfinite(out[3]))
    # the slot of weight zero is as good as masked
    mask = torch.ones((4, s.cap), dtype=torch.bool, device="cuda")
    mask[1, 5] = False
    assert torch.allclose(lc().cache_attend(s.cache, q, s.lengths, mask=mask)[1, 1].float(), out[1, 1].float(), atol=1e-2)
    # every logit -infinity: nothing is left
    t = Setup([3], heads=1, dim=64, kind="bf16", seed=5)
    t.k[:, :, :, 0] = math.inf
    q = t.queries(1).abs()
    q[..., 0] = -1.0
    lse = torch.empty((1, 1), device="cuda")
    out = lc().cache_attend(t.cache, q, t.lengths, lse=lse)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    no_device_error()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_attend_unaligned_pools(kind, shift):
    attend(Setup([0, 1, 50, 200], dim=64, kind=kind, seed=shift, shift=shift), 8, scores=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attend_strided_arguments(kind):
    s = Setup([20, 333, 64], heads=2, dim=96, kind=kind, order="token", seed=6)
    q = s.queries(4)
    wide = torch.zeros((3, 4, 3, 97), dtype=q.dtype, device="cuda")
    wide[:, :, 1, 1:] = q
    qs = wide[:, :, 1, 1:]
    out = torch.full((3, 5, 2, 96), 9.0, dtype=q.dtype, device="cuda")
    lse = torch.zeros((3, 9), device="cuda")
    sc = torch.zeros((3, 3, s.cap + 5), device="cuda")
    got = lc().cache_attend(s.cache, qs, s.lengths, out=out[:, :4, 1], lse=lse[:, 2:6], scores=sc[:, 1:, 3:-2])
    check_attend(s, q, got, lse[:, 2:6], sc[:, 1:, 3:-2], torch.zeros_like(sc[:, 1:, 3:-2]))
    assert torch.all(out[:, 4] == 9) and torch.all(out[:, :4, 0] == 9)
    assert torch.all(lse[:, :2] == 0) and torch.all(lse[:, 6:] == 0)
    assert torch.all(sc[:, 0] == 0) and torch.all(sc[:, 1:, :3] == 0) and torch.all(sc[:, 1:, -2:] == 0)


@pytest.mark.parametrize("kind,dim,n", [("bf16", 128, 20011), ("fp16", 64, 33000), ("e4m3", 128, 40001),
                                        ("bf16", 256, 9001)])
def test_attend_long(kind, dim, n):
    """One sequence over the whole GPU, split and joined; logits large enough that a few slots dominate."""
    attend(Setup([n], heads=1, dim=dim, kind=kind, seed=n, page=64), 5, scores=True, scale=0.4)
    attend(Setup([n // 2, 3, n // 3], heads=2, dim=dim, kind=kind, seed=n), 4, scores=True)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("dim,group", [(64, 3), (64, 12), (96, 8), (128, 9), (128, 20), (256, 2), (256, 16)])
def test_attend_units_cut_into_runs(kind, dim, group):
    """Units enough and long enough to be cut into runs, whole units among them, with windows and masks."""
    wide = 2 * dim * (1 if kind == "e4m3" else 2) > 256  # steps of 16 slots, else of 32
    n = 2100 if wide else 4200
    s = Setup([n, 35, 0, n // 2 + 1], heads=12, dim=dim, kind=kind, page=30, order="token", seed=dim + group)
    attend(s, 12 * group, scores=True)
    if group < 10:
        attend(s, 12 * group)
        mask = (torch.rand((4, s.cap), generator=s.g) < 0.5).cuda()
        mask[0, 100:1500] = False
        attend(s, 12 * group, scores=True, mask=mask, window=n - 7)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("dim,group", [(80, 8), (80, 12), (160, 3), (192, 16), (144, 9)])
def test_attend_between_padded_sizes_in_runs(kind, dim, group):
    """Head sizes that are padded to less than a power of two, units cut into many parts."""
    s = Setup([4300, 35, 0, 2051], heads=12, dim=dim, kind=kind, page=30, seed=dim + group)
    attend(s, 12 * group, scores=True)
    s = Setup([26001], heads=1, dim=dim, kind=kind, page=64, seed=dim)
    attend(s, group, window=25000)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("dim,group", [(64, 1), (64, 16), (80, 3), (128, 4), (128, 12), (192, 9), (256, 2), (256, 16)])
def test_attend_a_unit_a_warp(kind, dim, group):
    """Many units of few steps, of every length from none, their number no multiple of a block's."""
    s = Setup([(5 * i) % 67 for i in range(211)], heads=3, dim=dim, kind=kind, page=16, order="token", seed=dim + group)
    attend(s, 3 * group, scores=True)
    mask = (torch.rand((211, s.cap), generator=s.g) < 0.5).cuda()
    mask[::4] = False
    attend(s, 3 * group, scores=True, mask=mask, window=40)
    attend(s, 3 * group)


def test_attend_many_sequences():
    attend(Setup([(7 * i) % 97 for i in range(700)], heads=1, dim=64, seed=8), 2, scores=True)
    attend(Setup([(131 * i) % 900 for i in range(150)], heads=4, dim=128, seed=9), 16, scores=True)
    attend(Setup([0] * 40, heads=2, dim=64, per=4, seed=9), 2, scores=True)
    attend(Setup([0], heads=2, dim=64, per=4, seed=9), 2, scores=True)


def test_attend_growing_maximum():
    """Logits that rise along the sequence by more than exp's range: earlier sums vanish without a trace."""
    s = Setup([500], heads=1, dim=64, kind="fp16", seed=10)
    s.k.zero_()
    t = s.table.cpu()
    for j in range(500):
        s.k[int(t[0, j // 16]), 0, j % 16, 0] = j
    q = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda")
    q[0, 0, 0], q[0, 1, 0] = 1.0, -1.0
    lse = torch.empty((1, 2), device="cuda")
    out = lc().cache_attend(s.cache, q, s.lengths, scale=1.0, lse=lse)
    check_attend(s, q, out, lse, scale=1.0)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
def test_attend_many_small_weights_under_one_large(kind):
    """One slot's logit 18 above all the others': each of those weighs 2^-26 of it, together half a
    thousandth, which no 16-bit weight may lose."""
    n = 40000
    s = Setup([n], heads=1, dim=64, page=100, kind=kind, seed=15)
    table = s.table[0].long()
    if kind == "e4m3":
        s.k.view(torch.uint8).zero_()
        s.v.view(torch.uint8).copy_((torch.ones_like(s.v, dtype=torch.float32)).to(torch.float8_e4m3fn).view(torch.uint8))
        s.scales[0].fill_(1.0)
        s.scales[1].fill_(0.01)
    else:
        s.k.zero_()
        s.v.fill_(0.01)
    top = torch.full((64,), 2.25).to(s.k.dtype)
    at = (int(table[3]), 0, 17)
    (s.k.view(torch.uint8) if kind == "e4m3" else s.k)[at] = (top.view(torch.uint8) if kind == "e4m3" else top).cuda()
    s.v.view(torch.uint8 if kind == "e4m3" else s.v.dtype)[at] = 0
    q = torch.full((1, 2, 64), 1.0, dtype=IO[kind], device="cuda")
    lse = torch.empty((1, 2), device="cuda")
    out = lc().cache_attend(s.cache, q, s.lengths, scale=0.125, lse=lse)
    check_attend(s, q, out, lse, scale=0.125)
    assert torch.all(out > 0.01 * 5e-4)


def test_attend_offsets_past_32_bits():
    """Pages more than 2^32 elements apart."""
    gap = 2_500_000_000
    flat = torch.zeros(2 * gap + 4096, dtype=torch.bfloat16, device="cuda")
    s = Setup([40], heads=1, dim=64, page=16, seed=11)
    k = torch.as_strided(flat, (3, 1, 16, 64), (gap, 2048, 64, 1))
    v = torch.as_strided(flat, (3, 1, 16, 64), (gap, 2048, 64, 1), 1024)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    k.copy_(s.k[s.table[0].long()][[1, 2, 0]])
    v.copy_(s.v[s.table[0].long()][[1, 2, 0]])
    q = s.queries(2)
    want = lc().cache_attend(s.cache, q, s.lengths)
    cache = lc().PagedCache(k, v, table)
    assert torch.equal(lc().cache_attend(cache, q, s.lengths), want)
    new = torch.randn((1, 2, 1, 64), device="cuda").bfloat16()
    lc().cache_append(cache, new, new, torch.tensor([7], dtype=torch.int32, device="cuda"))
    assert torch.equal(k[2, 0, 7:9], new[0, :, 0]) and torch.equal(v[2, 0, 7:9], new[0, :, 0])
    sc = torch.arange(48, dtype=torch.float32, device="cuda").reshape(1, 1, 48)
    rows = torch.cat([k[i, 0] for i in (2, 0, 1)]).clone()
    kept, _, n = lc().cache_evict(cache, s.lengths, sc, 20, 4)
    assert int(n) == 20 and kept[0, 0].tolist() == list(range(20, 40))
    assert torch.equal(torch.cat([k[i, 0] for i in (2, 0, 1)])[:20], rows[20:40])
    no_device_error()


def test_attend_is_repeatable_and_runs_on_any_stream_and_in_graphs():
    s = Setup([3000, 17, 1200, 0], heads=2, dim=128, seed=12)
    q, out, lse, _ = attend(s, 8)
    for _ in range(5):
        assert torch.equal(lc().cache_attend(s.cache, q, s.lengths), out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lc().cache_attend(s.cache, q, s.lengths, stream=side)
    got2 = lc().cache_attend(s.cache, q, s.lengths, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, out) and torch.equal(got2, out)
    scores = torch.zeros((4, 2, s.cap), device="cuda")
    ws = lc().cache_attend_workspace(s.cache, 8, True)
    res, graph = torch.empty_like(out), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lc().cache_attend(s.cache, q, s.lengths, out=res, scores=scores, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(res, out)
    total = scores.sum(2)
    assert torch.allclose(total, torch.where(s.lengths > 0, 12.0, 0.0)[:, None].expand(4, 2), atol=1e-3)


def device_error_is(status):
    st, _ = lc().last_device_error()
    assert st == lc().STATUS[status]
    no_device_error()  # reading it cleared it


@pytest.mark.parametrize("kind,dim", [("bf16", 64), ("e4m3", 128), ("fp16", 33)])
def test_bad_device_indices_are_reported(kind, dim):
    """A length past the capacity is clamped, a page id outside the pool makes its slots unseen; both are recorded."""
    s = Setup([40, 40, 40], dim=dim, per=3, page=16, kind=kind, seed=13)
    q = s.queries(4)
    lens = torch.tensor([40, 1000, -5], dtype=torch.int32, device="cuda")
    out = lc().cache_attend(s.cache, q, lens)
    device_error_is("LC_ERR_CACHE_INDEX")
    check_attend(s, q, out, None, lengths=np.array([40, 48, 0]))
    table = s.table.clone()
    for bad in (-1, s.k.shape[0], 1 << 30, -(1 << 31)):
        t = table.clone()
        t[1, 1] = bad
        c = lc().PagedCache(s.k, s.v, t, *s.scales)
        out = lc().cache_attend(c, q, s.lengths)
        device_error_is("LC_ERR_CACHE_INDEX")
        mask = torch.ones((3, s.cap), dtype=torch.bool, device="cuda")
        mask[1, 16:32] = False
        check_attend(s, q, out, None, mask=mask)
        before = (s.k.view(torch.uint8) if kind == "e4m3" else s.k).clone()
        new = torch.randn((3, 4, 2, dim), device="cuda").to(IO[kind])
        n = lc().cache_append(c, new, new, torch.tensor([14, 14, 47], dtype=torch.int32, device="cuda"))
        device_error_is("LC_ERR_CACHE_INDEX")
        assert n.tolist() == [18, 18, 48]
        after = s.k.view(torch.uint8) if kind == "e4m3" else s.k
        changed = (before != after).flatten(1).any(1).nonzero().flatten().tolist()
        assert sorted(changed) == sorted(int(x) for x in (t[0, 0], t[0, 1], t[1, 0], t[2, 2]))
        sc = torch.rand((3, 2, s.cap), device="cuda")
        lc().cache_evict(c, s.lengths, sc, 20, 3)
        device_error_is("LC_ERR_CACHE_INDEX")


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def raw(x):
    return x.contiguous().view(torch.uint8 if x.element_size() == 1 else torch.int16).cpu().numpy()


def check_append(s, new, lengths, counts, got_lengths, before, before_scales):
    n, m = lengths.tolist(), ([new[0].shape[1]] * s.n_seq if counts is None else counts.tolist())
    to, want_len = oc.append_slots(n, m, s.cap)
    assert got_lengths.tolist() == want_len
    table = s.table.cpu().numpy()
    for x, pool, old, scale, old_scale in zip(new, (s.k, s.v), before, s.scales, before_scales):
        want, ws = raw(old), None if old_scale is None else old_scale.cpu().numpy().copy()
        xs = x.float().cpu().numpy()
        xr = raw(x)
        got = raw(pool)
        for b, t, j in to:
            p, r = table[b, j // s.page], j % s.page
            for h in range(s.heads):
                if s.kind == "e4m3":
                    vals, sc = oc.quantise(xs[b, t, h])
                    ws[p, h, r] = sc
                    if np.isnan(sc):
                        want[p, h, r] = got[p, h, r]  # the scale says it all
                    else:
                        mine = np.array([oc.e4m3_value(int(c)) for c in got[p, h, r]])
                        assert np.array_equal(mine, vals)
                        want[p, h, r] = got[p, h, r]
                else:
                    want[p, h, r] = xr[b, t, h]
        assert np.array_equal(got, want)
        if ws is not None:
            assert np.array_equal(scale.cpu().numpy(), ws, equal_nan=True)
    no_device_error()


@pytest.mark.parametrize("kind,io", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("dim,shift,order", [(64, 0, "head"), (128, 0, "token"), (256, 0, "head"), (80, 0, "token"),
                                             (1, 0, "head"), (33, 0, "token"), (72, 1, "head"), (255, 0, "head")])
def test_append(kind, io, dim, shift, order):
    s = Setup([0, 5, 30, 47, 12], dim=dim, per=3, page=16, kind=kind, order=order, seed=dim, shift=shift)
    for n_new, ragged in ((1, False), (7, True), (1, True)):
        new = [(torch.randn((5, n_new, 2, dim), generator=s.g) * 3).to(IO[io]).cuda() for _ in "kv"]
        new[0][1, 0] = 0
        if kind == "e4m3" and dim > 1:
            new[1][2, 0, 0, 1] = math.inf
            new[0][2, 0, 1, 0] = math.nan
            new[0][0, 0, 0] = new[0][0, 0, 0] * 1e-6
        counts = torch.tensor([0, n_new, 1, 1, max(1, n_new // 2)], dtype=torch.int32, device="cuda") if ragged else None
        lengths = s.lengths if ragged or n_new == 1 else s.lengths - n_new
        before = [x.clone() for x in (s.k, s.v)]
        scales = [None if x is None else x.clone() for x in s.scales]
        got = lc().cache_append(s.cache, new[0], new[1], lengths, counts)
        check_append(s, new, lengths, counts, got, before, scales)


def test_append_e4m3_rounds_as_torch_does():
    """Every bfloat16 magnitude beside a largest value of 448: the codes are torch's own conversion."""
    x = torch.arange(0, 0x43e1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # 0 .. 448
    rows = -(-x.numel() // 127)
    new = torch.zeros((rows, 128), dtype=torch.bfloat16)
    flat = torch.zeros(rows * 127, dtype=torch.bfloat16)
    flat[:x.numel()] = x
    new[:, :127] = flat.reshape(rows, 127)
    new[:, 127] = 448
    s = Setup([0], heads=1, dim=128, per=-(-rows // 16), kind="e4m3", seed=1)
    new = new.reshape(1, rows, 1, 128).cuda()
    lc().cache_append(s.cache, new, -new, s.lengths)
    for pool, sign in ((s.k, 1), (s.v, -1)):
        got = pool[s.table[0].long()].transpose(1, 2).reshape(-1, 128)[:rows]
        assert torch.equal(got.view(torch.uint8), (sign * new[0, :, 0].float()).to(torch.float8_e4m3fn).view(torch.uint8))
    assert torch.all(s.scales[0][s.table[0].long()].reshape(-1)[:rows] == 1)


def test_append_reports_what_does_not_fit():
    s = Setup([10, 46, 0], dim=64, per=3, seed=2)
    new = torch.randn((3, 4, 2, 64), device="cuda").bfloat16()
    before = [s.k.clone(), s.v.clone()]
    got = lc().cache_append(s.cache, new, new, s.lengths)
    device_error_is("LC_ERR_CACHE_INDEX")
    check_append(s, [new, new], s.lengths, None, got, before, [None, None])
    counts = torch.tensor([-3, 9, 2], dtype=torch.int32, device="cuda")  # clamped to 0 .. 4
    before = [s.k.clone(), s.v.clone()]
    got = lc().cache_append(s.cache, new, new, torch.zeros_like(s.lengths), counts)
    device_error_is("LC_ERR_CACHE_INDEX")
    check_append(s, [new, new], torch.zeros_like(s.lengths), counts.clamp(0, 4), got, before, [None, None])
    none = torch.empty((3, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(lc().cache_append(s.cache, none, none, s.lengths), s.lengths)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_strided_and_long(kind):
    s = Setup([0, 3], heads=3, dim=64, per=40, kind=kind, order="token", seed=3)
    wide = torch.randn((500, 2, 2, 3, 72), generator=s.g).bfloat16().cuda()
    k, v = (wide[:, :, i, :, :64].transpose(0, 1) for i in range(2))
    counts = torch.tensor([500, 499], dtype=torch.int32, device="cuda")
    before, scales = [s.k.clone(), s.v.clone()], [None if x is None else x.clone() for x in s.scales]
    got = lc().cache_append(s.cache, k, v, s.lengths, counts, stream=torch.cuda.current_stream())
    check_append(s, [k, v], s.lengths, counts, got, before, scales)


# ---------------------------------------------------------------------------
# evict
# ---------------------------------------------------------------------------

def check_evict(s, scores, budget, recent, **kw):
    n = s.lengths.tolist()
    table = s.table.cpu().numpy()
    pools = [s.k, s.v] + [x for x in s.scales if x is not None]
    want = [(raw(x) if x.dim() == 4 else x.cpu().numpy()).copy() for x in pools]
    sc = scores.cpu().numpy()
    kept, new_scores, new_n = lc().cache_evict(s.cache, s.lengths, scores, budget, recent, **kw)
    assert new_n.tolist() == [min(x, budget) for x in n]
    want_kept = np.full((s.n_seq, s.heads, budget), -1, np.int32)
    want_scores = np.zeros(sc.shape, np.float32)
    for b in range(s.n_seq):
        for h in range(s.heads):
            slots = oc.evict_kept(sc[b, h], n[b], budget, recent)
            want_kept[b, h, :len(slots)] = slots
            want_scores[b, h, :len(slots)] = sc[b, h, slots]
            for x in want:
                old = x.copy() if slots != list(range(len(slots))) else x
                for r, j in enumerate(slots):
                    if r != j:
                        x[table[b, r // s.page], h, r % s.page] = old[table[b, j // s.page], h, j % s.page]
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(new_scores.cpu().numpy(), want_scores, equal_nan=True)
    for x, w in zip(pools, want):
        assert np.array_equal(raw(x) if x.dim() == 4 else x.cpu().numpy(), w)
    no_device_error()
    return kept, new_scores, new_n


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("dim,shift,order", [(64, 0, "head"), (80, 0, "token"), (256, 0, "head"), (33, 0, "token"),
                                             (1, 0, "head"), (128, 1, "head"), (24, 0, "token")])
def test_evict(kind, dim, shift, order):
    for budget, recent in ((1, 0), (1, 1), (20, 0), (20, 5), (20, 20), (64, 3), (200, 10), (5000, 100)):
        s = Setup([0, 1, 20, 21, 63, 64, 65, 190], dim=dim, kind=kind, order=order, seed=budget, shift=shift)
        check_evict(s, torch.rand((8, 2, s.cap), generator=s.g).cuda(), budget, recent)


def test_evict_ties_and_odd_scores():
    """Equal scores keep the lowest slots; -0 is 0, NaN is the least, negatives and infinities are in order."""
    s = Setup([150, 150, 150, 150, 33], dim=64, seed=1)
    x = torch.randint(0, 3, (5, 2, s.cap), generator=s.g).float()
    x[1] = 0
    x[1, 0, 7], x[1, 0, 70] = -0.0, -1.0
    x[2] = torch.randn((2, s.cap), generator=s.g) * 1e-40  # subnormals
    x[3, 0, :50], x[3, 0, 50:80], x[3, 1, ::3] = math.nan, -math.inf, math.inf
    for budget, recent in ((1, 0), (31, 4), (100, 0), (120, 30), (149, 0)):
        check_evict(s, x.cuda(), budget, recent)


@pytest.mark.parametrize("n,budget,recent", [(20000, 7000, 100), (20000, 19999, 0), (33333, 12, 3), (9000, 4096, 4096)])
def test_evict_long(n, budget, recent):
    s = Setup([n, n // 2], heads=2, dim=16, page=64, seed=n)
    x = torch.exp(3 * torch.randn((2, 2, s.cap), generator=s.g))
    x[0, 1] = (x[0, 1] * 2).round()  # many ties
    check_evict(s, x.cuda(), budget, recent)


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3", 64), ("fp16", 32), ("e4m3", 16)])
@pytest.mark.parametrize("cap", [8192, 8208])
def test_evict_at_the_bound_of_one_launch(kind, dim, cap):
    """Capacities and budgets on both sides of what one launch takes, with short sequences beside the long one."""
    n = [cap, 1, 31, 32, 33, 64, 700, 2049]
    for budget, recent in ((1, 1), (33, 0), (255, 60), (257, 0), (2048, 16), (cap - 1, 0)):
        s = Setup(n, dim=dim, kind=kind, seed=budget + dim)
        x = torch.rand((8, 2, s.cap), generator=s.g)
        x[1:3] = (x[1:3] * 3).round()
        check_evict(s, x.cuda(), budget, recent)


def test_evict_more_slots_than_shared_memory_holds():
    """Units too many for clusters, of more slots than a block holds keys of."""
    n = [50001, 49500] + [30 + i for i in range(78)]
    s = Setup(n, heads=1, dim=8, page=50, seed=4)
    x = torch.exp(2 * torch.randn((80, 1, s.cap), generator=s.g))
    x[1] = (x[1] * 4).round()
    check_evict(s, x.cuda(), 4000, 50)
    s = Setup(n[1:2] + n[2:], heads=1, dim=8, page=50, seed=5)
    check_evict(s, (4 * x[1:]).round().cuda()[..., :s.cap].contiguous(), 40, 0)


@pytest.mark.parametrize("lengths,heads", [([430001, 9], 1), ([20000, 16500, 40], 90), ([40000] * 3, 60)])
def test_evict_clusters(lengths, heads):
    """More slots than a cluster's blocks hold keys of, and clusters of units too many for an SM a block."""
    s = Setup(lengths, heads=heads, dim=8, page=500, seed=heads)
    x = torch.exp(2 * torch.randn((len(lengths), heads, s.cap), generator=s.g))
    x[:, ::2] = (x[:, ::2] * 4).round()
    check_evict(s, x.cuda(), 700, 50)


def test_evict_strided_arguments_and_streams():
    s = Setup([100, 60], heads=2, dim=64, seed=2)
    wide = torch.rand((2, 3, s.cap + 3), generator=s.g).cuda()
    kept = torch.full((2, 3, 40), 5, dtype=torch.int32, device="cuda")
    new = torch.full((2, 3, s.cap + 3), 5.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_evict(s, wide[:, 1:, 1:-2], 37, 6, kept=kept[:, :2, 2:39], new_scores=new[:, 1:, 1:-2], stream=side)
    side.synchronize()
    assert torch.all(kept[:, 2] == 5) and torch.all(kept[:, :, :2] == 5) and torch.all(kept[:, :, 39:] == 5)
    assert torch.all(new[:, 0] == 5) and torch.all(new[..., 0] == 5) and torch.all(new[..., -2:] == 5)


def test_evict_many_sequences():
    s = Setup([(37 * i) % 120 for i in range(200)], heads=3, dim=32, seed=3)
    check_evict(s, torch.rand((200, 3, s.cap), generator=s.g).cuda(), 50, 8)


def test_no_sequences_and_no_capacity():
    s = Setup([5, 9], heads=2, dim=64)
    none = lc().PagedCache(s.k, s.v, s.table[:, :0])       # no slots: nothing fits, nothing is seen
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = s.queries(4)
    lse, scores = torch.zeros((2, 4), device="cuda"), torch.zeros((2, 2, 0), device="cuda")
    out = lc().cache_attend(none, q, zero, lse=lse, scores=scores)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    kept, new_scores, n = lc().cache_evict(none, zero, scores, 3)
    assert torch.all(kept == -1) and new_scores.shape == (2, 2, 0) and torch.equal(n, zero)
    empty = torch.zeros((2, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(lc().cache_append(none, empty, empty, zero), zero)
    no_device_error()
    one = empty.new_zeros((2, 1, 2, 64))
    assert torch.equal(lc().cache_append(none, one, one, zero), zero)
    device_error_is("LC_ERR_CACHE_INDEX")
    nobody = lc().PagedCache(s.k, s.v, s.table[:0])
    no = zero[:0]
    assert lc().cache_attend(nobody, q[:0], no).shape == (0, 4, 64)
    assert lc().cache_append(nobody, empty[:0], empty[:0], no).shape == (0,)
    assert lc().cache_evict(nobody, no, torch.zeros((0, 2, s.cap), device="cuda"), 3)[0].shape == (0, 2, 3)
    no_device_error()


# ---------------------------------------------------------------------------
# refusals of the Python entry points
# ---------------------------------------------------------------------------

def test_python_refusals():
    M = lc()
    s = Setup([10, 20], heads=2, dim=64)
    q = s.queries(4)
    ok = dict(k=s.k, v=s.v, page_table=s.table)
    for bad in (dict(k=s.k.cpu()), dict(k=s.k.float()), dict(v=s.v[:, :1]), dict(v=s.v.half()), dict(k=s.k[0]),
                dict(page_table=s.table.long()), dict(page_table=s.table[0]), dict(page_table=s.table.t()),
                dict(k=s.k.transpose(2, 3), v=s.v.transpose(2, 3)),
                dict(k_scale=torch.ones(s.k.shape[:3], device="cuda"), v_scale=torch.ones(s.k.shape[:3], device="cuda")),
                dict(k=s.k.to(torch.float8_e4m3fn), v=s.v.to(torch.float8_e4m3fn))):
        with pytest.raises(ValueError):
            M.PagedCache(**{**ok, **bad})
    for bad in (dict(q=q.half()), dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q[0]), dict(q=q.cpu()),
                dict(lengths=s.lengths.long()), dict(lengths=s.lengths[:1]),
                dict(mask=torch.ones((2, s.cap + 1), dtype=torch.bool, device="cuda")),
                dict(mask=torch.ones((2, s.cap), device="cuda")), dict(lse=torch.empty((2, 3), device="cuda")),
                dict(scores=torch.empty((2, 2, s.cap), dtype=torch.float64, device="cuda")),
                dict(scores=torch.empty((2, 4, s.cap), device="cuda")), dict(out=torch.empty_like(q).half()),
                dict(workspace=torch.empty(64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            M.cache_attend(s.cache, **{**dict(q=q, lengths=s.lengths), **bad})
    with pytest.raises(M.LayoutCopyError):
        M.cache_attend(s.cache, q, s.lengths, window=-1)
    with pytest.raises(M.LayoutCopyError):
        M.cache_attend(s.cache, q, s.lengths, out=torch.empty_like(q[:1]).expand_as(q))
    new = torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k=new.half()), dict(k=new.float(), v=new.float()), dict(k=new[:, 0]), dict(v=new[:, :, :1]),
                dict(lengths=s.lengths.long()), dict(counts=s.lengths[:1]), dict(new_lengths=s.lengths.long())):
        with pytest.raises(ValueError):
            M.cache_append(s.cache, **{**dict(k=new, v=new, lengths=s.lengths), **bad})
    for bad, status in ((dict(k=new.half(), v=new.half()), "LC_ERR_TYPE"), (dict(new_lengths=s.lengths), "LC_ERR_OVERLAP")):
        with pytest.raises(M.LayoutCopyError) as e:
            M.cache_append(s.cache, **{**dict(k=new, v=new, lengths=s.lengths), **bad})
        assert e.value.status == M.STATUS[status]
    sc = torch.zeros((2, 2, s.cap), device="cuda")
    for bad in (dict(scores=sc.double()), dict(scores=sc[:1]), dict(lengths=s.lengths.long()),
                dict(kept=torch.empty((2, 2, 7), dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            M.cache_evict(s.cache, **{**dict(lengths=s.lengths, scores=sc, budget=8), **bad})
    for bad, status in ((dict(budget=0), "LC_ERR_SHAPE"), (dict(recent=9), "LC_ERR_SHAPE"), (dict(recent=-1), "LC_ERR_SHAPE"),
                        (dict(new_scores=sc), "LC_ERR_OVERLAP"), (dict(new_lengths=s.lengths), "LC_ERR_OVERLAP")):
        with pytest.raises(M.LayoutCopyError) as e:
            M.cache_evict(s.cache, **{**dict(lengths=s.lengths, scores=sc, budget=8), **bad})
        assert e.value.status == M.STATUS[status]
    no_device_error()
