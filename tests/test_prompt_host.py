"""Refusals of the prompt, draft-tree and page-reservation entry points (no GPU): nothing is read from the addresses."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import movement_primitives_gb300
    return movement_primitives_gb300


BASE = 1 << 24  # an address, and far more bytes than any argument below has


def status(M, code):
    return M._lib.STATUS_NAMES[code]


def fill(x, kw):
    for k, y in kw.items():
        if isinstance(y, tuple):
            getattr(x, k)[:] = y
        else:
            setattr(x, k, y)


def prompt(M, **kw):
    """20 tokens of 4 query and 2 key heads of 64."""
    p = M._lib.CPrompt()
    p.q, p.k, p.v, p.out, p.lse, p.starts, p.k_starts = (i * BASE for i in range(1, 8))
    p.n_tokens, p.n_keys, p.type, p.n_seqs, p.n_q_heads, p.n_kv_heads, p.head_dim = 20, 20, 0, 3, 4, 2, 64
    p.causal, p.window, p.scale = 1, 0, 0.125
    p.q_stride[:] = p.out_stride[:] = (256, 64)
    p.k_stride[:] = p.v_stride[:] = (128, 64)
    p.lse_stride = 4
    fill(p, kw)
    return status(M, M._lib.lib().lc_prompt_attend(ctypes.byref(p), None))


@pytest.mark.parametrize("kw,want", [
    (dict(type=2), "LC_ERR_TYPE"), (dict(n_seqs=-1), "LC_ERR_SHAPE"), (dict(n_q_heads=3), "LC_ERR_SHAPE"),
    (dict(n_kv_heads=0), "LC_ERR_SHAPE"), (dict(head_dim=0), "LC_ERR_SHAPE"), (dict(head_dim=60), "LC_ERR_SHAPE"),
    (dict(head_dim=264), "LC_ERR_SHAPE"), (dict(n_tokens=-1), "LC_ERR_SHAPE"), (dict(window=-1), "LC_ERR_SHAPE"),
    (dict(scale=math.inf), "LC_ERR_SHAPE"), (dict(scale=math.nan), "LC_ERR_SHAPE"),
    (dict(n_tokens=(1 << 30) + 1), "LC_ERR_OVERFLOW"), (dict(n_keys=1 << 40), "LC_ERR_OVERFLOW"),
    (dict(q=None), "LC_ERR_NULL"), (dict(out=None), "LC_ERR_NULL"), (dict(starts=None), "LC_ERR_NULL"), (dict(k=None), "LC_ERR_NULL"),
    (dict(q_stride=(0, 64)), "LC_ERR_BAD_STRIDE"), (dict(k_stride=(128, 0)), "LC_ERR_BAD_STRIDE"),
    (dict(v_stride=(-128, 64)), "LC_ERR_BAD_STRIDE"), (dict(k_stride=(1 << 38, 64)), "LC_ERR_OVERFLOW"),
    (dict(q=BASE + 2), "LC_ERR_ALIGN"), (dict(k_stride=(132, 64)), "LC_ERR_ALIGN"), (dict(v=3 * BASE + 8), "LC_ERR_ALIGN"),
    (dict(out=4 * BASE + 1), "LC_ERR_ALIGN"), (dict(starts=6 * BASE + 2), "LC_ERR_ALIGN"),
    (dict(out_stride=(64, 64)), "LC_ERR_NOT_INJECTIVE"), (dict(lse_stride=3), "LC_ERR_NOT_INJECTIVE"),
    (dict(n_tokens=0), "LC_OK"), (dict(n_seqs=0), "LC_OK"),
])
def test_prompt_refusals(M, kw, want):
    assert prompt(M, **kw) == want


def test_prompt_refuses_an_output_over_its_inputs(M):
    size = 20 * 256 * 2
    for at in (2 - size, -512, -2, 2, 128, size - 2):
        assert prompt(M, out=BASE + at) == "LC_ERR_OVERLAP"
    for pool in (2, 3):
        for at in (2 - size, 0, 20 * 128 * 2 - 2):
            assert prompt(M, out=pool * BASE + at) == "LC_ERR_OVERLAP"
    # the queries' own rows in another order
    assert prompt(M, out=BASE, out_stride=(64, 64 * 20)) == "LC_ERR_OVERLAP"
    # one buffer of rows [q k v]: out may not reach the keys
    rows = dict(q_stride=(512, 64), k=BASE + 512, v=BASE + 768, k_stride=(512, 64), v_stride=(512, 64), out_stride=(512, 64))
    assert prompt(M, out=BASE + 2, **rows) == "LC_ERR_OVERLAP" == prompt(M, out=BASE + 512, **rows)


def cache(M, **kw):
    c = M._lib.CPagedCache()
    c.k, c.v, c.page_table = 8 * BASE, 9 * BASE, 10 * BASE
    c.type, c.n_seqs, c.n_kv_heads, c.page_size, c.head_dim, c.pages_per_seq, c.n_pages = 0, 2, 4, 16, 64, 3, 9
    c.table_stride = 3
    c.k_stride[:] = c.v_stride[:] = (4 * 16 * 64, 16 * 64, 64)
    fill(c, kw)
    return c


def tree(M, c=None, **kw):
    """Two sequences of 3 drafts of 8 heads of 64."""
    t = M._lib.CCacheTree()
    t.q, t.out, t.lengths, t.counts, t.parents, t.lse, t.workspace = (i * BASE for i in range(1, 8))
    t.type, t.n_q_heads, t.n_drafts, t.window, t.scale = 0, 8, 3, 0, 0.125
    t.q_stride[:] = t.out_stride[:] = (3 * 512, 512, 64)
    t.parents_stride, t.workspace_bytes = 3, 1 << 40
    t.lse_stride[:] = (24, 8)
    fill(t, kw)
    return status(M, M._lib.lib().lc_cache_attend_tree(ctypes.byref(c or cache(M)), ctypes.byref(t), None))


@pytest.mark.parametrize("kw,want", [
    (dict(type=1), "LC_ERR_TYPE"), (dict(n_q_heads=6), "LC_ERR_SHAPE"), (dict(n_q_heads=0), "LC_ERR_SHAPE"),
    (dict(n_drafts=65), "LC_ERR_SHAPE"), (dict(n_drafts=-1), "LC_ERR_SHAPE"), (dict(window=-1), "LC_ERR_SHAPE"),
    (dict(scale=math.nan), "LC_ERR_SHAPE"), (dict(q=None), "LC_ERR_NULL"), (dict(parents=None), "LC_ERR_NULL"),
    (dict(workspace=None), "LC_ERR_NULL"), (dict(workspace_bytes=1000), "LC_ERR_WORKSPACE"), (dict(workspace=7 * BASE + 16), "LC_ERR_ALIGN"),
    (dict(q=BASE + 1), "LC_ERR_ALIGN"), (dict(counts=4 * BASE + 2), "LC_ERR_ALIGN"), (dict(parents_stride=-3), "LC_ERR_BAD_STRIDE"),
    (dict(out_stride=(512, 512, 64)), "LC_ERR_NOT_INJECTIVE"), (dict(lse_stride=(8, 8)), "LC_ERR_NOT_INJECTIVE"),
    (dict(out=BASE), "LC_ERR_OVERLAP"), (dict(out=BASE + 2 * 3 * 1024 - 2), "LC_ERR_OVERLAP"), (dict(out=BASE - 2), "LC_ERR_OVERLAP"),
    (dict(n_q_heads=1 << 28, lse=None, out=1 << 50, q_stride=(3 << 34, 1 << 34, 64), out_stride=(3 << 34, 1 << 34, 64)), "LC_ERR_OVERFLOW"), (dict(n_drafts=0), "LC_OK"),
])
def test_tree_refusals(M, kw, want):
    assert tree(M, **kw) == want


def test_tree_refuses_more_steps_than_it_counts(M):
    assert tree(M, cache(M, n_seqs=100, pages_per_seq=1 << 26, table_stride=1 << 26)) == "LC_ERR_OVERFLOW"


def test_tree_workspace(M):
    size = lambda c, n, d: M._lib.lib().lc_cache_attend_tree_workspace(ctypes.byref(c), n, d)  # noqa: E731
    assert size(cache(M), 8, 3) > 0 and size(cache(M), 8, 64) >= size(cache(M), 8, 3)
    assert size(cache(M), 6, 3) == size(cache(M), 0, 3) == size(cache(M), 8, 65) == size(cache(M), 8, -1) == -1
    assert size(cache(M, head_dim=257), 8, 3) == -1


def accept(M, c=None, lengths=BASE, counts=2 * BASE, path=3 * BASE, path_stride=4, n_path=4, new=4 * BASE):
    return status(M, M._lib.lib().lc_cache_accept(ctypes.byref(c or cache(M)), lengths, counts, path, path_stride, n_path, new, None))


def test_accept_refusals(M):
    assert accept(M, n_path=65) == accept(M, n_path=-1) == "LC_ERR_SHAPE"
    assert accept(M, lengths=None) == accept(M, path=None) == accept(M, new=None) == "LC_ERR_NULL"
    assert accept(M, path=3 * BASE + 2) == accept(M, new=4 * BASE + 1) == "LC_ERR_ALIGN"
    assert accept(M, path_stride=-4) == "LC_ERR_BAD_STRIDE"
    for at in (-4, 0, 4):
        assert accept(M, new=BASE + at) == accept(M, new=2 * BASE + at) == "LC_ERR_OVERLAP"
    for at in (-4, 0, 28):
        assert accept(M, new=3 * BASE + at) == "LC_ERR_OVERLAP"
    assert accept(M, cache(M, n_seqs=0)) == "LC_OK"


def packed(M, c=None, k=BASE, v=2 * BASE, kind=0, stride=(256, 64), n=3, slots=3 * BASE):
    st = (ctypes.c_int64 * 2)(*stride)
    return status(M, M._lib.lib().lc_cache_append_packed(ctypes.byref(c or cache(M)), k, v, kind, st, st, n, slots, None))


def test_packed_append_refusals(M):
    assert packed(M, kind=1) == "LC_ERR_TYPE"
    assert packed(M, k=None) == packed(M, slots=None) == "LC_ERR_NULL"
    assert packed(M, slots=3 * BASE + 4) == "LC_ERR_ALIGN"
    assert packed(M, n=-1) == "LC_ERR_SHAPE"
    assert packed(M, stride=(-256, 64)) == "LC_ERR_BAD_STRIDE"
    assert packed(M, n=0) == "LC_OK"


def reserve(M, **kw):
    """Two sequences of up to three pages, five tokens."""
    r = M._lib.CCacheReservation()
    r.page_table, r.new_table, r.table_stride, r.new_table_stride = BASE, BASE, 3, 3
    (r.lengths, r.counts, r.free, r.n_free, r.new_n_free, r.new_lengths, r.starts, r.slots, r.positions,
     r.seqs) = (i * BASE for i in range(2, 12))
    r.free_size, r.n_seqs, r.pages_per_seq, r.page_size, r.max_tokens = 4, 2, 3, 16, 5
    fill(r, kw)
    return status(M, M._lib.lib().lc_cache_reserve(ctypes.byref(r), None))


@pytest.mark.parametrize("kw,want", [
    (dict(n_seqs=-1), "LC_ERR_SHAPE"), (dict(n_seqs=4097), "LC_ERR_SHAPE"), (dict(page_size=0), "LC_ERR_SHAPE"),
    (dict(pages_per_seq=-1), "LC_ERR_SHAPE"), (dict(max_tokens=-1), "LC_ERR_SHAPE"), (dict(free_size=-1), "LC_ERR_SHAPE"),
    (dict(page_size=1 << 30), "LC_ERR_OVERFLOW"), (dict(free_size=1 << 31), "LC_ERR_OVERFLOW"),
    (dict(n_free=None), "LC_ERR_NULL"), (dict(free=None), "LC_ERR_NULL"), (dict(slots=None), "LC_ERR_NULL"), (dict(page_table=None), "LC_ERR_NULL"),
    (dict(slots=9 * BASE + 4), "LC_ERR_ALIGN"), (dict(lengths=2 * BASE + 1), "LC_ERR_ALIGN"), (dict(table_stride=-3), "LC_ERR_BAD_STRIDE"),
    (dict(new_table=20 * BASE, new_table_stride=2), "LC_ERR_NOT_INJECTIVE"),
    (dict(new_table=BASE + 4), "LC_ERR_OVERLAP"), (dict(new_table_stride=4), "LC_ERR_OVERLAP"), (dict(new_lengths=2 * BASE + 4), "LC_ERR_OVERLAP"),
    (dict(new_n_free=5 * BASE), "LC_ERR_OVERLAP"), (dict(positions=9 * BASE + 16), "LC_ERR_OVERLAP"), (dict(starts=4 * BASE - 4), "LC_ERR_OVERLAP"),
    (dict(free=BASE + 20), "LC_ERR_OVERLAP"), (dict(seqs=3 * BASE), "LC_ERR_OVERLAP"),
])
def test_reserve_refusals(M, kw, want):
    assert reserve(M, **kw) == want


def test_null_structs_are_refused(M):
    lib = M._lib.lib()
    assert status(M, lib.lc_prompt_attend(None, None)) == status(M, lib.lc_cache_reserve(None, None)) == "LC_ERR_NULL"
    assert status(M, lib.lc_cache_attend_tree(ctypes.byref(cache(M)), None, None)) == "LC_ERR_NULL"
    assert status(M, lib.lc_cache_attend_tree(None, None, None)) == "LC_ERR_NULL"


def test_python_entry_points_refuse_cpu_tensors(M):
    torch = pytest.importorskip("torch")
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.prompt_attend(x, x, x, i)
    with pytest.raises(ValueError):
        M.cache_reserve(i.view(2, 1), i, i, i, i[:1], 16, 4)
