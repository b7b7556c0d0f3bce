"""Pins of the paged-cache oracle, and the ABI's refusals (no GPU)."""
import ctypes
import itertools
import math

import numpy as np
import pytest

from oracle import cache as oc


def test_attend_hand_worked():
    # two slots on two pages: weights 1/3 and 2/3 from logits 0 and log 2
    k = np.zeros((2, 1, 1, 1))
    k[1] = math.log(2.0)
    v = np.array([3.0, 6.0]).reshape(2, 1, 1, 1)
    table = np.array([[0, 1]])
    out, lse, w, _mag, _reach = oc.attend(np.ones((1, 1, 1)), k, v, table, [2], 1.0)
    assert np.allclose(w[0, 0], [1 / 3, 2 / 3]) and np.allclose(out, 5.0) and np.allclose(lse, math.log(3.0))
    # the table's order is the slots' order
    out2, _, w2, _, _ = oc.attend(np.ones((1, 1, 1)), k, v, table[:, ::-1], [2], 1.0)
    assert np.allclose(w2[0, 0], [2 / 3, 1 / 3]) and np.allclose(out2, out)


def test_attend_window_mask_and_empty():
    rng = np.random.default_rng(0)
    k, v, q = rng.standard_normal((5, 2, 4, 8)), rng.standard_normal((5, 2, 4, 8)), rng.standard_normal((3, 6, 8))
    table = np.array([[4, 2, 0], [1, 3, 0], [0, 0, 0]])
    lens = [11, 7, 0]
    out, lse, w, _, _ = oc.attend(q, k, v, table, lens, 0.3)
    assert np.allclose(w.sum(2), [[3, 3], [3, 3], [0, 0]])       # one per query head of the group
    assert np.all(out[2] == 0) and np.all(np.isneginf(lse[2]))
    # a window is a mask of the older slots
    mask = np.zeros((3, 12), bool)
    for b, n in enumerate(lens):
        mask[b, max(0, n - 4):n] = True
    for a, b in zip(oc.attend(q, k, v, table, lens, 0.3, window=4), oc.attend(q, k, v, table, lens, 0.3, mask=mask)):
        assert np.array_equal(a, b)
    # dense softmax of one head, written another way
    rows = [(table[0, j // 4], j % 4) for j in range(11)]
    x = np.array([0.3 * q[0, 4] @ k[p, 1, r] for p, r in rows])
    p = np.exp(x) / np.exp(x).sum()
    assert np.allclose(out[0, 4], sum(pi * v[pg, 1, r] for pi, (pg, r) in zip(p, rows)))


def test_e4m3_values_and_rounding():
    values = sorted(oc.e4m3_value(c) for c in range(127))
    assert values[0] == 0 and values[1] == 2.0 ** -9 and values[-1] == 448.0 and len(set(values)) == 127
    for c in range(127):
        assert oc.e4m3_round(oc.e4m3_value(c)) == oc.e4m3_value(c)
        assert oc.e4m3_round(-oc.e4m3_value(c)) == -oc.e4m3_value(c)
    by_code = [oc.e4m3_value(c) for c in range(127)]
    for c in range(126):  # midpoints go to the even code, either side of them to the nearer
        mid = (by_code[c] + by_code[c + 1]) / 2
        assert oc.e4m3_round(mid) == by_code[c + (c & 1)]
        assert oc.e4m3_round(mid * (1 + 1e-9)) == by_code[c + 1] and oc.e4m3_round(mid * (1 - 1e-9)) == by_code[c]
    assert oc.e4m3_round(1e9) == 448.0


def test_quantise_rows():
    x, s = oc.quantise([0.0, 0.0])
    assert s == np.float32(2.0 ** -126) and np.all(x == 0)
    x, s = oc.quantise([896.0, -448.0, 2.0])
    assert s == 2 and list(x) == [448.0, -224.0, 1.0]
    for bad in (math.inf, -math.inf, math.nan):
        assert math.isnan(oc.quantise([1.0, bad])[1])


def test_evict_against_enumeration():
    """The kept slots are the ones no other choice beats: by brute force on
    small integer scores with many ties."""
    rng = np.random.default_rng(1)
    for _ in range(300):
        n, budget = int(rng.integers(1, 9)), int(rng.integers(1, 9))
        recent = int(rng.integers(0, budget + 1))
        s = rng.integers(0, 3, n).astype(float)
        kept = oc.evict_kept(s, n, budget, recent)
        assert kept == sorted(set(kept)) and len(kept) == min(n, budget)
        if n > budget:
            assert kept[budget - recent:] == list(range(n - recent, n))
            best = max(itertools.combinations(range(n - recent), budget - recent),
                       key=lambda c: (sum(s[list(c)]), [-j for j in c]))
            got = kept[:budget - recent]
            assert sorted(s[list(best)]) == sorted(s[got])
            worst = min(s[got], default=None)
            for j in range(n - recent):  # of equal scores the lowest slots
                if j not in got and got:
                    assert s[j] < worst or (s[j] == worst and all(j > i for i in got if s[i] == worst))
    assert oc.evict_kept([1.0, math.nan, -math.inf, 0.5], 4, 2, 0) == [0, 3]
    assert oc.evict_kept([-0.0, 0.0, 0.0], 3, 2, 0) == [0, 1]


def test_append_slots_drop_past_capacity():
    assert oc.append_slots([0, 6], [2, 3], 8) == ([(0, 0, 0), (0, 1, 1), (1, 0, 6), (1, 1, 7)], [2, 8])


def test_planted_mistakes_are_caught(monkeypatch):
    real = oc.evict_kept
    monkeypatch.setattr(oc, "evict_kept", lambda s, n, b, r: real(list(s)[::-1], n, b, r))
    with pytest.raises(AssertionError):
        test_evict_against_enumeration()
    monkeypatch.setattr(oc, "evict_kept", real)
    real_seen = oc.seen_slots
    monkeypatch.setattr(oc, "seen_slots", lambda n, w=0, m=None: real_seen(n, w + 1 if w else 0, m))
    with pytest.raises(AssertionError):
        test_attend_window_mask_and_empty()
    monkeypatch.setattr(oc, "seen_slots", real_seen)
    monkeypatch.setattr(oc, "e4m3_round", lambda x: math.copysign(math.floor(abs(x)), x))
    with pytest.raises(AssertionError):
        test_e4m3_values_and_rounding()


# ---------------------------------------------------------------------------
# what the ABI refuses, before anything is launched
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import movement_primitives_gb300
    return movement_primitives_gb300


BASE = 1 << 20  # an address: nothing is read from it


def _cache(M, **kw):
    c = M._lib.CPagedCache()
    c.k, c.v, c.page_table = BASE, 2 * BASE, 3 * BASE
    c.type, c.n_seqs, c.n_kv_heads, c.page_size, c.head_dim, c.pages_per_seq, c.n_pages = 0, 2, 4, 16, 64, 3, 9
    c.table_stride = 3
    c.k_stride[:] = (4 * 16 * 64, 16 * 64, 64)
    c.v_stride[:] = (4 * 16 * 64, 16 * 64, 64)
    for k, x in kw.items():
        if isinstance(x, tuple):
            getattr(c, k)[:] = x
        else:
            setattr(c, k, x)
    return c


def _query(M, **kw):
    q = M._lib.CCacheQuery()
    q.q, q.out, q.lengths = 4 * BASE, 5 * BASE, 6 * BASE
    q.type, q.n_q_heads, q.scale = 0, 8, 0.125
    q.q_stride[:] = (8 * 64, 64)
    q.out_stride[:] = (8 * 64, 64)
    q.workspace, q.workspace_bytes = 16 * BASE, 1 << 40
    for k, x in kw.items():
        if isinstance(x, tuple):
            getattr(q, k)[:] = x
        else:
            setattr(q, k, x)
    return q


BAD_CACHES = [
    (dict(type=3), "LC_ERR_TYPE"), (dict(k=None), "LC_ERR_NULL"), (dict(v=None), "LC_ERR_NULL"),
    (dict(page_table=None), "LC_ERR_NULL"), (dict(type=2), "LC_ERR_NULL"),
    (dict(k_scale=BASE, v_scale=BASE), "LC_ERR_TYPE"), (dict(n_kv_heads=0), "LC_ERR_SHAPE"),
    (dict(page_size=0), "LC_ERR_SHAPE"), (dict(head_dim=0), "LC_ERR_SHAPE"), (dict(head_dim=257), "LC_ERR_SHAPE"),
    (dict(n_seqs=-1), "LC_ERR_SHAPE"), (dict(pages_per_seq=-1), "LC_ERR_SHAPE"), (dict(n_pages=-1), "LC_ERR_SHAPE"),
    (dict(n_pages=0), "LC_ERR_SHAPE"),
    (dict(k=BASE + 1), "LC_ERR_ALIGN"), (dict(page_table=BASE + 2), "LC_ERR_ALIGN"),
    (dict(k_stride=(4096, -1, 64)), "LC_ERR_BAD_STRIDE"), (dict(table_stride=-1), "LC_ERR_BAD_STRIDE"),
    (dict(v_stride=(1 << 61, 1024, 64)), "LC_ERR_OVERFLOW"),
    (dict(page_size=1 << 16, pages_per_seq=1 << 15), "LC_ERR_OVERFLOW"),
]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_operator_refuses_a_bad_cache(M, bad, status):
    lib, names, c = M._lib.lib(), M._lib.STATUS_NAMES, _cache(M, **bad)
    st = (ctypes.c_int64 * 3)(4 * 64, 4 * 64, 64)
    assert names[lib.lc_cache_append(ctypes.byref(c), BASE, BASE, 0, st, st, 1, None, BASE, 2 * BASE, None)] == status
    assert names[lib.lc_cache_attend(ctypes.byref(c), ctypes.byref(_query(M)), None)] == status
    e = M._lib.CCacheEviction()
    assert names[lib.lc_cache_evict(ctypes.byref(c), ctypes.byref(e), None)] == status
    assert lib.lc_cache_attend_workspace(ctypes.byref(c), 8, 0) == -1
    assert names[lib.lc_cache_attend(None, ctypes.byref(_query(M)), None)] == "LC_ERR_NULL"


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), "LC_ERR_NULL"), (dict(out=None), "LC_ERR_NULL"), (dict(lengths=None), "LC_ERR_NULL"),
    (dict(n_q_heads=7), "LC_ERR_SHAPE"), (dict(n_q_heads=0), "LC_ERR_SHAPE"), (dict(window=-1), "LC_ERR_SHAPE"),
    (dict(type=1), "LC_ERR_TYPE"), (dict(type=2), "LC_ERR_TYPE"), (dict(q=BASE + 1), "LC_ERR_ALIGN"),
    (dict(lse=BASE + 2, lse_stride=8), "LC_ERR_ALIGN"), (dict(q_stride=(-8, 64)), "LC_ERR_BAD_STRIDE"),
    (dict(out_stride=(512, 32)), "LC_ERR_NOT_INJECTIVE"), (dict(out_stride=(0, 64)), "LC_ERR_NOT_INJECTIVE"),
    (dict(scores=BASE, scores_stride=(48, 40)), "LC_ERR_NOT_INJECTIVE"),
    (dict(lse=BASE, lse_stride=7), "LC_ERR_NOT_INJECTIVE"),
    (dict(q_stride=(1 << 62, 64)), "LC_ERR_OVERFLOW"),
])
def test_attend_refusals(M, bad, status):
    c = _cache(M)
    got = M._lib.lib().lc_cache_attend(ctypes.byref(c), ctypes.byref(_query(M, **bad)), None)
    assert M._lib.STATUS_NAMES[got] == status


def test_attend_workspace_refusals(M):
    lib, names = M._lib.lib(), M._lib.STATUS_NAMES
    c = _cache(M, pages_per_seq=4096)
    need = lib.lc_cache_attend_workspace(ctypes.byref(c), 8, 1)
    assert need >= 0 and lib.lc_cache_attend_workspace(ctypes.byref(c), 7, 0) == -1
    if need:
        q = _query(M, scores=BASE, scores_stride=(4 * 65536, 65536))
        for bad, status in ((dict(workspace=None), "LC_ERR_NULL"), (dict(workspace=BASE + 16), "LC_ERR_ALIGN"),
                            (dict(workspace_bytes=need - 1), "LC_ERR_WORKSPACE")):
            for k, x in dict(workspace=BASE, workspace_bytes=need).items():
                setattr(q, k, bad.get(k, x))
            assert names[lib.lc_cache_attend(ctypes.byref(c), ctypes.byref(q), None)] == status


def test_writers_refuse_rows_that_overlap(M):
    """Attention may read a broadcast pool; append and evict may not write one."""
    lib, names = M._lib.lib(), M._lib.STATUS_NAMES
    st = (ctypes.c_int64 * 3)(4 * 64, 4 * 64, 64)
    e = M._lib.CCacheEviction()
    for bad in (dict(k_stride=(4096, 0, 64)), dict(v_stride=(4096, 1024, 63))):
        c = _cache(M, **bad)
        assert names[lib.lc_cache_append(ctypes.byref(c), BASE, BASE, 0, st, st, 1, None, BASE, 2 * BASE,
                                         None)] == "LC_ERR_NOT_INJECTIVE"
        assert names[lib.lc_cache_evict(ctypes.byref(c), ctypes.byref(e), None)] == "LC_ERR_NOT_INJECTIVE"


def test_append_refusals(M):
    lib, names = M._lib.lib(), M._lib.STATUS_NAMES

    def call(cache=None, k=4 * BASE, v=5 * BASE, type=0, strides=(2 * 256, 256, 64), n=2, counts=None, lengths=BASE,
             new=2 * BASE):
        st = (ctypes.c_int64 * 3)(*strides)
        return names[lib.lc_cache_append(ctypes.byref(cache or _cache(M)), k, v, type, st, st, n, counts, lengths,
                                         new, None)]
    assert call(k=None) == call(v=None) == call(lengths=None) == call(new=None) == "LC_ERR_NULL"
    assert call(type=1) == call(type=2) == "LC_ERR_TYPE"
    assert call(n=-1) == "LC_ERR_SHAPE"
    assert call(new=BASE) == "LC_ERR_OVERLAP"
    assert call(k=BASE + 1) == call(counts=BASE + 1) == "LC_ERR_ALIGN"
    assert call(strides=(-1, 256, 64)) == "LC_ERR_BAD_STRIDE"
    assert call(strides=(0, 0, 0), n=1 << 30) == "LC_ERR_OVERFLOW"


def test_evict_refusals(M):
    lib, names = M._lib.lib(), M._lib.STATUS_NAMES

    def call(cache=None, **kw):
        e = M._lib.CCacheEviction()
        e.lengths, e.scores, e.kept, e.new_scores, e.new_lengths = BASE, 2 * BASE, 3 * BASE, 4 * BASE, 5 * BASE
        e.scores_stride[:] = e.new_scores_stride[:] = (4 * 48, 48)
        e.kept_stride[:] = (4 * 8, 8)
        e.budget, e.recent = 8, 2
        e.workspace, e.workspace_bytes = 16 * BASE, lib.lc_cache_evict_workspace(ctypes.byref(_cache(M)), 8)
        for k, x in kw.items():
            if isinstance(x, tuple):
                getattr(e, k)[:] = x
            else:
                setattr(e, k, x)
        return names[lib.lc_cache_evict(ctypes.byref(_cache(M, **(cache or {}))), ctypes.byref(e), None)]
    for f in ("lengths", "scores", "kept", "new_scores", "new_lengths"):
        assert call(**{f: None}) == "LC_ERR_NULL"
        assert call(**{f: BASE * 9 + 2}) == "LC_ERR_ALIGN"
    assert call(budget=0) == call(recent=9) == call(recent=-1) == "LC_ERR_SHAPE"
    assert call(new_scores=2 * BASE) == call(new_lengths=BASE) == "LC_ERR_OVERLAP"
    assert call(kept_stride=(32, 7)) == call(new_scores_stride=(48, 47)) == "LC_ERR_NOT_INJECTIVE"
    assert call(scores_stride=(-1, 48)) == "LC_ERR_BAD_STRIDE"
    long = dict(pages_per_seq=2048, table_stride=2048)  # too long for the form that needs no workspace
    wide = dict(scores_stride=(4 * 32768, 32768), new_scores_stride=(4 * 32768, 32768))
    need = lib.lc_cache_evict_workspace(ctypes.byref(_cache(M, **long)), 8)
    assert need > 0 and lib.lc_cache_evict_workspace(ctypes.byref(_cache(M)), 0) == -1
    assert call(long, workspace=None, **wide) == "LC_ERR_NULL"
    assert call(long, workspace=BASE + 64, workspace_bytes=need, **wide) == "LC_ERR_ALIGN"
    assert call(long, workspace_bytes=need - 1, **wide) == "LC_ERR_WORKSPACE"
