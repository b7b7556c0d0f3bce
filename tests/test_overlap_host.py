"""Outputs that meet what a call reads or writes beside them, in the prompt and draft operators (no GPU)."""
import pytest

from test_prompt_host import BASE, M, accept, cache, prompt, tree  # noqa: F401  (M is a fixture)


def test_prompt_refuses_logs_over_anything(M):  # noqa: F811
    q, kv, logs = 20 * 256 * 2, 20 * 128 * 2, 20 * 4 * 4
    for base, size in ((BASE, q), (2 * BASE, kv), (3 * BASE, kv), (4 * BASE, q), (6 * BASE, 16), (7 * BASE, 16)):
        for at in (4 - logs, 0, size - 4):
            assert prompt(M, lse=base + at) == "LC_ERR_OVERLAP", (base // BASE, at)
    # over the queries that out takes the place of
    assert prompt(M, out=BASE, lse=BASE + 512) == "LC_ERR_OVERLAP"
    for at in (2 - q, 0, 14):
        assert prompt(M, out=6 * BASE + at) == prompt(M, out=7 * BASE + at) == "LC_ERR_OVERLAP"


def test_prompt_parts_of_one_buffer(M):  # noqa: F811
    """Rows [q k v out lse] of 784 elements, of which lse may only have its own columns (test_gpu_overlap.py runs that)."""
    rows = dict(q_stride=(784, 64), k_stride=(784, 64), v_stride=(784, 64), out_stride=(784, 64), lse_stride=392,
                k=BASE + 512, v=BASE + 768, out=BASE + 1024)
    for column in (1532, 1020, 756, 508, 4, 1568 - 4):
        assert prompt(M, lse=BASE + column, **rows) == "LC_ERR_OVERLAP", column


def test_tree_refuses_outputs_over_anything(M):  # noqa: F811
    size, logs = 2 * 3 * 512 * 2, 2 * 3 * 8 * 4
    for base, n in ((BASE, size), (2 * BASE, size), (3 * BASE, 8), (4 * BASE, 8), (5 * BASE, 24)):
        for at in (4 - logs, 0, n - 4):
            assert tree(M, lse=base + at) == "LC_ERR_OVERLAP", (base // BASE, at)
    for base, n in ((3 * BASE, 8), (4 * BASE, 8), (5 * BASE, 24)):
        for at in (4 - size, 0, n - 4):
            assert tree(M, out=base + at) == "LC_ERR_OVERLAP", (base // BASE, at)
    # a tree for all sequences, its row read by each
    assert tree(M, parents_stride=0, lse=5 * BASE + 8) == "LC_ERR_OVERLAP"


def test_accept_refuses_lengths_over_the_page_table(M):  # noqa: F811
    for at in (-4, 0, 8, 20):
        assert accept(M, new=10 * BASE + at) == "LC_ERR_OVERLAP"
    # in columns of the table's buffer that are not the table's
    c = cache(M, table_stride=8, n_seqs=1)
    assert accept(M, c, new=10 * BASE + 8) == "LC_ERR_OVERLAP"
