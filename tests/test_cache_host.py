"""Host-side behaviour of the paged-cache entry points (no GPU)."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT

PKG = os.path.join(ROOT, "movement_primitives_gb300")

FAILING_LAUNCH = r"""
#include <cuda_runtime.h>
static cudaError_t pending = cudaSuccess;
static cudaError_t fake_launch(const cudaLaunchConfig_t *, const void *, void **) {
    return pending = cudaErrorInvalidValue;
}
static cudaError_t fake_last() {
    const cudaError_t e = pending;
    pending = cudaSuccess;
    return e;
}
#define cudaLaunchKernelExC fake_launch
#define cudaGetLastError fake_last
#include "cache_common.cuh"
int main() {
    int arg = 0;
    if (lc::launch_after(nullptr, 1, 32, 0, nullptr, &arg) != LC_ERR_CUDA) return 1;
    return lc::finish_launch() == LC_OK ? 0 : 2;
}
"""


def test_a_failed_launch_leaves_no_error_for_the_next_call(tmp_path):
    """The runtime keeps a launch's error until it is read; the next call's check may not be the one that reads it."""
    from movement_primitives_gb300 import build
    src, exe = tmp_path / "launch.cu", tmp_path / "launch"
    src.write_text(FAILING_LAUNCH)
    subprocess.run([build.nvcc(), "-std=c++17", *build.ARCH, "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(PKG, "csrc"), str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0

ROWS_MEET = r"""
#include <cstdio>
#include <random>
#include <set>
#include "cache_common.cuh"
int main() {
    std::mt19937 rng(1);
    auto pick = [&](int lo, int hi) { return int64_t(std::uniform_int_distribution<int>(lo, hi)(rng)); };
    static int32_t memory[4096];
    int met = 0, near = 0;
    for (int k = 0; k < 400000; ++k) {
        const int64_t e[2] = {pick(1, 4), pick(1, 4)}, run = pick(1, 5);
        int64_t st[2], q[2];
        do {
            for (int i = 0; i < 2; ++i) {
                st[i] = pick(0, 24);
                q[i] = pick(0, 24);
            }
        } while (!lc::rows_apart(2, e, q, run));
        const int64_t pa = pick(0, 200), qa = pick(0, 200);
        std::set<int64_t> at;
        for (int i = 0; i < e[0] * e[1]; ++i)
            for (int x = 0; x < run; ++x) at.insert(pa + i / e[1] * st[0] + i % e[1] * st[1] + x);
        bool want = false;
        int64_t low = 1 << 30, high = 0;
        for (int i = 0; i < e[0] * e[1]; ++i)
            for (int x = 0; x < run; ++x) {
                const int64_t y = qa + i / e[1] * q[0] + i % e[1] * q[1] + x;
                want |= at.count(y) != 0;
                low = std::min(low, y);
                high = std::max(high, y);
            }
        met += want;
        near += !want && *at.begin() <= high && low <= *at.rbegin();
        if (lc::rows_meet(memory + pa, st, memory + qa, q, e, run) != want) {
            std::printf("e %d %d run %d p %d (%d %d) q %d (%d %d): %d\n", int(e[0]), int(e[1]), int(run), int(pa),
                        int(st[0]), int(st[1]), int(qa), int(q[0]), int(q[1]), int(want));
            return 1;
        }
    }
    if (met < 10000 || near < 10000) return 2;  // enough of both answers where ranges meet
    for (int i = 0; i < 20; ++i)
        for (int j = 0; j < 20; ++j)
            for (int n = 0; n < 6; ++n)
                if (lc::lists_meet(memory + i, memory + j, n) != (n > 0 && i < j + n && j < i + n)) return 3;
    return 0;
}
"""


def test_rows_that_meet_are_told_from_rows_that_do_not(tmp_path):
    """Against sets of elements, on random extents and strides."""
    from movement_primitives_gb300 import build
    src, exe = tmp_path / "rows.cu", tmp_path / "rows"
    src.write_text(ROWS_MEET)
    subprocess.run([build.nvcc(), "-O2", "-std=c++17", *build.ARCH, "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(PKG, "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import movement_primitives_gb300
    return movement_primitives_gb300


BASE = 1 << 20  # an address: nothing is read from it


@pytest.mark.parametrize("n_new", [0, 3])
def test_append_refuses_new_lengths_over_what_it_reads(M, n_new):
    """Two sequences: lists one element apart share one."""
    c = _cache(M)
    st = (ctypes.c_int64 * 3)(4 * 64 * 3, 4 * 64, 64)

    def call(lengths, counts, new):
        return M._lib.STATUS_NAMES[M._lib.lib().lc_cache_append(ctypes.byref(c), 4 * BASE, 5 * BASE, 0, st, st, n_new,
                                                                counts, lengths, new, None)]
    for at in (BASE + 4, BASE - 4):
        assert call(BASE, None, at) == call(2 * BASE, BASE, at) == call(BASE, 2 * BASE, at) == "LC_ERR_OVERLAP"
    if n_new:
        assert call(BASE, None, BASE) == call(2 * BASE, BASE, BASE) == "LC_ERR_OVERLAP"


def test_evict_refuses_outputs_over_what_it_reads(M):
    c = _cache(M)

    def call(**kw):
        e = M._lib.CCacheEviction()
        e.lengths, e.scores, e.kept, e.new_scores, e.new_lengths = BASE, 2 * BASE, 3 * BASE, 4 * BASE, 5 * BASE
        e.scores_stride[:] = e.new_scores_stride[:] = (4 * 48, 48)
        e.kept_stride[:] = (4 * 8, 8)
        e.budget, e.recent = 8, 2
        for k, x in kw.items():
            if isinstance(x, tuple):
                getattr(e, k)[:] = x
            else:
                setattr(e, k, x)
        return M._lib.STATUS_NAMES[M._lib.lib().lc_cache_evict(ctypes.byref(c), ctypes.byref(e), None)]
    size = 2 * 4 * 48 * 4
    for at in (BASE - 4, BASE, BASE + 4):
        assert call(new_lengths=at) == "LC_ERR_OVERLAP"
    for at in (4 - size, -48 * 4, 0, 4, 48 * 4, size - 4):
        assert call(new_scores=2 * BASE + at) == "LC_ERR_OVERLAP"
    # halves of one buffer, a slot into each other
    halves = dict(scores_stride=(8 * 48, 48), new_scores_stride=(8 * 48, 48))
    assert call(new_scores=2 * BASE + 4 * (4 * 48 - 1), **halves) == "LC_ERR_OVERLAP"


def _cache(M):
    c = M._lib.CPagedCache()
    c.k, c.v, c.page_table = 8 * BASE, 9 * BASE, 10 * BASE
    c.type, c.n_seqs, c.n_kv_heads, c.page_size, c.head_dim, c.pages_per_seq, c.n_pages = 0, 2, 4, 16, 64, 3, 9
    c.table_stride = 3
    c.k_stride[:] = c.v_stride[:] = (4 * 16 * 64, 16 * 64, 64)
    return c


def test_attend_refuses_an_output_over_the_queries(M):
    """Two sequences of eight heads of 64 16-bit elements: one element shared, or the same buffer in another order."""
    c = _cache(M)

    def call(out, stride=(8 * 64, 64), q_stride=(8 * 64, 64)):
        q = M._lib.CCacheQuery()
        q.q, q.out, q.lengths = 4 * BASE, out, 6 * BASE
        q.type, q.n_q_heads, q.scale = 0, 8, 0.125
        q.q_stride[:], q.out_stride[:] = q_stride, stride
        q.workspace, q.workspace_bytes = 16 * BASE, 1 << 40
        return M._lib.STATUS_NAMES[M._lib.lib().lc_cache_attend(ctypes.byref(c), ctypes.byref(q), None)]
    size = 2 * 8 * 64 * 2
    for at in (2 - size, -2, 2, 128, size - 2):
        assert call(4 * BASE + at) == "LC_ERR_OVERLAP"
    assert call(4 * BASE, stride=(64, 2 * 64)) == "LC_ERR_OVERLAP"
    assert call(4 * BASE + 2 * (64 - 1), (16 * 64, 2 * 64), (16 * 64, 2 * 64)) == "LC_ERR_OVERLAP"
