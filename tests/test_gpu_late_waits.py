"""Waits of the prompt and tree kernels under a limit of next to nothing, in processes of their own.

The work is ordinary; only LC_WAIT_TIMEOUT_NS is small, so warps give up on copies, products and one another that
would have come.  Whatever gave up, a call returns, the error word says so or the output is the usual one, and what
comes after runs as ever.
"""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HEAD = """
import os, sys
os.environ["LC_WAIT_TIMEOUT_NS"] = "%d"
sys.path[:0] = [%r, %r]
import torch
from test_gpu_cache import IO, Setup, lc
from test_gpu_tree import ints, queries, trees
g = torch.Generator().manual_seed(1)
late = lc().STATUS["LC_ERR_TIMEOUT"]

def run(call, right):
    out = call()
    status, _ = lc().last_device_error()
    assert status in (0, late), status
    assert status or right(out)
    return status == late
"""

PROMPTS = HEAD + """
late_ones = []
for dim in (64, 128, 192, 256):
    for tokens in ([1], [5], [61], [300, 17, 900], [40] * 50, [2000, 3]):
        n, starts = sum(tokens), [0]
        for t in tokens:
            starts.append(starts[-1] + t)
        x = torch.randn((n, 8, dim), generator=g).bfloat16().cuda()
        x[:, :4] = 0  # queries of zeros: the mean of what is seen
        q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
        want = torch.cat([v[a:b].float().cumsum(0) / torch.arange(1, b - a + 1, device="cuda")[:, None, None]
                          for a, b in zip(starts, starts[1:])]).repeat_interleave(2, 1)
        for _ in range(4):
            late_ones.append(run(lambda: lc().prompt_attend(q, k, v, ints(starts)),
                                 lambda out: torch.allclose(out.float(), want, rtol=2e-2, atol=2e-2)))
print("late", sum(late_ones), "of", len(late_ones))
"""


TREES = HEAD + """
late_ones = []
other = Setup([700, 90], heads=2, dim=64, seed=2)
oq = other.queries(4)
usual = lc().cache_attend(other.cache, oq, other.lengths)
for kind in ("bf16", "fp16", "e4m3"):
    for dim, page, lengths in ((64, 16, [5]), (64, 16, [70, 301]), (128, 64, [6000, 40, 2900]), (64, 3, [300, 9]),
                               (256, 16, [2500]), (128, 16, [100] * 200)):
        s = Setup(lengths, heads=2, dim=dim, page=page, kind=kind, seed=dim)
        n_seq, drafts = len(lengths), 5
        q = queries(s, drafts, 4)
        q[:] = 0  # the mean of what is seen
        v = s.v.float() if s.scales[1] is None else s.v.float() * s.scales[1][..., None]
        v = v[s.table.long()].transpose(2, 3).flatten(1, 2)  # [sequence, slot, head, dim]
        mean = v.cumsum(1) / torch.arange(1, v.shape[1] + 1, device="cuda")[:, None, None]
        at = s.lengths[:, None].long() - drafts + torch.arange(drafts, device="cuda")
        want = mean[torch.arange(n_seq, device="cuda")[:, None], at].repeat_interleave(2, 2)
        parents = trees(n_seq, drafts, g, "chain")
        for _ in range(4):
            late_ones.append(run(lambda: lc().cache_attend_tree(s.cache, q, s.lengths, parents),
                                 lambda out: torch.allclose(out.float(), want, rtol=2e-2, atol=2e-2)))
            assert torch.equal(lc().cache_attend(other.cache, oq, other.lengths), usual)
print("late", sum(late_ones), "of", len(late_ones))
"""


def run(code, library=None):
    """(late calls, calls)"""
    env = dict(os.environ, LC_LIBRARY_PATH=library) if library else None
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stderr[-2000:]
    words = r.stdout.split()
    return int(words[-3]), int(words[-1])


def filled(code, limit):
    return code % (limit, os.path.join(ROOT, "tests"), ROOT)


@pytest.mark.parametrize("limit", [1, 1000, 10000])
def test_prompts_return(limit):
    run(filled(PROMPTS, limit))


@pytest.fixture(scope="module")
def awake(tmp_path_factory):
    """A library whose polls do not sleep, so that short limits are kept; the same code else."""
    from movement_primitives_gb300 import build
    return build.build(out=str(tmp_path_factory.mktemp("awake") / "liblayoutcopy.so"), defines=["LC_POLLS_AWAKE"],
                       only=["k_%s_attend_%s.cu" % x for x in (("prompt", "bf16"), ("tree", "bf16"), ("tree", "f16"), ("tree", "e4m3"))])


@pytest.mark.parametrize("limit", [1, 300, 1000, 2000, 3000, 10000])
@pytest.mark.parametrize("code", [PROMPTS, TREES], ids=["prompts", "trees"])
def test_waits_that_run_out(awake, code, limit):
    """At a nanosecond all calls are late: a block's first reads take longer.  At more, some waits go through."""
    late, calls = run(filled(code, limit), awake)
    assert late == calls if limit == 1 else late <= calls


@pytest.mark.parametrize("code", [PROMPTS, TREES], ids=["prompts", "trees"])
def test_nothing_is_late_within_the_usual_limit(awake, code):
    assert run(filled(code, 2000000000))[0] == 0 == run(filled(code, 2000000000), awake)[0]
