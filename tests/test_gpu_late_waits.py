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
late, calls = lc().STATUS["LC_ERR_TIMEOUT"], 0

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


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    words = r.stdout.split()
    return int(words[-3]), int(words[-1])


@pytest.mark.parametrize("limit", [1, 1000, 10000])
def test_prompts_return(limit):
    run(PROMPTS % (limit, os.path.join(ROOT, "tests"), ROOT))
