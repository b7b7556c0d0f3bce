"""Paged key-value cache operators on the GPU: what their results may not depend on, and how near they come.

Cases beside those of ``test_gpu_cache.py``, whose caches and checks they use.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest

from conftest import ROOT
from oracle import cache as oc

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_cache import IO, Setup, attend, check_attend, lc, no_device_error  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("group", [1, 7, 16])
def test_weights_of_a_unit_over_a_cluster_repeat(kind, group):
    """Few units of some hundred slots: a cluster of blocks each, every block forms every row's log sum
    once.  Outputs, log sums and weights are the same bits each time."""
    s = Setup([700, 333, 0, 40], heads=2, dim=128, kind=kind, page=16, seed=group)
    q, out, lse, _ = attend(s, 2 * group, scores=True)
    first = torch.zeros((4, 2, s.cap), device="cuda")
    lc().cache_attend(s.cache, q, s.lengths, scores=first)
    for _ in range(20):
        again, logs = torch.zeros_like(first), torch.zeros_like(lse)
        assert torch.equal(lc().cache_attend(s.cache, q, s.lengths, scores=again, lse=logs), out)
        assert torch.equal(again, first) and torch.equal(logs, lse)
