"""Log sums of few keys under small scales, where nothing but their own roundings shows, against the 64-bit oracle.

An exponent below 32 is off by 2^-20 (the difference to the maximum, rounded), its power of two by 2^-22 of itself, and
so is the log sum: ln 2 * 2^-20 + 2^-22; beside that the logits are off as in test_gpu_prompt.py, the additions by
n 2^-24 and the result by 2^-22 of its size and 2^-24 (the logarithm, two products).
"""
import math

import numpy as np
import pytest

import test_gpu_prompt as tp
import test_gpu_tree as tt
from oracle import drafts as od, prompt as op
from test_gpu_cache import Setup, lc, no_device_error

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def check(got, want, reach, dim, n):
    tol = math.log(2) * 2.0 ** -20 + 2.0 ** -22 + 2 * (dim + 8) * 2.0 ** -24 * reach + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(want) + 2.0 ** -24
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("dtype", tp.TYPES)
@pytest.mark.parametrize("dim", [16, 64, 192])
@pytest.mark.parametrize("scale", [0.0, 1e-4, 1e-3, 1e-2])
def test_prompts(dtype, dim, scale):
    for n, heads in ((1, 128), (3, 128), (20, 64), (200, 8)):
        q, k, v = (tp.rows(n, h, dim, dtype, h + n) for h in (heads, 1, 1))
        lse = torch.empty((n, heads), device="cuda")
        lc().prompt_attend(q, k, v, tp.ints([0, n]), lse=lse, scale=scale)
        _, want, _, reach, _ = op.attend(*(x.double().cpu().numpy() for x in (q, k, v)), [0, n], None, scale)
        check(lse, want, reach, dim, n)
    no_device_error()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("scale", [0.0, 1e-4, 1e-3, 1e-2])
def test_trees(kind, page, scale):
    for n, drafts in ((3, 3), (20, 5), (1500, 2)):
        s = Setup([n], heads=2, dim=64, page=page, kind=kind, seed=n)
        q, parents = tt.queries(s, drafts, 64), tt.trees(1, drafts, s.g)
        lse = torch.empty(q.shape[:3], device="cuda")
        lc().cache_attend_tree(s.cache, q, s.lengths, parents, lse=lse, scale=scale)
        k, v = s.values()
        _, want, _, reach, _ = od.attend(q.double().cpu().numpy(), k, v, s.table.cpu().numpy(), [n], None, parents.cpu().numpy(), scale)
        check(lse, want, reach, 64, n)
    no_device_error()


@pytest.mark.parametrize("behind", [0.0, 5.25])
def test_sums_of_the_largest_values_stay_finite(behind):
    """The average of the type's largest values is no larger than they are, their sum past float32; `behind`: how much larger than
    the first key's the others' logits are, less than what makes the running maximum follow."""
    n = 6000
    q, k = (torch.zeros((n, h, 64), dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    q[..., 0], k[1:, :, 0] = 1.0, behind
    v = torch.full_like(k, torch.finfo(torch.bfloat16).max)
    v[::2, :, 1::2] *= -1
    out = lc().prompt_attend(q, k, v, tp.ints([0, n]), scale=1.0)
    tp.check(q, k, v, [0, n], None, out, None, scale=1.0)
    s = Setup([n], heads=1, dim=64, page=16, seed=1)
    table = s.table[0].long()
    s.k[table], s.v[table] = k[:, 0].view(-1, 1, 16, 64), v[:, 0].view(-1, 1, 16, 64)
    tq = q[:2].view(1, 2, 2, 64)
    out = torch.full_like(tq, 7.0)
    lc().cache_attend_tree(s.cache, tq, s.lengths, tt.ints([[-1, 0]]), out=out, scale=1.0)
    tt.check(s, tq, s.lengths, tt.ints([[-1, 0]]), None, out, None, 1.0)
