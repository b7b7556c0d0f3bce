"""Trees over E4M3 caches whose queries are zero or very small, with scales down to zero.

A row of q is divided by a power of two near its largest element, and the logits are multiplied by that and the scale:
a product that may be less than a float32 holds, where slots that are not seen still have to weigh nothing.  With
logits that are next to nothing every seen slot weighs the same.  Tolerances: test_gpu_tree.py.
"""
import pytest

from test_gpu_cache import Setup, lc, no_device_error
from test_gpu_tree import check, ints, queries, trees

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-30, -1e-30, 1e-8, None, 1e20])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -100, 2.0 ** -50, 2.0 ** -20])
def test_small_queries(kind, page, scale, size):
    if scale == 1e20:  # logits that a float32 sum still tells apart
        size = min(size, 2.0 ** -100)
    if kind == "fp16" and size < 2.0 ** -24:  # no float16 number but 0 is that small
        size = 0.0
    s = Setup([70, 5, 301], dim=64, kind=kind, page=page, seed=1)
    q, parents, counts = queries(s, 4, 4), trees(3, 4, s.g), ints([4, 4, 3])
    q[:, ::2] = (q[:, ::2].float().sign() * size).to(q.dtype)  # beside rows of ordinary ones
    if scale == 1e20:
        q[:, 1::2] = q[:, ::2]
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    lc().cache_attend_tree(s.cache, q, s.lengths, parents, counts, scale=scale, out=out, lse=lse)
    check(s, q, s.lengths, parents, counts, out, lse, scale)
    no_device_error()


def test_small_queries_across_cut_units():
    """The same where a sequence is many blocks' and its parts are joined."""
    s = Setup([9000], heads=1, dim=128, kind="e4m3", page=64, seed=2)
    q, parents = queries(s, 4, 4), trees(1, 4, s.g)
    q[:, 1] = 0
    for scale in (0.0, 1e-30, None):
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
        lc().cache_attend_tree(s.cache, q, s.lengths, parents, scale=scale, out=out, lse=lse)
        check(s, q, s.lengths, parents, None, out, lse, scale)
    no_device_error()
