"""Scales of next to nothing over dot products of any size a float32 holds: at 0 every seen key weighs the same, whatever
q and k hold.  Tolerances: test_gpu_prompt.py, test_gpu_tree.py."""
import pytest

import test_gpu_prompt as tp
import test_gpu_tree as tt
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


SCALES = [0.0, -0.0, 2.0 ** -149, -2.0 ** -140, 2.0 ** -126, 2.0 ** -118, -2.0 ** -110]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("scale", SCALES)
def test_prompts(dim, scale):
    starts = [0, 100, 101, 400]
    q, k, v = (tp.rows(400, h, dim, torch.bfloat16, h) for h in (4, 2, 2))
    q, k = q * 2.0 ** 58, k * 2.0 ** 57
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    lc().prompt_attend(q, k, v, tp.ints(starts), scale=scale, out=out, lse=lse)
    tp.check(q, k, v, starts, None, out, lse, scale=scale)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("scale", SCALES)
def test_trees(kind, page, scale):
    s = Setup([300, 7], dim=128, kind=kind, page=page, seed=3)
    q, parents = tt.queries(s, 4, 4) * 2.0 ** 58, tt.trees(2, 4, s.g)
    if kind == "e4m3":
        s.scales[0].mul_(2.0 ** 56)
    else:
        s.k.mul_(2.0 ** 57)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    lc().cache_attend_tree(s.cache, q, s.lengths, parents, scale=scale, out=out, lse=lse)
    tt.check(s, q, s.lengths, parents, None, out, lse, scale)
    no_device_error()
