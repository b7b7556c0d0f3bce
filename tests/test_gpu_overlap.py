"""Parts of one buffer as arguments of the prompt and draft operators: apart, they run; where they meet, they are refused."""
import pytest

from test_gpu_cache import Setup, lc, no_device_error
from test_gpu_tree import ints, queries, trees

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def refused(call):
    with pytest.raises(lc().LayoutCopyError) as e:
        call()
    assert e.value.status == lc().STATUS["LC_ERR_OVERLAP"]


def test_prompt_rows_of_one_buffer():
    """[q k v out lse], 784 elements of 16 bits a token."""
    n = 300
    flat = torch.randn((n, 784), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, k, v, out = (flat[:, a:b].unflatten(1, (-1, 64)) for a, b in ((0, 256), (256, 384), (384, 512), (512, 768)))
    logs = flat.view(torch.float32)
    starts = ints([0, 100, 300])
    want_lse = torch.empty((n, 4), device="cuda")
    want = lc().prompt_attend(q.contiguous(), k.contiguous(), v.contiguous(), starts, lse=want_lse)
    before = flat.clone()
    lc().prompt_attend(q, k, v, starts, out=out, lse=logs[:, 384:388])
    assert torch.equal(out, want) and torch.equal(logs[:, 384:388], want_lse)
    assert torch.equal(flat[:, :512], before[:, :512]) and torch.equal(flat[:, 776:], before[:, 776:])
    no_device_error()
    for column in (0, 127, 255, 300, 383):
        refused(lambda: lc().prompt_attend(q, k, v, starts, out=out, lse=logs[:, column:column + 4]))
    both = torch.cat([starts, torch.zeros(n * 4, dtype=torch.int32, device="cuda")])
    refused(lambda: lc().prompt_attend(q, k, v, both[:3], lse=both[2:2 + n * 4].view(torch.float32).view(n, 4)))
    lc().prompt_attend(q, k, v, both[:3], lse=both[3:].view(torch.float32).view(n, 4))
    assert torch.equal(both[3:].view(torch.float32).view(n, 4), want_lse)
    no_device_error()


def test_tree_rows_of_one_buffer():
    """[q out lse] a sequence: apart as columns.  Ranges of q and out meet all the same, which trees refuse; logs may lie among q's rows."""
    s = Setup([40, 9], heads=2, dim=64, seed=2)
    q, parents = queries(s, 3, 4), trees(2, 3, s.g)
    want_lse = torch.empty((2, 3, 4), device="cuda")
    want = lc().cache_attend_tree(s.cache, q, s.lengths, parents, lse=want_lse)
    flat = torch.zeros((2, 3 * 256 + 32), dtype=torch.bfloat16, device="cuda")
    mine, logs = flat[:, :768].unflatten(1, (3, 4, 64)), flat.view(torch.float32)
    mine.copy_(q)
    lse = logs[:, 384:396].unflatten(1, (3, 4))
    assert torch.equal(lc().cache_attend_tree(s.cache, mine, s.lengths, parents, lse=lse), want) and torch.equal(lse, want_lse)
    no_device_error()
    for column in (0, 380, 383):
        refused(lambda: lc().cache_attend_tree(s.cache, mine, s.lengths, parents, lse=logs[:, column:column + 12].unflatten(1, (3, 4))))
    refused(lambda: lc().cache_attend_tree(s.cache, q, s.lengths, parents, out=want, lse=want.view(torch.float32).flatten()[8:32].view(2, 3, 4)))
    lists = torch.zeros(64, dtype=torch.int32, device="cuda")
    lists[:2] = s.lengths
    refused(lambda: lc().cache_attend_tree(s.cache, q, lists[:2], parents, lse=lists[1:25].view(torch.float32).view(2, 3, 4)))
    assert torch.equal(lc().cache_attend_tree(s.cache, q, lists[:2], parents, lse=lists[2:26].view(torch.float32).view(2, 3, 4)), want)
    no_device_error()
