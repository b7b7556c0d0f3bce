"""Parts of one buffer as arguments of the prompt and draft operators: apart, they run; where they meet, they are refused."""
import pytest

from test_gpu_cache import lc, no_device_error
from test_gpu_tree import ints

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
