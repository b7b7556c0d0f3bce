"""Reservations with pages of up to 2^31 slots: sums that pass 31 bits on the way."""
import pytest

from test_gpu_pages import reservation

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("page,per", [(0x7fff0000, 1), (0x60000000, 1), (0x3fff8000, 2), (0x10000000, 7)])
@pytest.mark.parametrize("new", [False, True])
def test_reserve_pages_of_many_slots(page, per, new):
    cap = page * per
    for length, count in ((0, 1), (5, 7), (page // 2 + 1, 3), (page - 1, 1), (cap - 2, 2), (cap, 0), (cap // 2, 9)):
        held = min(-(-length // page), per)
        need = -(-(length + count) // page) - held
        reservation([list(range(held)) + [-1] * (per - held)] * 2, [length, 0], [count, min(count, 4)], [9, 8, 7][:need + 2], page, 16, spare=2 * per, new=new)
    reservation([[3] + [-1] * (per - 1)], [page // 2], [cap - page // 2 + 1], [5], page, 16, new=new, error=True)
