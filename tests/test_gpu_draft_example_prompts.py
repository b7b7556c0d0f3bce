"""Prompts of the drafting example that come in one after another, and sequences that get none."""
import pytest

from test_gpu_draft_example import example  # noqa: F401  (a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_prompts_one_after_another(example):  # noqa: F811
    """The second batch leaves the first's next tokens as they are; more tokens for a sequence that has some are refused."""
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.randint(0, 8, (70,), generator=g, device="cuda")
    both, turns = (example.Server(3, 100, q_heads=8, kv_heads=2, seed=4) for _ in range(2))
    want = both.prompt(tokens, ints([30, 5, 35]))
    near = lambda x, y: torch.allclose(x.float(), y.float(), rtol=2e-2, atol=2e-2)  # noqa: E731  (products of other sizes)
    first = turns.prompt(tokens[30:35], ints([0, 5, 0]))
    assert near(first, want[30:35]) and turns.next.tolist() == [0, int(turns.chosen(first[[0, 4, 4]])[1]), 0]
    for counts in ([0, 1, 0], [3, 2, 0]):
        with pytest.raises(ValueError):
            turns.prompt(tokens[:sum(counts)], ints(counts))
    assert turns.lengths.tolist() == [0, 5, 0]
    kept = int(turns.next[1])
    rest = turns.prompt(torch.cat([tokens[:30], tokens[35:]]), ints([30, 0, 35]))
    assert near(rest, torch.cat([want[:30], want[35:]])) and turns.lengths.tolist() == [30, 5, 35]
    choice = turns.chosen(rest[[29, 29, 64]]).tolist()
    assert turns.next.tolist() == [choice[0], kept, choice[2]]
    assert example.lc.last_device_error()[0] == 0
