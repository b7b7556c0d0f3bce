"""Scales that prompts and trees refuse (no GPU): what is not finite in float32 once it is in powers of two."""
import pytest

from test_prompt_host import M, prompt, tree  # noqa: F401  (M is a fixture)

MOST = float.fromhex("0x1.fffffep127")  # the largest float32


@pytest.mark.parametrize("scale", [MOST, -MOST, 2.4e38, -2.4e38])
def test_scales_whose_powers_of_two_overflow_are_refused(M, scale):  # noqa: F811
    assert prompt(M, scale=scale) == tree(M, scale=scale) == "LC_ERR_SHAPE"
    # one that does not is looked at no further where there is nothing to do
    assert prompt(M, scale=scale / 2, n_tokens=0) == tree(M, scale=scale / 2, n_drafts=0) == "LC_OK"
