"""Calls of the mixers' bindings that no tensor or sizes can be read from are refused by ValueError or TypeError, as the
other calls are (no GPU needed)."""
import pytest
import torch

from linear_attention_sequence_mshortconv_b200 import build, gdn

z = torch.zeros

@pytest.mark.parametrize("which", [1, 3, 4])
def test_a_step_without_an_input(which):
    build.build()
    x = [z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), z(4, 2), z(4, 2)]
    x[which] = None
    with pytest.raises(TypeError, match=("q", "k", "v", "g", "beta")[which] + " must be"):
        gdn.step(*x, z(4, 2, 64, 64))
