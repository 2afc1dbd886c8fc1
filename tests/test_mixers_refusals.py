"""Calls of the mixers' bindings that no tensor or sizes can be read from are refused by ValueError or TypeError, as the
other calls are (no GPU needed)."""
import pytest
import torch

from linear_attention_sequence_mshortconv_b200 import attention, build, gdn, kda

z = torch.zeros
CALLS = {
    "attention.forward": lambda q: attention.forward(q, z(1, 4, 2, 64), z(1, 4, 2, 64)),
    "attention.forward_varlen": lambda q: attention.forward_varlen(q, z(4, 2, 64), z(4, 2, 64), [0, 4]),
    "attention.backward": lambda q: attention.backward(q, *[z(1, 4, 2, 64)] * 3, z(1, 4, 2), z(1, 4, 2, 64)),
    "attention.backward_varlen": lambda q: attention.backward_varlen(q, *[z(4, 2, 64)] * 3, z(4, 2), z(4, 2, 64), [0, 4]),
    "gdn.forward": lambda q: gdn.forward(q, z(1, 4, 2, 64), z(1, 4, 2, 64), z(1, 4, 2), z(1, 4, 2)),
    "gdn.forward_varlen": lambda q: gdn.forward_varlen(q, z(4, 2, 64), z(4, 2, 64), z(4, 2), z(4, 2), [0, 4]),
    "gdn.backward": lambda q: gdn.backward(q, z(1, 4, 2, 64), z(1, 4, 2, 64), z(1, 4, 2), z(1, 4, 2), z(1, 4, 2, 64)),
    "gdn.backward_varlen": lambda q: gdn.backward_varlen(q, z(4, 2, 64), z(4, 2, 64), z(4, 2), z(4, 2), z(4, 2, 64), [0, 4]),
    "gdn.step": lambda q: gdn.step(q, z(4, 2, 64), z(4, 2, 64), z(4, 2), z(4, 2), z(4, 2, 64, 64)),
}


@pytest.mark.parametrize("q", [None, [1.0, 2.0], torch.zeros(()), torch.zeros(64), torch.zeros(2, 64), torch.zeros(1, 1, 4, 2, 64)],
                         ids=["None", "list", "0-d", "1-d", "2-d", "5-d"])
@pytest.mark.parametrize("call", CALLS, ids=str)
def test_q_is_no_tensor_of_the_calls_shape(call, q):
    build.build()
    with pytest.raises((TypeError, ValueError)):
        CALLS[call](q)


@pytest.mark.parametrize("which", [1, 3, 4])
def test_a_step_without_an_input(which):
    build.build()
    x = [z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), z(4, 2), z(4, 2)]
    x[which] = None
    with pytest.raises(TypeError, match=("q", "k", "v", "g", "beta")[which] + " must be"):
        gdn.step(*x, z(4, 2, 64, 64))


@pytest.mark.parametrize("cu", [[0, 2 ** 32 + 4], [0, 2 ** 32 + 2, 4], [2 ** 32, 4], [0, -2 ** 32 + 4], [0, 2 ** 31]], ids=str)
def test_offsets_beyond_32_bits(cu):
    """Their low 32 bits would be offsets of 4 tokens (or negative ones)."""
    build.build()
    q, gate = z(4, 2, 64), z(4, 2)
    for call in (lambda: gdn.forward_varlen(q, q, q, gate, gate, cu), lambda: gdn.backward_varlen(q, q, q, gate, gate, q, cu),
                 lambda: attention.forward_varlen(q, q, q, cu), lambda: attention.backward_varlen(q, q, q, q, gate, q, cu),
                 lambda: gdn.varlen_workspace_size(cu, 2, 2, 64, 64), lambda: kda.varlen_workspace_size(cu, 2, 64, 64)):
        with pytest.raises(ValueError):
            call()
