"""Workspaces that the library states for the gated delta rule (no GPU needed): what the kernels that run put there."""
import pytest
import torch

from linear_attention_sequence_mshortconv_b200 import build, gdn

RECORD = 4 * 12 * 512 + 5 * 64 * 4   # bytes of a chunk's factors: two planes of T and of P, ten blocks and two of zeros each, and the gates


def kept(Dk, Dv):   # of what the gradients keep of a chunk: two planes of S, D, U and dY, one of R
    return 2 * (4 * Dv * Dk + 5 * Dv * 64)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", [(4, 4352, 16, 16, 128, 128), (1, 32768, 16, 16, 128, 64), (2, 6016, 4, 8, 64, 128), (3, 640, 2, 2, 128, 32)])
def test_gradients_take_what_the_tensor_core_kernels_need(B, T, Hk, Hv, Dk, Dv):
    slots = B * T // 64 + B
    need = slots * Hv * (RECORD + kept(Dk, Dv))
    assert need <= gdn.backward_workspace_size(B, T, Hk, Hv, Dk, Dv) <= need + 256
    cu = [i * T for i in range(B + 1)]
    assert need <= gdn.backward_varlen_workspace_size(cu, Hk, Hv, Dk, Dv) <= need + 256
    # fp32: the entry states of chunks of 16 tokens, and dq and dk of every value head
    need = 4 * ((B * T // 16 + B) * Hv * Dk * Dv + 2 * B * T * Hv * Dk)
    assert gdn.backward_workspace_size(B, T, Hk, Hv, Dk, Dv, torch.float32) == need


@pytest.mark.parametrize("T", [1, 17, 63])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_short_rows_take_no_chunk_each(T, dtype):
    """65535 rows, each of less than a chunk: 4 GiB at most, or what 255 rows need."""
    for Hk, Hv, Dk, Dv in ((16, 16, 128, 128), (1, 1, 64, 64), (4, 8, 128, 32)):
        for size in (gdn.backward_workspace_size, gdn.workspace_size):
            most = max(2 ** 32, size(255, T, Hk, Hv, Dk, Dv, dtype))
            assert size(65535, T, Hk, Hv, Dk, Dv, dtype) <= most + 2 ** 20
