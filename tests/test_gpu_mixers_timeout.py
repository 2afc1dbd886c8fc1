"""Device-side failure path of the mixers' tcgen05 kernels, exercised without a fault.

With the test hook kda_debug_drop_handoff one barrier of each kernel expects an arrival that never comes, so the wait of
the warp that issues the MMAs runs out (2 s): the kernel records a timeout in the device's status word, every role runs to
its end, the copies and MMAs in flight end before the CTA leaves, and the host reads KDA_ERR_TIMEOUT.  The same call
without the hook then gives the bits that it gave before."""
import pytest
import torch

import mixers_ref as R
from linear_attention_sequence_mshortconv_b200 import attention, gdn, kda
from test_gpu_attention import make as make_attention
from test_gpu_gdn import cuda, make

pytestmark = pytest.mark.gpu
KDA_ERR_TIMEOUT = 4


def times_out_and_recovers(call):
    want = call()
    torch.cuda.synchronize()
    assert kda.last_device_error() == 0
    kda.debug_drop_handoff(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        kda.debug_drop_handoff(False)
    assert kda.last_device_error() == KDA_ERR_TIMEOUT
    assert kda.last_device_error() == 0          # reading the word clears it
    got = call()
    torch.cuda.synchronize()
    assert kda.last_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# 100, 200 tokens: every copy of keys is issued before any wait; 1000: the ring goes round.  Groups of 3 heads are no boxes.
@pytest.mark.parametrize("lens,H,Hkv,D", [([100], 1, 1, 64), ([200, 40], 4, 2, 64), ([1000, 65], 2, 1, 128), ([700], 3, 1, 64)], ids=str)
def test_attention_forward(lens, H, Hkv, D):
    q, k, v, _ = cuda(make_attention(lens, H, Hkv, D, torch.bfloat16, seed=1))
    times_out_and_recovers(lambda: attention.forward_varlen(q, k, v, R.offsets(lens)))


@pytest.mark.parametrize("lens,H,Hkv,D", [([200, 40], 4, 2, 128), ([1000, 65], 3, 1, 64)], ids=str)
def test_attention_backward(lens, H, Hkv, D):
    q, k, v, do = cuda(make_attention(lens, H, Hkv, D, torch.bfloat16, seed=2))
    o, lse = attention.forward_varlen(q, k, v, R.offsets(lens))
    times_out_and_recovers(lambda: attention.backward_varlen(q, k, v, o, lse, do, R.offsets(lens)))


# whole heads (with ragged last chunks, whole ones, and samples of one chunk), and the pieces of a long sample
@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [([130, 64, 1, 192], 16, 32, 128, 64), ([100, 192], 32, 64, 64, 128), ([6000], 1, 2, 64, 64)], ids=str)
def test_gdn_forward(lens, Hk, Hv, Dk, Dv):
    x, S0, _, _ = make(lens, Hk, Hv, Dk, Dv, torch.bfloat16, seed=3, g_scale=0.02)
    x, S0 = cuda(x), S0.cuda()
    times_out_and_recovers(lambda: gdn.forward_varlen(*x, R.offsets(lens), S0))


# whole heads, and columns of heads (of whose kernels the gradients' alone has such waits)
@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [([130, 64, 320], 16, 32, 128, 128), ([100, 192], 32, 64, 64, 64), ([150, 64], 1, 2, 128, 64)], ids=str)
def test_gdn_backward(lens, Hk, Hv, Dk, Dv):
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, torch.bfloat16, seed=4)
    x, S0, do, dS = cuda(x), S0.cuda(), do.cuda(), dS.cuda()
    times_out_and_recovers(lambda: gdn.backward_varlen(*x, do, R.offsets(lens), S0, dS))
