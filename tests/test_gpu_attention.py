"""Causal grouped attention on the GPU against the plain 64-bit form (tests/mixers_ref.py), on the stored inputs.

Tolerances, fixed from the arithmetic, in the 2-norm.  bf16 forward: the weights are rounded to bf16 for the product
with v and the output is rounded once, 2^-8 each.  bf16 gradients: the weights or the score gradients are rounded
once, the output once, and the row sums do.o use the bf16 o (2^-8 of each term): 3 * 2^-8.  lse and fp32 outputs:
sums of at most 128 terms and of one term per key in fp32, exponentials to a few units in the last place:
128 * 2^-24 for outputs of random-sign terms, and 16 * 2^-24 times the largest score's magnitude for lse.
"""
import numpy as np
import pytest
import torch

import mixers_ref as R
from linear_attention_sequence_mshortconv_b200 import attention, kda

pytestmark = pytest.mark.gpu
FWD, GRAD, FP32 = 2 * 2.0 ** -8, 3 * 2.0 ** -8, 128 * 2.0 ** -24


def make(lens, H, Hkv, D, dtype, seed=0, spare=0, size=1.0):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens) + spare
    n = lambda *s: (size * torch.randn(*s, generator=gen)).to(dtype)   # noqa: E731
    return n(T, H, D), n(T, Hkv, D), n(T, Hkv, D), n(T, H, D)


def cuda(ts):
    return [t.cuda() for t in ts]


CASES = [  # lens, H, Hkv, D
    ([1], 1, 1, 32), ([1, 2, 3, 0, 5], 2, 1, 64), ([64, 128, 127, 129], 2, 2, 128), ([63, 65, 1, 0, 200], 4, 2, 64),
    ([300, 7], 6, 2, 128), ([257], 3, 1, 32), ([0, 0, 130], 1, 1, 64), ([513, 31, 384], 2, 1, 128), ([640], 8, 1, 64)]


def check_forward(o, lse, q, k, v, lens, dtype, scale=None):
    ref_o, ref_l = R.attention(*map(R.f64, (q, k, v)), lens, scale)
    T = sum(lens)
    assert R.norm_error(o[:T], ref_o[:T]) <= (FP32 if dtype == torch.float32 else FWD)
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    top = max(1.0, float(abs(scale) * q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()))
    assert np.abs(R.f64(lse)[:T] - ref_l[:T]).max() <= 16 * 2.0 ** -24 * top


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_varlen(case, dtype):
    lens, H, Hkv, D = case
    q, k, v, _ = make(lens, H, Hkv, D, dtype, seed=len(lens))
    o, lse = attention.forward_varlen(*cuda((q, k, v)), R.offsets(lens))
    assert o.dtype == dtype and lse.dtype == torch.float32
    check_forward(o, lse, q, k, v, lens, dtype)
    assert kda.last_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward_varlen(case, dtype):
    lens, H, Hkv, D = case
    q, k, v, do = make(lens, H, Hkv, D, dtype, seed=3 + len(lens))
    x = cuda((q, k, v))
    o, lse = attention.forward_varlen(*x, R.offsets(lens))
    got = attention.backward_varlen(*x, o, lse, do.cuda(), R.offsets(lens))
    ref = R.attention_backward(*map(R.f64, (q, k, v, do)), lens)
    for name, a, b in zip(("dq", "dk", "dv"), got, ref):
        assert a.dtype == dtype
        # a sample of one token has dq = dk = 0: compare against the scale of its dv
        err = np.linalg.norm(R.f64(a) - b)
        assert err <= (FP32 if dtype == torch.float32 else GRAD) * max(np.linalg.norm(b), 0.05 * np.linalg.norm(ref[2])), name
    assert kda.last_device_error() == 0


@pytest.mark.parametrize("case", [([1100, 5, 300], 3, 1, 64), ([900, 70], 5, 1, 128), ([40, 1, 33], 64, 1, 128),
                                  ([40, 1, 33], 65, 1, 64), ([130, 2], 128, 1, 64), ([1500], 10, 2, 64)], ids=str)
def test_shared_heads(case):
    """Group sizes that no tile is a multiple of, large ones, and more heads than a tile has rows."""
    lens, H, Hkv, D = case
    q, k, v, do = make(lens, H, Hkv, D, torch.bfloat16, seed=60 + H)
    o, lse = attention.forward_varlen(*cuda((q, k, v)), R.offsets(lens))
    check_forward(o, lse, q, k, v, lens, torch.bfloat16)
    got = attention.backward_varlen(*cuda((q, k, v)), o, lse, do.cuda(), R.offsets(lens))
    for a, b in zip(got, R.attention_backward(*map(R.f64, (q, k, v, do)), lens)):
        assert R.norm_error(a, b) <= GRAD
    assert kda.last_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,H,Hkv,D", [(2, 200, 4, 2, 64), (1, 1, 2, 1, 128), (3, 128, 2, 2, 128), (2, 77, 1, 1, 32)])
def test_rows_equal_packed_samples(B, T, H, Hkv, D, dtype):
    q, k, v, do = cuda(make([T] * B, H, Hkv, D, dtype, seed=5))
    cu = R.offsets([T] * B)
    rows = lambda t: t.view(B, T, *t.shape[1:])   # noqa: E731
    o, lse = attention.forward(rows(q), rows(k), rows(v))
    o2, lse2 = attention.forward_varlen(q, k, v, cu)
    assert torch.equal(o.view_as(o2), o2) and torch.equal(lse.view_as(lse2), lse2)
    g = attention.backward(rows(q), rows(k), rows(v), o, lse, rows(do))
    for a, b in zip(g, attention.backward_varlen(q, k, v, o2, lse2, do, cu)):
        assert torch.equal(a.view_as(b), b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.3, 1.0), (1.0, 3.0), (1e-3, 1.0)])
def test_scales(scale, size, D, dtype):
    """No scale, a negative one, scores in the hundreds (one key takes the row), and nearly none."""
    lens = [200, 65]
    q, k, v, do = make(lens, 2, 1, D, dtype, seed=6, size=size)
    x = cuda((q, k, v))
    cu = R.offsets(lens)
    o, lse = attention.forward_varlen(*x, cu, scale=scale)
    check_forward(o, lse, q, k, v, lens, dtype, scale)
    if scale == 1.0:
        return   # the weights' own rounding of scores in the hundreds is not a gradient's tolerance
    got = attention.backward_varlen(*x, o, lse, do.cuda(), cu, scale=scale)
    for a, b in zip(got, R.attention_backward(*map(R.f64, (q, k, v, do)), lens, scale)):
        assert R.norm_error(a, b) <= (FP32 if dtype == torch.float32 else GRAD) or np.linalg.norm(b) == 0


def test_growing_scores():
    """The running maximum moves at every tile: keys that score higher and higher, from far below zero."""
    T, D = 700, 64
    q = torch.zeros(T, 1, D)
    q[..., 0] = 8.0
    k = torch.zeros(T, 1, D)
    k[:, 0, 0] = torch.linspace(-60, 60, T)
    v = torch.randn(T, 1, D, generator=torch.Generator().manual_seed(1))
    for dtype in (torch.float32, torch.bfloat16):
        x = [t.to(dtype) for t in (q, k, v)]
        o, lse = attention.forward_varlen(*cuda(x), [0, T])
        check_forward(o, lse, *x, [T], dtype)


def test_backward_is_the_forwards_derivative():
    """Central differences along random directions, forward and backward both on the GPU in fp32; the third-order
    term at step 1e-2 and the forward's rounding (128 * 2^-24 of the loss over the step) stay below 2e-3 of the
    gradient's norm."""
    lens = [70, 33]
    q, k, v, do = cuda(make(lens, 2, 1, 64, torch.float32, seed=2))
    cu = R.offsets(lens)
    o, lse = attention.forward_varlen(q, k, v, cu)
    grads = attention.backward_varlen(q, k, v, o, lse, do, cu)
    loss = lambda x: float((attention.forward_varlen(*x, cu)[0].double() * do.double()).sum())   # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(5)
    for i in range(3):
        d = torch.randn((q, k, v)[i].shape, generator=gen, device="cuda")
        d /= d.norm()
        y = []
        for s in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + s * 1e-2 * d
            y.append(loss(x))
        assert abs((y[0] - y[1]) / 2e-2 - float((grads[i].double() * d.double()).sum())) <= 2e-3 * float(grads[i].double().norm())


def test_samples_do_not_touch_each_other_nor_the_rows_behind():
    lens, spare = [65, 1, 130], 40
    for dtype in (torch.float32, torch.bfloat16):
        for D in (64, 128):
            q, k, v, do = cuda(make(lens, 2, 1, D, dtype, seed=4, spare=spare))
            cu = R.offsets(lens)
            o, lse = attention.forward_varlen(q, k, v, cu)
            g = attention.backward_varlen(q, k, v, o, lse, do, cu)
            bad = [t.clone() for t in (q, k, v, do)]
            for t in bad:
                t[66:] = float("nan")
            o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
            attention.forward_varlen(*bad[:3], cu, o=o2, lse=lse2)
            assert torch.equal(o2[:66], o[:66]) and torch.equal(lse2[:66], lse[:66])
            assert bool((o2[sum(lens):] == 7.0).all()) and bool((lse2[sum(lens):] == 7.0).all())
            out = tuple(torch.full_like(t, 7.0) for t in g)
            attention.backward_varlen(*bad[:3], o2, lse2, bad[3], cu, out=out)
            for a, b in zip(out, g):
                assert torch.equal(a[:66], b[:66]) and bool((a[sum(lens):] == 7.0).all())


def test_unaligned_tensors():
    lens = [150, 20]
    x = make(lens, 2, 1, 64, torch.bfloat16, seed=9)

    def shift(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.flatten().cuda()
        return buf[1:].view(t.shape)

    q, k, v, do = map(shift, x)
    o, lse = attention.forward_varlen(q, k, v, R.offsets(lens))
    check_forward(o, lse, *x[:3], lens, torch.bfloat16)
    got = attention.backward_varlen(q, k, v, o, lse, do, R.offsets(lens))
    for a, b in zip(got, R.attention_backward(*map(R.f64, x), lens)):
        assert R.norm_error(a, b) <= GRAD


def test_more_samples_than_one_launch_takes():
    lens = [(7 * i) % 5 for i in range(600)]
    q, k, v, do = make(lens, 2, 1, 64, torch.bfloat16, seed=6)
    x = cuda((q, k, v))
    o, lse = attention.forward_varlen(*x, R.offsets(lens))
    check_forward(o, lse, q, k, v, lens, torch.bfloat16)
    got = attention.backward_varlen(*x, o, lse, do.cuda(), R.offsets(lens))
    for a, b in zip(got, R.attention_backward(*map(R.f64, (q, k, v, do)), lens)):
        assert R.norm_error(a, b) <= GRAD


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_calls_replay(dtype):
    lens, cu = [200, 65], R.offsets([200, 65])
    a, b = (cuda(make(lens, 4, 2, 128, dtype, seed=s)) for s in (1, 2))

    def call(x):
        o, lse = attention.forward_varlen(*x[:3], cu)
        return (o, lse, *attention.backward_varlen(*x[:3], o, lse, x[3], cu))

    static = [t.clone() for t in a]
    eager = call(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(static)
    for s, t in zip(static, b):
        s.copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, call(b)))
    assert all(torch.equal(x, y) for x, y in zip(eager, call(a)))


def test_two_streams_at_once():
    lens, cu = [300, 100], R.offsets([300, 100])
    sets = [cuda(make(lens, 4, 2, 128, torch.bfloat16, seed=20 + i)) for i in range(2)]

    def call(x, stream=None):
        o, lse = attention.forward_varlen(*x[:3], cu, stream=stream)
        return (o, lse, *attention.backward_varlen(*x[:3], o, lse, x[3], cu, stream=stream))

    want = [call(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [call(x, s) for x, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_hybrid_pair_of_layers():
    """Both mixers over the same packed samples, one after the other, with their gradients, as a hybrid stack
    runs them: attention's output is the delta rule's value."""
    from linear_attention_sequence_mshortconv_b200 import gdn
    lens, H, Hkv, D = [70, 1, 130], 4, 2, 64
    cu, T = R.offsets(lens), sum(lens)
    gen = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
    aq, ak, av = n(T, H, D), n(T, Hkv, D), n(T, Hkv, D)
    q, k, g, beta, do = unit(n(T, 2, D)), unit(n(T, 2, D)), -0.1 * torch.rand(T, H, generator=gen), torch.sigmoid(n(T, H)), n(T, H, D)
    ref_v, _ = R.attention(*map(R.f64, (aq, ak, av)), lens)
    ref_o, _ = R.gdn(R.f64(q), R.f64(k), ref_v, R.f64(g), R.f64(beta), lens)
    ref_d = R.gdn_backward(R.f64(q), R.f64(k), ref_v, R.f64(g), R.f64(beta), R.f64(do), lens)
    ref_a = R.attention_backward(*map(R.f64, (aq, ak, av)), ref_d[2], lens)
    aq, ak, av, q, k, g, beta, do = cuda((aq, ak, av, q, k, g, beta, do))
    v, lse = attention.forward_varlen(aq, ak, av, cu)
    o, _ = gdn.forward_varlen(q, k, v, g, beta, cu, want_state=False)
    d = gdn.backward_varlen(q, k, v, g, beta, do, cu, want_dS0=False)
    a = attention.backward_varlen(aq, ak, av, v, lse, d[2], cu)
    assert R.norm_error(o, ref_o) <= FP32
    for x, y in zip((*d[:5], *a), (*ref_d[:5], *ref_a)):
        assert R.norm_error(x, y) <= FP32
