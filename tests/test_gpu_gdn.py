"""The gated delta rule on the GPU against the plain 64-bit recurrence (tests/mixers_ref.py), on the stored
(rounded) inputs.

Tolerances, fixed from the arithmetic.  A bf16 output is rounded once (half a step, 2^-8 of its value), and on the
tensor cores one operand of each output's last product is rounded to bf16 too (another 2^-8 of each term): 2-norms
are within 2 * 2^-8 of the reference's.  A gradient there passes through one more bf16 operand (the pair products
dO U^T, dY U^T): 3 * 2^-8.  fp32 outputs and states: products of at most 128 terms, summed in fp32 in any order, are
within 128 * 2^-24 of the sum of the terms' magnitudes; the terms here have random signs (the sum of magnitudes is
about sqrt(128) times the norm), which chains through a few such products per token and decays: 128 * 2^-24 in
the 2-norm covers it (7.6e-6).
"""
import numpy as np
import pytest
import torch

import mixers_ref as R
from linear_attention_sequence_mshortconv_b200 import attention, gdn, kda

pytestmark = pytest.mark.gpu
BF16_TOL, BF16_GRAD_TOL, FP32_TOL = 2 * 2.0 ** -8, 3 * 2.0 ** -8, 128 * 2.0 ** -24


def make(lens, Hk, Hv, Dk, Dv, dtype, seed=0, g_scale=0.1, spare=0):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens) + spare
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
    x = (unit(n(T, Hk, Dk)), unit(n(T, Hk, Dk)), n(T, Hv, Dv), -g_scale * torch.rand(T, Hv, generator=gen), torch.sigmoid(n(T, Hv)))
    return [t.to(dtype) for t in x], n(len(lens), Hv, Dk, Dv), n(T, Hv, Dv).to(dtype), n(len(lens), Hv, Dk, Dv)


def check_grads(got, ref, x, tolerance):
    """Each gradient within the tolerance of the reference's 2-norm.  dg is a difference: a token's gate gets
    q.dq + k.(row part of dk) - k.(column part of dk) from its token and the later ones, terms that cancel wholly
    where nothing came before (the first token's dg is 0, the terms are q.dq and its negative).  Each term carries
    the tolerance of its own size, so dg's is taken of |dg| + |q.dq| in the 2-norm.  Below 2^-126, fp32's smallest
    normal number (alpha = e^-90 is), values are subnormal and have an absolute precision only: each entry may be off
    by that much whatever its size."""
    q = R.f64(x[0])
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, ref):
        size = np.linalg.norm(b) + (np.linalg.norm((q * ref[0]).sum(-1)) if name == "dg" else 0.0)
        assert np.linalg.norm(R.f64(a) - b) <= tolerance * size + 2.0 ** -126 * b.size ** 0.5, name


def cuda(ts):
    return [t.cuda() for t in ts]


def tol(dtype, grad=False):
    return FP32_TOL if dtype == torch.float32 else BF16_GRAD_TOL if grad else BF16_TOL


CASES = [  # lens, Hk, Hv, Dk, Dv
    ([1], 1, 1, 32, 32), ([2, 0, 1], 1, 2, 64, 32), ([64], 2, 2, 128, 128), ([63, 65, 1, 0, 128, 17], 2, 4, 128, 64),
    ([200, 3, 129], 1, 3, 64, 128), ([16, 15, 31, 33], 2, 2, 32, 128), ([300], 3, 3, 128, 32), ([0, 0, 130], 1, 1, 64, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_s0", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_varlen(case, with_s0, dtype):
    lens, Hk, Hv, Dk, Dv = case
    x, S0, _, _ = make(lens, Hk, Hv, Dk, Dv, dtype, seed=len(lens))
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, R.f64(S0) if with_s0 else None)
    o, S = gdn.forward_varlen(*cuda(x), R.offsets(lens), S0.cuda() if with_s0 else None)
    assert o.dtype == dtype and S.dtype == torch.float32
    assert R.norm_error(o, ref_o) <= tol(dtype)
    assert R.norm_error(S, ref_S) <= FP32_TOL


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", [(2, 130, 2, 2, 128, 128), (3, 64, 1, 4, 64, 64), (1, 1, 2, 2, 128, 128), (2, 77, 1, 1, 32, 32)])
def test_forward_rows_equal_packed_samples(B, T, Hk, Hv, Dk, Dv, dtype):
    x, S0, _, _ = make([T] * B, Hk, Hv, Dk, Dv, dtype, seed=3)
    x, S0 = cuda(x), S0.cuda()
    o, S = gdn.forward(*[t.view(B, T, *t.shape[1:]) for t in x], S0)
    o2, S2 = gdn.forward_varlen(*x, R.offsets([T] * B), S0)
    assert torch.equal(o.view_as(o2), o2) and torch.equal(S, S2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_states", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward_varlen(case, with_states, dtype):
    lens, Hk, Hv, Dk, Dv = case
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, dtype, seed=7 + len(lens))
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, *((R.f64(S0), R.f64(dS)) if with_states else ()))
    got = gdn.backward_varlen(*cuda(x), do.cuda(), R.offsets(lens), *((S0.cuda(), dS.cuda()) if with_states else ()))
    assert [a.dtype for a in got] == [dtype] * 5 + [torch.float32]
    check_grads(got, ref, x, tol(dtype, grad=True))


def test_backward_is_the_forwards_derivative():
    """Central differences of L = sum(do o) + sum(dS S_T) along random directions, forward and backward both on
    the GPU in fp32.  With step e the difference is off by e^2 |L'''| / 6 (about 1e-4 of it at e = 1e-2) and by
    the forward's rounding, 2 * 128 * 2^-24 * |L| / (2 e) with |L| at most a few hundred times the slope's scale."""
    lens, Hk, Hv, Dk, Dv = [70, 33], 1, 2, 64, 32
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, torch.float32, seed=1)
    x, S0, do, dS = cuda(x), S0.cuda(), do.cuda(), dS.cuda()
    cu = R.offsets(lens)
    grads = gdn.backward_varlen(*x, do, cu, S0, dS)

    def loss(x, S0):
        o, S = gdn.forward_varlen(*x, cu, S0)
        return float((o.double() * do.double()).sum() + (S.double() * dS.double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(5)
    for i in range(6):
        t = (x + [S0])[i]
        d = torch.randn(t.shape, generator=gen, device="cuda")
        d = d / d.norm()
        e = 1e-2 * (0.1 if i in (3, 4) else 1.0)
        shifted = []
        for sgn in (1, -1):
            y = x + [S0]
            y[i] = t + sgn * e * d
            shifted.append(loss(y[:5], y[5]))
        slope, want = (shifted[0] - shifted[1]) / (2 * e), float((grads[i].double() * d.double()).sum())
        scale = float(grads[i].double().norm())
        assert abs(slope - want) <= 2e-3 * scale, (i, slope, want, scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [-0.5, -8.0, -90.0, float("-inf")])
def test_strong_gates(g, dtype):
    """Any gate down to alpha = 0, on some tokens and on all of them."""
    lens, Hk, Hv, Dk, Dv = [150, 70], 2, 2, 64, 64
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, dtype, seed=11)
    x[3][::7] = g
    x[3][150:] = g
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, R.f64(S0))
    o, S = gdn.forward_varlen(*cuda(x), R.offsets(lens), S0.cuda())
    assert R.norm_error(o, ref_o) <= tol(dtype) and R.norm_error(S, ref_S) <= FP32_TOL
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, R.f64(S0), R.f64(dS))
    got = gdn.backward_varlen(*cuda(x), do.cuda(), R.offsets(lens), S0.cuda(), dS.cuda())
    check_grads(got, ref, x, tol(dtype, grad=True))


def test_repeated_keys_without_decay():
    """beta = 1 and the same unit key at every token: each token overwrites the last (A is all ones below the
    diagonal, the worst case of the chunk inverse)."""
    T, D = 192, 64
    k = torch.zeros(T, 1, D)
    k[:, :, 3] = 1.0
    v = torch.randn(T, 1, D, generator=torch.Generator().manual_seed(2))
    for dtype in (torch.float32, torch.bfloat16):
        x = cuda([t.to(dtype) for t in (k, k, v, torch.zeros(T, 1), torch.ones(T, 1))])
        o, S = gdn.forward_varlen(*x, [0, T])
        assert R.norm_error(o, R.f64(x[2])) <= tol(dtype)
        assert R.norm_error(S[0, 0, 3], R.f64(x[2][-1, 0])) <= FP32_TOL


def test_samples_do_not_touch_each_other_nor_the_rows_behind():
    lens, spare = [65, 1, 130], 40
    x, S0, do, _ = make(lens, 1, 2, 128, 64, torch.bfloat16, seed=4, spare=spare)
    x, do, cu = cuda(x), do.cuda(), R.offsets(lens)
    want_o, want_S = gdn.forward_varlen(*x, cu)
    want_g = gdn.backward_varlen(*x, do, cu)
    bad = [t.clone() for t in x]
    for t in bad:
        t[66:] = float("nan")   # the third sample and the spare rows
    o = torch.full_like(want_o, 7.0)
    S = torch.full_like(want_S, 7.0)
    gdn.forward_varlen(*bad, cu, o=o, S_T=S)
    assert torch.equal(o[:66], want_o[:66]) and torch.equal(S[:2], want_S[:2])
    assert bool((o[sum(lens):] == 7.0).all())
    out = tuple(torch.full_like(t, 7.0) for t in want_g)
    gdn.backward_varlen(*bad, do, cu, out=out)
    for a, b in zip(out[:5], want_g):
        assert torch.equal(a[:66], b[:66]) and bool((a[sum(lens):] == 7.0).all())


def test_unaligned_tensors():
    """Views one element into their storage: contiguous, but not 16-byte aligned."""
    lens = [70, 20]
    x, S0, do, dS = make(lens, 1, 2, 64, 64, torch.bfloat16, seed=9)

    def shift(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.flatten().cuda()
        return buf[1:].view(t.shape)

    y = [shift(t) for t in x]
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens)
    o, S = gdn.forward_varlen(*y, R.offsets(lens))
    assert R.norm_error(o, ref_o) <= BF16_TOL and R.norm_error(S, ref_S) <= FP32_TOL
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens)
    check_grads(gdn.backward_varlen(*y, shift(do), R.offsets(lens)), ref, x, BF16_GRAD_TOL)


def test_more_samples_than_one_launch_takes():
    lens = [(7 * i) % 5 for i in range(600)]
    x, S0, do, _ = make(lens, 1, 1, 64, 64, torch.bfloat16, seed=6)
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, R.f64(S0))
    o, S = gdn.forward_varlen(*cuda(x), R.offsets(lens), S0.cuda())
    assert R.norm_error(o, ref_o) <= BF16_TOL and R.norm_error(S, ref_S) <= FP32_TOL
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, R.f64(S0))
    check_grads(gdn.backward_varlen(*cuda(x), do.cuda(), R.offsets(lens), S0.cuda()), ref, x, BF16_GRAD_TOL)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_calls_replay(dtype):
    """Forward and backward in one CUDA graph, replayed on new inputs, while an eager call's outputs live."""
    lens = [100, 65]
    x, S0, do, dS = make(lens, 1, 2, 128, 128, dtype, seed=8)
    y, S02, do2, dS2 = make(lens, 1, 2, 128, 128, dtype, seed=9)
    cu = R.offsets(lens)
    static = cuda(x) + [S0.cuda(), do.cuda(), dS.cuda()]
    call = lambda s: (*gdn.forward_varlen(*s[:5], cu, s[5]), *gdn.backward_varlen(*s[:5], s[6], cu, s[5], s[7]))   # noqa: E731
    eager = call(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(static)
    for s, t in zip(static, cuda(y) + [S02.cuda(), do2.cuda(), dS2.cuda()]):
        s.copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, call(cuda(y) + [S02.cuda(), do2.cuda(), dS2.cuda()])):
        assert torch.equal(a, b)
    for a, b in zip(eager, call(cuda(x) + [S0.cuda(), do.cuda(), dS.cuda()])):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    lens = [260, 100]
    sets = [make(lens, 2, 4, 128, 128, torch.bfloat16, seed=20 + i) for i in range(2)]
    cu = R.offsets(lens)
    sets = [(cuda(x), S0.cuda(), do.cuda()) for x, S0, do, _ in sets]
    want = [(*gdn.forward_varlen(*x, cu, S0), *gdn.backward_varlen(*x, do, cu, S0)) for x, S0, do in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(5):
        got = [(*gdn.forward_varlen(*x, cu, S0, stream=s), *gdn.backward_varlen(*x, do, cu, S0, stream=s))
               for (x, S0, do), s in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, w) for u, w in zip(a, b))


def test_workspace_of_the_stated_size():
    lens = [130, 64]
    x, S0, do, _ = make(lens, 1, 2, 128, 128, torch.bfloat16, seed=12)
    x, do, cu = cuda(x), do.cuda(), R.offsets(lens)
    for need, call in ((gdn.varlen_workspace_size(cu, 1, 2, 128, 128), lambda w: gdn.forward_varlen(*x, cu, workspace=w)),
                       (gdn.backward_varlen_workspace_size(cu, 1, 2, 128, 128), lambda w: gdn.backward_varlen(*x, do, cu, workspace=w))):
        guard = 4096
        buf = torch.full((need + guard,), 0xA5, dtype=torch.uint8, device="cuda")
        got, want = call(buf[:need]), call(None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool((buf[need:] == 0xA5).all())
        if need:
            with pytest.raises(kda.KdaError):
                call(buf[:need - 256])


@pytest.mark.parametrize("which", [1, 2, 3, 4])
def test_inputs_of_fewer_tokens_are_refused(which):
    """k, v, g or beta one token shorter than q."""
    x, S0, do, _ = make([8], 1, 2, 64, 64, torch.bfloat16)
    x, do = cuda(x), do.cuda()
    bad = [t[:-1].contiguous() if i == which else t for i, t in enumerate(x)]
    rows = [t[None] for t in bad]
    for call in (lambda: gdn.forward_varlen(*bad, [0, 7]), lambda: gdn.forward(*rows), lambda: gdn.step(*bad, torch.zeros(8, 2, 64, 64, device="cuda")),
                 lambda: gdn.backward_varlen(*bad, do, [0, 7]), lambda: gdn.backward(*rows, do[None])):
        with pytest.raises(ValueError):
            call()


# ---- many heads or samples: whole heads to a CTA in the scan, two column tiles in the reverse one ----------------------
WIDE = [  # lens, Hk, Hv, Dk, Dv
    ([64] * 10, 4, 8, 128, 128), ([130, 70, 0, 1, 129], 16, 32, 128, 64), ([65] * 6 + [3], 2, 6, 64, 128),
    ([63, 1, 200, 64, 130], 32, 32, 64, 64), ([191] + [128, 127] * 5, 2, 6, 128, 128)]
NARROW = [([40, 65] * 10, 4, 8, 64, 32), ([1, 129, 64] * 6, 1, 9, 128, 32)]   # Dv = 32: columns of heads, two tiles to a CTA


def kernels(names, call):
    """The call's result, and which of the named kernels it launched."""
    for n in names:
        kda.profile_collect(n)
    kda.profile_enable(True)
    try:
        out = call()
        torch.cuda.synchronize()
    finally:
        kda.profile_enable(False)
    return out, {n for n in names if kda.profile_collect(n)}


@pytest.mark.parametrize("with_states", [False, True])
@pytest.mark.parametrize("case", WIDE + NARROW, ids=str)
def test_many_heads(case, with_states):
    lens, Hk, Hv, Dk, Dv = case
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, torch.bfloat16, seed=40 + len(lens))
    states = (S0, dS) if with_states else ()
    cu, whole = R.offsets(lens), Dv > 32
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, *map(R.f64, states[:1]))
    (o, S), ran = kernels(["gdn_chain", "gdn_scan"], lambda: gdn.forward_varlen(*cuda(x), cu, *cuda(states[:1])))
    assert ran == {"gdn_chain" if whole else "gdn_scan"}
    assert R.norm_error(o, ref_o) <= BF16_TOL and R.norm_error(S, ref_S) <= FP32_TOL
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, *map(R.f64, states))
    got, ran = kernels(["gdn_chain_keep", "gdn_scan_keep"], lambda: gdn.backward_varlen(*cuda(x), do.cuda(), cu, *cuda(states)))
    assert ran == {"gdn_chain_keep" if whole else "gdn_scan_keep"}
    check_grads(got, ref, x, BF16_GRAD_TOL)
    assert kda.last_device_error() == 0


@pytest.mark.parametrize("case", [([64, 65, 3] * 60, 2, 2, 64, 64), ([130, 1] * 20, 1, 8, 128, 128), ([100] * 80, 2, 6, 128, 64)], ids=str)
def test_more_chunks_than_sms(case):
    """The gradients' kernel takes several chunks to an SM, ragged ones among them, and groups of many heads."""
    lens, Hk, Hv, Dk, Dv = case
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, torch.bfloat16, seed=90 + Hv)
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, R.f64(S0), R.f64(dS))
    got = gdn.backward_varlen(*cuda(x), do.cuda(), R.offsets(lens), S0.cuda(), dS.cuda())
    check_grads(got, ref, x, BF16_GRAD_TOL)
    assert kda.last_device_error() == 0


@pytest.mark.parametrize("case", [([2000, 1, 777, 2048], 4, 4, 128, 128), ([700, 100, 1333], 2, 6, 128, 64), ([900] * 9, 2, 4, 64, 128),
                                  ([12000], 2, 2, 64, 64)], ids=str)
def test_the_same_call_gives_the_same_bits(case):
    """Nothing depends on which warp, block or copy comes first."""
    lens, Hk, Hv, Dk, Dv = case
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, torch.bfloat16, seed=95)
    x, S0, do, dS, cu = cuda(x), S0.cuda(), do.cuda(), dS.cuda(), R.offsets(lens)
    call = lambda: (*gdn.forward_varlen(*x, cu, S0), *gdn.backward_varlen(*x, do, cu, S0, dS))   # noqa: E731
    want = call()
    for _ in range(15):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert all(bool(torch.isfinite(t.float()).all()) for t in want)


@pytest.mark.parametrize("Dv", [32, 64])
def test_gradients_of_tokens_that_write_nothing(Dv):
    """beta is 0, or far below any rounding, on some tokens and in whole samples."""
    lens, Hk, Hv, Dk = [130, 70, 64], 1, 2, 64
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, torch.bfloat16, seed=33)
    x[4][::5] = 0.0
    x[4][1::5] = 2.0 ** -40
    x[4][2::7] = -2.0 ** -30
    x[4][130:200] = 0.0
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, R.f64(S0), R.f64(dS))
    got = gdn.backward_varlen(*cuda(x), do.cuda(), R.offsets(lens), S0.cuda(), dS.cuda())
    check_grads(got, ref, x, BF16_GRAD_TOL)
    # dbeta of the tokens with beta = 0 by themselves: it does not depend on their own beta
    rows = np.arange(sum(lens)) % 5 == 0
    a, b = R.f64(got[4])[rows], ref[4][rows]
    assert np.linalg.norm(a - b) <= BF16_GRAD_TOL * np.linalg.norm(b)


@pytest.mark.parametrize("g", [-0.5, -8.0, -90.0, float("-inf")])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64)])
def test_many_heads_strong_gates(Dk, Dv, g):
    lens, Hk, Hv = [150, 70, 130], 16, 32
    x, S0, do, dS = make(lens, Hk, Hv, Dk, Dv, torch.bfloat16, seed=11)
    x[3][::7] = g
    x[3][150:] = g
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, R.f64(S0))
    o, S = gdn.forward_varlen(*cuda(x), R.offsets(lens), S0.cuda())
    assert R.norm_error(o, ref_o) <= BF16_TOL and R.norm_error(S, ref_S) <= FP32_TOL
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, R.f64(S0), R.f64(dS))
    got = gdn.backward_varlen(*cuda(x), do.cuda(), R.offsets(lens), S0.cuda(), dS.cuda())
    check_grads(got, ref, x, BF16_GRAD_TOL)


def test_many_heads_repeated_keys_without_decay():
    T, H, D = 192, 48, 128
    k = torch.zeros(T, H, D)
    k[:, :, 3] = 1.0
    v = torch.randn(T, H, D, generator=torch.Generator().manual_seed(2))
    x = cuda([t.to(torch.bfloat16) for t in (k, k, v, torch.zeros(T, H), torch.ones(T, H))])
    o, S = gdn.forward_varlen(*x, [0, T])
    assert R.norm_error(o, R.f64(x[2])) <= BF16_TOL
    assert R.norm_error(S[0, :, 3], R.f64(x[2][-1])) <= FP32_TOL


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (128, 32)])
def test_many_heads_samples_do_not_touch_each_other_nor_the_rows_behind(Dk, Dv):
    lens, spare = [65, 1, 130], 70
    x, S0, do, dS = make(lens, 16, 64, Dk, Dv, torch.bfloat16, seed=4, spare=spare)
    x, do, cu, S0, dS = cuda(x), do.cuda(), R.offsets(lens), S0.cuda(), dS.cuda()
    want_o, want_S = gdn.forward_varlen(*x, cu, S0)
    want_g = gdn.backward_varlen(*x, do, cu, S0, dS)
    for lo, hi in ((66, None), (0, 66)):   # the third sample and the spare rows; the first two
        bad = [t.clone() for t in x]
        for t in bad:
            t[lo:hi] = float("nan")
        keep, seqs = (slice(0, 66), slice(0, 2)) if lo else (slice(66, 196), slice(2, 3))
        o, S = torch.full_like(want_o, 7.0), torch.full_like(want_S, 7.0)
        gdn.forward_varlen(*bad, cu, S0, o=o, S_T=S)
        assert torch.equal(o[keep], want_o[keep]) and torch.equal(S[seqs], want_S[seqs])
        assert bool((o[sum(lens):] == 7.0).all())
        out = tuple(torch.full_like(t, 7.0) for t in want_g)
        gdn.backward_varlen(*bad, do, cu, S0, dS, out=out)
        for a, b in zip(out[:5], want_g):
            assert torch.equal(a[keep], b[keep]) and bool((a[sum(lens):] == 7.0).all())
        assert torch.equal(out[5][seqs], want_g[5][seqs])


def test_many_heads_captured_and_on_two_streams():
    lens = [100, 65, 64]
    cu = R.offsets(lens)
    sets = [make(lens, 16, 32, 128, 128, torch.bfloat16, seed=50 + i) for i in range(2)]
    sets = [cuda(x) + [S0.cuda(), do.cuda(), dS.cuda()] for x, S0, do, dS in sets]
    call = lambda s, **kw: (*gdn.forward_varlen(*s[:5], cu, s[5], **kw), *gdn.backward_varlen(*s[:5], s[6], cu, s[5], s[7], **kw))   # noqa: E731
    want = [call(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [call(s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, w) for u, w in zip(a, b))
    static = [t.clone() for t in sets[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(static)
    for s, t in zip(static, sets[1]):
        s.copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(out, want[1]))
    assert kda.last_device_error() == 0


def test_beside_attention_on_another_stream():
    """Kernels of both mixers, each with all of its tensor memory, at once."""
    lens = [1000, 65, 300]
    cu = R.offsets(lens)
    x, S0, do, dS = make(lens, 16, 32, 128, 128, torch.bfloat16, seed=70)
    x, S0, do, dS = cuda(x), S0.cuda(), do.cuda(), dS.cuda()
    gen = torch.Generator().manual_seed(71)
    q, k, v, dO = (torch.randn(sum(lens), H, 128, generator=gen).to(torch.bfloat16).cuda() for H in (16, 4, 4, 16))
    lse_o = attention.forward_varlen(q, k, v, cu)

    def both(a, b):
        return ((*gdn.forward_varlen(*x, cu, S0, stream=a), *gdn.backward_varlen(*x, do, cu, S0, dS, stream=a)),
                (*attention.forward_varlen(q, k, v, cu, stream=b), *attention.backward_varlen(q, k, v, *lse_o, dO, cu, stream=b)))

    want = both(None, None)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(6):
        got = both(a, b)
        torch.cuda.synchronize()
        assert all(torch.equal(u, w) for g, n in zip(got, want) for u, w in zip(g, n))
    assert kda.last_device_error() == 0


def test_many_heads_workspace_of_the_stated_size():
    lens = [130, 64]
    x, S0, do, _ = make(lens, 16, 64, 128, 128, torch.bfloat16, seed=12)
    x, do, cu = cuda(x), do.cuda(), R.offsets(lens)
    for need, call in ((gdn.varlen_workspace_size(cu, 16, 64, 128, 128), lambda w: gdn.forward_varlen(*x, cu, workspace=w)),
                       (gdn.backward_varlen_workspace_size(cu, 16, 64, 128, 128), lambda w: gdn.backward_varlen(*x, do, cu, workspace=w))):
        buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        got, want = call(buf[:need]), call(None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool((buf[need:] == 0xA5).all())


# ---- few heads and long samples: the samples cut into pieces ------------------------------------------------------------
LONG = [([6000, 0, 70, 3001], 1, 2, 64, 128), ([6107], 2, 2, 128, 64), ([5120, 64], 1, 1, 128, 128), ([9000], 2, 6, 64, 64)]
PIECES = {"gdn_chain", "gdn_chain_state", "gdn_chain_transition", "gdn_carry"}


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_samples(case):
    lens, Hk, Hv, Dk, Dv = case
    x, S0, _, _ = make(lens, Hk, Hv, Dk, Dv, torch.bfloat16, seed=70 + len(lens), g_scale=0.02)
    cu = R.offsets(lens)
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, R.f64(S0))
    x, S0 = cuda(x), S0.cuda()
    (o, S), ran = kernels([*PIECES, "gdn_scan"], lambda: gdn.forward_varlen(*x, cu, S0))
    assert ran == PIECES
    assert R.norm_error(o, ref_o) <= BF16_TOL and R.norm_error(S, ref_S) <= FP32_TOL
    o2, none = gdn.forward_varlen(*x, cu, S0, want_state=False)
    assert none is None and torch.equal(o, o2)
    need = gdn.varlen_workspace_size(cu, Hk, Hv, Dk, Dv)
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    o3, S3 = gdn.forward_varlen(*x, cu, S0, workspace=buf[:need])
    assert torch.equal(o, o3) and torch.equal(S, S3) and bool((buf[need:] == 0xA5).all())
    assert kda.last_device_error() == 0


@pytest.mark.parametrize("g", [-0.5, -90.0, float("-inf")])
def test_long_samples_strong_gates(g):
    lens = [6000]
    x, S0, _, _ = make(lens, 1, 2, 64, 64, torch.bfloat16, seed=13, g_scale=0.01)
    x[3][::701] = g
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, R.f64(S0))
    (o, S), ran = kernels(PIECES, lambda: gdn.forward(*[t[None].cuda() for t in x], S0.cuda()))
    assert ran == PIECES
    assert R.norm_error(o[0], ref_o) <= BF16_TOL and R.norm_error(S, ref_S) <= FP32_TOL


def test_long_samples_without_decay():
    """No gate closes and every key is one of eight: what the pieces hand on is all there is."""
    T, D = 6016, 64
    k = torch.zeros(T, 1, D)
    at = torch.randint(0, 8, (T,), generator=torch.Generator().manual_seed(3))
    k[torch.arange(T), 0, at] = 1.0
    k[:64] = 0.0
    k[torch.arange(64), 0, torch.arange(64)] = 1.0   # the other keys are written once, in the first chunk
    v = torch.randn(T, 1, D, generator=torch.Generator().manual_seed(2))
    x = [t.to(torch.bfloat16) for t in (k, k, v, torch.zeros(T, 1), torch.ones(T, 1))]
    ref_o, ref_S = R.gdn(*map(R.f64, x), [T])
    o, S = gdn.forward_varlen(*cuda(x), [0, T])
    assert R.norm_error(o, ref_o) <= BF16_TOL and R.norm_error(S, ref_S) <= FP32_TOL


def test_long_samples_do_not_touch_each_other_nor_the_rows_behind():
    lens, spare = [6000, 5000, 1], 70
    x, S0, _, _ = make(lens, 1, 2, 128, 64, torch.bfloat16, seed=4, spare=spare, g_scale=0.02)
    x, cu, S0 = cuda(x), R.offsets(lens), S0.cuda()
    want_o, want_S = gdn.forward_varlen(*x, cu, S0)
    for bad_rows, good in (((6000, 11000), [0, 2]), ((0, 6000), [1, 2])):
        bad = [t.clone() for t in x]
        for t in bad:
            t[bad_rows[0]:bad_rows[1]] = float("nan")
            t[sum(lens):] = float("nan")
        o, S = torch.full_like(want_o, 7.0), torch.full_like(want_S, 7.0)
        gdn.forward_varlen(*bad, cu, S0, o=o, S_T=S)
        for i in good:
            assert torch.equal(o[cu[i]:cu[i + 1]], want_o[cu[i]:cu[i + 1]]) and torch.equal(S[i], want_S[i])
        assert bool((o[sum(lens):] == 7.0).all())


def test_long_samples_with_states_off_alignment():
    """States one float into their storage: contiguous, but not 16-byte aligned."""
    lens = [0] * 100 + [6000]
    x, S0, _, _ = make(lens, 1, 2, 64, 64, torch.bfloat16, seed=14, g_scale=0.02)
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, R.f64(S0))
    buf = torch.zeros(2, S0.numel() + 1, device="cuda")
    first, last = (b[1:].view(S0.shape) for b in buf)
    first.copy_(S0)
    need = gdn.varlen_workspace_size(R.offsets(lens), 1, 2, 64, 64)
    for S, out in ((first, None), (S0.cuda(), last), (first, last), (S0.cuda(), None)):
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        o, S_T = gdn.forward_varlen(*cuda(x), R.offsets(lens), S, S_T=out, workspace=ws[:need])
        assert R.norm_error(o, ref_o) <= BF16_TOL and R.norm_error(S_T, ref_S) <= FP32_TOL
        assert bool((ws[need:] == 0xA5).all())


def test_long_samples_captured():
    x, S0, _, _ = make([6000], 2, 2, 64, 64, torch.bfloat16, seed=8, g_scale=0.02)
    y, S1, _, _ = make([6000], 2, 2, 64, 64, torch.bfloat16, seed=9, g_scale=0.02)
    static, other = cuda(x) + [S0.cuda()], cuda(y) + [S1.cuda()]
    call = lambda s: gdn.forward_varlen(*s[:5], [0, 6000], s[5])   # noqa: E731
    want = call(other)
    call(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(static)
    for s, t in zip(static, other):
        s.copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(out, want))


# ---- one token per request --------------------------------------------------------------------------------------
def make_step(n, slots, Hk, Hv, Dk, Dv, dtype, seed=0):
    x, _, _, _ = make([n], Hk, Hv, Dk, Dv, dtype, seed=seed)
    gen = torch.Generator().manual_seed(seed + 100)
    return x, torch.randn(slots, Hv, Dk, Dv, generator=gen), torch.randperm(slots, generator=gen)[:n].to(torch.int32)


def step_ref(x, state, slots):
    q, k, v, g, beta = map(R.f64, x)
    S, o = R.f64(state), np.zeros(v.shape)
    for i, s in enumerate(slots):
        if s >= 0:
            a, b = R.gdn(q[i:i + 1], k[i:i + 1], v[i:i + 1], g[i:i + 1], beta[i:i + 1], [1], S[s:s + 1])
            o[i], S[s] = a[0], b[0]
    return o, S


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,slots,Hk,Hv,Dk,Dv", [(1, 1, 1, 1, 128, 128), (5, 9, 2, 4, 64, 128), (3, 3, 1, 3, 128, 32), (17, 40, 2, 2, 32, 64), (300, 301, 1, 1, 64, 32)])
def test_step(n, slots, Hk, Hv, Dk, Dv, dtype):
    x, state, at = make_step(n, slots, Hk, Hv, Dk, Dv, dtype)
    ref_o, ref_S = step_ref(x, state, at.tolist())
    S = state.cuda()
    o = gdn.step(*cuda(x), S, at.cuda())
    assert R.norm_error(o, ref_o) <= (FP32_TOL if dtype == torch.float32 else 2.0 ** -8)
    assert R.norm_error(S, ref_S) <= FP32_TOL
    untouched = sorted(set(range(slots)) - set(at.tolist()))
    assert torch.equal(S.cpu()[untouched], state[untouched])
    if n == slots:
        S2 = state.cuda()
        o2 = gdn.step(*cuda(x), S2)
        ref_o2, ref_S2 = step_ref(x, state, range(n))
        assert R.norm_error(o2, ref_o2) <= (FP32_TOL if dtype == torch.float32 else 2.0 ** -8)
        assert R.norm_error(S2, ref_S2) <= FP32_TOL
    assert kda.last_device_error() == 0


def test_step_with_padding_and_bad_slots():
    x, state, _ = make_step(6, 4, 1, 2, 64, 64, torch.float32)
    for slots, used, code in (([2, -1, 0, -5, 1, 3], [2, -1, 0, -1, 1, 3], 0),
                              ([2, 0, 2, 1, -1, 0], [2, 0, -1, 1, -1, -1], 1),   # named twice: the first has it
                              ([2, 4, 0, 1000, -1, 1], [2, -1, 0, -1, -1, 1], 1)):   # outside the pool
        ref_o, ref_S = step_ref(x, state, used)
        S = state.cuda()
        o = gdn.step(*cuda(x), S, torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert kda.last_device_error() == code
        assert R.norm_error(o, ref_o) <= FP32_TOL and R.norm_error(S, ref_S) <= FP32_TOL
        assert all(float(o[i].abs().max()) == 0.0 for i, s in enumerate(used) if s < 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_then_tokens(dtype):
    """As they are used: a packed batch of prompts, its final states kept in a pool, then single tokens; the
    outputs are those of the whole sequences at once.  In bf16 the two ways round the same values once."""
    lens, extra, Hk, Hv, D = [70, 1, 129], 9, 1, 2, 128
    whole = [n + extra for n in lens]
    x, _, _, _ = make(whole, Hk, Hv, D, D, dtype, seed=30)
    ref_o, ref_S = R.gdn(*map(R.f64, x), whole)
    at = R.offsets(whole)
    x = cuda(x)
    prompt = [torch.cat([t[at[i]:at[i] + n] for i, n in enumerate(lens)]) for t in x]
    _, S = gdn.forward_varlen(*prompt, R.offsets(lens))
    pool = torch.zeros(5, Hv, D, D, device="cuda")
    slots = torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    for s in range(extra):
        rows = torch.tensor([at[i] + n + s for i, n in enumerate(lens)], device="cuda")
        o = gdn.step(*[t[rows].contiguous() for t in x], pool, slots)
        assert R.norm_error(o, ref_o[rows.cpu().numpy()]) <= (FP32_TOL if dtype == torch.float32 else 2.0 ** -8)
    assert R.norm_error(pool[slots.long()], ref_S) <= FP32_TOL


def test_step_in_a_graph():
    x, state, at = make_step(4, 6, 1, 2, 128, 128, torch.bfloat16)
    x, at, S = cuda(x), at.cuda(), state.cuda()
    gdn.step(*x, state.cuda(), at)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.step(*x, S, at)
    S.copy_(state)
    want = state.cuda()
    for _ in range(3):
        graph.replay()
        assert torch.equal(o, gdn.step(*x, want, at))
    assert torch.equal(S, want)
