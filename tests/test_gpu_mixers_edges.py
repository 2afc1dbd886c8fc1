"""The gated delta rule and causal attention on the GPU where they can go wrong.  Tolerances as in test_gpu_gdn.py and
test_gpu_attention.py, or derived beside the test."""
import numpy as np
import pytest
import torch

import mixers_ref as R
from linear_attention_sequence_mshortconv_b200 import attention, gdn, kda
from test_gpu_attention import FP32, FWD, GRAD
from test_gpu_attention import make as make_attention
from test_gpu_gdn import PIECES, check_grads, cuda, kernels, make, make_step, tol

pytestmark = pytest.mark.gpu


# ---- a gate that is not a number ---------------------------------------------------------------------------------------
def same_where_finite(got, clean, nan, free):
    """`got` is NaN where `nan` says so and bit-equal to `clean` elsewhere; entries marked `free` may be either."""
    got, clean = R.f64(got), R.f64(clean)
    assert np.isnan(got[nan & ~free]).all() and (got == clean)[~nan & ~free].all() and not np.isnan(clean).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,Dk,Dv", [(2, 32, 32), (2, 64, 128), (2, 128, 32), (40, 64, 64), (40, 128, 128)])
def test_a_gate_that_is_not_a_number(H, Dk, Dv, dtype):
    """One NaN gate: by the recurrence the state and the outputs of its head are NaN from its token on, and every
    gradient that passes through one of the states.  The rest of its 64-token chunk may be as well; nothing else."""
    lens, at, chunk = [150, 70], 75, slice(64, 128)
    x, S0, do, dS = make(lens, H, H, Dk, Dv, dtype, seed=17)
    args = lambda t: (*cuda(t), do.cuda(), R.offsets(lens), S0.cuda(), dS.cuda())   # noqa: E731
    clean = gdn.backward_varlen(*args(x))
    clean_o, clean_S = gdn.forward_varlen(*cuda(x), R.offsets(lens), S0.cuda())
    x[3][at, 1] = float("nan")
    ref_o, ref_S = R.gdn(*map(R.f64, x), lens, R.f64(S0))
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, R.f64(S0), R.f64(dS))
    assert np.isnan(ref_S[0, 1]).all() and np.isnan(ref_o[at:150, 1]).all() and np.isnan(ref[3][:150, 1]).all()
    o, S = gdn.forward_varlen(*cuda(x), R.offsets(lens), S0.cuda())
    for a, b, want in ((o, clean_o, ref_o), *zip(gdn.backward_varlen(*args(x))[:5], clean, ref)):
        free = np.zeros(want.shape, bool)
        free[chunk, 1] = True
        same_where_finite(a, b, np.isnan(want), free)
    assert np.isnan(R.f64(o)[at:150, 1]).all()
    same_where_finite(S, clean_S, np.isnan(ref_S), np.zeros(ref_S.shape, bool))
    assert kda.last_device_error() == 0


def test_a_gate_that_is_not_a_number_in_a_long_sample():
    lens, at = [6000], 3000
    x, S0, _, _ = make(lens, 2, 2, 64, 64, torch.bfloat16, seed=18, g_scale=0.02)
    (clean, clean_S), ran = kernels(PIECES, lambda: gdn.forward_varlen(*cuda(x), R.offsets(lens), S0.cuda()))
    assert ran == PIECES
    x[3][at, 1] = float("nan")
    o, S = gdn.forward_varlen(*cuda(x), R.offsets(lens), S0.cuda())
    first = at // 64 * 64
    assert torch.equal(o[:, 0], clean[:, 0]) and torch.equal(o[:first, 1], clean[:first, 1]) and torch.equal(S[0, 0], clean_S[0, 0])
    assert bool(o[at:, 1].isnan().all()) and bool(S[0, 1].isnan().all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_gate_that_is_not_a_number_in_a_step(dtype):
    x, state, at = make_step(3, 5, 2, 2, 64, 64, dtype)
    x[3][1, 0] = float("nan")
    S = state.cuda()
    o = gdn.step(*cuda(x), S, at.cuda())
    assert bool(o[1, 0].isnan().all()) and bool(S[int(at[1]), 0].isnan().all())
    assert int(o.isnan().sum()) == 64 and int(S.isnan().sum()) == 64 * 64


# ---- scores of minus infinity ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,H,masked,value,scale", [
    (64, 2, 130, -np.inf, None), (128, 4, 64, -np.inf, None), (64, 3, 200, -np.inf, -0.1), (128, 2, 1, -np.inf, 0.2),
    (64, 2, 130, torch.finfo(torch.bfloat16).min, None), (64, 2, 130, torch.finfo(torch.bfloat16).min, 1.0)], ids=str)
def test_keys_scored_minus_infinity(D, H, masked, value, scale, dtype):
    """The first keys score minus infinity (or the type's lowest value) with every query, over whole blocks: the rows that
    see other keys take those alone, and the rows that see none have no sum."""
    lens = [300]
    q, k, v, _ = make_attention(lens, H, 1, D, dtype, seed=21)
    q[..., 0] = 1.0 if (scale or 1) > 0 else -1.0
    k[:masked, :, 0] = value
    far = k.clone()
    far[:masked, :, 0] = -1e5   # e^-10000 is 0 in 64 bits too
    ref_o, ref_lse = R.attention(*map(R.f64, (q, far, v)), lens, scale)
    o, lse = attention.forward_varlen(*cuda((q, k, v)), R.offsets(lens), scale=scale)
    assert R.norm_error(o[masked:], ref_o[masked:]) <= (FP32 if dtype == torch.float32 else FWD)
    top = float(max(1.0, np.abs(ref_lse[masked:]).max(), abs(scale or D ** -0.5) * q.double().norm(dim=-1).max() * k[masked:].double().norm(dim=-1).max()))
    assert np.abs(R.f64(lse)[masked:] - ref_lse[masked:]).max() <= 16 * 2.0 ** -24 * top
    if value == -np.inf:
        assert bool((lse[:masked] == -np.inf).all()) and bool(o[:masked].isnan().all())
    assert kda.last_device_error() == 0


# ---- the gradients over equal rows -------------------------------------------------------------------------------------
ROWS = [  # B, T, Hk, Hv, Dk, Dv
    (2, 130, 2, 2, 128, 128), (3, 64, 1, 4, 64, 64), (1, 1, 2, 2, 128, 128), (2, 77, 1, 1, 32, 32), (4, 65, 1, 3, 64, 32),
    (5, 63, 16, 32, 128, 64), (3, 193, 16, 32, 64, 128), (7, 129, 8, 24, 128, 32), (100, 1, 1, 2, 64, 64), (90, 65, 1, 2, 128, 64), (255, 64, 1, 1, 64, 32)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_gradients_of_rows_equal_packed_samples(case, dtype):
    B, T, Hk, Hv, Dk, Dv = case
    x, S0, do, dS = make([T] * B, Hk, Hv, Dk, Dv, dtype, seed=B + T)
    x, S0, do, dS = cuda(x), S0.cuda(), do.cuda(), dS.cuda()
    rows = lambda t: t.view(B, T, *t.shape[1:])   # noqa: E731
    got = gdn.backward(*map(rows, x), rows(do), S0, dS)
    for a, b in zip(got, gdn.backward_varlen(*x, do, R.offsets([T] * B), S0, dS)):
        assert torch.equal(a.view_as(b), b)
    o, S = gdn.forward(*map(rows, x), S0)
    o2, S2 = gdn.forward_varlen(*x, R.offsets([T] * B), S0)
    assert torch.equal(o.view_as(o2), o2) and torch.equal(S, S2)
    assert kda.last_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Dk,Dv", [(300, 1, 64, 64), (300, 63, 64, 128), (300, 64, 128, 64), (300, 65, 64, 32), (700, 17, 128, 128), (1111, 3, 64, 64)])
def test_many_rows(B, T, Dk, Dv, dtype):
    """More rows than a launch takes packed samples."""
    x, S0, do, dS = make([T] * B, 1, 1, Dk, Dv, dtype, seed=B + T)
    rows = lambda t: t.view(B, T, *t.shape[1:]).cuda()   # noqa: E731
    ref_o, ref_S = R.gdn(*map(R.f64, x), [T] * B, R.f64(S0))
    o, S = gdn.forward(*map(rows, x), S0.cuda())
    assert R.norm_error(o.flatten(0, 1), ref_o) <= tol(dtype) and R.norm_error(S, ref_S) <= tol(torch.float32)
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), [T] * B, R.f64(S0), R.f64(dS))
    got = gdn.backward(*map(rows, x), rows(do), S0.cuda(), dS.cuda())
    check_grads([t.flatten(0, 1) for t in got[:5]] + [got[5]], ref, x, tol(dtype, grad=True))
    assert kda.last_device_error() == 0


@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv,dtype", [(2800, 2, 4, 16, 64, 64, torch.bfloat16), (2300, 33, 2, 8, 128, 128, torch.bfloat16),
                                                    (2300, 1, 8, 32, 64, 32, torch.bfloat16), (4200, 1, 4, 16, 128, 128, torch.float32)])
def test_many_short_rows_of_many_heads(B, T, Hk, Hv, Dk, Dv, dtype):
    """Rows that go in several groups, for their workspace: the bits of packed samples (255 to a launch)."""
    gen = torch.Generator(device="cuda").manual_seed(B)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
    x = [t.to(dtype) for t in (unit(n(B * T, Hk, Dk)), unit(n(B * T, Hk, Dk)), n(B * T, Hv, Dv), -0.1 * n(B * T, Hv).abs(), torch.sigmoid(n(B * T, Hv)))]
    S0, do, dS = n(B, Hv, Dk, Dv), n(B * T, Hv, Dv).to(dtype), n(B, Hv, Dk, Dv)
    rows = lambda t: t.view(B, T, *t.shape[1:])   # noqa: E731
    ws = torch.full((gdn.backward_workspace_size(B, T, Hk, Hv, Dk, Dv, dtype) + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for a, b in zip(gdn.backward(*map(rows, x), rows(do), S0, dS, workspace=ws[:-4096]), gdn.backward_varlen(*x, do, R.offsets([T] * B), S0, dS)):
        assert torch.equal(a.view_as(b), b)
    assert bool((ws[-4096:] == 0xA5).all())
    o, S = gdn.forward(*map(rows, x), S0)
    o2, S2 = gdn.forward_varlen(*x, R.offsets([T] * B), S0)
    assert torch.equal(o.view_as(o2), o2) and torch.equal(S, S2)
    assert kda.last_device_error() == 0


# ---- workspaces ----------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (128, 32)])
@pytest.mark.parametrize("lens", [[70, 20], [130, 0, 1, 640]], ids=str)
def test_unaligned_gradients_with_a_workspace_of_the_stated_size(lens, Dk, Dv):
    """What is stated is for aligned tensors: views one element into their storage take another kernel, which may need more,
    and write nothing behind the workspace."""
    x, S0, do, dS = make(lens, 1, 2, Dk, Dv, torch.bfloat16, seed=44)

    def shift(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.flatten().cuda()
        return buf[1:].view(t.shape)

    cu = R.offsets(lens)
    need = gdn.backward_varlen_workspace_size(cu, 1, 2, Dk, Dv)
    ref = R.gdn_backward(*map(R.f64, x), R.f64(do), lens, R.f64(S0), R.f64(dS))
    for move in (shift, lambda t: t.cuda()):
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        got = gdn.backward_varlen(*map(move, x), move(do), cu, S0.cuda(), dS.cuda(), workspace=ws[:need])
        check_grads(got, ref, x, tol(torch.bfloat16, grad=True))
        assert bool((ws[need:] == 0xA5).all())
        with pytest.raises(kda.KdaError):
            gdn.backward_varlen(*map(move, x), move(do), cu, S0.cuda(), dS.cuda(), workspace=ws[:need - 256])


# ---- gradients of flat and of peaked softmaxes ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_gradients_without_a_scale(D, dtype):
    """scale = 0: q and k have no part in the output, and their gradients are exactly zero."""
    lens = [200, 65, 400]
    x = make_attention(lens, 2, 1, D, dtype, seed=6)
    q, k, v, do = cuda(x)
    o, lse = attention.forward_varlen(q, k, v, R.offsets(lens), scale=0.0)
    dq, dk, dv = attention.backward_varlen(q, k, v, o, lse, do, R.offsets(lens), scale=0.0)
    assert bool((dq == 0).all()) and bool((dk == 0).all())
    assert R.norm_error(dv, R.attention_backward(*map(R.f64, x), lens, 0.0)[2]) <= (FP32 if dtype == torch.float32 else GRAD)


def magnitudes(q, k, v, do, lens, scale):
    """Per entry of dq, dk, dv the sum of the magnitudes of its terms, the score gradient p (do.v - delta) counted as
    p (|do.v| + |delta|)."""
    T, H, D = q.shape
    r = H // k.shape[1]
    out = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    at = 0
    for n in lens:
        sl = slice(at, at + n)
        for h in range(H):
            s = np.where(np.tril(np.ones((n, n), bool)), scale * q[sl, h] @ k[sl, h // r].T, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            dp = do[sl, h] @ v[sl, h // r].T
            ds = abs(scale) * p * (np.abs(dp) + np.abs((p * dp).sum(1, keepdims=True)))
            out[0][sl, h] = ds @ np.abs(k[sl, h // r])
            out[1][sl, h // r] += ds.T @ np.abs(q[sl, h])
            out[2][sl, h // r] += p.T @ np.abs(do[sl, h])
        at += n
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", [[200, 65], [600]], ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_scores_in_the_hundreds(D, lens, dtype):
    """One key takes most of each row.  A weight e^{s - lse} is off by the errors of s and of lse, 16 * 2^-24 times the
    largest |q||k| each (as the forward's test has them); a term of dq or dk is that, and in bf16 a rounding of the weight or
    of the score gradient and delta's from the rounded o, 2^-8 each; and each sum is rounded once.  The terms of a
    peaked row cancel, so the bound is of the sum of their magnitudes: 3 * 2^-8 + 32 * 2^-24 |q||k| in bf16,
    128 * 2^-24 + 32 * 2^-24 |q||k| in fp32."""
    x = make_attention(lens, 2, 1, D, dtype, seed=6, size=3.0)
    q, k, v, do = cuda(x)
    o, lse = attention.forward_varlen(q, k, v, R.offsets(lens), scale=1.0)
    got = attention.backward_varlen(q, k, v, o, lse, do, R.offsets(lens), scale=1.0)
    f = list(map(R.f64, x))
    top = np.linalg.norm(f[0], axis=-1).max() * np.linalg.norm(f[1], axis=-1).max()
    bound = 32 * 2.0 ** -24 * top + (FP32 if dtype == torch.float32 else GRAD)
    for name, a, b, size in zip(("dq", "dk", "dv"), got, R.attention_backward(*f, lens, 1.0), magnitudes(*f, lens, 1.0)):
        assert np.linalg.norm(R.f64(a) - b) <= bound * np.linalg.norm(size), name


# ---- calls without a tensor that they need -------------------------------------------------------------------------------
@pytest.mark.parametrize("which", range(5))
def test_a_step_without_an_input_is_refused(which):
    x, state, at = make_step(3, 5, 2, 2, 64, 64, torch.bfloat16)
    x = cuda(x)
    x[which] = None
    with pytest.raises((TypeError, ValueError)):
        gdn.step(*x, state.cuda(), at.cuda())
