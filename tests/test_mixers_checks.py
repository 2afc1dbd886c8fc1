"""CPU checks of the gated delta rule and of causal attention: the 64-bit forms the GPU tests compare against are
pinned by automatic differentiation and by identities, and the library and its binding refuse bad calls before any
launch (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import mixers_ref as R
from linear_attention_sequence_mshortconv_b200 import attention, gdn, kda
from linear_attention_sequence_mshortconv_b200 import build as B

P, D = None, ctypes.c_void_p(256)   # a null pointer; one that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return kda.load_library()


def cu(*offs):
    return (ctypes.c_int32 * len(offs))(*offs)


# ---- the 64-bit forms -----------------------------------------------------------------------------------------
def _random(lens, Hk, Hv, Dk, Dv):
    gen = torch.Generator().manual_seed(1)
    T = sum(lens)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)   # noqa: E731
    return [n(T, Hk, Dk) * 0.3, n(T, Hk, Dk) * 0.3, n(T, Hv, Dv), -torch.rand(T, Hv, generator=gen, dtype=torch.float64),
            torch.rand(T, Hv, generator=gen, dtype=torch.float64), n(len(lens), Hv, Dk, Dv)]


def test_gdn_gradients_equal_autograd():
    lens, Hk, Hv, Dk, Dv = [3, 0, 5], 2, 4, 5, 3
    x = _random(lens, Hk, Hv, Dk, Dv)
    gen = torch.Generator().manual_seed(2)
    do = torch.randn(sum(lens), Hv, Dv, generator=gen, dtype=torch.float64)
    dS = torch.randn(len(lens), Hv, Dk, Dv, generator=gen, dtype=torch.float64)
    leaves = [t.clone().requires_grad_() for t in x]
    q, k, v, g, beta, S0 = leaves
    loss, at = 0.0, 0
    for i, n in enumerate(lens):
        S = S0[i]
        for t in range(at, at + n):
            kt, qt = (z[t].repeat_interleave(Hv // Hk, 0) for z in (k, q))
            I = torch.eye(Dk, dtype=torch.float64) - beta[t][:, None, None] * kt[:, :, None] * kt[:, None, :]
            S = torch.exp(g[t])[:, None, None] * (I @ S) + beta[t][:, None, None] * kt[:, :, None] * v[t][:, None, :]
            loss = loss + (torch.einsum("hkv,hk->hv", S, qt) * do[t]).sum()
        loss = loss + (S * dS[i]).sum()
        at += n
    want = torch.autograd.grad(loss, leaves)
    got = R.gdn_backward(*[t.numpy() for t in x[:5]], do.numpy(), lens, x[5].numpy(), dS.numpy())
    for a, b in zip(got, want):
        assert np.allclose(a, b.numpy(), rtol=1e-10, atol=1e-12)
    o, S = R.gdn(*[t.numpy() for t in x[:5]], lens, x[5].numpy())
    assert np.isclose((o * do.numpy()).sum() + (S * dS.numpy()).sum(), float(loss), rtol=1e-12)


def test_gdn_is_the_oracles_scan_with_one_gate_for_all_channels():
    from oracle import oracle as O
    T, H, D_ = 12, 2, 32
    q, k, v, g, beta, S0 = _random([T], H, H, D_, D_)
    f = [t.float() for t in (q, k, v, g, beta, S0)]
    o, S = O.kda_forward(f[0][None], f[1][None], f[2][None], f[3][None, ..., None].expand(1, T, H, D_).contiguous(), f[4][None], S0=f[5])
    o2, S2 = R.gdn(*[R.f64(t) for t in f[:5]], [T], R.f64(f[5]))
    assert np.allclose(o[0], o2, rtol=1e-10, atol=1e-12) and np.allclose(S, S2, rtol=1e-10, atol=1e-12)


def test_attention_gradients_equal_autograd():
    lens, H, Hkv, W = [4, 1, 0, 6], 4, 2, 3
    gen = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)   # noqa: E731
    T = sum(lens)
    x = [n(T, H, W), n(T, Hkv, W), n(T, Hkv, W)]
    do = n(T, H, W)
    leaves = [t.clone().requires_grad_() for t in x]
    q, k, v = leaves
    loss, at, outs = 0.0, 0, []
    for m in lens:
        K, V = (z[at:at + m].repeat_interleave(H // Hkv, 1) for z in (k, v))
        s = torch.einsum("ihd,jhd->hij", q[at:at + m], K) * 0.4
        s = s.masked_fill(torch.ones(m, m, dtype=torch.bool).triu(1), -torch.inf)
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), V))
        at += m
    loss = (torch.cat(outs) * do).sum()
    want = torch.autograd.grad(loss, leaves)
    for a, b in zip(R.attention_backward(*[t.numpy() for t in x], do.numpy(), lens, 0.4), want):
        assert np.allclose(a, b.numpy(), rtol=1e-10, atol=1e-12)
    o, lse = R.attention(*[t.numpy() for t in x], lens, 0.4)
    assert np.allclose(o, torch.cat(outs).detach().numpy(), rtol=1e-12) and lse.shape == (T, H)


# ---- refusals of the library ------------------------------------------------------------------------------------
def test_gdn_forward_refuses(lib):
    full = lambda q=D, o=D: (q, D, D, D, D, P, o, P)   # noqa: E731
    sizes = lambda B=1, T=8, Hk=1, Hv=1, Dk=64, Dv=64, dt=1: (B, T, Hk, Hv, Dk, Dv, dt, P, 0, P)   # noqa: E731
    f = lib.gdn_forward
    assert f(*full(q=P), *sizes()) == 1 and f(*full(o=P), *sizes()) == 1
    assert f(*full(), *sizes(B=-1)) == 1 and f(*full(), *sizes(T=-1)) == 1
    assert f(*full(), *sizes(Hk=2, Hv=3)) == 1 and f(*full(), *sizes(Hk=0)) == 1
    assert f(*full(), *sizes(dt=2)) == 1
    assert f(*full(), *sizes(Dk=48)) == 2 and f(*full(), *sizes(Dv=256)) == 2
    assert f(*full(), *sizes(B=65536)) == 2 and f(*full(), *sizes(B=60000, T=60000)) == 2
    assert f(*full(), *sizes(Hk=1, Hv=65536)) == 2
    assert f(*full(q=P, o=P), *sizes(B=0)) == 0
    assert lib.gdn_forward_workspace_size(1, 8, 1, 1, 48, 64, 1) == 0
    v = lib.gdn_forward_varlen
    tail = (1, 1, 64, 64, 1, P, 0, P)
    assert v(*full(), P, 1, *tail) == 1                          # no offsets
    assert v(*full(), cu(1, 4), 1, *tail) == 1                   # does not start at 0
    assert v(*full(), cu(0, 4, 3), 2, *tail) == 1                # decreasing
    assert v(*full(), cu(0), -1, *tail) == 1
    assert v(*full(q=P), cu(0, 4), 1, *tail) == 1
    assert v(*full(q=P, o=P), cu(0), 0, *tail) == 0              # no samples
    assert lib.gdn_forward_varlen_workspace_size(cu(0, 4, 3), 2, 1, 1, 64, 64, 1) == 0


def test_gdn_backward_refuses(lib):
    full = lambda q=D, g=D, do=D: (q, D, D, D, D, P, do, P, D, D, D, g, D, P)   # noqa: E731
    sizes = lambda B=1, T=8, Hk=1, Hv=1, Dk=64, Dv=64, dt=1: (B, T, Hk, Hv, Dk, Dv, dt, P, 0, P)   # noqa: E731
    f = lib.gdn_backward
    assert f(*full(q=P), *sizes()) == 1 and f(*full(g=P), *sizes()) == 1 and f(*full(do=P), *sizes()) == 1
    assert f(*full(), *sizes(Hk=2, Hv=3)) == 1 and f(*full(), *sizes(Dk=96)) == 2
    assert f(*full(), 1, 8, 1, 1, 64, 64, 1, D, 16, P) == 5      # a workspace that is too small
    assert f(*full(), 1, 8, 1, 1, 64, 64, 1, ctypes.c_void_p(264), 1 << 40, P) == 1   # and one that is not aligned
    assert lib.gdn_backward_workspace_size(1, 8, 1, 1, 64, 64, 1) > 0
    assert lib.gdn_backward_varlen(*full(), cu(0, 4, 3), 2, 1, 1, 64, 64, 1, P, 0, P) == 1


def test_gdn_step_refuses(lib):
    f = lib.gdn_step
    args = lambda q=D, state=D, slots=D, n=4, ns=8, Hk=1, Hv=1, Dk=64, Dv=64, dt=1: (   # noqa: E731
        q, D, D, D, D, state, slots, D, n, ns, Hk, Hv, Dk, Dv, dt, P)
    assert f(*args(q=P)) == 1 and f(*args(state=P)) == 1 and f(*args(n=-1)) == 1 and f(*args(ns=-1)) == 1
    assert f(*args(slots=P, n=9)) == 1                           # more requests than states
    assert f(*args(state=ctypes.c_void_p(264))) == 1             # state not 16-byte aligned
    assert f(*args(Hk=2, Hv=3)) == 1 and f(*args(dt=5)) == 1
    assert f(*args(Dk=16)) == 2 and f(*args(n=65536, ns=70000)) == 2
    assert f(*args(q=P, n=0)) == 0


def test_attention_refuses(lib):
    f = lib.attn_forward
    args = lambda q=D, o=D, B=1, T=8, H=2, Hkv=1, W=64, scale=0.1, dt=1: (q, D, D, o, P, B, T, H, Hkv, W, scale, dt, P)   # noqa: E731
    assert f(*args(q=P)) == 1 and f(*args(o=P)) == 1 and f(*args(B=-1)) == 1 and f(*args(T=-1)) == 1
    assert f(*args(H=3, Hkv=2)) == 1 and f(*args(Hkv=0)) == 1 and f(*args(dt=3)) == 1
    assert f(*args(scale=float("nan"))) == 1 and f(*args(scale=float("inf"))) == 1
    assert f(*args(W=80)) == 2 and f(*args(B=65536)) == 2 and f(*args(B=60000, T=60000)) == 2
    assert f(*args(q=P, T=0)) == 0 and f(*args(q=P, B=0)) == 0
    assert lib.attn_forward_varlen(D, D, D, D, P, cu(0, 5, 4), 2, 2, 1, 64, 0.1, 1, P) == 1
    assert lib.attn_forward_varlen(D, D, D, D, P, P, 2, 2, 1, 64, 0.1, 1, P) == 1
    b = lambda lse=D, dk=D, W=64: (D, D, D, D, lse, D, D, dk, D, 1, 8, 2, 1, W, 0.1, 1, P, 0, P)   # noqa: E731
    assert lib.attn_backward(*b(lse=P)) == 1 and lib.attn_backward(*b(dk=P)) == 1 and lib.attn_backward(*b(W=96)) == 2
    assert lib.attn_backward_varlen(D, D, D, D, D, D, D, D, D, cu(0, 5, 4), 2, 2, 1, 64, 0.1, 1, P, 0, P) == 1


# ---- refusals of the binding ------------------------------------------------------------------------------------
def test_binding_refuses(lib):
    z = torch.zeros
    x = [z(1, 4, 2, 64), z(1, 4, 2, 64), z(1, 4, 2, 64), z(1, 4, 2), z(1, 4, 2)]
    with pytest.raises(TypeError):
        gdn.forward(*x)                                          # CPU tensors
    with pytest.raises(ValueError):
        gdn.forward(x[0][0], *x[1:])                             # dimensions
    with pytest.raises(ValueError):
        gdn.forward(z(1, 4, 3, 64), z(1, 4, 3, 64), *x[2:])      # 2 value heads, 3 key heads
    flat = [t[0] for t in x]
    with pytest.raises(ValueError):
        gdn.forward_varlen(*flat, [0, 5])                        # offsets past the tokens
    with pytest.raises(ValueError):
        gdn.backward_varlen(*flat, flat[2], [])
    with pytest.raises(TypeError):
        gdn.step(*flat, z(4, 2, 64, 64))
    with pytest.raises(ValueError):
        gdn.step(*flat, z(4, 2, 64))
    with pytest.raises(TypeError):
        gdn.forward(*[t.half() for t in x])                      # neither bf16 nor fp32
    with pytest.raises(TypeError):
        attention.forward(x[0], x[1], x[2])
    with pytest.raises(ValueError):
        attention.forward(z(1, 4, 3, 64), x[1], x[2])
    with pytest.raises(ValueError):
        attention.forward_varlen(flat[0], flat[1], flat[2], [0, 9])


@pytest.mark.gpu
def test_binding_refuses_on_the_device(lib):
    n = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    x = [n(1, 4, 2, 64), n(1, 4, 2, 64), n(1, 4, 2, 64), n(1, 4, 2), n(1, 4, 2)]
    with pytest.raises(TypeError):
        gdn.forward(*x[:3], x[3].float(), x[4])                  # mixed types
    with pytest.raises(ValueError):
        gdn.forward(x[0].transpose(1, 2).contiguous().transpose(1, 2), *x[1:])   # strided
    with pytest.raises(ValueError):
        gdn.forward(*x, n(1, 2, 64, 32, dt=torch.float32))       # S0's shape
    with pytest.raises(TypeError):
        gdn.forward(*x, n(1, 2, 64, 64))                         # S0's type
    with pytest.raises(ValueError):
        gdn.forward(*x[:4], x[4].cpu().cuda()[:, :3])            # beta's shape
    with pytest.raises(TypeError):
        gdn.forward(*x[:4], x[4].cpu())                          # beta on the CPU
    flat = [t[0] for t in x]
    with pytest.raises(TypeError):
        gdn.step(*flat, n(4, 2, 64, 64, dt=torch.float32), torch.arange(4, device="cuda"))   # int64 slots
    with pytest.raises(ValueError):
        attention.backward(x[0], x[1], x[2], x[0], None, x[0])
    with pytest.raises(TypeError):
        attention.forward(x[0], x[1], x[2].float())
