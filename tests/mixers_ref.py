"""Plain 64-bit forms of the gated delta rule and of causal attention, token by token and row by row on the
CPU (numpy), and the bounds their tests share."""
import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def f64(t):
    return t.detach().double().cpu().numpy()


def gdn(q, k, v, g, beta, lens, S0=None):
    """q, k [T,Hk,Dk], v [T,Hv,Dv], g, beta [T,Hv] on one token axis -> o [T,Hv,Dv], S [n,Hv,Dk,Dv]."""
    T, Hv, Dv = v.shape
    r, Dk = Hv // q.shape[1], q.shape[2]
    o = np.zeros((T, Hv, Dv))
    S_T = np.zeros((len(lens), Hv, Dk, Dv))
    at = 0
    for i, n in enumerate(lens):
        S = np.zeros((Hv, Dk, Dv)) if S0 is None else S0[i].copy()
        for t in range(at, at + n):
            kt, qt = np.repeat(k[t], r, 0), np.repeat(q[t], r, 0)
            S = np.exp(g[t])[:, None, None] * S
            S = S + (beta[t][:, None] * kt)[:, :, None] * (v[t] - np.einsum("hk,hkv->hv", kt, S))[:, None, :]
            o[t] = np.einsum("hk,hkv->hv", qt, S)
        S_T[i] = S
        at += n
    return o, S_T


def gdn_backward(q, k, v, g, beta, do, lens, S0=None, dS_T=None):
    """Reverse sweep of gdn(): dq, dk, dv, dg, dbeta, dS0."""
    T, Hv, Dv = v.shape
    r, Dk = Hv // q.shape[1], q.shape[2]
    dq, dk, dv, dg, db = np.zeros((T, Hv, Dk)), np.zeros((T, Hv, Dk)), np.zeros_like(v), np.zeros_like(g), np.zeros_like(g)
    dS0 = np.zeros((len(lens), Hv, Dk, Dv))
    at = 0
    for i, n in enumerate(lens):
        S = np.zeros((Hv, Dk, Dv)) if S0 is None else S0[i].copy()
        kept = []
        for t in range(at, at + n):
            kt = np.repeat(k[t], r, 0)
            kept.append(S)
            S = np.exp(g[t])[:, None, None] * S
            S = S + (beta[t][:, None] * kt)[:, :, None] * (v[t] - np.einsum("hk,hkv->hv", kt, S))[:, None, :]
        D = np.zeros((Hv, Dk, Dv)) if dS_T is None else dS_T[i].copy()
        for t in reversed(range(at, at + n)):
            kt, qt = np.repeat(k[t], r, 0), np.repeat(q[t], r, 0)
            a = np.exp(g[t])[:, None, None]
            A = a * kept.pop()
            w = v[t] - np.einsum("hk,hkv->hv", kt, A)
            after = A + (beta[t][:, None] * kt)[:, :, None] * w[:, None, :]
            D = D + qt[:, :, None] * do[t][:, None, :]
            dq[t] = np.einsum("hkv,hv->hk", after, do[t])
            kD = np.einsum("hk,hkv->hv", kt, D)
            db[t] = (kD * w).sum(-1)
            dv[t] = beta[t][:, None] * kD
            dk[t] = beta[t][:, None] * np.einsum("hkv,hv->hk", D, w) - np.einsum("hkv,hv->hk", A, dv[t])
            D = D - kt[:, :, None] * dv[t][:, None, :]
            dg[t] = (D * A).sum((-1, -2))
            D = a * D
        dS0[i] = D
        at += n
    group = lambda x: x.reshape(T, Hv // r, r, Dk).sum(2)   # noqa: E731
    return group(dq), group(dk), dv, dg, db, dS0


def attention(q, k, v, lens, scale=None):
    """q [T,H,D], k, v [T,Hkv,D] -> o [T,H,D], lse [T,H]."""
    T, H, D = q.shape
    r = H // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    o, lse = np.zeros_like(q), np.zeros((T, H))
    at = 0
    for n in lens:
        for h in range(H):
            s = scale * q[at:at + n, h] @ k[at:at + n, h // r].T
            s = np.where(np.tril(np.ones((n, n), bool)), s, -np.inf)
            if n:
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                z = p.sum(1, keepdims=True)
                o[at:at + n, h] = (p / z) @ v[at:at + n, h // r]
                lse[at:at + n, h] = (m + np.log(z))[:, 0]
        at += n
    return o, lse


def attention_backward(q, k, v, do, lens, scale=None):
    T, H, D = q.shape
    r = H // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    at = 0
    for n in lens:
        sl = slice(at, at + n)
        for h in range(H if n else 0):
            Q, K, V, G = q[sl, h], k[sl, h // r], v[sl, h // r], do[sl, h]
            s = np.where(np.tril(np.ones((n, n), bool)), scale * Q @ K.T, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            dp = G @ V.T
            ds = scale * p * (dp - (p * dp).sum(1, keepdims=True))
            dq[sl, h] = ds @ K
            dk[sl, h // r] += ds.T @ Q
            dv[sl, h // r] += p.T @ G
        at += n
    return dq, dk, dv


def offsets(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def norm_error(x, ref):
    """2-norm of the difference over the reference's (0 where both are 0)."""
    x = f64(x) if isinstance(x, torch.Tensor) else x
    d, n = np.linalg.norm((x - ref).ravel()), np.linalg.norm(ref.ravel())
    return d / n if n else (0.0 if d == 0 else np.inf)
