"""The token mixers of a hybrid stack over rows or packed samples, as cases to be timed and compared:

  gdn_forward   the gated delta rule over whole sequences,
                    S_t = a_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   a_t = exp(g_t),   o_t = S_t^T q_t,
                with one gate per value head and several value heads to a query/key head
  gdn_backward  its gradients
  gdn_step      one token per request, the requests' states in a pool, updated in place
  attn_forward  causal softmax attention with grouped heads over the same rows or packed samples
  attn_backward its gradients, from the outputs that the forward kept

`run` computes the plain form in elementary torch operations where `own` is false, and calls the framework's
operators where it is true.  `exact` is the definition token by token (the delta rule) and row by row (attention)
in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64
DEVICE = "cuda"


def _dt(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ---- cases ----------------------------------------------------------------------------------------------------
def listed():
    return [
        # the fp32 parity workload (text 64): the smallest call, where only latency counts
        dict(name="gdn_forward tiny fp32", op="gdn_forward", lens="64", packed=False, hk=2, hv=2, dk=32, dv=32, dtype="fp32", s0=False),
        # prompts of one to a few thousand tokens packed on one axis, continuing from kept states; two value heads to a key head
        dict(name="gdn_forward packed", op="gdn_forward", lens="1,777,64,2049,130,63,1500,3,512,901,65,333", packed=True, hk=4, hv=8, dk=128, dv=128, dtype="bf16", s0=True),
        # one text + video row (512 + 21 x 32 x 48 tokens): few heads, a long serial axis
        dict(name="gdn_forward video clip", op="gdn_forward", lens="32768", packed=False, hk=16, hv=16, dk=128, dv=128, dtype="bf16", s0=False),
        # training on packed samples with shared key heads and narrow keys
        dict(name="gdn_backward packed", op="gdn_backward", lens="700,1,1333,64,255,1024", packed=True, hk=4, hv=8, dk=64, dv=128, dtype="bf16", s0=False),
        # training on a batch of text + image rows (256 + 64 x 64 tokens)
        dict(name="gdn_backward image stream", op="gdn_backward", lens="4352,4352,4352,4352", packed=False, hk=16, hv=16, dk=128, dv=128, dtype="bf16", s0=False),
        # one request answered token by token
        dict(name="gdn_step one request", op="gdn_step", n=1, slots=4, hk=16, hv=16, dk=128, dv=128, dtype="bf16"),
        # a full serving batch out of a larger pool of states
        dict(name="gdn_step batch", op="gdn_step", n=256, slots=300, hk=16, hv=32, dk=128, dv=128, dtype="bf16"),
        # one short text prompt (the text part of a video row)
        dict(name="attn_forward text", op="attn_forward", lens="512", packed=True, hq=16, hkv=4, d=128, dtype="bf16"),
        # ragged prompts, one token among them, narrow heads
        dict(name="attn_forward packed", op="attn_forward", lens="1,777,64,2049,130,63,1500,3,512,901,65,333", packed=True, hq=8, hkv=2, d=64, dtype="bf16"),
        # one long row
        dict(name="attn_forward long", op="attn_forward", lens="16384", packed=False, hq=16, hkv=4, d=128, dtype="bf16"),
        # training on packed samples, narrow heads
        dict(name="attn_backward packed", op="attn_backward", lens="700,1,1333,64,255,1024", packed=True, hq=8, hkv=2, d=64, dtype="bf16"),
        # training on the image-stream batch
        dict(name="attn_backward image stream", op="attn_backward", lens="4352,4352,4352,4352", packed=False, hq=16, hkv=4, d=128, dtype="bf16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_lens(rng, total, most_seqs):
    """(lens, packed): equal rows or ragged samples of about `total` tokens in all."""
    n = min(_logint(rng, 1, most_seqs), total)
    if rng.random() < 0.3:
        return [max(1, total // n)] * n, False
    w = [rng.uniform(0.02, 1.0) ** 2 for _ in range(n)]
    return [max(1, int(total * x / sum(w))) for x in w], True


def draw(rng):
    op = rng.choice(("gdn_forward", "gdn_forward", "gdn_backward", "gdn_step", "attn_forward", "attn_backward"))
    if op == "gdn_step":
        n = _logint(rng, 1, 256)
        hk = rng.choice((1, 2, 4, 6, 8, 16))
        return dict(op=op, n=n, slots=n + rng.randrange(0, 40), hk=hk, hv=hk * rng.choice((1, 2)), dk=rng.choice((64, 128)),
                    dv=rng.choice((64, 128)), dtype="bf16")
    if op in ("attn_forward", "attn_backward"):
        lens, packed = _draw_lens(rng, _logint(rng, 100, 12000), 16)
        hkv = rng.choice((1, 2, 3, 4))
        return dict(op=op, lens=",".join(map(str, lens)), packed=packed, hq=hkv * rng.choice((1, 2, 3, 4)), hkv=hkv,
                    d=rng.choice((64, 128)), dtype="bf16")
    if op == "gdn_forward" and rng.random() < 0.15:
        lens, packed = _draw_lens(rng, _logint(rng, 16, 500), 4)
        d = rng.choice((32, 64))
        return dict(op=op, lens=",".join(map(str, lens)), packed=packed, hk=2, hv=2, dk=d, dv=d, dtype="fp32", s0=rng.random() < 0.5)
    lens, packed = _draw_lens(rng, _logint(rng, 100, 12000), 16)
    hk = rng.choice((1, 2, 3, 4, 8))
    return dict(op=op, lens=",".join(map(str, lens)), packed=packed, hk=hk, hv=hk * rng.choice((1, 2, 3)) if hk < 8 else rng.choice((8, 16)),
                dk=rng.choice((64, 128)), dv=rng.choice((64, 128)), dtype="bf16", s0=op == "gdn_forward" and rng.random() < 0.5)


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("attn_forward", "attn_backward"):
        t, h, hk, d = sum(_lens(case)), case["hq"], case["hkv"], case["d"]
        pairs = sum(n * (n + 1) // 2 for n in _lens(case))
        if case["op"] == "attn_backward":
            return {"bytes": 4 * t * h * d * e + 4 * t * hk * d * e + 4 * t * h, "flops": 10 * pairs * h * d}
        return {"bytes": 2 * t * h * d * e + 2 * t * hk * d * e + 4 * t * h, "flops": 4 * pairs * h * d}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    if case["op"] == "gdn_step":
        n = case["n"]
        return {"bytes": 8 * n * hv * dk * dv + e * n * (2 * hk * dk + 2 * hv * dv + 2 * hv), "flops": 7 * n * hv * dk * dv}
    t, n = sum(_lens(case)), len(_lens(case))
    row = e * (2 * hk * dk + hv * dv + 2 * hv)  # q, k, v, g, beta of one token
    if case["op"] == "gdn_forward":
        return {"bytes": t * (row + e * hv * dv) + (1 + case["s0"]) * 4 * n * hv * dk * dv, "flops": 7 * t * hv * dk * dv}
    return {"bytes": t * (2 * row + e * hv * dv), "flops": 20 * t * hv * dk * dv}


# ---- inputs ---------------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = _dt(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    def unit(*shape):
        x = normal(*shape)
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

    if case["op"] in ("attn_forward", "attn_backward"):
        lens = _lens(case)
        lead = (sum(lens),) if case["packed"] else (len(lens), lens[0])
        s = {"q": normal(*lead, case["hq"], case["d"]).to(dt), "k": normal(*lead, case["hkv"], case["d"]).to(dt),
             "v": normal(*lead, case["hkv"], case["d"]).to(dt)}
    else:
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        if case["op"] == "gdn_step":
            lead, rows = (case["n"],), case["slots"]
        else:
            lens = _lens(case)
            lead, rows = ((sum(lens),) if case["packed"] else (len(lens), lens[0])), len(lens)
        s = {"q": unit(*lead, hk, dk), "k": unit(*lead, hk, dk), "v": normal(*lead, hv, dv).to(dt),
             "g": (-0.001 - 0.099 * torch.rand(*lead, hv, generator=gen, device=DEVICE)).to(dt),
             "beta": torch.sigmoid(normal(*lead, hv)).to(dt)}
        if case["op"] == "gdn_step":
            s["state"] = normal(rows, hv, dk, dv)
            s["slots"] = torch.randperm(rows, generator=gen, device=DEVICE)[: case["n"]].to(torch.int32)
        if case["op"] == "gdn_forward":
            s["S0"] = normal(rows, hv, dk, dv) if case["s0"] else None
        if case["op"] == "gdn_backward":
            s["do"] = (0.01 * normal(*lead, hv, dv)).to(dt)
    s["op"], s["packed"] = case["op"], case.get("packed", False)
    if case["op"] != "gdn_step":
        s["lens"], s["cu"] = lens, [sum(lens[:i]) for i in range(len(lens) + 1)]
    if case["op"] == "attn_backward":
        s["o"], s["lse"] = _plain_attention(s)  # what the forward pass of the training step kept
        s["do"] = (0.01 * normal(*lead, case["hq"], case["d"])).to(dt)
    return s


# ---- plain forms ----------------------------------------------------------------------------------------------
def _chunk_table(lens):
    """Tokens of each chunk ([chunks, 64], -1 past a sample's end), and per step the chunks of the samples still
    running, the longest sample first."""
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    start = [sum(lens[:i]) for i in range(len(lens))]
    count = [-(-lens[i] // CHUNK) for i in order]
    first = [sum(count[:j]) for j in range(len(order))]
    begin = torch.tensor([start[i] for i in order]).repeat_interleave(torch.tensor(count))
    size = torch.tensor([lens[i] for i in order]).repeat_interleave(torch.tensor(count))
    local = torch.arange(sum(count)) - torch.tensor(first).repeat_interleave(torch.tensor(count))
    at = local[:, None] * CHUNK + torch.arange(CHUNK)
    token = torch.where(at < size[:, None], begin[:, None] + at, -1).to(DEVICE)
    live = [sum(c > s for c in count) for s in range(max(count))]
    return token, torch.tensor(first, device=DEVICE), live, torch.tensor(order, device=DEVICE)


def _gdn_chunked(q, k, v, g, beta, S0, lens):
    """o [tokens, hv, dv] and the final states [samples, hv, dk, dv] in fp32, from fp32 tensors on one token axis."""
    token, first, live, order = _chunk_table(lens)
    r = v.shape[1] // q.shape[1]
    inside = (token >= 0)[:, None, :, None]

    def chunks(x):  # [tokens, h, d] -> [chunks, h, 64, d], zero past a sample's end
        return torch.where(inside, x[token.clamp_min(0)].transpose(1, 2), 0.0)

    Q, K = (chunks(x).repeat_interleave(r, 1) for x in (q, k))
    V, G, Bt = chunks(v), chunks(g[..., None]), chunks(beta[..., None])
    b = G.double().cumsum(2)
    low = torch.ones(CHUNK, CHUNK, device=q.device).tril()
    decay = torch.exp(torch.where(low > 0, b - b.transpose(2, 3), -math.inf)).float()
    N = -(Bt * decay * (K @ K.transpose(2, 3))).tril(-1)
    eye = torch.eye(CHUNK, device=q.device)
    T = eye + N
    for _ in range(5):  # (I - N)^-1 = (I + N)(I + N^2)(I + N^4) ...: N^64 = 0
        N = N @ N
        T = T + T @ N
    grow, end = torch.exp(b).float(), torch.exp(b[:, :, -1:] - b).float()
    U0, W = T @ (Bt * V), T @ (Bt * grow * K)
    P, Qg, Ke = decay * (Q @ K.transpose(2, 3)), grow * Q, (end * K).transpose(2, 3)
    last = grow[:, :, -1:]
    S = torch.zeros(len(lens), v.shape[1], q.shape[2], v.shape[2], device=q.device) if S0 is None else S0[order]
    done, outs, where = [], [], []
    for step, n in enumerate(live):
        at = first[:n] + step
        if n < len(S):
            done.append(S[n:])
            S = S[:n]
        U = U0[at] - W[at] @ S
        outs.append(Qg[at] @ S + P[at] @ U)
        where.append(at)
        S = last[at] * S + Ke[at] @ U
    states = torch.cat([S] + done[::-1])
    O = torch.cat(outs).transpose(1, 2)  # [chunks in the order run, 64, h, d]
    ran = token[torch.cat(where)]
    o = torch.zeros_like(v).index_put((ran[ran >= 0],), O[ran >= 0])
    return o, torch.zeros_like(states).index_put((order,), states)


def _flat(x, packed):
    return x if packed else x.flatten(0, 1)


def _plain_gdn(s, grads):
    names = ("q", "k", "v", "g", "beta")
    x = [_flat(s[n], s["packed"]).float() for n in names]
    if not grads:
        o, S = _gdn_chunked(*x, s["S0"], s["lens"])
        return o.to(s["v"].dtype).view_as(s["v"]), S
    with torch.enable_grad():
        x = [t.detach().requires_grad_() for t in x]
        o, _ = _gdn_chunked(*x, None, s["lens"])
        d = torch.autograd.grad(o, x, _flat(s["do"], s["packed"]).float())
    return tuple(t.to(s[n].dtype).view_as(s[n]) for n, t in zip(names, d))


def _plain_step(s):
    r = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(r, 1)[..., None] for n in ("q", "k"))
    v, g, beta = s["v"].float()[:, :, None], s["g"].float()[..., None, None], s["beta"].float()[..., None, None]
    at = s["slots"].long()
    S = s["state"][at] * torch.exp(g)
    S = S + beta * k * (v - (k * S).sum(2, keepdim=True))
    s["state"][at] = S
    return (q * S).sum(2).to(s["v"].dtype), s["state"]


def _plain_attention(s):
    q, k, v = (_flat(s[n], s["packed"]) for n in ("q", "k", "v"))
    h, d, hk = q.shape[1], q.shape[2], k.shape[1]
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[0], h, device=q.device)
    for at, n in zip(s["cu"], s["lens"]):
        K, V = k[at:at + n].float().transpose(0, 1), v[at:at + n].float().transpose(0, 1)
        rows = 1024  # query rows at a time: the scores of a long row would not fit
        for i in range(0, n, rows):
            m = min(n, i + rows)
            Q = q[at + i:at + m].float().view(m - i, hk, h // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
            x = (Q @ K[:, :m].transpose(1, 2) / math.sqrt(d)).view(hk, h // hk, m - i, m)
            x = torch.where(torch.arange(m, device=q.device) <= torch.arange(i, m, device=q.device)[:, None], x, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            z = p.sum(-1, keepdim=True)
            y = (p.view(hk, -1, m) @ V[:, :m]).view(hk, h // hk, m - i, d) / z
            o[at + i:at + m] = y.permute(2, 0, 1, 3).reshape(m - i, h, d).to(q.dtype)
            lse[at + i:at + m] = (top + torch.log(z))[..., 0].permute(2, 0, 1).reshape(m - i, h)
    return o.view_as(s["q"]), lse.view(s["q"].shape[:-1])


def _plain_attention_backward(s):
    q, k, v, do = (_flat(s[n], s["packed"]) for n in ("q", "k", "v", "do"))
    h, d, hk = q.shape[1], q.shape[2], k.shape[1]
    r = h // hk
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for at, n in zip(s["cu"], s["lens"]):
        K, V = k[at:at + n].float().transpose(0, 1), v[at:at + n].float().transpose(0, 1)
        gK, gV = torch.zeros_like(K), torch.zeros_like(V)
        rows = 1024
        for i in range(0, n, rows):
            m = min(n, i + rows)
            Q, G = (t[at + i:at + m].float().view(m - i, hk, r, d).permute(1, 2, 0, 3).reshape(hk, -1, d) for t in (q, do))
            x = (Q @ K[:, :m].transpose(1, 2) / math.sqrt(d)).view(hk, r, m - i, m)
            x = torch.where(torch.arange(m, device=q.device) <= torch.arange(i, m, device=q.device)[:, None], x, -math.inf)
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = (p / p.sum(-1, keepdim=True)).view(hk, -1, m)
            gp = G @ V[:, :m].transpose(1, 2)
            gx = p * (gp - (p * gp).sum(-1, keepdim=True)) / math.sqrt(d)
            gV[:, :m] += p.transpose(1, 2) @ G
            gK[:, :m] += gx.transpose(1, 2) @ Q
            dq[at + i:at + m] = (gx @ K[:, :m]).view(hk, r, m - i, d).permute(2, 0, 1, 3).reshape(m - i, h, d).to(q.dtype)
        dk[at:at + n], dv[at:at + n] = gK.transpose(0, 1).to(k.dtype), gV.transpose(0, 1).to(v.dtype)
    return dq.view_as(s["q"]), dk.view_as(s["k"]), dv.view_as(s["v"])


# ---- the framework's operators --------------------------------------------------------------------------------
def _own(s):
    from linear_attention_sequence_mshortconv_b200 import attention, gdn

    if s["op"] == "gdn_step":
        return gdn.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["slots"]), s["state"]
    if s["op"] == "attn_forward":
        if s["packed"]:
            return attention.forward_varlen(s["q"], s["k"], s["v"], s["cu"])
        return attention.forward(s["q"], s["k"], s["v"])
    if s["op"] == "attn_backward":
        x = [s[n] for n in ("q", "k", "v", "o", "lse", "do")]
        return attention.backward_varlen(*x, s["cu"]) if s["packed"] else attention.backward(*x)
    x = [s[n] for n in ("q", "k", "v", "g", "beta")]
    if s["op"] == "gdn_forward":
        return gdn.forward_varlen(*x, s["cu"], s["S0"]) if s["packed"] else gdn.forward(*x, s["S0"])
    d = gdn.backward_varlen(*x, s["do"], s["cu"], want_dS0=False) if s["packed"] else gdn.backward(*x, s["do"], want_dS0=False)
    return d[:5]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "gdn_step":
        return _plain_step(state)
    if state["op"] == "attn_forward":
        return _plain_attention(state)
    if state["op"] == "attn_backward":
        return _plain_attention_backward(state)
    return _plain_gdn(state, state["op"] == "gdn_backward")


# ---- the definitions in 64 bits -------------------------------------------------------------------------------
def _side_by_side(x, lens):
    """[tokens, h, d] -> [longest, samples, h, d] in 64 bits, zeros behind a sample's end: a zero key, gate and
    strength leave the state as it is."""
    out = torch.zeros(max(lens), len(lens), *x.shape[1:], dtype=torch.float64, device=x.device)
    at = 0
    for i, n in enumerate(lens):
        out[:n, i] = x[at:at + n].double()
        at += n
    return out


def _end_to_end(x, lens):
    return torch.cat([x[:n, i] for i, n in enumerate(lens)])


def _exact_gdn(s, grads):
    lens, packed = s["lens"], s["packed"]
    r = s["v"].shape[-2] // s["q"].shape[-2]
    q, k = (_side_by_side(_flat(s[n], packed), lens).repeat_interleave(r, 2) for n in ("q", "k"))
    v = _side_by_side(_flat(s["v"], packed), lens)
    g, beta = (_side_by_side(_flat(s[n], packed)[..., None], lens)[..., 0] for n in ("g", "beta"))
    a = torch.exp(g)
    n, h, dk, dv = len(lens), v.shape[2], q.shape[3], v.shape[3]
    S = torch.zeros(n, h, dk, dv, dtype=torch.float64, device=q.device)
    if s.get("S0") is not None:
        S = s["S0"].double()
    o, kept = torch.empty_like(v), []
    for t in range(max(lens)):
        if grads:
            kept.append(S)
        S = a[t, :, :, None, None] * S
        e = beta[t, :, :, None] * (v[t] - torch.einsum("nhk,nhkv->nhv", k[t], S))
        S = S + k[t][..., None] * e[..., None, :]
        o[t] = torch.einsum("nhk,nhkv->nhv", q[t], S)
    if not grads:
        return _end_to_end(o, lens).view(s["v"].shape), S
    do = _side_by_side(_flat(s["do"], packed), lens)
    dq, dk_, dv_, dg, db = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g), torch.empty_like(g)
    D = torch.zeros_like(S)
    for t in reversed(range(max(lens))):
        before = kept.pop()
        A = a[t, :, :, None, None] * before
        w = v[t] - torch.einsum("nhk,nhkv->nhv", k[t], A)
        after = A + (beta[t, :, :, None] * k[t])[..., None] * w[..., None, :]
        D = D + q[t][..., None] * do[t][..., None, :]
        dq[t] = torch.einsum("nhkv,nhv->nhk", after, do[t])
        kD = torch.einsum("nhk,nhkv->nhv", k[t], D)
        db[t] = (kD * w).sum(-1)
        dw = beta[t, :, :, None] * kD
        dv_[t] = dw
        dk_[t] = beta[t, :, :, None] * torch.einsum("nhkv,nhv->nhk", D, w) - torch.einsum("nhkv,nhv->nhk", A, dw)
        D = D - k[t][..., None] * dw[..., None, :]
        dg[t] = (D * A).sum((-1, -2))
        D = a[t, :, :, None, None] * D
    hk = h // r
    dq, dk_ = (x.view(*x.shape[:2], hk, r, dk).sum(3) for x in (dq, dk_))
    return tuple(_end_to_end(x, lens).view(s[m].shape) for m, x in zip(("q", "k", "v", "g", "beta"), (dq, dk_, dv_, dg, db)))


def _exact_step(s):
    r = s["v"].shape[1] // s["q"].shape[1]
    state, o = s["state"].double(), torch.empty(s["v"].shape, dtype=torch.float64, device=DEVICE)
    at = s["slots"].long()
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    for h in range(v.shape[1]):
        S = torch.exp(s["g"][:, h].double())[:, None, None] * state[at, h]
        e = s["beta"][:, h].double()[:, None] * (v[:, h] - torch.einsum("nk,nkv->nv", k[:, h // r], S))
        S = S + torch.einsum("nk,nv->nkv", k[:, h // r], e)
        o[:, h] = torch.einsum("nk,nkv->nv", q[:, h // r], S)
        state[at, h] = S
    return o, state


def _exact_attention(s):
    q, k, v = (_flat(s[n], s["packed"]) for n in ("q", "k", "v"))
    r = q.shape[1] // k.shape[1]
    o = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:-1], dtype=torch.float64, device=q.device)
    for at, n in zip(s["cu"], s["lens"]):
        for h in range(q.shape[1]):
            for i in range(0, n, 4096):
                m = min(n, i + 4096)
                x = q[at + i:at + m, h].double() @ k[at:at + m, h // r].double().T * q.shape[2] ** -0.5
                x.masked_fill_(torch.ones(m - i, m, dtype=torch.bool, device=q.device).triu(i + 1), -math.inf)
                lse[at + i:at + m, h] = torch.logsumexp(x, -1)
                o[at + i:at + m, h] = torch.exp(x - lse[at + i:at + m, h, None]) @ v[at:at + m, h // r].double()
    return o.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def _exact_attention_backward(s):
    q, k, v, do = (_flat(s[n], s["packed"]) for n in ("q", "k", "v", "do"))
    r, c = q.shape[1] // k.shape[1], q.shape[2] ** -0.5
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=x.device) for x in (q, k, v))
    for at, n in zip(s["cu"], s["lens"]):
        for h in range(q.shape[1]):
            for i in range(0, n, 4096):
                m = min(n, i + 4096)
                Q, K, V, G = q[at + i:at + m, h].double(), k[at:at + m, h // r].double(), v[at:at + m, h // r].double(), do[at + i:at + m, h].double()
                p = torch.softmax((Q @ K.T * c).masked_fill_(torch.ones(m - i, m, dtype=torch.bool, device=q.device).triu(i + 1), -math.inf), -1)
                dv[at:at + m, h // r] += p.T @ G
                y = G @ V.T
                y = c * p * (y - (G * (p @ V)).sum(-1, keepdim=True))
                dq[at + i:at + m, h] = y @ K
                dk[at:at + m, h // r] += y.T @ Q
    return dq.view(s["q"].shape), dk.view(s["k"].shape), dv.view(s["v"].shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn_backward":
        return _exact_attention_backward(s)
    if case["op"] == "gdn_step":
        return _exact_step(s)
    if case["op"] == "attn_forward":
        return _exact_attention(s)
    return _exact_gdn(s, case["op"] == "gdn_backward")
