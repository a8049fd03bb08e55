"""The standalone operators from their definitions in 64 bits, for the GPU tests.
Gradients come from automatic differentiation of the definition."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def act(z, kind):
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2.0)))
    return z


def group_norm(x, gamma, beta, groups, eps, kind):
    """x [batch, rows, channels]; gamma / beta may be None. Returns y, mean, rstd."""
    n, r, c = x.shape
    g = x.reshape(n, r, groups, c // groups)
    mean = g.mean(dim=(1, 3), keepdim=True)
    var = ((g - mean) ** 2).mean(dim=(1, 3), keepdim=True)
    rstd = (var + eps) ** -0.5
    xh = ((g - mean) * rstd).reshape(n, r, c)
    z = xh if gamma is None else xh * gamma
    z = z if beta is None else z + beta
    return act(z, kind), mean.reshape(n, groups), rstd.reshape(n, groups)


def gated_ff(x, w1, b1, w2, b2, kind):
    pre = x @ w1.T
    pre = pre if b1 is None else pre + b1
    f = w2.shape[1]
    y = (pre[:, :f] * act(pre[:, f:], kind)) @ w2.T
    return (y if b2 is None else y + b2), pre


def visible(b, q_len, k_len, causal=False, k_lens=None, prefix=None, q_doc=None, k_doc=None):
    """[q_len, k_len] for sequence b: which keys each query sees; and the positions of the queries."""
    n = k_len if k_lens is None else min(max(int(k_lens[b]), 0), k_len)
    j = torch.arange(k_len)
    pos = torch.arange(q_len) + (n - q_len)
    see = (j < n)[None, :].expand(q_len, k_len).clone()
    if causal:
        ok = j[None, :] <= pos[:, None]
        if prefix is not None:
            ok = ok | (j[None, :] < int(prefix[b]))
        see &= ok
    if q_doc is not None:
        see &= q_doc[b].cpu()[:, None] == k_doc[b].cpu()[None, :]
    return see, pos


def attention(q, k, v, scale=0.0, softcap=0.0, slopes=None, **masks):
    """q [B, q_len, H, D], k and v [B, k_len, KV, D], 64 bits. Returns o, lse [B, H, q_len].
    Rows that see nothing: o = 0, lse = -inf, no gradient. Hidden values never enter."""
    B, nq, H, D = q.shape
    nk, KV = k.shape[1], k.shape[2]
    scale = scale or D ** -0.5
    outs, lses = [], []
    for b in range(B):
        see, pos = visible(b, nq, nk, **masks)
        see, pos = see.to(q.device), pos.to(q.device)
        used = see.any(dim=0)
        dist = (pos[:, None] - torch.arange(nk, device=q.device)[None, :]).abs().double()
        some = see.any(dim=1, keepdim=True)
        for h in range(H):
            kk = torch.where(used[:, None], k[b, :, h // (H // KV)], 0.0)
            vv = torch.where(used[:, None], v[b, :, h // (H // KV)], 0.0)
            s = (q[b, :, h] @ kk.T) * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - slopes[h].double() * dist
            s = torch.where(see, s, -math.inf)
            m = torch.where(some, s.amax(dim=1, keepdim=True) if nk else torch.zeros(nq, 1).to(s), 0.0).detach()
            e = torch.where(see, torch.exp(torch.where(see, s, 0.0) - m), 0.0)
            t = e.sum(dim=1, keepdim=True)
            outs.append((e / torch.where(some, t, 1.0)) @ vv)
            lses.append(torch.where(some, torch.log(torch.where(some, t, 1.0)) + m, -math.inf).squeeze(1))
    o = torch.stack(outs).reshape(B, H, nq, D).permute(0, 2, 1, 3)
    return o, torch.stack(lses).reshape(B, H, nq)


def rel(got, want):
    """2-norm of the difference over the 2-norm of the result."""
    got, want = got.detach().double(), want.detach().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    assert torch.isfinite(got).all()
    d, n = (got - want).norm().item(), want.norm().item()
    return d / n if n else d
