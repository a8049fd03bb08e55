"""The operators of a trainable transformer and residual block, on real sizes:
group norm with an activation (channels last), the gated feed-forward block, and
attention with capped scores, a distance bias, document, prefix and padding masks.

``run`` computes them in plain torch operations in 32 bits (``own = False``) or
through the library's entry points (``own = True``); ``exact`` is the definition
in 64 bits, with gradients by automatic differentiation.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # GroupNorm + SiLU in front of a convolution at the deepest level of the 96x96 U-Net step: latency
        gn("gn_fwd_12x12x1280", "fwd", "bf16", 1, 144, 1280, 32, "silu"),
        # the last level of the VAE decoder for a 768x768 image: the largest tensor the framework normalises
        gn("gn_fwd_768x768x128", "fwd", "bf16", 1, 589824, 128, 32, "silu"),
        # a training step's GroupNorm + SiLU at the U-Net's first level, four images
        gn("gn_train_b4_96x96x320", "train", "f16", 4, 9216, 320, 32, "silu"),
        # odd sizes in full precision: 3 channels a group, rows in no multiple of anything
        gn("gn_train_b3_1001x96", "train", "f32", 3, 1001, 96, 32, "none"),
        # one token through the widest feed-forward: the weights' bytes
        ff("ff_token_1280", "fwd", "bf16", 1, 1280, 5120, "gelu"),
        # the feed-forward of the 96x96 step's first level
        ff("ff_fwd_9216x320", "fwd", "bf16", 9216, 320, 1280, "gelu"),
        # fifteen prompts of 77 tokens, a training step with SiLU gates
        ff("ff_train_1155x640", "train", "f16", 1155, 640, 2560, "silu"),
        # sixteen images of 32x32 tokens at the widest level, a training step
        ff("ff_train_16384x1280", "train", "bf16", 16384, 1280, 5120, "gelu"),
        # one new token of each of eight sequences over caches of unequal lengths, shared heads, distance bias
        attn("attn_token_b8_4096", "fwd", "f16", 8, 1, 4096, 16, 4, 128, lens=True, causal=True, slopes=True),
        # three images packed into one sequence of 9216 tokens, each attending to itself
        attn("attn_fwd_docs_9216", "fwd", "bf16", 1, 9216, 9216, 5, 5, 64, docs=3),
        # image tokens on padded prompts of up to 77 tokens, a training step
        attn("attn_train_cross_4096x77", "train", "bf16", 4, 4096, 77, 10, 10, 64, lens=True),
        # prompt tokens as a prefix that all see, then one after another; capped scores, shared heads
        attn("attn_train_prefix_2047", "train", "bf16", 2, 2047, 2047, 8, 2, 80, causal=True, prefix=True, slopes=True,
             cap=30.0),
    ]


def gn(name, what, dtype, batch, rows, channels, groups, act):
    return {"name": name, "op": "gn", "pass": what, "dtype": dtype, "batch": batch, "rows": rows, "channels": channels,
            "groups": groups, "act": act}


def ff(name, what, dtype, tokens, d_model, d_hidden, act):
    return {"name": name, "op": "ff", "pass": what, "dtype": dtype, "tokens": tokens, "d_model": d_model,
            "d_hidden": d_hidden, "act": act}


def attn(name, what, dtype, batch, q_len, k_len, heads, kv_heads, head_dim, lens=False, causal=False, prefix=False,
         docs=0, slopes=False, cap=0.0):
    return {"name": name, "op": "attn", "pass": what, "dtype": dtype, "batch": batch, "q_len": q_len, "k_len": k_len,
            "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "lens": lens, "causal": causal,
            "prefix": prefix, "docs": docs, "slopes": slopes, "cap": cap}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["gn", "ff", "attn"])
    if op == "gn":
        groups = rng.choice([8, 16, 32, 32])
        channels = groups * rng.choice([1, 2, 3, 4, 5, 8, 10, 12, 16, 20, 30, 40])
        total = _log(rng, 2000, 70e6)
        batch = min(rng.randint(1, 9), max(1, total // channels))
        rows = max(1, total // (channels * batch))
        c = gn("", rng.choice(["fwd", "train"]), rng.choice(["bf16", "f16", "f32"]), batch, rows, channels, groups,
               rng.choice(["none", "silu", "silu", "gelu"]))
    elif op == "ff":
        d = 8 * _log(rng, 8, 160)
        c = ff("", rng.choice(["fwd", "train"]), rng.choice(["bf16", "f16"]), _log(rng, 1, 16384), d,
               8 * _log(rng, 8, 4 * d // 8), rng.choice(["gelu", "silu", "silu"]))
    else:
        what = rng.choice(["fwd", "train"])
        causal = rng.random() < 0.5
        heads, kv = rng.choice([(1, 1), (3, 3), (5, 5), (8, 2), (8, 8), (10, 10), (6, 2), (16, 4), (12, 1)])
        q_len = 1 if what == "fwd" and rng.random() < 0.3 else _log(rng, 2, 6000)
        k_len = rng.choice([q_len, 77, _log(rng, 1, 16384)])
        batch = max(1, min(rng.randint(1, 8), int(2.5e8 / (heads * q_len * k_len))))
        if heads * q_len * k_len > 2.5e8:
            q_len = max(1, int(2.5e8 / (heads * k_len)))
        c = attn("", what, rng.choice(["bf16", "f16"]), batch, q_len, k_len, heads, kv,
                 rng.choice([40, 64, 64, 80, 128]), lens=rng.random() < 0.5, causal=causal,
                 prefix=causal and rng.random() < 0.5, docs=rng.choice([0, 0, 2, 5]), slopes=rng.random() < 0.4,
                 cap=rng.choice([0.0, 0.0, 20.0, 50.0]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _norm(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def prepare(case, seed):
    g, t = _gen(seed), DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if case["op"] == "gn":
        n, r, c = case["batch"], case["rows"], case["channels"]
        # activations with a mean of their own in every channel, as convolutions leave them
        s["x"] = (torch.randn(n, r, c, generator=g, device="cuda") * 1.5
                  + torch.randn(c, generator=g, device="cuda")).to(t)
        s["gamma"], s["beta"] = _norm(g, (c,), t, 0.1, 1.0), _norm(g, (c,), t, 0.1)
        if case["pass"] == "train":
            s["dy"] = _norm(g, (n, r, c), t)
    elif case["op"] == "ff":
        m, d, f = case["tokens"], case["d_model"], case["d_hidden"]
        s["x"] = _norm(g, (m, d), t)
        s["w1"], s["b1"] = _norm(g, (2 * f, d), t, d ** -0.5), _norm(g, (2 * f,), t, 0.1)
        s["w2"], s["b2"] = _norm(g, (d, f), t, f ** -0.5), _norm(g, (d,), t, 0.1)
        if case["pass"] == "train":
            s["dy"] = _norm(g, (m, d), t)
    else:
        b, nq, nk, h, kv, d = (case[k] for k in ("batch", "q_len", "k_len", "heads", "kv_heads", "head_dim"))
        # [batch, tokens, heads, head_dim], as the projections leave them
        s["q"], s["k"], s["v"] = (_norm(g, (b, n, m, d), t) for n, m in ((nq, h), (nk, kv), (nk, kv)))
        if case["pass"] == "train":
            s["do"] = _norm(g, (b, nq, h, d), t)
        i32 = dict(dtype=torch.int32, device="cuda")
        s["lens"] = torch.randint(max(1, nk // 2), nk + 1, (b,), generator=g, **i32) if case["lens"] else None
        s["prefix"] = torch.randint(0, nk // 2 + 1, (b,), generator=g, **i32) if case["prefix"] else None
        s["q_doc"] = s["k_doc"] = None
        if case["docs"]:
            # sequences packed one behind the other: ids rise along the tokens, cut at random places
            cut = torch.rand(b, case["docs"] - 1, generator=g, device="cuda").sort(dim=1).values
            at = lambda n: (torch.arange(n, device="cuda") + 0.5) / n  # noqa: E731
            s["q_doc"], s["k_doc"] = ((at(n)[None, :, None] > cut[:, None, :]).sum(dim=2).to(torch.int32)
                                      for n in (nq, nk))
        s["slopes"] = (torch.arange(1, h + 1, device="cuda").float() * (-4.0 / h)).exp2() * 0.1 if case["slopes"] else None
    return s


# ---------------------------------------------------------------- the plain form, in 32 bits


def _act(z, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return z * sg, sg * (1 + z * (1 - sg))
    if kind == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return z, torch.ones_like(z)


def _plain_gn(s, c):
    n, r, ch, g, t = c["batch"], c["rows"], c["channels"], c["groups"], s["x"].dtype
    x = s["x"].float().view(n, r, g, ch // g)
    mean = x.mean(dim=(1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(dim=(1, 3), keepdim=True) + 1e-5)
    xh = (x - mean) * rstd
    gamma, beta = s["gamma"].float().view(g, ch // g), s["beta"].float().view(g, ch // g)
    y, slope = _act(xh * gamma + beta, c["act"])
    if c["pass"] == "fwd":
        return {"y": y.view(n, r, ch).to(t)}
    dz = s["dy"].float().view(n, r, g, ch // g) * slope
    dxh = dz * gamma
    dx = rstd * (dxh - dxh.mean(dim=(1, 3), keepdim=True) - xh * (dxh * xh).mean(dim=(1, 3), keepdim=True))
    return {"y": y.view(n, r, ch).to(t), "dx": dx.view(n, r, ch).to(t),
            "dgamma": (dz * xh).sum(dim=(0, 1)).view(ch), "dbeta": dz.sum(dim=(0, 1)).view(ch)}


def _plain_ff(s, c):
    f, t = c["d_hidden"], s["x"].dtype
    x, w1, w2 = s["x"].float(), s["w1"].float(), s["w2"].float()
    pre = x @ w1.T + s["b1"].float()
    v, z = pre[:, :f], pre[:, f:]
    a, slope = _act(z, c["act"])
    hid = v * a
    y = hid @ w2.T + s["b2"].float()
    if c["pass"] == "fwd":
        return {"y": y.to(t)}
    dy = s["dy"].float()
    dh = dy @ w2
    dpre = torch.cat([dh * a, dh * v * slope], dim=1)
    return {"y": y.to(t), "dx": (dpre @ w1).to(t), "dw1": (dpre.T @ x).to(t), "db1": dpre.sum(dim=0).to(t),
            "dw2": (dy.T @ hid).to(t), "db2": dy.sum(dim=0).to(t)}


def _visible(s, c):
    """[batch, 1, 1, q_len, k_len]: which keys a query sees, and the distance between them."""
    nq, nk = c["q_len"], c["k_len"]
    n = s["lens"].long() if s["lens"] is not None else torch.full((c["batch"],), nk, device="cuda")
    pos = torch.arange(nq, device="cuda")[None, :] + (n - nq)[:, None]  # the queries are the last of the sequence
    j = torch.arange(nk, device="cuda")
    see = (j[None, :] < n[:, None])[:, None, :].expand(-1, nq, -1)
    if c["causal"]:
        ok = j[None, None, :] <= pos[:, :, None]
        if s["prefix"] is not None:
            ok = ok | (j[None, :] < s["prefix"][:, None])[:, None, :]
        see = see & ok
    if s["q_doc"] is not None:
        see = see & (s["q_doc"][:, :, None] == s["k_doc"][:, None, :])
    return see[:, None, None], (pos[:, :, None] - j[None, None, :]).abs().float()[:, None, None]


def _plain_attn(s, c):
    b, nq, h, kv, d, t = c["batch"], c["q_len"], c["heads"], c["kv_heads"], c["head_dim"], s["q"].dtype
    scale, cap, grp = d ** -0.5, c["cap"], h // kv
    q = s["q"].float().view(b, nq, kv, grp, d).permute(0, 2, 3, 1, 4)
    k, v = (s[n].float().permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))
    see, dist = _visible(s, c)
    w = (q @ k.transpose(-1, -2)) * scale
    th = torch.tanh(w / cap) if cap else None
    w = th * cap if cap else w
    if s["slopes"] is not None:
        w = w - s["slopes"].view(1, kv, grp, 1, 1) * dist
    w = w.masked_fill(~see, -math.inf)
    top = w.amax(dim=-1, keepdim=True)
    p = torch.exp(w - top.masked_fill(top == -math.inf, 0.0))
    del w, dist
    p = p / p.sum(dim=-1, keepdim=True).clamp_min(1e-30)  # a row that sees nothing gives zeros
    o = p @ v
    back = lambda a: a.permute(0, 3, 1, 2, 4).reshape(b, nq, h, d).to(t)  # noqa: E731
    if c["pass"] == "fwd":
        return {"o": back(o)}
    do = s["do"].float().view(b, nq, kv, grp, d).permute(0, 2, 3, 1, 4)
    ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(dim=-1, keepdim=True))
    ds = ds * (1 - th * th) if cap else ds
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q).sum(dim=2) * scale
    dv = (p.transpose(-1, -2) @ do).sum(dim=2)
    return {"o": back(o), "dq": back(dq), "dk": dk.permute(0, 2, 1, 3).contiguous().to(t),
            "dv": dv.permute(0, 2, 1, 3).contiguous().to(t)}


# ---------------------------------------------------------------- the library's entry points


def _lib_plan(s, c):
    """The configuration and the workspace that a program keeps."""
    if "cfg" not in s:
        from latent_diffusion_net_b200 import binding as B
        act = {"none": B.SD_ACT_NONE, "silu": B.SD_ACT_SILU, "gelu": B.SD_ACT_GELU}
        dt = {"bf16": B.SD_DTYPE_BF16, "f16": B.SD_DTYPE_F16, "f32": B.SD_DTYPE_F32}[c["dtype"]]
        if c["op"] == "gn":
            cfg = B.group_norm_cfg(c["batch"], c["rows"], c["channels"], groups=c["groups"], act=act[c["act"]], dtype=dt)
            n = B.sd_group_norm_workspace_size(cfg)
        elif c["op"] == "ff":
            cfg = B.gated_ff_cfg(c["tokens"], c["d_model"], c["d_hidden"], act=act[c["act"]], dtype=dt)
            n = B.sd_gated_ff_workspace_size(cfg)
        else:
            cfg = B.attention_cfg(c["batch"], c["q_len"], c["k_len"], c["heads"], c["kv_heads"], c["head_dim"], dtype=dt,
                                  softcap=c["cap"], causal=c["causal"])
            s["masks"] = B.attention_masks(k_lens=s["lens"], prefix=s["prefix"], q_doc=s["q_doc"], k_doc=s["k_doc"],
                                           slopes=s["slopes"])
            n = B.sd_attention_workspace_size(cfg)
        s["B"], s["ws"], s["cfg"] = B, torch.empty(n, dtype=torch.uint8, device="cuda"), cfg
    return s["B"], s["cfg"], s["ws"], torch.cuda.current_stream()


def _own_gn(s, c):
    B, cfg, ws, st = _lib_plan(s, c)
    x, train = s["x"], c["pass"] == "train"
    y = torch.empty_like(x)
    stats = torch.empty(c["batch"], c["groups"], 2, device="cuda") if train else None
    B.sd_group_norm_fwd(cfg, x, s["gamma"], s["beta"], y, stats, ws, ws.numel(), st)
    if not train:
        return {"y": y}
    dx, dgamma = torch.empty_like(x), torch.empty(c["channels"], device="cuda")
    dbeta = torch.empty_like(dgamma)
    B.sd_group_norm_bwd(cfg, x, s["gamma"], s["beta"], stats, s["dy"], dx, dgamma, dbeta, ws, ws.numel(), st)
    return {"y": y, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _own_ff(s, c):
    B, cfg, ws, st = _lib_plan(s, c)
    x, train = s["x"], c["pass"] == "train"
    y = torch.empty_like(x)
    pre = torch.empty(c["tokens"], 2 * c["d_hidden"], dtype=x.dtype, device="cuda") if train else None
    B.sd_gated_ff_fwd(cfg, s["w1"], s["b1"], s["w2"], s["b2"], x, pre, y, ws, ws.numel(), st)
    if not train:
        return {"y": y}
    dx, dw1, db1, dw2, db2 = (torch.empty_like(s[n]) for n in ("x", "w1", "b1", "w2", "b2"))
    B.sd_gated_ff_bwd(cfg, s["w1"], s["w2"], x, pre, s["dy"], dx, dw1, db1, dw2, db2, ws, ws.numel(), st)
    return {"y": y, "dx": dx, "dw1": dw1, "db1": db1, "dw2": dw2, "db2": db2}


def _own_attn(s, c):
    B, cfg, ws, st = _lib_plan(s, c)
    q, k, v, train = s["q"], s["k"], s["v"], c["pass"] == "train"
    o = torch.empty_like(q)
    lse = torch.empty(c["batch"], c["heads"], c["q_len"], device="cuda") if train else None
    B.sd_attention_fwd(cfg, q, k, v, s["masks"], o, lse, ws, ws.numel(), st)
    if not train:
        return {"o": o}
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    B.sd_attention_bwd(cfg, q, k, v, s["masks"], o, lse, s["do"], dq, dk, dv, ws, ws.numel(), st)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    c = state["case"]
    if own:
        return {"gn": _own_gn, "ff": _own_ff, "attn": _own_attn}[c["op"]](state, c)
    return {"gn": _plain_gn, "ff": _plain_ff, "attn": _plain_attn}[c["op"]](state, c)


# ---------------------------------------------------------------- floors


def work(case):
    e, train = (4 if case["dtype"] == "f32" else 2), case["pass"] == "train"
    if case["op"] == "gn":
        n = case["batch"] * case["rows"] * case["channels"]
        # forward: x in, y out; backward: dy in, dx out as well (x was read)
        return {"bytes": n * e * (4 if train else 2) + 4 * case["channels"] * e, "flops": n * (30 if train else 12)}
    if case["op"] == "ff":
        m, d, f = case["tokens"], case["d_model"], case["d_hidden"]
        weights, acts = 3 * d * f + 2 * f + d, 2 * m * d
        return {"bytes": e * ((2 if train else 1) * weights + (2 if train else 1) * acts),
                "flops": (18 if train else 6) * m * d * f}
    b, nq, nk, h, kv, d = (case[k] for k in ("batch", "q_len", "k_len", "heads", "kv_heads", "head_dim"))
    n = 0.75 * nk if case["lens"] else nk  # the lengths are drawn evenly from the upper half
    pairs = nq * n
    if case["causal"]:
        m = min(nq, n)
        pairs = m * (n - m / 2) + (min(nq, n) * n / 32 if case["prefix"] else 0)
    if case["docs"]:
        pairs *= 2 / (case["docs"] + 1)  # the expected sum of squares of random cuts
    return {"bytes": e * b * d * ((2 * nq * h + 2 * n * kv) * (2 if train else 1)),
            "flops": (14 if train else 4) * b * h * d * pairs}


# ---------------------------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        return {"gn": _exact_gn, "ff": _exact_ff, "attn": _exact_attn}[case["op"]](s, case)


_EXACT_ACT = {"none": lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}


def _leaf(t):
    return t.double().requires_grad_()


def _exact_gn(s, c):
    x, gamma, beta = (_leaf(s[k]) for k in ("x", "gamma", "beta"))
    y = _EXACT_ACT[c["act"]](torch.nn.functional.group_norm(x.transpose(1, 2), c["groups"], gamma, beta, 1e-5)
                             .transpose(1, 2))
    if c["pass"] == "fwd":
        return {"y": y.detach()}
    y.backward(s["dy"].double())
    return {"y": y.detach(), "dx": x.grad, "dgamma": gamma.grad, "dbeta": beta.grad}


def _exact_ff(s, c):
    x, w1, b1, w2, b2 = (_leaf(s[k]) for k in ("x", "w1", "b1", "w2", "b2"))
    value, gate = torch.nn.functional.linear(x, w1, b1).chunk(2, dim=1)
    y = torch.nn.functional.linear(value * _EXACT_ACT[c["act"]](gate), w2, b2)
    if c["pass"] == "fwd":
        return {"y": y.detach()}
    y.backward(s["dy"].double())
    return {"y": y.detach(), "dx": x.grad, "dw1": w1.grad, "db1": b1.grad, "dw2": w2.grad, "db2": b2.grad}


def _exact_attn(s, c):
    q, k, v = (_leaf(s[n]) for n in ("q", "k", "v"))
    nq, nk, grp = c["q_len"], c["k_len"], c["heads"] // c["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    row, col = torch.arange(nq, device="cuda")[:, None], torch.arange(nk, device="cuda")[None, :]
    for b in range(c["batch"]):
        n = int(s["lens"][b]) if c["lens"] else nk
        pos = row + n - nq
        hidden = (col >= n).expand(nq, nk)
        if c["causal"]:
            hidden = hidden | ((col > pos) & (col >= (int(s["prefix"][b]) if c["prefix"] else 0)))
        if c["docs"]:
            hidden = hidden | (s["q_doc"][b][:, None] != s["k_doc"][b][None, :])
        empty = hidden.all(dim=1, keepdim=True)
        for h in range(c["heads"]):
            kk, vv = k[b, :, h // grp], v[b, :, h // grp]
            sc = torch.matmul(q[b, :, h], kk.T) / math.sqrt(c["head_dim"])
            if c["cap"]:
                sc = c["cap"] * torch.tanh(sc / c["cap"])
            if c["slopes"]:
                sc = sc - s["slopes"][h].double() * (pos - col).abs().double()
            p = torch.softmax(sc.masked_fill(hidden & ~empty, -math.inf), dim=1)
            o = torch.matmul(p.masked_fill(empty, 0.0), vv)
            if c["pass"] == "train":
                o.backward(s["do"][b, :, h].double())
            out[b, :, h] = o.detach()
    if c["pass"] == "fwd":
        return {"o": out}
    return {"o": out, "dq": q.grad, "dk": k.grad, "dv": v.grad}
