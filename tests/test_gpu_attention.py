"""Attention with capped scores, a distance bias and document, prefix, causal and
length masks, and its gradients, on a B200 against the definition in 64 bits.

Tolerances count roundings to the type, each at most half a step u of a value and
independent of each other, as relative 2-norms: o and dv have P's and their own
(2 u); dq and dk have the saved o's (in delta), dS's and their own, and P's way
through delta (4 u). FP32 scores, exponentials and sums add less than 1e-5 (a cap of
50 leaves 50 * 2^-22 in a score)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import operator_refs as R  # noqa: E402
from latent_diffusion_net_b200 import binding as B  # noqa: E402

DT = {"bf16": (torch.bfloat16, B.SD_DTYPE_BF16), "f16": (torch.float16, B.SD_DTYPE_F16)}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def inputs(batch, nq, nk, h, kv, d, dt, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DT[dt][0]
    n = lambda tok, m: (torch.randn(batch, tok, m, d, generator=g, device="cuda") * std).to(t)  # noqa: E731
    return n(nq, h), n(nk, kv), n(nk, kv), n(nq, h)


def call(q, k, v, do=None, scale=0.0, softcap=0.0, causal=False, slopes=None, strides=None, cfg_h=None, stream=None,
         ws=None, **masks):
    """o, lse and (with do) dq, dk, dv through the entry points."""
    batch, nq, h, d = q.shape
    nk, kv = k.shape[1], k.shape[2]
    code = {torch.bfloat16: B.SD_DTYPE_BF16, torch.float16: B.SD_DTYPE_F16}[q.dtype]
    st = {}
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_contiguous():
            st[name + "_stride"] = t.stride()[:3]
    cfg = B.attention_cfg(batch, nq, nk, h, kv, d, dtype=code, causal=causal, scale=scale, softcap=softcap, **st)
    n = B.sd_attention_workspace_size(cfg)
    if ws is None:
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    assert ws.numel() >= n > 0
    m = B.attention_masks(slopes=slopes, **masks)
    o = torch.full((batch, nq, h, d), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full((batch, h, nq), float("nan"), device="cuda")
    B.sd_attention_fwd(cfg, q, k, v, m, o, lse, ws, ws.numel(), stream)
    out = {"o": o, "lse": lse}
    if do is not None:
        # gradients have the strides of q, k and v
        for name, t in (("dq", q), ("dk", k), ("dv", v)):
            out[name] = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").fill_(float("nan"))
        B.sd_attention_bwd(cfg, q, k, v, m, o, lse, do, out["dq"], out["dk"], out["dv"], ws, ws.numel(), stream)
    if stream is None:
        assert B.sd_query_device_status(ws) == 0
    return out


def reference(q, k, v, do=None, **kw):
    leaf = [t.double().detach().requires_grad_() for t in (q, k, v)]
    o, lse = R.attention(*leaf, **kw)
    out = {"o": o.detach(), "lse": lse.detach()}
    if do is not None:
        o.backward(do.double())
        zero = lambda t: torch.zeros_like(t) if t.grad is None else t.grad  # noqa: E731
        out.update(dq=zero(leaf[0]), dk=zero(leaf[1]), dv=zero(leaf[2]))
    return out


def compare(got, want, t):
    u = R.HALF_STEP[t]
    for name in want:
        if name == "lse":
            some = want["lse"] > -math.inf
            assert (got["lse"][~some] == -math.inf).all()
            assert (got["lse"][some].double() - want["lse"][some]).abs().max().item() < 1e-4 if some.any() else True
        else:
            tol = (2 if name in ("o", "dv") else 4) * u + 1e-5
            err = R.rel(got[name], want[name])
            assert err < tol, (name, err, tol)
    empty = want["lse"] == -math.inf  # [B, H, q]
    assert not got["o"].permute(0, 2, 1, 3)[empty].any()
    if "dq" in got:
        assert not got["dq"].permute(0, 2, 1, 3)[empty].any()


def check(batch, nq, nk, h, kv, d, dt="bf16", seed=1, backward=True, std=1.0, **kw):
    q, k, v, do = inputs(batch, nq, nk, h, kv, d, dt, seed, std)
    do = do if backward else None
    compare(call(q, k, v, do, **kw), reference(q, k, v, do, **kw), q.dtype)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", [8, 16, 40, 64, 72, 80, 104, 128])
def test_head_dims_and_types(dt, d):
    check(2, 150, 200, 3, 3, d, dt, seed=d)


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 77), (2, 128), (127, 129), (128, 128), (129, 127), (300, 1), (5, 1000),
                                   (640, 640)])
def test_lengths(nq, nk):
    check(1, nq, nk, 2, 2, 64, seed=nq)
    check(2, nq, nk, 2, 1, 128, "f16", seed=nk)


@pytest.mark.parametrize("h,kv", [(8, 2), (6, 2), (5, 1), (12, 4), (32, 1), (48, 1), (128, 1)])
@pytest.mark.parametrize("nq", [1, 37, 200])
def test_shared_heads(h, kv, nq):
    check(2, nq, 200, h, kv, 64, seed=h + nq, causal=True)


@pytest.mark.parametrize("nq,nk", [(200, 200), (1, 300), (64, 500), (500, 64), (257, 1025)])
@pytest.mark.parametrize("d", [64, 128])
def test_causal(nq, nk, d):
    """With more queries than keys the first queries see nothing."""
    check(2, nq, nk, 2, 2, d, seed=nq, causal=True)


@pytest.mark.parametrize("d", [40, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_key_lengths(d, causal):
    lens = i32([0, 1, 127, 128, 129, 300, 1000, -5])  # clamped to 0 .. 300
    check(8, 140, 300, 2, 1, d, seed=d, causal=causal, k_lens=lens)
    check(8, 1, 300, 2, 1, d, seed=d, causal=causal, k_lens=lens)


@pytest.mark.parametrize("d", [64, 80])
def test_prefix(d):
    check(4, 300, 300, 4, 2, d, seed=3, causal=True, prefix=i32([0, 50, 128, 300]))
    check(4, 100, 300, 4, 2, d, seed=4, causal=True, prefix=i32([-3, 299, 260, 1000]), k_lens=i32([300, 300, 250, 90]))


def packed(lens, total):
    ids = []
    for n, m in enumerate(lens):
        ids += [n] * m
    return ids + [10 ** 6] * (total - len(ids))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_documents(d, causal):
    doc = i32([packed([128, 128, 200], 500), packed([1, 3, 250, 100], 500)])
    check(2, 500, 500, 4, 2, d, seed=5, causal=causal, q_doc=doc, k_doc=doc)
    # other ids for the keys, in no order: some queries see nothing
    g = torch.Generator(device="cuda").manual_seed(1)
    qd = torch.randint(-2, 6, (2, 300), generator=g, device="cuda", dtype=torch.int32)
    kd = torch.randint(0, 9, (2, 200), generator=g, device="cuda", dtype=torch.int32)
    check(2, 300, 200, 4, 2, d, seed=6, causal=causal, q_doc=qd, k_doc=kd, k_lens=i32([200, 150]))


def test_documents_that_share_no_tile():
    qd, kd = i32([[0] * 128 + [5] * 128]), i32([[5] * 128 + [7] * 128])
    check(1, 256, 256, 2, 2, 64, seed=2, q_doc=qd, k_doc=kd)
    check(1, 256, 256, 2, 2, 64, seed=2, q_doc=qd, k_doc=kd + 100)  # no query sees any key


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("cap", [0.0, 5.0, 50.0])
def test_cap_and_bias(d, dt, cap):
    slopes = torch.tensor([0.5, 0.01, 0.0, 2.0], device="cuda")
    check(2, 260, 330, 4, 2, d, dt, seed=7, softcap=cap, slopes=slopes, std=2.0)
    check(2, 260, 330, 4, 2, d, dt, seed=8, softcap=cap, causal=True, slopes=slopes, prefix=i32([10, 200]),
          k_lens=i32([330, 280]))
    check(2, 1, 330, 4, 2, d, dt, seed=9, softcap=cap, causal=True, slopes=slopes)


def test_all_masks_at_once():
    doc = i32([packed([150, 200, 100], 512), packed([512], 512)])
    check(2, 512, 512, 6, 2, 72, "f16", seed=11, causal=True, softcap=20.0, prefix=i32([20, 300]),
          k_lens=i32([460, 512]), q_doc=doc, k_doc=doc, slopes=torch.linspace(0.0, 0.3, 6, device="cuda"))


def test_given_scale():
    check(1, 100, 200, 2, 2, 64, scale=0.5, seed=12)


@pytest.mark.parametrize("nq,nk,h,kv,d", [(1, 4096, 16, 4, 128), (1, 16000, 2, 2, 64), (3, 5000, 8, 1, 64),
                                          (130, 8192, 1, 1, 128)])
def test_few_rows_over_many_keys(nq, nk, h, kv, d):
    check(2, nq, nk, h, kv, d, seed=nk, causal=True, k_lens=i32([nk, nk // 3]))


@pytest.mark.parametrize("nq,nk,h,d", [(4096, 77, 2, 64), (9216, 77, 1, 64), (2300, 2300, 2, 64), (1500, 1500, 2, 128)])
def test_long(nq, nk, h, d):
    check(1, nq, nk, h, h, d, seed=nq)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_growing_scores_rescale(dt):
    """Scores that rise along the keys by far more than 2^8: the running maximum moves in many tiles."""
    q, k, v, do = inputs(1, 256, 1024, 2, 2, 64, dt, 13)
    k = (k.float() * torch.linspace(0.1, 6.0, 1024, device="cuda")[None, :, None, None]).to(k.dtype)
    compare(call(q, k, v, do), reference(q, k, v, do), q.dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_behind_the_last_key_are_never_used(d, bad):
    lens = [200, 130, 0]
    q, k, v, do = inputs(3, 150, 300, 4, 2, d, "bf16", 14)
    clean = call(q, k, v, do, k_lens=i32(lens), causal=True)
    for b, n in enumerate(lens):
        k[b, n:] = bad
        v[b, n:] = bad
    dirty = call(q, k, v, do, k_lens=i32(lens), causal=True)
    for name in clean:
        assert torch.equal(clean[name], dirty[name]), name
    for b, n in enumerate(lens):
        assert not dirty["dk"][b, n:].any() and not dirty["dv"][b, n:].any()


def test_strided_projection():
    """q, k and v as columns of one projection output, with padding between tokens; what lies between stays."""
    h, kv, d, n = 6, 2, 40, 200
    wide = h * d + 2 * kv * d + 24
    g = torch.Generator(device="cuda").manual_seed(15)
    buf = torch.randn(2, n, wide, generator=g, device="cuda").to(torch.bfloat16)
    q = buf[:, :, :h * d].view(2, n, h, d)
    k = buf[:, :, h * d:(h + kv) * d].view(2, n, kv, d)
    v = buf[:, :, (h + kv) * d:(h + 2 * kv) * d].view(2, n, kv, d)
    do = torch.randn(2, n, h, d, generator=g, device="cuda").to(torch.bfloat16)
    want = reference(q, k, v, do, causal=True)
    cfg = B.attention_cfg(2, n, n, h, kv, d, causal=True, q_stride=q.stride()[:3], k_stride=k.stride()[:3],
                          v_stride=v.stride()[:3])
    ws = torch.empty(B.sd_attention_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty(2, n, h, d, dtype=q.dtype, device="cuda"), torch.empty(2, h, n, device="cuda")
    gbuf = torch.full_like(buf, 3.0)
    dq, dk, dv = (gbuf[:, :, a:b].view(2, n, -1, d) for a, b in ((0, h * d), (h * d, (h + kv) * d),
                                                               ((h + kv) * d, (h + 2 * kv) * d)))
    B.sd_attention_fwd(cfg, q, k, v, None, o, lse, ws, ws.numel())
    B.sd_attention_bwd(cfg, q, k, v, None, o, lse, do, dq, dk, dv, ws, ws.numel())
    compare({"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, want, q.dtype)
    assert (gbuf[:, :, (h + 2 * kv) * d:] == 3).all()


def test_head_major_tensors():
    """[batch][head][token][head_dim] storage, seen through strides."""
    q, k, v, do = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in inputs(2, 150, 170, 4, 2, 64, "f16", 16))
    do = do.contiguous()
    compare(call(q, k, v, do, causal=True), reference(q, k, v, do, causal=True), q.dtype)


def test_no_keys_or_no_queries():
    q, k, v, do = inputs(2, 50, 60, 2, 2, 64, "bf16", 17)
    cfg = B.attention_cfg(2, 50, 0, 2, 2, 64)
    ws = torch.empty(B.sd_attention_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    o, lse, dq = torch.ones_like(q), torch.ones(2, 2, 50, device="cuda"), torch.ones_like(q)
    B.sd_attention_fwd(cfg, q, None, None, None, o, lse, ws, ws.numel())
    B.sd_attention_bwd(cfg, q, None, None, None, o, lse, do, dq, None, None, ws, ws.numel())
    assert B.sd_query_device_status(ws) == 0
    assert not o.any() and (lse == -math.inf).all() and not dq.any()
    cfg = B.attention_cfg(2, 0, 60, 2, 2, 64)
    ws = torch.full((B.sd_attention_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    dk, dv = torch.ones_like(k), torch.ones_like(v)
    B.sd_attention_fwd(cfg, None, k, v, None, None, None, ws, ws.numel())
    B.sd_attention_bwd(cfg, None, k, v, None, None, None, None, None, dk, dv, ws, ws.numel())
    assert B.sd_query_device_status(ws) == 0
    assert not dk.any() and not dv.any()


def test_gradient_against_differences():
    """Central differences of the 64-bit forward are good to 1e-7 here; the FP16 gradients are off by 4 u."""
    q, k, v, do = inputs(1, 5, 9, 2, 1, 16, "f16", 18)
    kw = dict(causal=True, softcap=4.0, slopes=torch.tensor([0.2, 0.7], device="cuda"))
    got = call(q, k, v, do, **kw)
    x = [t.double() for t in (q, k, v)]
    for n, name in enumerate(("dq", "dk", "dv")):
        flat, g = x[n].reshape(-1), got[name].reshape(-1)
        for i in (0, flat.numel() // 2, flat.numel() - 1):
            keep, val = flat[i].item(), []
            for e in (1e-4, -1e-4):
                flat[i] = keep + e
                val.append((R.attention(*x, **kw)[0] * do.double()).sum().item())
            flat[i] = keep
            assert abs((val[0] - val[1]) / 2e-4 - g[i].item()) < 4 * 2.0 ** -11 * 4 * got[name].abs().max().item(), name


def test_repeatable_and_captured_with_separate_workspaces():
    a, b = inputs(2, 700, 900, 4, 2, 64, "bf16", 19), inputs(2, 700, 900, 4, 2, 64, "bf16", 20)
    kw = dict(causal=True, k_lens=i32([900, 650]))
    want = [call(*t, **kw) for t in (a, b)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs, outs, spaces = [], [], []
    cfg = B.attention_cfg(2, 700, 900, 4, 2, 64, causal=True)
    for i, t in enumerate((a, b)):
        spaces.append(torch.empty(B.sd_attention_workspace_size(cfg), dtype=torch.uint8, device="cuda"))
        graph = torch.cuda.CUDAGraph()
        s[i].wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s[i]):
            outs.append(call(*t, stream=s[i], ws=spaces[i], **kw))
        graphs.append(graph)
    for _ in range(4):
        for i in (0, 1):
            with torch.cuda.stream(s[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        for name in want[i]:
            assert torch.equal(want[i][name], outs[i][name]), name


def test_lse_may_be_absent():
    q, k, v, _ = inputs(1, 200, 300, 2, 2, 64, "bf16", 21)
    cfg = B.attention_cfg(1, 200, 300, 2, 2, 64)
    ws = torch.empty(B.sd_attention_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(q)
    B.sd_attention_fwd(cfg, q, k, v, None, o, None, ws, ws.numel())
    assert torch.equal(o, call(q, k, v)["o"])


def test_empty_tiles_between_documents():
    """Units without a visible tile between units with some (short rows, many heads): outputs of every kind follow one
    another in the same CTAs."""
    qd = i32([[0] * 128 + [9] * 128 + [1] * 128 + [8] * 200 + [2] * 100] * 3)
    kd = i32([[0] * 100 + [1] * 200 + [2] * 90 + [3] * 300] * 3)
    for d in (64, 128):
        check(3, 684, 690, 60, 60, d, seed=30 + d, q_doc=qd, k_doc=kd)


def test_items_cut_by_group():
    """More query and key tiles than the GPU holds at once, not a multiple: the last ones are computed in parts. The
    documents leave some of the parts without a visible tile, and the last sequence's keys end early."""
    qd = i32([[0] * 700 + [1] * 708])
    kd = i32([[0] * 600 + [1] * 3300 + [2] * 196])
    check(1, 1408, 4096, 30, 30, 64, seed=41)
    check(1, 1408, 4096, 30, 30, 64, seed=42, backward=False, q_doc=qd, k_doc=kd)
    check(1, 4000, 1408, 30, 30, 40, seed=43, k_lens=i32([1300]))


@pytest.mark.parametrize("d", [64, 80])
def test_long_walks_cut_shorter(d):
    """A causal mask with few items of unequal lengths: the longest are computed in two to eight parts."""
    check(2, 2047, 2047, 8, 2, d, seed=44, causal=True, prefix=i32([300, 0]), slopes=torch.linspace(0.01, 0.2, 8).cuda())
    check(1, 600, 3000, 6, 1, d, seed=45, causal=True, k_lens=i32([2900]))


def test_outputs_on_16_byte_boundaries():
    """Addresses and strides that are multiples of 16 bytes and not of 32 give the same bits."""
    def shifted(t):
        return torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[8:].view(t.shape)

    q, k, v, do = inputs(2, 300, 410, 4, 2, 64, "bf16", 51)
    want = call(q, k, v, do)
    cfg = B.attention_cfg(2, 300, 410, 4, 2, 64)
    n = B.sd_attention_workspace_size(cfg)
    ws, lse = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), torch.empty(2, 4, 300, device="cuda")
    o, dq, dk, dv = shifted(q), shifted(q), shifted(k), shifted(v)
    B.sd_attention_fwd(cfg, q, k, v, None, o, lse, ws, n)
    B.sd_attention_bwd(cfg, q, k, v, None, o, lse, do, dq, dk, dv, ws, n)
    # rows 16 bytes longer than their heads
    tall = torch.full((2, 300, 4 * 64 + 8), float("nan"), dtype=q.dtype, device="cuda")
    odd = B.attention_cfg(2, 300, 410, 4, 2, 64, o_stride=(300 * 264, 264, 64))
    B.sd_attention_fwd(odd, q, k, v, None, tall, lse, ws, n)
    torch.cuda.synchronize()
    for name, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(t, want[name]), name
    assert torch.equal(tall[:, :, :256].reshape(2, 300, 4, 64), want["o"])
    assert torch.isnan(tall[:, :, 256:]).all()
