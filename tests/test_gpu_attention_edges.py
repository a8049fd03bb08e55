"""Attention at the edges of what its description allows, on a B200: values that are not numbers, padding that holds
anything, loss-scaled FP16 gradients, saturated caps, strided outputs. Tolerances as in test_gpu_attention.py, with
what a test adds written beside it."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import operator_refs as R  # noqa: E402
from latent_diffusion_net_b200 import binding as B  # noqa: E402
from test_gpu_attention import call, compare, i32, inputs, packed, reference  # noqa: E402


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_documents_cut_anywhere_in_long_rows(d, causal):
    """Tiles of one document, tiles with a cut inside and tiles that nobody sees in turns, through many more steps than
    the documents' ring has places, in CTAs that take several units and end after any kind of step."""
    cuts = [[0, 130, 131, 700, 1280, 1900, 2600], [0, 1, 64, 1000, 1024, 2000, 2690]]
    n = 2700
    doc = torch.zeros(2, n, dtype=torch.int32, device="cuda")
    for b, at in enumerate(cuts):
        for i, c in enumerate(at):
            doc[b, c:] = (i * 5) % 7  # ids in no order
    q, k, v, do = inputs(2, n, n, 6, 2, d, "bf16", 75)
    kw = dict(causal=causal, q_doc=doc, k_doc=doc, k_lens=i32([n, 2650]))
    compare(call(q, k, v, do, **kw), reference(q, k, v, do, **kw), q.dtype)


# one query on many keys: computed in parts; 300 and 200 queries: whole
NAN_SHAPES = [(1, 4096, 16, 4, 128), (3, 5000, 4, 4, 64), (300, 300, 2, 2, 64), (200, 260, 4, 2, 128)]


@pytest.mark.parametrize("nq,nk,h,kv,d", NAN_SHAPES)
def test_nan_in_a_query_stays_in_its_row(nq, nk, h, kv, d):
    """Whether keys are taken in parts or not: the row's output and lse are NaN, all others as without it."""
    q, k, v, _ = inputs(2, nq, nk, h, kv, d, "bf16", 61)
    clean = call(q, k, v)
    q[1, nq - 1, h - 1, 3] = math.nan
    got = call(q, k, v)
    bad = torch.zeros(2, nq, h, dtype=torch.bool, device="cuda")
    bad[1, nq - 1, h - 1] = True
    assert torch.isnan(got["o"][bad]).all() and torch.equal(got["o"][~bad], clean["o"][~bad])
    bad = bad.permute(0, 2, 1)
    assert torch.isnan(got["lse"][bad]).all() and torch.equal(got["lse"][~bad], clean["lse"][~bad])


@pytest.mark.parametrize("nq,nk,h,kv,d", NAN_SHAPES)
def test_nan_in_visible_keys_is_not_dropped(nq, nk, h, kv, d):
    """The newest half of the keys of one head: whole tiles and whole parts whose scores are all NaN."""
    q, k, v, do = inputs(2, nq, nk, h, kv, d, "bf16", 62)
    clean = call(q, k, v, do)
    k[1, nk // 2:, kv - 1] = math.nan
    got = call(q, k, v, do)
    g = h // kv
    assert torch.isnan(got["o"][1, :, -g:]).all() and torch.isnan(got["lse"][1, -g:]).all()
    assert torch.isnan(got["dq"][1, :, -g:]).all() and torch.isnan(got["dv"][1, :, -1]).all()
    for name, at in (("o", 2), ("lse", 1), ("dq", 2)):
        keep = torch.ones_like(clean[name], dtype=torch.bool)
        keep[1].narrow(at - 1, h - g, g).fill_(False)
        assert torch.equal(got[name][keep], clean[name][keep]), name
    assert torch.equal(got["dv"][0], clean["dv"][0]) and torch.equal(got["dk"][0], clean["dk"][0])


def test_nan_only_in_the_newest_key():
    """One key in a tile of its own (and, for one query, perhaps in a part of its own)."""
    for nq, nk in ((1, 4097), (1, 129), (140, 385)):
        q, k, v, _ = inputs(1, nq, nk, 2, 2, 64, "f16", 63)
        k[0, nk - 1, 1] = math.nan
        got = call(q, k, v)
        assert torch.isnan(got["o"][0, :, 1]).all() and torch.isnan(got["lse"][0, 1]).all()
        assert torch.isfinite(got["o"][0, :, 0]).all() and torch.isfinite(got["lse"][0, 0]).all()


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (64, "f16"), (80, "bf16"), (128, "f16")])
@pytest.mark.parametrize("cap,std", [(5.0, 2.0), (50.0, 0.3)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_capped_scores_of_padding_are_never_used(d, dt, cap, std, bias, bad):
    """Large and small capped scores over keys and values that hold anything behind the lengths."""
    lens = [200, 130, 0]
    q, k, v, do = inputs(3, 150, 300, 4, 2, d, dt, 64, std)
    kw = dict(softcap=cap, causal=True, slopes=torch.tensor([0.1, 0.0, 0.02, 0.3], device="cuda") if bias else None)
    want = reference(q, k, v, do, k_lens=i32(lens), **kw)
    for b, n in enumerate(lens):
        k[b, n:] = bad
        v[b, n:] = bad
    got = call(q, k, v, do, k_lens=i32(lens), **kw)
    for name in ("o", "dq", "dk", "dv"):
        assert torch.isfinite(got[name]).all(), name
    compare(got, want, q.dtype)
    for b, n in enumerate(lens):
        assert not got["dk"][b, n:].any() and not got["dv"][b, n:].any()


def f16_gradients(scale, nq, nk, d, seed, h=2, kv=1, **kw):
    """Against 64 bits with dO of that size. The gradients' own subnormal numbers end at 2^-24: half a step of it an
    element comes on top of the roundings."""
    q, k, v, do = inputs(1, nq, nk, h, kv, d, "f16", seed)
    do = (do.float() * scale).half()
    got, want = call(q, k, v, do, **kw), reference(q, k, v, do, **kw)
    for name in ("dq", "dk", "dv"):
        w = want[name]
        assert w.abs().max().item() < 3e4, "the true gradient has to fit"
        assert torch.isfinite(got[name]).all(), name
        tol = (2 if name == "dv" else 4) * 2.0 ** -11 + 1e-5 + 2.0 ** -25 * w.numel() ** 0.5 / w.norm().item()
        err = R.rel(got[name], w)
        assert err < tol, (name, err, tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nk", [4096, 16384])
@pytest.mark.parametrize("scale", [2.0 ** -8, 1.0, 4096.0])
def test_f16_gradients_over_long_rows(scale, nk, d):
    """Rows that see all keys, and rows of the same call that see four (large probabilities)."""
    f16_gradients(scale, 200, nk, d, 65)
    doc = i32([packed([4] * 32 + [nk // 2], nk)])
    rows = torch.arange(200, device="cuda", dtype=torch.int32)[None] % 34
    f16_gradients(scale / 4, 200, nk, d, 66, q_doc=rows, k_doc=doc)


def test_f16_gradients_with_one_large_row():
    """A row of dO 2^12 times the others, peaked and capped scores, parts of long walks, shared heads."""
    q, k, v, do = inputs(2, 700, 9000, 6, 2, 64, "f16", 67, 1.5)
    do[1, 600, 4] *= 2.0 ** 12
    for kw in (dict(causal=True), dict(causal=True, softcap=30.0, k_lens=i32([9000, 8000]))):
        got, want = call(q, k, v, do, **kw), reference(q, k, v, do, **kw)
        for name in ("dq", "dk", "dv"):
            assert torch.isfinite(got[name]).all(), name
            w = want[name]
            tol = (2 if name == "dv" else 4) * 2.0 ** -11 + 1e-5 + 2.0 ** -25 * w.numel() ** 0.5 / w.norm().item()
            assert R.rel(got[name], w) < tol, (name, R.rel(got[name], w), tol)
        # the other rows of dq by themselves: their factor is their own
        g, w = got["dq"].double().clone(), want["dq"].clone()
        g[1, 600, 4] = w[1, 600, 4] = 0
        assert R.rel(g, w) < 4 * 2.0 ** -11 + 1e-5 + 2.0 ** -25 * w.numel() ** 0.5 / w.norm().item()


def test_f16_gradients_ignore_values_that_no_key_holds():
    """What lies behind the lengths, or in the dO of rows that see nothing, takes no part in any scaling."""
    q, k, v, do = inputs(2, 300, 500, 4, 2, 64, "f16", 68)
    kw = dict(k_lens=i32([500, 200]), causal=True)
    do[1, :100] = 0
    want = call(q, k, v, do, **kw)
    k[1, 200:] = v[1, 200:] = 6e4
    do[1, :100] = 3e4  # positions below zero
    got = call(q, k, v, do, **kw)
    for name in want:
        assert torch.equal(got[name], want[name]), name
    v[1, 200:] = math.inf
    got = call(q, k, v, do, **kw)
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (128, "f16")])
def test_capped_results_do_not_depend_on_padding(d, dt):
    """Small scores beside the cap, and padding whose scores would be large: the same bits for every padding."""
    lens = [200, 130]
    q, k, v, do = inputs(2, 150, 300, 4, 2, d, dt, 69, 0.5)
    outs = []
    for fill in (0.0, 200.0, -3.0, math.nan):
        for b, n in enumerate(lens):
            k[b, n:] = fill
            v[b, n:] = fill
        outs.append(call(q, k, v, do, softcap=8.0, k_lens=i32(lens)))
        outs.append(call(q, k, v, do, softcap=8.0, k_lens=i32(lens), causal=True, prefix=i32([40, 0])))
    for i, got in enumerate(outs[2:]):
        for name in got:
            assert torch.equal(got[name], outs[i % 2][name]), (i, name)


@pytest.mark.parametrize("h,kv,d", [(3, 1, 64), (12, 1, 64), (6, 2, 128), (5, 1, 80)])
def test_capped_results_do_not_depend_on_earlier_calls(h, kv, d):
    """A tile of 128 / 3 (or 5, 12) tokens leaves rows over, whose place in the chip's memory holds what the last call
    left there."""
    q, k, v, do = inputs(2, 512, 640, h, kv, d, "bf16", 70, 0.5)
    before = inputs(4, 1280, 640, 16, 16, d, "bf16", 71)
    outs = []
    for size in (0.0, 300.0, 1.0):
        call((before[0].float() * size).bfloat16(), before[1], before[2])
        outs.append(call(q, k, v, do, softcap=8.0))
    for got in outs[1:]:
        for name in got:
            assert torch.equal(got[name], outs[0][name]), name


def test_prefix_of_any_negative_number_is_none():
    q, k, v, do = inputs(3, 300, 300, 2, 2, 64, "bf16", 72)
    want = call(q, k, v, do, causal=True)
    got = call(q, k, v, do, causal=True, prefix=i32([-2 ** 31, -1, 0]))
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_saturated_cap_keeps_its_gradient(d, dt, sign):
    """All scores far beyond the cap: the slope 1 - tanh^2 is near 4 e^-14 and has to be right relative to itself. Scores
    are near 14 c for a cap of 2 c: x = 7 with a small spread. FP32 scores (sums of D products, 2^-22 of 14 c) move
    ln(slope) by less than 1e-5.

    q and k lie close to one direction, so that dq = scale sum_j dS_ij k_j adds long vectors to a short one. Roundings of
    dS are independent and at most u each: as a 2-norm they move dq by u scale (sum_ij dS_ij^2 |k_j|^2)^1/2, which is A u
    relative to |dq| with A from the 64-bit dS. dS is rounded once, its slope once (FP16 pairs), and dP takes in v and do
    unrounded; P's rounding enters through delta's correction, once more: 3 A u, and the result's own u. dk likewise with q."""
    c = 1.0 if dt == "bf16" else 0.5
    g = torch.Generator(device="cuda").manual_seed(73)
    t = torch.bfloat16 if dt == "bf16" else torch.float16
    base = torch.sign(torch.randn(d, generator=g, device="cuda"))
    n = lambda tok: (base + 0.05 * torch.randn(1, tok, 2, d, generator=g, device="cuda"))  # noqa: E731
    q, k = n(140).to(t), (sign * n(200)).to(t)
    v, do = (torch.randn(1, tok, 2, d, generator=g, device="cuda") for tok in (200, 140))
    v, do = v.to(t), (do * (8192.0 if dt == "f16" else 1.0)).to(t)  # gradients well above FP16's smallest numbers
    kw = dict(scale=14 * c / d, softcap=2 * c)
    got, want = call(q, k, v, do, **kw), reference(q, k, v, do, **kw)
    q8, k8, v8, do8 = (x[0].double().transpose(0, 1) for x in (q, k, v, do))  # [H, tokens, D]
    th = torch.tanh(q8 @ k8.transpose(1, 2) * (kw["scale"] / kw["softcap"]))
    p = torch.softmax(kw["softcap"] * th, dim=-1)
    dp = do8 @ v8.transpose(1, 2)
    ds2 = (p * (dp - (p * dp).sum(-1, keepdim=True)) / torch.cosh(torch.atanh(th)) ** 2) ** 2
    u = R.HALF_STEP[t]
    assert R.rel(got["o"], want["o"]) < 2 * u + 1e-5 and R.rel(got["dv"], want["dv"]) < 2 * u + 1e-5
    for name, other in (("dq", ds2 @ (k8 ** 2).sum(-1, keepdim=True)),
                        ("dk", ds2.transpose(1, 2) @ (q8 ** 2).sum(-1, keepdim=True))):
        a = kw["scale"] * other.sum().sqrt().item() / want[name].norm().item()
        err = R.rel(got[name], want[name])
        print(name, "A", a, "err", err, "tol", (1 + 3 * a) * u + 1e-5)
        assert err < (1 + 3 * a) * u + 1e-5, (name, err, a)


def test_f16_small_probabilities_of_short_rows():
    """Keys far below a row's largest score: P near 2^-20, below FP16's normal numbers, is all that their dv and dk come
    from. Each such gradient against 64 bits by itself, as large as the others through a large dO."""
    q, k, v, do = inputs(1, 130, 100, 2, 2, 64, "f16", 76, 0.1)
    q[..., 0] = 4.0
    k[:, :50, :, 0], k[:, 50:, :, 0] = 14.0, -14.0  # scores +-7, so that P falls by e^-14
    do = (do.float() * 2.0 ** 14).half()
    got, want = call(q, k, v, do), reference(q, k, v, do)
    for name, rounds in (("dv", 2), ("dk", 4)):
        for part in (slice(0, 50), slice(50, 100)):
            w = want[name][:, part]
            if name == "dk":
                w, g = w[..., 1:], got[name][:, part, :, 1:]  # q's first column is the same everywhere: it adds up dS
            else:
                g = got[name][:, part]
            tol = rounds * 2.0 ** -11 + 1e-5 + 2.0 ** -25 * w.numel() ** 0.5 / w.norm().item()
            assert R.rel(g, w) < tol, (name, part, R.rel(g, w), tol)


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (128, "bf16"), (80, "f16")])
@pytest.mark.parametrize("cap", [0.0, 10.0])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_queries_that_see_nothing_may_hold_anything(d, dt, cap, bad):
    """Rows before a sequence's first key, and rows whose document no key has: nothing of their q and dO goes anywhere."""
    q, k, v, do = inputs(2, 400, 300, 4, 2, d, dt, 77)
    doc = torch.zeros(2, 400, dtype=torch.int32, device="cuda")
    doc[0, 350:370] = 9
    kw = dict(causal=True, k_lens=i32([300, 180]), q_doc=doc, k_doc=doc[:, :300] * 0, softcap=cap)
    want = call(q, k, v, do, **kw)
    dead = torch.isneginf(want["lse"])[:, 0]  # [batch, q]
    assert 300 < dead.sum() < 500 and (dead == torch.isneginf(want["lse"]).all(dim=1)).all()
    q[dead], do[dead] = bad, bad
    got = call(q, k, v, do, **kw)
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_strided_output_and_its_gradient(dt):
    """o and d_o as columns of a wider tensor: read and written in place, what lies between stays."""
    q, k, v, do = inputs(2, 190, 210, 4, 2, 64, dt, 74)
    want = reference(q, k, v, do, causal=True)
    wide = 4 * 64 + 40
    buf = torch.full((2, 190, wide), 3.0, dtype=q.dtype, device="cuda")
    o = buf[:, :, 16:16 + 256].view(2, 190, 4, 64)
    gbuf = torch.full((2, 190, wide), math.nan, dtype=q.dtype, device="cuda")
    gbuf[:, :, 16:16 + 256] = do.view(2, 190, 256)
    d_o = gbuf[:, :, 16:16 + 256].view(2, 190, 4, 64)
    cfg = B.attention_cfg(2, 190, 210, 4, 2, 64, dtype=B.SD_DTYPE_BF16 if dt == "bf16" else B.SD_DTYPE_F16, causal=True,
                          o_stride=o.stride()[:3])
    ws = torch.full((B.sd_attention_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    lse = torch.empty(2, 4, 190, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    B.sd_attention_fwd(cfg, q, k, v, None, o, lse, ws, ws.numel())
    B.sd_attention_bwd(cfg, q, k, v, None, o, lse, d_o, dq, dk, dv, ws, ws.numel())
    compare({"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, want, q.dtype)
    assert (buf[:, :, :16] == 3).all() and (buf[:, :, 272:] == 3).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_workspace_on_a_16_byte_boundary(dt):
    """A workspace taken out of a larger buffer, with documents and with rows computed in parts: the same bits, and
    nothing written outside it."""
    q, k, v, do = inputs(2, 300, 3000, 6, 2, 72, dt, 78)
    doc = torch.zeros(2, 3000, dtype=torch.int32, device="cuda")
    doc[:, 1111:] = 1
    kw = dict(causal=True, q_doc=doc[:, 2700:].contiguous(), k_doc=doc, k_lens=i32([3000, 2900]))
    want = call(q, k, v, do, **kw)
    cfg = B.attention_cfg(2, 300, 3000, 6, 2, 72, dtype=B.SD_DTYPE_BF16 if dt == "bf16" else B.SD_DTYPE_F16, causal=True)
    n = B.sd_attention_workspace_size(cfg)
    for offset in (16, 48, 240):
        buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        got = call(q, k, v, do, ws=buf[offset:offset + n], **kw)
        for name in want:
            assert torch.equal(got[name], want[name]), name
        assert (buf[:offset] == 0xA5).all() and (buf[offset + n:] == 0xA5).all()


def test_f16_backward_captured_and_replayed_with_other_sizes_of_gradient():
    """The factors of dS come from the tensors at the time of the replay."""
    q, k, v, do = inputs(2, 300, 700, 4, 2, 64, "f16", 79)
    cfg = B.attention_cfg(2, 300, 700, 4, 2, 64, dtype=B.SD_DTYPE_F16, softcap=15.0)
    ws = torch.full((B.sd_attention_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(2, 4, 300, device="cuda")
    out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v)}
    given, s = do.clone(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.sd_attention_fwd(cfg, q, k, v, None, o, lse, ws, ws.numel(), torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.sd_attention_bwd(cfg, q, k, v, None, o, lse, given, out["dq"], out["dk"], out["dv"], ws, ws.numel(), s)
    for scale in (2.0 ** -6, 4096.0, 1.0):
        given.copy_(do.float() * scale)
        want = call(q, k, v, given, softcap=15.0)
        graph.replay()
        torch.cuda.synchronize()
        for name in out:
            assert torch.isfinite(out[name]).all() and torch.equal(out[name], want[name]), (scale, name)


def test_f16_infinite_gradient_stays_in_its_row_of_dq():
    q, k, v, do = inputs(1, 300, 400, 4, 2, 64, "f16", 80)
    want = reference(q, k, v, do)
    do[0, 100, 3] = math.inf
    got = call(q, k, v, do)
    assert not torch.isfinite(got["dq"][0, 100, 3]).any()
    keep = torch.ones_like(do, dtype=torch.bool)
    keep[0, 100, 3] = False
    assert R.rel(got["dq"][keep], want["dq"][keep]) < 4 * 2.0 ** -11 + 1e-5
    # the other key head's gradients
    assert R.rel(got["dk"][:, :, 0], want["dk"][:, :, 0]) < 4 * 2.0 ** -11 + 1e-5
    assert R.rel(got["dv"][:, :, 0], want["dv"][:, :, 0]) < 2 * 2.0 ** -11 + 1e-5
