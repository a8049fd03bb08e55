"""The gated feed-forward block and its gradients on a B200 against the definition
in 64 bits.

Tolerances count roundings to the type, each at most half a step u of a value, as
relative 2-norms: y has h and itself (2 u). Backward starts from the rounded v and
z (u each; the activation's slope magnifies z's by at most 2), rounds dv, dz and h
(u) and the result (u): 5 u. The FP32 sums add less than 1e-5."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import operator_refs as R  # noqa: E402
from latent_diffusion_net_b200 import binding as B  # noqa: E402

DT = {"bf16": (torch.bfloat16, B.SD_DTYPE_BF16), "f16": (torch.float16, B.SD_DTYPE_F16)}
ACT = {"none": B.SD_ACT_NONE, "silu": B.SD_ACT_SILU, "gelu": B.SD_ACT_GELU}
NAMES = ("x", "w1", "b1", "w2", "b2")


def make(m, d, f, do, dt, bias=True, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DT[dt][0]
    n = lambda shape, std=1.0: (torch.randn(shape, generator=g, device="cuda") * std).to(t)  # noqa: E731
    p = {"x": n((m, d)), "w1": n((2 * f, d), d ** -0.5), "w2": n((do, f), f ** -0.5)}
    p["b1"], p["b2"] = (n((2 * f,), 0.3), n((do,), 0.3)) if bias else (None, None)
    return p, n((m, do))


def plan(m, d, f, do, act, dt):
    cfg = B.gated_ff_cfg(m, d, f, do, act=ACT[act], dtype=DT[dt][1])
    ws = torch.full((B.sd_gated_ff_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    return cfg, ws


def forward(p, cfg, ws, pre=None, stream=None):
    y = torch.full((p["x"].shape[0], p["w2"].shape[0]), float("nan"), dtype=p["x"].dtype, device="cuda")
    B.sd_gated_ff_fwd(cfg, p["w1"], p["b1"], p["w2"], p["b2"], p["x"], pre, y, ws, ws.numel(), stream)
    return y


def backward(p, cfg, ws, pre, dy, stream=None):
    g = {k: torch.full_like(p[k], float("nan")) for k in NAMES if p[k] is not None}
    B.sd_gated_ff_bwd(cfg, p["w1"], p["w2"], p["x"], pre, dy, g["x"], g["w1"], g.get("b1"), g["w2"], g.get("b2"), ws,
                      ws.numel(), stream)
    return g


def reference(p, dy, act):
    leaf = {k: v.double().requires_grad_() if v is not None else None for k, v in p.items()}
    y, pre = R.gated_ff(leaf["x"], leaf["w1"], leaf["b1"], leaf["w2"], leaf["b2"], act)
    y.backward(dy.double())
    return y, pre, {k: v.grad for k, v in leaf.items() if v is not None}


def check(m, d, f, do, act, dt, bias=True, seed=1):
    u = R.HALF_STEP[DT[dt][0]]
    p, dy = make(m, d, f, do, dt, bias, seed)
    cfg, ws = plan(m, d, f, do, act, dt)
    want, pre_w, grads = reference(p, dy, act)
    y = forward(p, cfg, ws)
    assert R.rel(y, want) < 2 * u + 1e-5
    pre = torch.full((m, 2 * f), float("nan"), dtype=y.dtype, device="cuda")
    assert torch.equal(forward(p, cfg, ws, pre), y)
    assert R.rel(pre, pre_w) < u + 1e-5
    got = backward(p, cfg, ws, pre, dy)
    for k, g in got.items():
        assert R.rel(g, grads[k]) < 5 * u + 1e-5, (k, R.rel(g, grads[k]))
    assert B.sd_query_device_status(ws) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("m,d,f,do", [(300, 320, 1280, 320), (77, 64, 200, 72)])
def test_types_and_activations(m, d, f, do, act, dt):
    check(m, d, f, do, act, dt)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 7, 8, 9, 16, 31, 64, 127, 128, 129, 255, 256, 257, 1000])
def test_token_counts(m):
    check(m, 128, 264, 128, "silu", "bf16", seed=m)


@pytest.mark.parametrize("m,d,f,do", [
    (1, 1280, 5120, 1280),       # one token
    (4, 640, 2560, 640),
    (2, 8, 8, 8),                # the smallest
    (513, 8, 24, 16),            # reductions shorter than one block
    (1155, 640, 2560, 640),
    (9216, 320, 1280, 320),      # weight gradients split over the tokens
    (40, 1000, 1496, 56),        # widths in no multiple of a tile
    (3000, 72, 5000, 1160),
])
def test_sizes(m, d, f, do):
    check(m, d, f, do, "gelu", "bf16", seed=7)


def test_no_bias():
    check(200, 64, 136, 64, "silu", "f16", bias=False)
    check(3, 64, 136, 64, "silu", "f16", bias=False)


def test_single_gradients():
    """Each gradient alone equals the same one of a whole call, and the others stay untouched."""
    p, dy = make(300, 64, 192, 64, "bf16")
    cfg, ws = plan(300, 64, 192, 64, "gelu", "bf16")
    pre = torch.empty(300, 384, dtype=torch.bfloat16, device="cuda")
    forward(p, cfg, ws, pre)
    whole = backward(p, cfg, ws, pre, dy)
    order = ("x", "w1", "b1", "w2", "b2")
    for k in order:
        one = torch.full_like(p[k], float("nan"))
        args = [one if k == o else None for o in order]
        B.sd_gated_ff_bwd(cfg, p["w1"], p["w2"], p["x"], pre, dy, *args, ws, ws.numel())
        assert torch.equal(one, whole[k]), k


def test_gradient_against_differences():
    """d(sum y dy)/dx by central differences of the 64-bit block, good to 1e-6; dx is rounded to FP16: 5 u."""
    p, dy = make(6, 16, 32, 16, "f16", seed=4)
    cfg, ws = plan(6, 16, 32, 16, "silu", "f16")
    pre = torch.empty(6, 64, dtype=torch.float16, device="cuda")
    forward(p, cfg, ws, pre)
    got = backward(p, cfg, ws, pre, dy)
    q = {k: v.double() for k, v in p.items()}
    for name in ("x", "w1", "b1", "w2", "b2"):
        flat = q[name].reshape(-1)
        scale = got[name].abs().max().item()
        for i in (0, flat.numel() // 2, flat.numel() - 1):
            keep = flat[i].item()
            vals = []
            for e in (1e-4, -1e-4):
                flat[i] = keep + e
                vals.append((R.gated_ff(q["x"], q["w1"], q["b1"], q["w2"], q["b2"], "silu")[0] * dy.double()).sum().item())
            flat[i] = keep
            assert abs((vals[0] - vals[1]) / 2e-4 - got[name].reshape(-1)[i].item()) < 5 * 2.0 ** -11 * 4 * scale, name


def test_repeatable_and_captured():
    p, dy = make(1000, 128, 512, 128, "bf16")
    cfg, ws = plan(1000, 128, 512, 128, "gelu", "bf16")
    pre = torch.empty(1000, 1024, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = forward(p, cfg, ws, pre, s)
        g = backward(p, cfg, ws, pre, dy, s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y2 = forward(p, cfg, ws, pre, s)
            g2 = backward(p, cfg, ws, pre, dy, s)
        for _ in range(3):
            y2.zero_()
            graph.replay()
            s.synchronize()
            assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)


def test_nothing_to_do():
    cfg, ws = plan(0, 64, 64, 64, "silu", "bf16")
    p, _ = make(1, 64, 64, 64, "bf16")
    g = {k: torch.ones_like(p[k]) for k in NAMES}
    B.sd_gated_ff_fwd(cfg, None, None, None, None, None, None, None, None, 0)
    B.sd_gated_ff_bwd(cfg, None, None, None, None, None, None, g["w1"], g["b1"], g["w2"], g["b2"], None, 0)
    torch.cuda.synchronize()
    assert not any(g[k].any() for k in ("w1", "b1", "w2", "b2"))


@pytest.mark.parametrize("m", [3, 300])
def test_tensors_on_16_byte_boundaries(m):
    """Every tensor at a multiple of 16 bytes that is none of 32: the same bits."""
    def shifted(t):
        return torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[8:].view(t.shape).copy_(t)

    p, dy = make(m, 128, 192, 160, "bf16")
    cfg, ws = plan(m, 128, 192, 160, "gelu", "bf16")
    pre = torch.empty(m, 384, dtype=dy.dtype, device="cuda")
    y = forward(p, cfg, ws, pre)
    want = backward(p, cfg, ws, pre, dy)
    q = {k: shifted(v) for k, v in p.items()}
    pre2, y2 = shifted(torch.zeros_like(pre)), shifted(torch.zeros_like(y))
    B.sd_gated_ff_fwd(cfg, q["w1"], q["b1"], q["w2"], q["b2"], q["x"], pre2, y2, ws, ws.numel())
    got = {k: shifted(torch.zeros_like(v)) for k, v in p.items()}
    B.sd_gated_ff_bwd(cfg, q["w1"], q["w2"], q["x"], pre2, shifted(dy), got["x"], got["w1"], got["b1"], got["w2"],
                      got["b2"], ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(pre2, pre)
    for name in want:
        assert torch.equal(got[name], want[name]), name
