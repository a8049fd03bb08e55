"""Group norm with an activation and its gradients on a B200 against the
definition in 64 bits.

Tolerances. Sums are FP32 over per-thread runs and a tree: their relative error
stays below 2^-20 here. An element of y or dx is then rounded once to its type
(half a step of its value), on top of an FP32 error of a few 2^-22 of the largest
term; 2^-17 of the tensor's largest value covers those terms. Parameter gradients
are FP32 sums, compared in the 2-norm with 1e-5."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import operator_refs as R  # noqa: E402
from latent_diffusion_net_b200 import binding as B  # noqa: E402

DT = {"bf16": (torch.bfloat16, B.SD_DTYPE_BF16), "f16": (torch.float16, B.SD_DTYPE_F16),
      "f32": (torch.float32, B.SD_DTYPE_F32)}
ACT = {"none": B.SD_ACT_NONE, "silu": B.SD_ACT_SILU, "gelu": B.SD_ACT_GELU}


def close(got, want, t, what):
    want = want.detach()
    tol = R.HALF_STEP[t] * want.abs() + 2.0 ** -17 * want.abs().max()
    worst = ((got.double() - want).abs() - tol).max().item()
    assert torch.isfinite(got).all() and worst <= 0, (what, worst)


def make(n, r, c, dt, seed, ld=0, mean=0.5, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DT[dt][0]
    buf = torch.full((n, r, ld or c), float("nan"), dtype=t, device="cuda")
    x = buf[:, :, :c]
    x.copy_(torch.randn(n, r, c, generator=g, device="cuda") * std + mean)
    return buf, x, g


def run(n, r, c, groups, act, dt, ld_x=0, ld_y=0, affine=True, mean=0.5, std=1.5, seed=1, backward=True):
    t, code = DT[dt]
    xb, x, g = make(n, r, c, dt, seed, ld_x, mean, std)
    dyb, dy, _ = make(n, r, c, dt, seed + 1, ld_y, 0.1, 1.0)
    gamma = (1 + 0.1 * torch.randn(c, generator=g, device="cuda")).to(t) if affine else None
    beta = (0.1 * torch.randn(c, generator=g, device="cuda")).to(t) if affine else None
    cfg = B.group_norm_cfg(n, r, c, groups=groups, act=ACT[act], dtype=code, ld_x=ld_x, ld_y=ld_y)
    ws = torch.full((B.sd_group_norm_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    yb = torch.full((n, r, ld_y or c), 7.0, dtype=t, device="cuda")
    stats = torch.empty(n, groups, 2, device="cuda")
    B.sd_group_norm_fwd(cfg, xb, gamma, beta, yb, stats, ws, ws.numel())
    leaf = [a.double().detach().requires_grad_() if a is not None else None for a in (x, gamma, beta)]
    want, mean_w, rstd_w = R.group_norm(leaf[0], leaf[1], leaf[2], groups, 1e-5, act)
    out = {"y": yb[:, :, :c], "stats": stats, "want": want, "mean": mean_w, "rstd": rstd_w, "ypad": yb[:, :, c:]}
    if backward:
        dxb = torch.full((n, r, ld_x or c), 7.0, dtype=t, device="cuda")
        dg, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
        B.sd_group_norm_bwd(cfg, xb, gamma, beta, stats, dyb, dxb, dg, db, ws, ws.numel())
        want.backward(dy.double())
        out.update(dx=dxb[:, :, :c], dxpad=dxb[:, :, c:], dgamma=dg, dbeta=db, dx_w=leaf[0].grad,
                   dgamma_w=leaf[1].grad if affine else None, dbeta_w=leaf[2].grad if affine else None)
    assert B.sd_query_device_status(ws) == 0
    return out


def check(o, t):
    close(o["y"], o["want"], t, "y")
    assert R.rel(o["stats"][..., 0], o["mean"]) < 1e-5 and R.rel(o["stats"][..., 1], o["rstd"]) < 1e-5
    if "dx" in o:
        close(o["dx"], o["dx_w"], t, "dx")
        if o["dgamma_w"] is not None:
            assert R.rel(o["dgamma"], o["dgamma_w"]) < 1e-5 and R.rel(o["dbeta"], o["dbeta_w"]) < 1e-5


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("n,r,c,groups", [(1, 144, 1280, 32), (2, 1000, 320, 32), (3, 257, 96, 32), (1, 1, 64, 8),
                                          (2, 33, 60, 20), (1, 4099, 128, 1)])
def test_types_and_sizes(dt, act, n, r, c, groups):
    check(run(n, r, c, groups, act, dt), DT[dt][0])


@pytest.mark.parametrize("n,r,c,groups,dt", [
    (1, 9216, 320, 32, "bf16"),     # the single-kernel range of one image
    (4, 9216, 320, 32, "f16"),
    (1, 65536, 128, 32, "bf16"),    # several passes over L2-sized data
    (1, 300, 2560, 32, "f32"),      # more channel vectors than threads
    (2, 50, 8192, 32, "bf16"),      # the widest tensor
    (1, 7, 7, 7, "f16"),            # no 16-byte row, one channel a group
    (300, 3, 64, 32, "f32"),        # more images than rows
    (1, 2, 8192, 1, "f32"),
    (700, 1, 8, 2, "bf16"),
])
def test_ranges(n, r, c, groups, dt):
    check(run(n, r, c, groups, "silu", dt, seed=3), DT[dt][0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("ld_x,ld_y", [(72, 0), (0, 80), (67, 65), (128, 96)])
def test_row_strides(dt, ld_x, ld_y):
    o = run(2, 129, 64, 8, "silu", dt, ld_x=ld_x, ld_y=ld_y, seed=5)
    check(o, DT[dt][0])
    assert (o["ypad"] == 7).all() and (o["dxpad"] == 7).all()  # what lies between the rows stays


def test_no_affine():
    check(run(2, 100, 96, 8, "gelu", "f32", affine=False), torch.float32)


@pytest.mark.parametrize("mean,std", [(1000.0, 1.0), (-3e4, 10.0), (0.0, 1e-6), (0.0, 1e4)])
def test_mean_far_from_zero(mean, std):
    """FP32 inputs: x - mean is exact to 2^-24 of |mean|, so xh may be off by 2^-23 |mean| / std."""
    o = run(1, 3000, 64, 8, "none", "f32", mean=mean, std=std, backward=False)
    err = (o["y"].double() - o["want"]).abs().max().item()
    assert err < 1e-5 + 2.0 ** -22 * abs(mean) / std, err


def test_constant_input_has_no_variance():
    cfg = B.group_norm_cfg(1, 64, 32, groups=4, act=B.SD_ACT_NONE, dtype=B.SD_DTYPE_F32)
    ws = torch.empty(B.sd_group_norm_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    x = torch.full((1, 64, 32), 123.456, device="cuda")
    y, stats = torch.empty_like(x), torch.empty(1, 4, 2, device="cuda")
    B.sd_group_norm_fwd(cfg, x, None, None, y, stats, ws, ws.numel())
    assert y.abs().max().item() < 1e-2  # at most a rounding of the mean (2^-17) times 1/sqrt(eps)
    assert torch.isfinite(stats).all()


def test_gradient_against_differences():
    """The analytic dx against central differences of the 64-bit forward at random places, and of the
    kernel's own dx: the difference quotient is good to about 1e-6 with step 1e-4."""
    o = run(1, 20, 32, 4, "silu", "f32", seed=9)
    x = make(1, 20, 32, "f32", 9)[1].double()
    g = torch.Generator(device="cuda").manual_seed(9)
    torch.randn(1, 20, 32, generator=g, device="cuda")
    gamma = (1 + 0.1 * torch.randn(32, generator=g, device="cuda")).double()
    beta = (0.1 * torch.randn(32, generator=g, device="cuda")).double()
    dy = make(1, 20, 32, "f32", 10, 0, 0.1, 1.0)[1].double()
    f = lambda a: (R.group_norm(a, gamma, beta, 4, 1e-5, "silu")[0] * dy).sum().item()  # noqa: E731
    for r, c in [(0, 0), (3, 17), (19, 31), (11, 8)]:
        e = torch.zeros_like(x)
        e[0, r, c] = 1e-4
        assert abs((f(x + e) - f(x - e)) / 2e-4 - o["dx"][0, r, c].item()) < 1e-4


def test_in_place_repeatable_and_captured():
    cfg = B.group_norm_cfg(2, 500, 64, groups=8)
    ws = torch.empty(B.sd_group_norm_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    _, x, g = make(2, 500, 64, "bf16", 11)
    gamma = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.sd_group_norm_fwd(cfg, x, gamma, None, y, None, ws, ws.numel(), s)
        graph = torch.cuda.CUDAGraph()
        z = torch.empty_like(x)
        with torch.cuda.graph(graph, stream=s):
            B.sd_group_norm_fwd(cfg, x, gamma, None, z, None, ws, ws.numel(), s)
        for _ in range(3):
            z.zero_()
            graph.replay()
            s.synchronize()
            assert torch.equal(y, z)
        w = x.clone()
        B.sd_group_norm_fwd(cfg, w, gamma, None, w, None, ws, ws.numel(), s)
        s.synchronize()
    assert torch.equal(w, y)


def test_nothing_to_do():
    for n, r in [(0, 5), (3, 0)]:
        cfg = B.group_norm_cfg(n, r, 64)
        dg, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
        B.sd_group_norm_fwd(cfg, None, None, None, None, None, None, 0)
        B.sd_group_norm_bwd(cfg, None, None, None, None, None, None, dg, db, None, 0)
        torch.cuda.synchronize()
        assert not dg.any() and not db.any()
