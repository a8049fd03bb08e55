"""Group norm at the edges of what its description allows, on a B200: outliers and steps in the data, results in place,
other eps."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import operator_refs as R  # noqa: E402
from latent_diffusion_net_b200 import binding as B  # noqa: E402
from test_gpu_group_norm import ACT, DT, close, make  # noqa: E402


def forward(x, groups, act="none", eps=1e-5):
    n, r, c = x.shape
    code = {torch.bfloat16: B.SD_DTYPE_BF16, torch.float16: B.SD_DTYPE_F16, torch.float32: B.SD_DTYPE_F32}[x.dtype]
    cfg = B.group_norm_cfg(n, r, c, groups=groups, eps=eps, act=ACT[act], dtype=code)
    ws = torch.full((B.sd_group_norm_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    y, stats = torch.empty_like(x), torch.empty(n, groups, 2, device="cuda")
    B.sd_group_norm_fwd(cfg, x, None, None, y, stats, ws, ws.numel())
    return y, stats


# one kernel in clusters, two kernels with whole vectors, two kernels element by element
PIVOT_SHAPES = [(1, 3000, 64, 8), (1, 9216, 320, 32), (1, 150000, 128, 32), (2, 40000, 60, 20)]


def statistics_hold(x, groups, where):
    """Sums are FP32 over per-thread runs and a tree, of positive terms only: rstd within 2^-18, the mean within 2^-18 of
    the standard deviation; y - away from the outliers - within 2^-18 of its size and of the mean's error."""
    y, stats = forward(x, groups)
    want, mean, rstd = R.group_norm(x.double(), None, None, groups, 1e-5, "none")
    assert ((stats[..., 1].double() / rstd - 1).abs().max().item()) < 2.0 ** -18
    far = (mean.abs() * rstd).max().item()
    assert (((stats[..., 0].double() - mean) * rstd).abs().max().item()) < 2.0 ** -18 + 2.0 ** -23 * far
    err = (y.double() - want).abs() - 2.0 ** -18 * (1 + want.abs()) - 2.0 ** -22 * far
    assert err[where].max().item() < 0, err[where].max().item()


@pytest.mark.parametrize("n,r,c,groups", PIVOT_SHAPES)
@pytest.mark.parametrize("size", [30.0, 100.0, 1000.0])
def test_outlier_in_the_first_place(n, r, c, groups, size):
    """One value far from all others, wherever a pass over the rows begins."""
    _, x, _ = make(n, r, c, "f32", 21, mean=0.0, std=1.0)
    where = torch.ones_like(x, dtype=torch.bool)
    for row in (0, r // 2, r - 1):
        x[:, row, ::c // groups] = size
        where[:, row] = False
    statistics_hold(x, groups, where)


@pytest.mark.parametrize("n,r,c,groups", PIVOT_SHAPES)
@pytest.mark.parametrize("border", [1, 40, 700])
def test_padded_border(n, r, c, groups, border):
    """Zeros in the first and last rows, values far from zero between them: x - mean is exact to 2^-24 of the mean, so y
    carries 2^-22 |mean| rstd more."""
    _, x, _ = make(n, r, c, "f32", 22, mean=100.0, std=1.0)
    x[:, :border] = 0
    x[:, r - border:] = 0
    statistics_hold(x, groups, torch.ones_like(x, dtype=torch.bool))


@pytest.mark.parametrize("n,r,c", [(2, 500, 64), (1, 60000, 128)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradient_in_place(n, r, c, dt):
    """dx in the place of x, and of dy: the same bits as beside them."""
    _, x, g = make(n, r, c, dt, 23)
    _, dy, _ = make(n, r, c, dt, 24, 0, 0.1, 1.0)
    gamma = (1 + 0.1 * torch.randn(c, generator=g, device="cuda")).to(x.dtype)
    cfg = B.group_norm_cfg(n, r, c, groups=8, dtype=DT[dt][1])
    ws = torch.full((B.sd_group_norm_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    y, stats = torch.empty_like(x), torch.empty(n, 8, 2, device="cuda")
    B.sd_group_norm_fwd(cfg, x, gamma, None, y, stats, ws, ws.numel())
    outs = []
    for place in (None, "x", "dy"):
        a, b = x.clone(), dy.clone()
        dx = {"x": a, "dy": b, None: torch.empty_like(x)}[place]
        dg, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
        B.sd_group_norm_bwd(cfg, a, gamma, None, stats, b, dx, dg, db, ws, ws.numel())
        outs.append((dx, dg, db))
    torch.cuda.synchronize()
    for other in outs[1:]:
        assert all(torch.equal(s, t) for s, t in zip(outs[0], other))


@pytest.mark.parametrize("eps", [1e-12, 1e-3, 0.5, 30.0])
def test_eps(eps):
    for r in (300, 60000):
        _, x, _ = make(1, r, 64, "f32", 25, mean=0.3, std=0.7)
        y, stats = forward(x, 8, "silu", eps)
        want, mean, rstd = R.group_norm(x.double(), None, None, 8, eps, "silu")
        close(y, want, torch.float32, "y")
        assert R.rel(stats[..., 1], rstd) < 1e-5


@pytest.mark.parametrize("n,r,c", [(3, 500, 64), (1, 60000, 128), (2, 3000, 60)])
def test_workspace_on_a_16_byte_boundary(n, r, c):
    """A workspace taken out of a larger buffer: the same bits, and nothing written outside it."""
    _, x, _ = make(n, r, c, "bf16", 26)
    _, dy, _ = make(n, r, c, "bf16", 27, 0, 0.1, 1.0)
    cfg = B.group_norm_cfg(n, r, c, groups=4)
    size = B.sd_group_norm_workspace_size(cfg)
    outs = []
    for offset in (0, 16, 240):
        buf = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        ws = buf[offset:offset + size]
        y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(n, 4, 2, device="cuda")
        dg, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
        B.sd_group_norm_fwd(cfg, x, None, None, y, stats, ws, size)
        B.sd_group_norm_bwd(cfg, x, None, None, stats, dy, dx, dg, db, ws, size)
        assert B.sd_query_device_status(ws) == 0
        assert (buf[:offset] == 0xA5).all() and (buf[offset + size:] == 0xA5).all()
        outs.append((y, stats, dx, dg, db))
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
