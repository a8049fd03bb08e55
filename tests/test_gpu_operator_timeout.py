"""The bounded waits of the operators' tensor-core kernels run out, without a fault: sd_debug_inject_timeout lets the
loading threads of the next launches wait for what never comes. Every other role then gives up its own waits (barriers
among them), and the kernel ends. The status is reported once, and the next call is right."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from latent_diffusion_net_b200 import binding as B  # noqa: E402
from test_gpu_attention import i32, inputs  # noqa: E402
from test_gpu_gated_ff import NAMES, make  # noqa: E402

TIMEOUT = 8


def gives_up(run, outs, ws, launches):
    """`run` without and with `launches` kernels held; what it leaves the first and the third time is the same."""
    run()
    assert B.sd_query_device_status(ws) == 0
    want = [t.clone() for t in outs]
    try:
        B.sd_debug_inject_timeout(launches, 1000)
        run()
        assert B.sd_query_device_status(ws) == TIMEOUT
    finally:
        B.sd_debug_inject_timeout(0, 0)
    assert B.sd_query_device_status(ws) == 0
    for t in outs:
        t.zero_()
    run()
    assert B.sd_query_device_status(ws) == 0
    for t, w in zip(outs, want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("m,d,f", [(300, 128, 512), (5, 1280, 5120), (9216, 320, 1280)])
def test_gated_ff(m, d, f):
    p, dy = make(m, d, f, d, "bf16", seed=81)
    cfg = B.gated_ff_cfg(m, d, f, act=B.SD_ACT_GELU)
    ws = torch.full((B.sd_gated_ff_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    y, pre = torch.empty_like(p["x"]), torch.empty(m, 2 * f, dtype=dy.dtype, device="cuda")
    g = [torch.empty_like(p[k]) for k in NAMES]

    def forward():
        B.sd_gated_ff_fwd(cfg, p["w1"], p["b1"], p["w2"], p["b2"], p["x"], pre, y, ws, ws.numel())

    def backward():
        B.sd_gated_ff_bwd(cfg, p["w1"], p["w2"], p["x"], pre, dy, *g, ws, ws.numel())

    for n in (1, 2):
        gives_up(forward, [y, pre], ws, n)
    for n in (1, 4):
        gives_up(backward, g, ws, n)


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16")])
@pytest.mark.parametrize("cap", [0.0, 10.0])
@pytest.mark.parametrize("nq,nk,h", [(200, 300, 2), (1500, 1500, 40), (1, 4096, 8)])
def test_attention(nq, nk, h, cap, d, dt):
    q, k, v, do = inputs(2, nq, nk, h, h // 2, d, dt, 82)
    cfg = B.attention_cfg(2, nq, nk, h, h // 2, d, dtype=B.SD_DTYPE_F16 if dt == "f16" else B.SD_DTYPE_BF16, causal=True,
                          softcap=cap)
    lens = i32([nk, nk - 50])
    masks = B.attention_masks(k_lens=lens)
    ws = torch.full((B.sd_attention_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(2, h, nq, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)

    def forward():
        B.sd_attention_fwd(cfg, q, k, v, masks, o, lse, ws, ws.numel())

    def backward():
        B.sd_attention_bwd(cfg, q, k, v, masks, o, lse, do, dq, dk, dv, ws, ws.numel())

    gives_up(forward, [o, lse], ws, 1)
    for n in (1, 2):  # dq alone, dq and dk / dv
        gives_up(backward, [dq, dk, dv], ws, n)
