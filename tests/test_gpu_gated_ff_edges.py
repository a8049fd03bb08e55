"""The gated feed-forward at the edges of what its description allows, on a B200."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from latent_diffusion_net_b200 import binding as B  # noqa: E402
from test_gpu_gated_ff import backward, forward, make, plan  # noqa: E402


@pytest.mark.parametrize("offset", [16, 48, 240])
@pytest.mark.parametrize("m,d,f", [(5, 1280, 5120), (77, 320, 1280), (1155, 640, 2560), (3, 640, 640)])
def test_workspace_on_a_16_byte_boundary(m, d, f, offset):
    """A workspace taken out of a larger buffer, products split over their reduction among them: the same bits, and
    nothing written outside it."""
    p, dy = make(m, d, f, d, "bf16", seed=31)
    cfg, ws = plan(m, d, f, d, "gelu", "bf16")
    n = B.sd_gated_ff_workspace_size(cfg)
    pre = torch.empty(m, 2 * f, dtype=dy.dtype, device="cuda")
    y = forward(p, cfg, ws, pre)
    want = backward(p, cfg, ws, pre, dy)
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    part = buf[offset:offset + n]
    assert part.data_ptr() % 32 == 16
    pre2 = torch.empty_like(pre)
    assert torch.equal(forward(p, cfg, part, pre2), y) and torch.equal(pre2, pre)
    got = backward(p, cfg, part, pre, dy)
    assert B.sd_query_device_status(part) == 0
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert (buf[:offset] == 0xA5).all() and (buf[offset + n:] == 0xA5).all()


@pytest.mark.parametrize("m", [1, 2, 4])
def test_input_written_by_the_call_before(m):
    """Few tokens through a chain of blocks without anything between the calls: each block reads what the one before it
    has just written, and h within a block."""
    blocks = [make(m, 256, 1024, 256, "bf16", seed=40 + i)[0] for i in range(6)]
    cfg, ws = plan(m, 256, 1024, 256, "silu", "bf16")
    spaces = [torch.empty_like(ws) for _ in blocks]
    x0 = blocks[0]["x"]
    step, want = x0, []
    for p in blocks:
        y = forward({**p, "x": step}, cfg, ws)
        torch.cuda.synchronize()
        want.append(y)
        step = y
    for _ in range(20):
        outs = [torch.zeros_like(x0) for _ in blocks]
        src = x0
        for p, space, y in zip(blocks, spaces, outs):
            B.sd_gated_ff_fwd(cfg, p["w1"], p["b1"], p["w2"], p["b2"], src, None, y, space, space.numel())
            src = y
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w)
