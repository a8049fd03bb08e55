"""Group norm, attention and the gated feed-forward after one another, forward and backward, as the blocks of the
denoiser use them: one stream, one workspace, directly and as a captured graph, against the chain in 64 bits.

Tolerance as a relative 2-norm: each rounding to the type moves a value by at most half a step u, and the norm of what
it moves behind it by as much. Forward, y: h, P, o, v and z of the feed-forward (one), v act(z), y: 6 u, and q and k's
through scores of size one into P: 2 u. Backward: dpre, dh of the product (one), d o, dS, dq, dk, dv, their sum, dx:
9 u on top of those 8 of the values that the gradients are taken at."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import operator_refs as R  # noqa: E402
from latent_diffusion_net_b200 import binding as B  # noqa: E402

BATCH, ROWS, HEADS, D = 2, 333, 5, 64
C, HIDDEN, GROUPS, EPS = HEADS * D, 4 * HEADS * D, 32, 1e-5
DT = {"bf16": (torch.bfloat16, B.SD_DTYPE_BF16), "f16": (torch.float16, B.SD_DTYPE_F16)}


def tensors(t):
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(t)  # noqa: E731
    p = {"x": n(BATCH, ROWS, C) + 0.5, "gamma": 1 + n(C, std=0.1), "beta": n(C, std=0.1), "w1": n(2 * HIDDEN, C, std=C ** -0.5),
         "b1": n(2 * HIDDEN, std=0.1), "w2": n(C, HIDDEN, std=HIDDEN ** -0.5), "b2": n(C, std=0.1), "dy": n(BATCH, ROWS, C)}
    doc = torch.zeros(BATCH, ROWS, dtype=torch.int32, device="cuda")
    doc[:, 150:] = 1
    lens = torch.tensor([ROWS, ROWS - 60], dtype=torch.int32, device="cuda")
    return p, doc, lens


class Block:
    def __init__(self, dt, p, doc, lens):
        t, code = DT[dt]
        self.p = p
        self.gn = B.group_norm_cfg(BATCH, ROWS, C, groups=GROUPS, eps=EPS, act=B.SD_ACT_SILU, dtype=code)
        self.at = B.attention_cfg(BATCH, ROWS, ROWS, HEADS, HEADS, D, dtype=code)
        self.ff = B.gated_ff_cfg(BATCH * ROWS, C, HIDDEN, act=B.SD_ACT_GELU, dtype=code)
        self.masks = B.attention_masks(k_lens=lens, q_doc=doc, k_doc=doc)
        self.keep = (doc, lens)
        n = max(B.sd_group_norm_workspace_size(self.gn), B.sd_attention_workspace_size(self.at),
                B.sd_gated_ff_workspace_size(self.ff))
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        e = lambda *s, t=t: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        f = torch.float32
        self.h, self.o, self.y, self.do, self.dh, self.dx = (e(BATCH, ROWS, C) for _ in range(6))
        self.dq, self.dk, self.dv = (e(BATCH, ROWS, C) for _ in range(3))
        self.pre, self.stats, self.lse = e(BATCH * ROWS, 2 * HIDDEN), e(BATCH, GROUPS, 2, t=f), e(BATCH, HEADS, ROWS, t=f)
        self.dgamma, self.dbeta = e(C, t=f), e(C, t=f)
        self.dw1, self.db1, self.dw2, self.db2 = (torch.full_like(p[n], float("nan")) for n in ("w1", "b1", "w2", "b2"))

    def run(self, st):
        p, w, n = self.p, self.ws, self.ws.numel()
        B.sd_group_norm_fwd(self.gn, p["x"], p["gamma"], p["beta"], self.h, self.stats, w, n, st)
        B.sd_attention_fwd(self.at, self.h, self.h, self.h, self.masks, self.o, self.lse, w, n, st)
        B.sd_gated_ff_fwd(self.ff, p["w1"], p["b1"], p["w2"], p["b2"], self.o, self.pre, self.y, w, n, st)
        B.sd_gated_ff_bwd(self.ff, p["w1"], p["w2"], self.o, self.pre, p["dy"], self.do, self.dw1, self.db1, self.dw2,
                          self.db2, w, n, st)
        B.sd_attention_bwd(self.at, self.h, self.h, self.h, self.masks, self.o, self.lse, self.do, self.dq, self.dk,
                           self.dv, w, n, st)
        self.dh.copy_(self.dq.float() + self.dk.float() + self.dv.float())
        B.sd_group_norm_bwd(self.gn, p["x"], p["gamma"], p["beta"], self.stats, self.dh, self.dx, self.dgamma, self.dbeta,
                            w, n, st)
        return {n: getattr(self, n) for n in ("y", "dx", "dgamma", "dbeta", "dw1", "db1", "dw2", "db2")}


def reference(p, doc, lens):
    leaf = {n: t.double().requires_grad_() for n, t in p.items() if n != "dy"}
    h, _, _ = R.group_norm(leaf["x"], leaf["gamma"], leaf["beta"], GROUPS, EPS, "silu")
    qkv = h.reshape(BATCH, ROWS, HEADS, D)
    o, _ = R.attention(qkv, qkv, qkv, k_lens=lens, q_doc=doc, k_doc=doc)
    y, _ = R.gated_ff(o.reshape(BATCH * ROWS, C), leaf["w1"], leaf["b1"], leaf["w2"], leaf["b2"], "gelu")
    y = y.reshape(BATCH, ROWS, C)
    y.backward(p["dy"].double())
    return {"y": y.detach(), **{"d" + n: t.grad for n, t in leaf.items()}}


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_block_forward_and_backward(dt):
    t = DT[dt][0]
    p, doc, lens = tensors(t)
    block = Block(dt, p, doc, lens)
    got = block.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert B.sd_query_device_status(block.ws) == 0
    want, u = reference(p, doc, lens), R.HALF_STEP[t]
    for name, value in want.items():
        err, tol = R.rel(got[name], value), (8 if name == "y" else 17) * u
        assert err < tol, (name, err, tol)

    # the same calls captured, on new inputs in the same places
    first = {n: v.clone() for n, v in got.items()}
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        got = block.run(s)
    x = p["x"].clone()
    p["x"].copy_(x.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    other = {n: v.clone() for n, v in got.items()}
    assert not torch.equal(other["y"], first["y"])
    p["x"].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    for name, value in first.items():
        assert torch.equal(got[name], value), name
    assert B.sd_query_device_status(block.ws) == 0
