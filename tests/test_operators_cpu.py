"""The standalone operators refuse bad calls on the host, before any launch; their
workspace sizes are host arithmetic. No GPU is needed: a call whose arguments
are in order ends with SD_ERR_NOT_SM100 or SD_ERR_LAUNCH where there is none."""
import pytest

from latent_diffusion_net_b200 import binding as B

P = 4096  # an aligned address that is never read: every call here is refused, or meets no device
OK, NULL, SHAPE, UNSUPPORTED, MISALIGNED, SMALL = 0, 1, 2, 3, 4, 5
NO_DEVICE = (6, 7)


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_diffusion_net_b200 import build
    build.build()
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where there is no GPU")


def gn_fwd(cfg, x=P, y=P, ws=P, n=None, stats=None):
    n = B.sd_group_norm_workspace_size(cfg) if n is None else n
    return B.sd_group_norm_fwd(cfg, x, None, None, y, stats, ws, n, check=False)


def gn_bwd(cfg, x=P, stats=P, dy=P, dx=P, ws=P, n=None):
    n = B.sd_group_norm_workspace_size(cfg) if n is None else n
    return B.sd_group_norm_bwd(cfg, x, None, None, stats, dy, dx, None, None, ws, n, check=False)


def test_group_norm_refusals():
    ok = B.group_norm_cfg(2, 100, 64)
    size = B.sd_group_norm_workspace_size(ok)
    assert size > 0
    assert gn_fwd(ok) in NO_DEVICE and gn_bwd(ok) in NO_DEVICE
    assert gn_fwd(ok, x=None) == NULL and gn_fwd(ok, y=None) == NULL and gn_fwd(ok, ws=None) == NULL
    assert gn_bwd(ok, stats=None) == NULL and gn_bwd(ok, dy=None) == NULL and gn_bwd(ok, dx=None) == NULL
    assert gn_fwd(ok, x=P + 8) == MISALIGNED and gn_fwd(ok, stats=P + 4) == MISALIGNED
    assert gn_fwd(ok, n=size - 1) == SMALL and gn_bwd(ok, n=0) == SMALL
    for bad, code in [(B.group_norm_cfg(-1, 100, 64), SHAPE), (B.group_norm_cfg(1, -1, 64), SHAPE),
                      (B.group_norm_cfg(1, 10, 0), SHAPE), (B.group_norm_cfg(1, 10, 65), SHAPE),
                      (B.group_norm_cfg(1, 10, 64, groups=0), SHAPE), (B.group_norm_cfg(1, 10, 64, eps=0.0), SHAPE),
                      (B.group_norm_cfg(1, 10, 64, eps=float("nan")), SHAPE),
                      (B.group_norm_cfg(1, 10, 64, ld_x=63), SHAPE), (B.group_norm_cfg(1, 10, 64, ld_y=8), SHAPE),
                      (B.group_norm_cfg(1, 10, 8224), UNSUPPORTED), (B.group_norm_cfg(1, 10, 64, act=3), UNSUPPORTED),
                      (B.group_norm_cfg(1, 10, 64, dtype=3), UNSUPPORTED),
                      (B.group_norm_cfg(1, 10, 64, act=-1), UNSUPPORTED)]:
        assert gn_fwd(bad, n=1 << 30) == code and gn_bwd(bad, n=1 << 30) == code
        assert B.sd_group_norm_workspace_size(bad) == 0
    assert gn_fwd(B.group_norm_cfg(0, 10, 64), x=None, y=None, ws=None) == OK
    assert B.lib().sd_group_norm_fwd(None, P, None, None, P, None, P, 1, None) == NULL


def ff_fwd(cfg, w1=P, w2=P, x=P, y=P, ws=P, n=None, b1=None, pre=None):
    n = B.sd_gated_ff_workspace_size(cfg) if n is None else n
    return B.sd_gated_ff_fwd(cfg, w1, b1, w2, None, x, pre, y, ws, n, check=False)


def ff_bwd(cfg, w1=P, w2=P, x=P, pre=P, dy=P, dx=P, ws=P, n=None, db1=None):
    n = B.sd_gated_ff_workspace_size(cfg) if n is None else n
    return B.sd_gated_ff_bwd(cfg, w1, w2, x, pre, dy, dx, None, db1, None, None, ws, n, check=False)


def test_gated_ff_refusals():
    ok = B.gated_ff_cfg(100, 64, 128)
    size = B.sd_gated_ff_workspace_size(ok)
    assert ff_fwd(ok) in NO_DEVICE and ff_bwd(ok) in NO_DEVICE
    for name in ("w1", "w2", "x", "y", "ws"):
        assert ff_fwd(ok, **{name: None}) == NULL, name
    for name in ("w1", "w2", "x", "pre", "dy", "ws"):
        assert ff_bwd(ok, **{name: None}) == NULL, name
    assert ff_fwd(ok, b1=P + 2) == MISALIGNED and ff_fwd(ok, pre=P + 8) == MISALIGNED
    assert ff_bwd(ok, db1=P + 2) == MISALIGNED
    assert ff_fwd(ok, n=size - 1) == SMALL and ff_bwd(ok, n=size - 1) == SMALL
    assert ff_bwd(ok, dx=None) == OK  # no gradient asked for
    for bad, code in [(B.gated_ff_cfg(-1, 64, 128), SHAPE), (B.gated_ff_cfg(1, 0, 128), SHAPE),
                      (B.gated_ff_cfg(1, 64, 0), SHAPE), (B.gated_ff_cfg(1, 64, 128, d_out=0), SHAPE),
                      (B.gated_ff_cfg(1, 60, 128), UNSUPPORTED), (B.gated_ff_cfg(1, 64, 132), UNSUPPORTED),
                      (B.gated_ff_cfg(1, 64, 128, d_out=4), UNSUPPORTED),
                      (B.gated_ff_cfg(1, 64, 128, dtype=B.SD_DTYPE_F32), UNSUPPORTED),
                      (B.gated_ff_cfg(1, 64, 128, act=7), UNSUPPORTED)]:
        assert ff_fwd(bad, n=1 << 40) == code and ff_bwd(bad, n=1 << 40) == code
        assert B.sd_gated_ff_workspace_size(bad) == 0
    assert ff_fwd(B.gated_ff_cfg(0, 64, 128), w1=None, w2=None, x=None, y=None, ws=None) == OK


def test_workspaces_cover_every_size():
    """Sizes grow with nothing hidden: a call's scratch is part of what the size function says."""
    for m in (1, 77, 4096, 1 << 20):
        cfg = B.gated_ff_cfg(m, 320, 1280)
        assert B.sd_gated_ff_workspace_size(cfg) >= m * 1280 * 2 * 3
    for n, r in ((1, 1), (64, 4096), (4096, 1)):
        cfg = B.group_norm_cfg(n, r, 320)
        assert B.sd_group_norm_workspace_size(cfg) >= n * 32 * 8


def at_fwd(cfg, q=P, k=P, v=P, o=P, ws=P, n=None, masks=None, lse=None):
    n = B.sd_attention_workspace_size(cfg) if n is None else n
    return B.sd_attention_fwd(cfg, q, k, v, masks, o, lse, ws, n, check=False)


def at_bwd(cfg, q=P, k=P, v=P, o=P, lse=P, d_o=P, dq=P, dk=P, dv=P, ws=P, n=None, masks=None):
    n = B.sd_attention_workspace_size(cfg) if n is None else n
    return B.sd_attention_bwd(cfg, q, k, v, masks, o, lse, d_o, dq, dk, dv, ws, n, check=False)


def test_attention_refusals():
    ok = B.attention_cfg(2, 100, 200, 8, 2, 64, causal=True)
    size = B.sd_attention_workspace_size(ok)
    assert at_fwd(ok) in NO_DEVICE and at_bwd(ok) in NO_DEVICE
    for name in ("q", "k", "v", "o", "ws"):
        assert at_fwd(ok, **{name: None}) == NULL, name
    for name in ("q", "k", "v", "o", "lse", "d_o", "dq", "dk", "dv", "ws"):
        assert at_bwd(ok, **{name: None}) == NULL, name
        assert at_bwd(ok, **{name: P + 8}) == MISALIGNED, name
    assert at_fwd(ok, lse=P + 4) == MISALIGNED
    assert at_fwd(ok, n=size - 1) == SMALL and at_bwd(ok, n=size - 1) == SMALL
    c = B.attention_cfg
    for bad, code in [(c(-1, 1, 1, 1), SHAPE), (c(1, -1, 1, 1), SHAPE), (c(1, 1, -1, 1), SHAPE), (c(1, 1, 1, 0), SHAPE),
                      (c(1, 1, 1, 8, 3), SHAPE), (c(1, 1, 1, 8, 0), SHAPE), (c(1, 1, 1, 1, 1, 0), SHAPE),
                      (c(1, 1, 1, 1, 1, 64, scale=-1.0), SHAPE), (c(1, 1, 1, 1, 1, 64, scale=float("nan")), SHAPE),
                      (c(1, 1, 1, 1, 1, 64, scale=1e30), SHAPE), (c(1, 1, 1, 1, 1, 64, softcap=-1.0), SHAPE),
                      (c(1, 1, 1, 1, 1, 64, softcap=float("inf")), SHAPE),
                      (c(1, 1, 1, 1, 1, 60), UNSUPPORTED), (c(1, 1, 1, 1, 1, 136), UNSUPPORTED),
                      (c(1, 1, 1, 256, 1, 64), UNSUPPORTED), (c(1, 1, (1 << 20) + 1, 1), UNSUPPORTED),
                      (c(1, (1 << 20) + 1, 1, 1), UNSUPPORTED), (c(1, 1, 1, 1, dtype=B.SD_DTYPE_F32), UNSUPPORTED),
                      # strides: steps of 16 bytes, never backwards, never in place where there is more than one
                      (c(2, 4, 4, 2, q_stride=(512, 128, 60)), SHAPE), (c(2, 4, 4, 2, k_stride=(512, 0, 64)), SHAPE),
                      (c(2, 4, 4, 2, v_stride=(-512, 128, 64)), SHAPE),
                      (c(2, 4, 4, 2, o_stride=(1 << 40, 128, 64)), SHAPE)]:
        assert at_fwd(bad, n=1 << 40) == code and at_bwd(bad, n=1 << 40) == code
        assert B.sd_attention_workspace_size(bad) == 0
    # a stride that is never stepped may be anything
    assert at_fwd(c(1, 1, 4, 2, q_stride=(0, 0, 64)), n=1 << 40) in NO_DEVICE
    m = B.attention_masks
    assert at_fwd(ok, masks=m(q_doc=P)) == NULL and at_fwd(ok, masks=m(k_doc=P)) == NULL
    assert at_fwd(ok, masks=m(k_lens=P + 4)) == MISALIGNED and at_bwd(ok, masks=m(slopes=P + 4)) == MISALIGNED
    assert at_fwd(c(2, 100, 200, 8, 2, 64), masks=m(prefix=P)) == SHAPE  # a prefix without a causal mask
    assert at_fwd(ok, masks=m(prefix=P, k_lens=P, q_doc=P, k_doc=P, slopes=P)) in NO_DEVICE
    assert at_fwd(c(0, 4, 4, 1), q=None, k=None, v=None, o=None, ws=None) == OK
    assert at_fwd(c(1, 0, 4, 1), q=None, k=None, v=None, o=None, ws=None) == OK


def test_attention_sizes_beyond_the_grid_are_refused():
    """Query rows and key rows of all sequences and heads together have to stay countable."""
    for cfg in (B.attention_cfg(4096, 1, 1 << 20, 4096, 4096, 8), B.attention_cfg(4096, 1 << 20, 1, 4096, 1, 8),
                B.attention_cfg(1 << 13, 1, 1, 1 << 12, 1, 8)):
        assert B.sd_attention_workspace_size(cfg) == 0
