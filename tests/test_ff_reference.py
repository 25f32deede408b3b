"""The 64-bit reference of the feed-forward operators (tests/_ff.py) on the
CPU: the 8-bit format against torch's own 8-bit types, the gradients against
differences; and what the entry points refuse before any launch."""
import pytest
import torch

from tests import _ff as ff


@pytest.mark.parametrize("fmt,dtype", [(0, torch.float8_e4m3fn), (1, torch.float8_e5m2)])
def test_codes_are_torchs(fmt, dtype):
    every = torch.arange(256, dtype=torch.uint8)
    want = every.view(dtype).double()
    got = ff.code_values(every, fmt)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(got[fine], want[fine])
    g = torch.Generator().manual_seed(fmt)
    v = torch.randn(7, 400, generator=g).to(torch.bfloat16).double()
    v[1] *= 2.0 ** -60
    v[2, :128] = 0
    v[3, 5] = 448.0
    v[4, 200] = -57344.0
    q, s = ff.encode(v, fmt)
    e = ff.read_scales(s, 7, 400)
    want = (v * ff.pow2(-e).repeat_interleave(128, 1)[:, :400]).float().to(dtype).view(torch.uint8)
    assert torch.equal(q, want)
    a = ff.blocks(v).abs().amax(2)
    assert bool((a <= ff.FMAX[fmt] * ff.pow2(e)).all())
    assert bool(((a > ff.FMAX[fmt] * ff.pow2(e - 1)) | (e == -127)).all())


def test_scale_tiles_are_a_permutation():
    at = ff.tile_index(256, 1024, "cpu").flatten()
    assert sorted(at.tolist()) == list(range(4 * 512))
    # (row 33, block 2) of a narrow matrix: lane 1, second group of rows, third byte
    assert int(ff.tile_index(40, 384, "cpu")[33, 2]) == 16 + 4 + 2


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_gated_gradient_against_differences(kind):
    g = torch.Generator().manual_seed(kind)
    x, w, dh = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 24), (32, 24), (5, 16)))
    _, gg, u, _, _ = ff.gated_fwd(x, w, kind)
    dx, dw, _, _ = ff.gated_bwd(dh, x, gg, u, w, kind)
    for which, grad in ((0, dx), (1, dw)):
        v = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        t = 1e-6
        up, dn = ((x + t * v, w) if which == 0 else (x, w + t * v) for t in (t, -t))
        diff = ((ff.gated_fwd(*up, kind)[0] - ff.gated_fwd(*dn, kind)[0]) * dh).sum() / (2 * t)
        assert abs(float((grad * v).sum() - diff)) < 1e-6 * float(grad.norm() * v.norm())


def test_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(4)
    s, dy, dsum = (torch.randn(3, 40, generator=g, dtype=torch.float64) for _ in range(3))
    gamma = torch.randn(40, generator=g, dtype=torch.float64)
    _, r = ff.norm_fwd(s, gamma, 1e-5)
    dx, dgamma = ff.norm_bwd(dy, dsum, s, gamma, r)
    v, vg = torch.randn(3, 40, generator=g, dtype=torch.float64), torch.randn(40, generator=g, dtype=torch.float64)

    def loss(s, gamma):
        return float((ff.norm_fwd(s, gamma, 1e-5)[0] * dy).sum() + (s * dsum).sum())

    t = 1e-6
    assert abs((loss(s + t * v, gamma) - loss(s - t * v, gamma)) / (2 * t) - float((dx * v).sum())) < 1e-6 * float(dx.norm() * v.norm())
    assert abs((loss(s, gamma + t * vg) - loss(s, gamma - t * vg)) / (2 * t) - float((dgamma * vg).sum())) < 1e-6 * float(dgamma.norm() * vg.norm())


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def ax():
    from deep_cnn_image_b200 import alexnet
    return alexnet


P, BIG = 4096, 1 << 40  # an aligned stand-in for a pointer, more than any workspace


def test_sizes(ax):
    assert ax.f8_scale_bytes(1, 16) == 512
    assert ax.f8_scale_bytes(129, 528) == 2 * 2 * 512
    for r, c in ((0, 16), (1, 0), (1, 24), (-1, 16)):
        assert ax.f8_scale_bytes(r, c) == 0
    assert ax.rmsnorm_workspace_bytes(1, 8) > 0
    for r, c in ((0, 8), (1, 12), (1, 65544), (1 << 31, 8)):
        assert ax.rmsnorm_workspace_bytes(r, c) == 0
    assert ax.fc_f8_workspace_bytes(1, 16, 8) > 0
    for s in ((0, 16, 8), (1, 24, 8), (1, 16, 12), (1, 0, 8), (1, 1 << 25, 8), ((1 << 30) + 1, 16, 8)):
        assert ax.fc_f8_workspace_bytes(*s) == 0
    assert ax.gated_workspace_bytes(1, 8, 8) > 0
    for s in ((0, 8, 8), (1, 12, 8), (1, 8, 12), (1, 1 << 25, 8), (1, 8, 1 << 25), ((1 << 30) + 1, 8, 8)):
        assert ax.gated_workspace_bytes(*s) == 0


def _refused(ax, name, good, changes, unsupported=()):
    f = getattr(ax.lib, name)
    for i, v in changes:
        a = list(good)
        a[i] = v
        assert f(*a) == ax.ERR_INVALID_ARG, (name, i, v)
    for i, v in unsupported:
        a = list(good)
        a[i] = v
        assert f(*a) == ax.ERR_UNSUPPORTED, (name, i, v)


def test_refusals(ax):
    _refused(ax, "alexnet_op_f8_quant", [P, 4, 16, 0, P, P, None],
             [(0, None), (0, P + 8), (1, 0), (2, 0), (2, 24), (3, 2), (3, -1), (4, None), (4, P + 2), (5, None), (5, P + 4)])
    _refused(ax, "alexnet_op_f8_dequant", [P, P, 4, 16, 0, P, None],
             [(0, None), (0, P + 8), (1, None), (1, P + 1), (2, 0), (3, 8), (4, 2), (5, None), (5, P + 2)])
    _refused(ax, "alexnet_op_rmsnorm_fwd", [P, P, P, 4, 16, 1e-5, P, P, P, P, P, None],
             [(0, None), (0, P + 2), (1, P + 2), (2, None), (2, P + 4), (3, 0), (4, 0), (4, 24), (4, 12), (5, 0.0), (5, -1.0),
              (5, float("nan")), (6, P + 2), (7, P + 2), (8, P + 4), (9, None), (9, P + 1), (10, None), (10, P + 1)],
             [(4, 65552), (3, 1 << 31)])
    _refused(ax, "alexnet_op_rmsnorm_bwd", [P, P, P, P, P, 4, 16, P, P, P, BIG, None],
             [(0, None), (0, P + 2), (1, P + 2), (2, None), (3, None), (4, None), (5, 0), (6, 12), (7, None), (7, P + 2), (8, P + 4),
              (9, None), (9, P + 4), (10, 0)],
             [(6, 65544), (5, 1 << 31)])
    _refused(ax, "alexnet_op_fc_f8_fwd", [P, P, 0, 4, 32, P, P, 1, 8, 1, P, P, BIG, None],
             [(0, None), (0, P + 8), (1, None), (1, P + 8), (2, 2), (3, 0), (4, 24), (4, 0), (5, None), (5, P + 8), (6, None), (6, P + 8),
              (7, -1), (8, 12), (8, 0), (9, 2), (10, None), (10, P + 8), (11, None), (11, P + 8), (12, 0)],
             [(3, (1 << 30) + 1), (4, 1 << 25), (8, 1 << 25)])
    _refused(ax, "alexnet_op_gated_fwd", [P, 4, 16, P, 8, 0, P, 1, P, P, BIG, None],
             [(0, None), (0, P + 8), (1, 0), (2, 12), (2, 0), (3, None), (3, P + 8), (4, 12), (4, 0), (5, 3), (5, -1), (6, None), (6, P + 8),
              (7, 2), (8, P + 8), (9, None), (9, P + 8), (10, 0)],
             [(2, 1 << 25), (4, 1 << 25)])
    _refused(ax, "alexnet_op_gated_bwd", [P, P, 0, P, 4, 16, P, 8, 0, P, P, P, BIG, None],
             [(0, None), (0, P + 8), (1, None), (1, P + 8), (2, -1), (3, None), (3, P + 8), (4, 0), (5, 12), (6, None), (7, 12), (8, 3),
              (9, P + 8), (10, P + 8), (11, None), (11, P + 8), (12, 0)],
             [(4, (1 << 30) + 1), (5, 1 << 25), (7, 1 << 25)])
    _refused(ax, "alexnet_op_gated_fwd_ckpt8", [P, 4, 16, P, 16, 0, P, P, P, P, BIG, None],
             [(0, None), (1, 0), (2, 24), (3, None), (4, 24), (5, 3), (6, None), (7, None), (7, P + 8), (8, None), (8, P + 8), (9, None),
              (10, 0)],
             [(2, 1 << 25), (4, 1 << 25)])
    _refused(ax, "alexnet_op_gated_bwd_ckpt8", [P, P, P, P, P, 4, 16, P, 16, 0, P, P, P, BIG, None],
             [(0, None), (1, None), (1, P + 8), (2, None), (2, P + 8), (3, None), (4, None), (5, 0), (6, 24), (7, None), (8, 24), (9, -1),
              (10, P + 8), (11, P + 8), (12, None), (13, 0)],
             [(6, 1 << 25), (8, 1 << 25)])
