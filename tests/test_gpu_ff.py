"""The feed-forward operators on the GPU against their formulas in 64 bits
(tests/_ff.py, which also derives the bounds), element by element: every
variant's sizes, odd and ragged ones, values that are not finite, streams,
captured graphs, and a run of all of them together."""
import pytest

from tests import _ff as ff

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def ax():
    from deep_cnn_image_b200 import alexnet
    return alexnet


class Buf:
    """A tensor between two guard regions of 0xA5 (or NaN for inputs: a read
    outside shows in the result)."""
    made = []

    def __init__(self, shape, dtype, fill=0xA5, like=None):
        import torch
        n = 1
        for d in shape:
            n *= d
        size = n * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((256 + size + 256,), fill, dtype=torch.uint8, device="cuda")
        self.size, self.fill = size, fill
        self.t = self.raw[256:256 + size].view(dtype).view(*shape)
        if like is not None:
            self.t.copy_(like)
        Buf.made.append(self)

    def intact(self):
        return bool((self.raw[:256] == self.fill).all()) and bool((self.raw[256 + self.size:] == self.fill).all())


@pytest.fixture(autouse=True)
def guards():
    Buf.made.clear()
    yield
    import torch
    torch.cuda.synchronize()
    assert all(b.intact() for b in Buf.made), "a guard region was written"
    Buf.made.clear()


def bf16(t):
    import torch
    return Buf(t.shape, torch.bfloat16, 0xFF, t.to(torch.bfloat16)).t


def u8(t):
    import torch
    return Buf(t.shape, torch.uint8, 0xFF, t).t


def f32(t):
    import torch
    return Buf(t.shape, torch.float32, 0xFF, t).t


def out(shape, dtype="bfloat16"):
    import torch
    return Buf(shape, getattr(torch, dtype)).t


def work(n):
    return out((n,), "uint8")


def randn(seed, *shape, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * scale


def spread(seed, rows, cols):
    """Normal values with some columns and rows far larger or smaller."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + 99)
    c = torch.exp2(torch.randint(-6, 7, (cols,), generator=g, device="cuda").float())
    r = torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g, device="cuda").float())
    return randn(seed, rows, cols) * c * r


def within(got, want, slack, unit=ff.U_BF16):
    """got = want rounded to a type of the given unit, computed to within
    `slack` before the rounding."""
    import torch
    got = got.double()
    tol = slack * (1 + unit) + unit * want.abs() + 2.0 ** -133
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), "%d of %d outside, worst %.3g of its bound" % (
        int(bad.sum()), bad.numel(), float(((got - want).abs() / tol).nan_to_num(nan=float("inf")).max()))
    assert bool(torch.isfinite(got).all())


def status(ws):
    import torch
    torch.cuda.synchronize()
    return int(ws[:4].clone().view(torch.int32)[0])


# ------------------------------------------------------------------ 8-bit rows
ROWS = [(1, 16), (1, 4096), (3, 144), (127, 512), (129, 528), (300, 1008), (17, 9216), (1000, 128)]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("R,C", ROWS)
def test_quant_dequant(ax, R, C, fmt):
    import torch
    v = spread(R + C, R, C)
    v[R // 2, : min(C, 128)] = 0
    v[R - 1, C - 1] = ff.FMAX[fmt]
    x = bf16(v)
    q, s, y = out((R, C), "uint8"), out((ax.f8_scale_bytes(R, C),), "uint8"), out((R, C))
    before = s.clone()
    ax.op_f8_quant(x, R, C, fmt, q, s)
    ax.op_f8_dequant(q, s, R, C, fmt, y)
    wq, ws = ff.encode(x.double(), fmt)
    assert torch.equal(q, wq)
    at = ff.tile_index(R, C, "cuda").flatten()
    assert torch.equal(s[at], ws[at])
    rest = torch.ones_like(s, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(s[rest], before[rest])
    assert torch.equal(y.double(), ff.values(q, s, fmt))


@pytest.mark.parametrize("fmt", [0, 1])
def test_quant_extremes(ax, fmt):
    """NaN stays, an infinity becomes NaN, neither counts for the scale; the
    largest and smallest blocks; subnormal inputs."""
    import torch
    R, C = 6, 272
    v = randn(3, R, C)
    v[0, 5], v[0, 200], v[1, 7], v[1, 271] = float("nan"), float("nan"), float("inf"), float("-inf")
    v[2] = float("nan")
    v[3, :128] = 3.3895e38
    v[4] *= 2.0 ** -133
    v[5] *= 2.0 ** -120
    x = bf16(v)
    q, s, y = out((R, C), "uint8"), out((ax.f8_scale_bytes(R, C),), "uint8"), out((R, C))
    ax.op_f8_quant(x, R, C, fmt, q, s)
    ax.op_f8_dequant(q, s, R, C, fmt, y)
    d = x.double()
    lost = ~torch.isfinite(d)
    at = ff.tile_index(R, C, "cuda")
    e = ff.exponents(d, fmt)
    assert torch.equal(s[at].int() - 127, e)
    fine = torch.where(lost, torch.zeros_like(d), d)
    wq, _ = ff.encode(fine, fmt)
    assert torch.equal(q[~lost], wq[~lost])
    assert bool(torch.isnan(ff.code_values(q, fmt)[lost]).all()) and bool(torch.isnan(y[lost]).all())
    # what lies under bf16's normal range may be rounded once more, and the
    # code of the largest block, 256 * 2^120 = 2^128, is past bf16's largest value
    want = ff.values(q, s, fmt)
    over = (want.abs() >= 2.0 ** 128) & ~lost
    assert bool(over[3, :128].all()) and bool((y[over].double() == torch.sign(want[over]) * float("inf")).all())
    assert bool(((y.double() - want).abs() <= 2.0 ** -134)[~lost & ~over].all())


# ------------------------------------------------------------------ norm
NORM = [(1, 8), (1, 4096), (5, 72), (33, 256), (9, 520), (17, 1024), (7, 1040), (65, 2048), (6, 4112), (3, 8192), (2, 9216),
        (2, 16400), (2, 40000), (1, 65536), (700, 64)]


def _norm_in(R, C):
    x, res = bf16(randn(R, R, C)), bf16(spread(C, R, C) * 0.25)
    return x, res, f32(1 + 0.3 * randn(7, C))


@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("R,C", NORM)
def test_norm_forward(ax, R, C, with_res):
    import torch
    x, res, gamma = _norm_in(R, C)
    res = res if with_res else None
    eight = C % 16 == 0
    s, y, r = out((R, C)), out((R, C)), out((R,), "float32")
    q = out((R, C), "uint8") if eight else None
    sc = out((ax.f8_scale_bytes(R, C),), "uint8") if eight else None
    ax.op_rmsnorm_fwd(x, res, gamma, R, C, EPS, s, y, r, q, sc)
    want = x.double() + (res.double() if with_res else 0)
    within(s, want, U32 * want.abs())
    # the statistic of the stored s: a sum of C squares, the quotient, the root
    d = s.double()
    wy, wr = ff.norm_fwd(d, gamma.double(), EPS)
    rel = (C // 8 / 32 + 40) * ff.U_F32
    within(r, wr, rel * wr, unit=ff.U_F32)
    slack = (rel + 4 * ff.U_F32) * wy.abs()
    within(y, wy, slack)
    if eight:
        e, we = ff.read_scales(sc, R, C), ff.exponents(wy)
        a = ff.blocks(wy).abs().amax(2)
        for shift in (-1, 1):  # another scale only where the maximum is next to its border
            other = e == we + shift
            edge = ff.FMAX[0] * ff.pow2(torch.minimum(e, we))
            assert bool((((a - edge).abs() <= 2 * rel * edge) | ~other).all())
        assert bool(((e - we).abs() <= 1).all())
        assert bool(((ff.values(q, sc) - wy).abs() <= (1 + ff.U_E4M3) * slack + ff.U_E4M3 * wy.abs() + ff.code_slack(e, C)).all())


U32 = ff.U_F32


@pytest.mark.parametrize("R,C", [(4096, 4096), (30000, 256), (20000, 512), (500, 16400), (100, 65536), (65536, 16)])
def test_norm_codes_are_rounded_once(ax, R, C):
    """Codes and scales are those of y in 64 bits, next to a border between
    two of them as well: y comes from a sum of squares in 64 bits and a
    reciprocal root good to 2^-42.  A border every 2^-4 of a value at the
    closest: of 2^24 values 2^24 * 2 * 2^-42 * 2^4, one in 8000 runs, may lie
    that near to one; in 32 bits about ten do."""
    import torch
    x, res, gamma = _norm_in(R, C)
    x[R // 2] = 0
    res[R // 2] = 0
    s, y, y2 = out((R, C)), out((R, C)), out((R, C))
    q, sc = out((R, C), "uint8"), out((ax.f8_scale_bytes(R, C),), "uint8")
    ax.op_rmsnorm_fwd(x, res, gamma, R, C, EPS, s, y, None, q, sc)
    ax.op_rmsnorm_fwd(x, res, gamma, R, C, EPS, None, y2, None, None, None)
    eps = torch.tensor(EPS, dtype=torch.float32).item()  # as the call hands it over
    wy, _ = ff.norm_fwd(s.double(), gamma.double(), eps)
    wq, ws = ff.encode(wy)
    assert torch.equal(ff.read_scales(sc, R, C), ff.read_scales(ws, R, C))
    assert torch.equal(q, wq)
    assert torch.equal(y, y2)  # asking for codes changes nothing else


@pytest.mark.parametrize("C", [64, 512, 4096, 9216, 40000])
def test_norm_range_and_values_not_finite(ax, C):
    """Rows far outside what squares fit in 32 bits; a NaN takes its row, an
    infinity leaves 1/inf = 0 of the others and 0 * inf of itself; a y beyond
    32 bits (through gamma) is NaN among the codes and nothing of the rest."""
    import torch
    R, eps = 7, 2.0 ** -120
    x = randn(C, R, C)
    x[0, 3] = float("nan")
    x[1, 5] = float("inf")
    x[2] *= 2.0 ** 100
    x[3] *= 2.0 ** -70
    x[4] = 0
    x[5, 9] = -0.0
    x, gamma = bf16(x), f32(1 + 0.3 * randn(7, C).abs())
    s, y, r = out((R, C)), out((R, C)), out((R,), "float32")
    q, sc = out((R, C), "uint8"), out((ax.f8_scale_bytes(R, C),), "uint8")
    ax.op_rmsnorm_fwd(x, None, gamma, R, C, eps, s, y, r, q, sc)
    wy, wr = ff.norm_fwd(x.double(), gamma.double(), eps)
    assert bool(torch.isnan(r[0])) and float(r[1]) == 0
    within(r[1:], wr[1:], 2 * U32 * wr[1:], unit=U32)
    lost = torch.isnan(wy)
    assert bool(lost[0].all()) and int(lost[1].sum()) == 1 and not bool(lost[2:].any())
    assert torch.equal(torch.isnan(y), lost) and torch.equal(torch.isnan(ff.code_values(q)), lost)
    wq, ws = ff.encode(torch.where(lost, torch.zeros_like(wy), wy))
    assert torch.equal(ff.read_scales(sc, R, C), ff.read_scales(ws, R, C))
    assert torch.equal(q[~lost], wq[~lost])
    within(y[~lost], wy[~lost], 4 * U32 * wy[~lost].abs())
    gamma[2], gamma[C - 3] = 3e38, -3e38
    x[6, 2], x[6, C - 3] = 300.0, 300.0
    ax.op_rmsnorm_fwd(x, None, gamma, R, C, eps, s, y, r, q, sc)
    wy, _ = ff.norm_fwd(x.double(), gamma.double(), eps)
    over = torch.tensor([2, C - 3], device="cuda")
    assert bool((wy[6, over].abs() > 3.41e38).all())
    assert bool(torch.isinf(y[6, over]).all()) and bool(torch.isnan(ff.code_values(q)[6, over]).all())
    assert int(torch.isnan(ff.code_values(q)[6]).sum()) == 2 and int(torch.isinf(y[6]).sum()) == 2


def test_norm_forward_in_place(ax):
    import torch
    R, C = 19, 1536
    x, res, gamma = _norm_in(R, C)
    want, y1, y2 = out((R, C)), out((R, C)), out((R, C))
    ax.op_rmsnorm_fwd(x, res, gamma, R, C, EPS, want, y1, None, None, None)
    for target in (x, res):
        a, b = x.clone(), res.clone()
        t = a if target is x else b
        ax.op_rmsnorm_fwd(a, b, gamma, R, C, EPS, t, y2, None, None, None)
        assert torch.equal(t, want) and torch.equal(y1, y2)


@pytest.mark.parametrize("with_sum", [True, False])
@pytest.mark.parametrize("R,C", NORM + [(1500, 1032), (1, 24)])
def test_norm_backward(ax, R, C, with_sum):
    import torch
    s, dy, dsum = bf16(spread(R, R, C)), bf16(randn(C, R, C)), bf16(randn(C + 1, R, C))
    gamma = f32(1 + 0.3 * randn(7, C))
    d = s.double()
    _, wr = ff.norm_fwd(d, gamma.double(), EPS)
    r = f32(wr.float())
    ws = work(ax.rmsnorm_workspace_bytes(R, C))
    dx, dg = out((R, C)), out((C,), "float32")
    ax.op_rmsnorm_bwd(dy, dsum if with_sum else None, s, gamma, r, R, C, dx, dg, ws)
    rd, g = r.double(), gamma.double()
    wx, wg = ff.norm_bwd(dy.double(), dsum.double() if with_sum else None, d, g, rd)
    t = dy.double() * g
    # the mean: each of C products and sums off by at most (C/256 + 40) units of the sum of magnitudes
    n = (C // 256 + 40) * ff.U_F32
    mag = rd[:, None] * (t.abs() + d.abs() * (rd ** 2)[:, None] * (t * d).abs().mean(1, keepdim=True))
    within(dx, wx, n * (mag + (dsum.double().abs() if with_sum else 0)))
    terms = (dy.double() * d * rd[:, None]).abs().sum(0)
    assert bool(((dg.double() - wg).abs() <= (R + 16) * ff.U_F32 * terms + 1e-37).all())
    # without dgamma the same dx; dx over dy and over dsum
    dx2 = out((R, C))
    ax.op_rmsnorm_bwd(dy, dsum if with_sum else None, s, gamma, r, R, C, dx2, None, ws)
    assert torch.equal(dx, dx2)
    over = dy.clone()
    ax.op_rmsnorm_bwd(over, dsum if with_sum else None, s, gamma, r, R, C, over, dg, ws)
    assert torch.equal(dx, over)
    if with_sum:
        over = dsum.clone()
        ax.op_rmsnorm_bwd(dy, over, s, gamma, r, R, C, over, dg, ws)
        assert torch.equal(dx, over)


# ------------------------------------------------------------------ 8-bit product
FC = [(1, 16, 8), (1, 4096, 1000), (2, 9216, 4096), (5, 528, 264), (16, 1024, 128), (17, 2064, 520), (33, 144, 1000), (64, 512, 2048),
      (65, 656, 136), (128, 9216, 512), (129, 1040, 136), (300, 2064, 520), (513, 384, 2056), (1025, 256, 2048), (2100, 1296, 1160)]


def _fc_in(B, In, Out, xf, wf):
    import torch
    xq, xs = ff.encode(spread(B, B, In).to(torch.bfloat16).double(), xf)
    wq, ws = ff.encode(randn(Out, Out, In).to(torch.bfloat16).double(), wf)
    return u8(xq), u8(xs), u8(wq), u8(ws)


@pytest.mark.parametrize("xf,wf", [(0, 0), (1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("B,In,Out", FC)
def test_fc_f8(ax, B, In, Out, xf, wf):
    import torch
    xq, xs, wq, ws = _fc_in(B, In, Out, xf, wf)
    x, w = ff.values(xq, xs, xf), ff.values(wq, ws, wf)
    want = x @ w.t()
    slack = ff.steps(In) * ff.ACC * (x.abs() @ w.abs().t())
    scratch = work(ax.fc_f8_workspace_bytes(B, In, Out))
    y = out((B, Out))
    ax.op_fc_f8_fwd(xq, xs, xf, B, In, wq, ws, wf, Out, ax.BF16, y, scratch)
    within(y, want, slack)
    y32 = out((B, Out), "float32")
    ax.op_fc_f8_fwd(xq, xs, xf, B, In, wq, ws, wf, Out, ax.FP32, y32, scratch)
    within(y32, want, slack, unit=ff.U_F32)
    assert torch.equal(y32.to(torch.bfloat16), y)
    assert status(scratch) == 0


@pytest.mark.parametrize("B", [3, 200])
def test_fc_f8_lost_values_stay_in_their_row(ax, B):
    import torch
    In, Out = 1040, 264
    xq, xs, wq, ws = _fc_in(B, In, Out, 0, 0)
    x, w = ff.values(xq, xs), ff.values(wq, ws)
    xq[1, 1030] = 127  # NaN
    wq[260, 0] = 255
    y = out((B, Out))
    ax.op_fc_f8_fwd(xq, xs, 0, B, In, wq, ws, 0, Out, ax.BF16, y, work(ax.fc_f8_workspace_bytes(B, In, Out)))
    lost = torch.zeros(B, Out, dtype=torch.bool, device="cuda")
    lost[1], lost[:, 260] = True, True
    assert torch.equal(torch.isnan(y), lost)
    slack = ff.steps(In) * ff.ACC * (x.abs() @ w.abs().t())
    within(torch.where(lost, torch.zeros_like(y), y), torch.where(lost, torch.zeros_like(slack), x @ w.t()), slack)


def test_fc_f8_extreme_scales(ax):
    """Scales at both ends of their range: 2^-127 (blocks of zeros and next to
    nothing) and 2^120."""
    import torch
    B, In, Out = 9, 512, 136
    x = randn(1, B, In).double()
    x[:, :128] *= 2.0 ** -124
    x[:, 128:256] = 0
    x[:, 256:384] *= 2.0 ** 100
    w = randn(2, Out, In).double()
    w[:, 256:384] *= 2.0 ** -100
    w[:, :128] *= 2.0 ** 100
    xq, xs = ff.encode(x)
    wq, ws = ff.encode(w)
    x, w = ff.values(xq, xs), ff.values(wq, ws)
    y = out((B, Out))
    ax.op_fc_f8_fwd(u8(xq), u8(xs), 0, B, In, u8(wq), u8(ws), 0, Out, ax.BF16, y, work(ax.fc_f8_workspace_bytes(B, In, Out)))
    within(y, x @ w.t(), ff.steps(In) * ff.ACC * (x.abs() @ w.abs().t()))


# ------------------------------------------------------------------ gated block
GATED = [(1, 8, 8), (1, 4096, 1024), (2, 1000, 328), (3, 72, 40), (16, 512, 128), (17, 136, 264), (50, 2056, 136), (64, 64, 2048),
         (65, 200, 72), (128, 1000, 1000), (129, 1000, 328), (257, 72, 2056), (300, 520, 1032), (700, 512, 768), (1100, 264, 1160)]


def _gated_in(B, In, F):
    return (bf16(spread(B, B, In)), bf16(randn(F, 2 * F, In, scale=In ** -0.5)), bf16(randn(In, B, F)))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("B,In,F", GATED)
def test_gated(ax, B, In, F, kind, dtype):
    import torch
    x, w, dh = _gated_in(B, In, F)
    ws = work(ax.gated_workspace_bytes(B, In, F))
    T = ax.FP32 if dtype == "float32" else ax.BF16
    h, gu, h2 = out((B, F)), out((B, 2 * F), dtype), out((B, F))
    ax.op_gated_fwd(x, B, In, w, F, kind, h, T, gu, ws)
    ax.op_gated_fwd(x, B, In, w, F, kind, h2, T, None, ws)
    assert torch.equal(h, h2)
    want, g, u, dz, slack = ff.gated_fwd(x.double(), w.double(), kind)
    within(h, want, slack)
    within(gu, torch.cat([g, u], 1), dz, unit=ff.U_BF16 if T == ax.BF16 else ff.U_F32)
    dx, dw = out((B, In)), out((2 * F, In))
    ax.op_gated_bwd(dh, x, T, gu, B, In, w, F, kind, dx, dw, ws)
    d = gu.double()
    wx, ww, ex, ew = ff.gated_bwd(dh.double(), x.double(), d[:, :F], d[:, F:], w.double(), kind)
    within(dx, wx, ex)
    within(dw, ww, ew)
    # one gradient alone
    dx2, dw2 = out((B, In)), out((2 * F, In))
    ax.op_gated_bwd(dh, x, T, gu, B, In, w, F, kind, dx2, None, ws)
    ax.op_gated_bwd(dh, x, T, gu, B, In, w, F, kind, None, dw2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    assert status(ws) == 0


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("B,In,F", [s for s in GATED if s[1] % 16 == 0 and s[2] % 16 == 0] +
                         [(1, 16, 16), (2, 1008, 336), (129, 1008, 528), (130, 80, 1040), (300, 528, 144)])
def test_gated_ckpt8(ax, B, In, F, kind):
    import torch
    x, w, dh = _gated_in(B, In, F)
    ws = work(ax.gated_workspace_bytes(B, In, F))
    h, hb = out((B, F)), out((B, F))
    n = ax.f8_scale_bytes(B, F)
    guq, gus = out((2, B, F), "uint8"), out((2, n), "uint8")
    before = gus.clone()
    ax.op_gated_fwd_ckpt8(x, B, In, w, F, kind, h, guq, gus, ws)
    ax.op_gated_fwd(x, B, In, w, F, kind, hb, ax.FP32, None, ws)
    assert torch.equal(h, hb)
    _, g, u, dz, _ = ff.gated_fwd(x.double(), w.double(), kind)
    at = ff.tile_index(B, F, "cuda").flatten()
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    for k, (p, e) in enumerate(((g, dz[:, :F]), (u, dz[:, F:]))):
        got = ff.values(guq[k], gus[k])
        ex = ff.read_scales(gus[k], B, F)
        assert bool(((got - p).abs() <= (1 + ff.U_E4M3) * e + ff.U_E4M3 * p.abs() + ff.code_slack(ex, F)).all())
        a, off = ff.blocks(p).abs().amax(2), ff.blocks(e).amax(2)
        assert bool((a - off <= ff.FMAX[0] * ff.pow2(ex)).all())
        assert bool(((a + off > ff.FMAX[0] * ff.pow2(ex - 1)) | (ex == -127)).all())
        assert torch.equal(gus[k][rest], before[k][rest])
    xq, xs = out((B, In), "uint8"), out((ax.f8_scale_bytes(B, In),), "uint8")
    ax.op_f8_quant(x, B, In, ax.E4M3, xq, xs)
    dx, dw = out((B, In)), out((2 * F, In))
    ax.op_gated_bwd_ckpt8(dh, xq, xs, guq, gus, B, In, w, F, kind, dx, dw, ws)
    wx, ww, ex, ew = ff.gated_bwd(dh.double(), ff.values(xq, xs), ff.values(guq[0], gus[0]), ff.values(guq[1], gus[1]), w.double(), kind)
    within(dx, wx, ex)
    within(dw, ww, ew)
    dx2, dw2 = out((B, In)), out((2 * F, In))
    ax.op_gated_bwd_ckpt8(dh, xq, xs, guq, gus, B, In, w, F, kind, dx2, None, ws)
    ax.op_gated_bwd_ckpt8(dh, xq, xs, guq, gus, B, In, w, F, kind, None, dw2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    assert status(ws) == 0


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_gated_large_projections(ax, kind):
    """Gate values far out on both sides: neither an overflow in exp nor one in
    gelu's cube makes a NaN, forward or backward."""
    import torch
    B, In, F = 4, 16, 64
    x = torch.zeros(B, In, device="cuda")
    x[:, 0] = torch.tensor([1.0, -1.0, 1e4, -1e4])
    w = torch.zeros(2 * F, In, device="cuda")
    w[:F, 0] = torch.linspace(-6, 16, F, device="cuda").exp2()
    w[F:, 0] = 1.0
    x, w = bf16(x), bf16(w)
    ws = work(ax.gated_workspace_bytes(B, In, F))
    h, gu = out((B, F)), out((B, 2 * F))
    ax.op_gated_fwd(x, B, In, w, F, kind, h, ax.BF16, gu, ws)
    want, _, _, _, slack = ff.gated_fwd(x.double(), w.double(), kind)
    within(h, want, slack)
    dh = bf16(torch.ones(B, F, device="cuda"))
    dx, dw = out((B, In)), out((2 * F, In))
    ax.op_gated_bwd(dh, x, ax.BF16, gu, B, In, w, F, kind, dx, dw, ws)
    d = gu.double()
    wx, ww, ex, ew = ff.gated_bwd(dh.double(), x.double(), d[:, :F], d[:, F:], w.double(), kind)
    within(dx, wx, ex)
    within(dw, ww, ew)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("B", [4, 150, 600])
def test_gated_lost_values_stay_in_their_row(ax, B, kind):
    import torch
    In, F = 136, 200
    x, w, dh = _gated_in(B, In, F)
    ws = work(ax.gated_workspace_bytes(B, In, F))
    h, gu, dx, dw = out((B, F)), out((B, 2 * F)), out((B, In)), out((2 * F, In))
    ax.op_gated_fwd(x, B, In, w, F, kind, h, ax.BF16, gu, ws)
    ax.op_gated_bwd(dh, x, ax.BF16, gu, B, In, w, F, kind, dx, dw, ws)
    clean, cleanx = h.clone(), dx.clone()
    x[2, 135] = float("nan")
    x[B - 1, 0] = float("inf")
    ax.op_gated_fwd(x, B, In, w, F, kind, h, ax.BF16, gu, ws)
    ax.op_gated_bwd(dh, x, ax.BF16, gu, B, In, w, F, kind, dx, None, ws)
    keep = [i for i in range(B) if i not in (2, B - 1)]
    assert torch.equal(h[keep], clean[keep]) and torch.equal(dx[keep], cleanx[keep])
    assert bool(torch.isnan(h[2]).all()) and bool(torch.isnan(dx[2]).all())
    # +-inf * +-inf of the projections, or a gate of -inf: never a finite value
    # but for relu's gates at -inf, which are 0 * inf = NaN
    assert not bool(torch.isfinite(h[B - 1]).any())


@pytest.mark.parametrize("B", [3, 200])
def test_ckpt8_lost_values_stay_in_their_row(ax, B):
    """A NaN or an infinity in one row's projections: NaN codes there, nothing
    in the other rows' codes, scales and gradients."""
    import torch
    In, F = 144, 272
    x, w, dh = _gated_in(B, In, F)
    ws = work(ax.gated_workspace_bytes(B, In, F))
    n = ax.f8_scale_bytes(B, F)
    h, guq, gus, dx = out((B, F)), out((2, B, F), "uint8"), out((2, n), "uint8"), out((B, In))
    xq, xs = out((B, In), "uint8"), out((ax.f8_scale_bytes(B, In),), "uint8")

    def go():
        ax.op_f8_quant(x, B, In, ax.E4M3, xq, xs)
        ax.op_gated_fwd_ckpt8(x, B, In, w, F, 0, h, guq, gus, ws)
        ax.op_gated_bwd_ckpt8(dh, xq, xs, guq, gus, B, In, w, F, 0, dx, None, ws)
        return [t.clone() for t in (h, guq, gus, dx)]

    clean = go()
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    bad = go()
    keep = [i for i in range(B) if i not in (1, 2)]
    assert torch.equal(bad[0][keep], clean[0][keep]) and torch.equal(bad[3][keep], clean[3][keep])
    assert torch.equal(bad[1][:, keep], clean[1][:, keep])
    at = ff.tile_index(B, F, "cuda")[keep].flatten()
    assert torch.equal(bad[2][:, at], clean[2][:, at])
    assert bool(torch.isnan(ff.code_values(bad[1][:, [1, 2]])).all())
    assert bool(torch.isnan(bad[3][[1, 2]]).all())


def test_gated_gradient_against_differences(ax):
    """<dx, v> and <dw, v> of the kernels against central differences of the
    64-bit loss, to within the elementwise bounds summed over v (the loss is
    smooth: a step of 2^-10 leaves a third-order term far below them)."""
    import torch
    B, In, F = 24, 96, 160
    x, w, dh = _gated_in(B, In, F)
    x.copy_(randn(5, B, In))
    for kind in (0, 1):
        ws = work(ax.gated_workspace_bytes(B, In, F))
        h, gu, dx, dw = out((B, F)), out((B, 2 * F)), out((B, In)), out((2 * F, In))
        ax.op_gated_fwd(x, B, In, w, F, kind, h, ax.BF16, gu, ws)
        ax.op_gated_bwd(dh, x, ax.BF16, gu, B, In, w, F, kind, dx, dw, ws)
        X, W, H = x.double(), w.double(), dh.double()
        _, g, u, _, _ = ff.gated_fwd(X, W, kind)
        # the saved projections are rounded: their part of the bound
        a, d = ff.act(g, kind)
        ez = ff.U_BF16 * torch.cat([(H * u * d).abs() + (H * u * g).abs(), (H * a).abs() + (H * g).abs() * ff.LIPSCHITZ], 1)
        wx, ww, ex, ew = ff.gated_bwd(H, X, g, u, W, kind)
        ex, ew = ex + ez @ W.abs() + ff.U_BF16 * wx.abs(), ew + ez.t() @ X.abs() + ff.U_BF16 * ww.abs()
        t = 2.0 ** -10
        for grad, bound, of in ((dx, ex, 0), (dw, ew, 1)):
            v = randn(9 + of, *grad.shape).double()
            v = v / v.norm()
            up, dn = (((X + k * v, W) if of == 0 else (X, W + k * v)) for k in (t, -t))
            diff = float(((ff.gated_fwd(*up, kind)[0] - ff.gated_fwd(*dn, kind)[0]) * H).sum()) / (2 * t)
            assert abs(float((grad.double() * v).sum()) - diff) <= float((bound * v.abs()).sum())


# ------------------------------------------------------------------ together, streams, graphs
def _block(ax, seed, B, In, F):
    """A normalised gated block with its gradient, and the 8-bit product of its
    output: buffers and the calls in the order in which a program makes them."""
    import torch
    b = {"x": bf16(randn(seed, B, In)), "res": bf16(randn(seed + 1, B, In)), "gamma": f32(1 + 0.1 * randn(seed + 2, In)),
         "w": bf16(randn(seed + 3, 2 * F, In, scale=In ** -0.5)), "dy": bf16(randn(seed + 4, B, In))}
    down = randn(seed + 5, In, F, scale=F ** -0.5).to(torch.bfloat16).double()
    wq, wsc = ff.encode(down)
    b.update(down=down, wq=u8(wq), wsc=u8(wsc), dh=bf16(randn(seed + 6, B, F)))
    for k in ("s", "y", "dx", "dy2", "o"):
        b[k] = out((B, In))
    b.update(h=out((B, F)), dw=out((2 * F, In)), r=out((B,), "float32"), dgamma=out((In,), "float32"))
    b.update(yq=out((B, In), "uint8"), ys=out((ax.f8_scale_bytes(B, In),), "uint8"), guq=out((2, B, F), "uint8"),
             gus=out((2, ax.f8_scale_bytes(B, F)), "uint8"), hq=out((B, F), "uint8"), hs=out((ax.f8_scale_bytes(B, F),), "uint8"))
    b.update(w1=work(ax.gated_workspace_bytes(B, In, F)), w2=work(ax.fc_f8_workspace_bytes(B, F, In)),
             w3=work(ax.rmsnorm_workspace_bytes(B, In)))

    def go(stream=None):
        ax.op_rmsnorm_fwd(b["x"], b["res"], b["gamma"], B, In, EPS, b["s"], b["y"], b["r"], b["yq"], b["ys"], stream)
        ax.op_gated_fwd_ckpt8(b["y"], B, In, b["w"], F, ax.SILU, b["h"], b["guq"], b["gus"], b["w1"], stream)
        ax.op_f8_quant(b["h"], B, F, ax.E4M3, b["hq"], b["hs"], stream)
        ax.op_fc_f8_fwd(b["hq"], b["hs"], ax.E4M3, B, F, b["wq"], b["wsc"], ax.E4M3, In, ax.BF16, b["o"], b["w2"], stream)
        ax.op_gated_bwd_ckpt8(b["dh"], b["yq"], b["ys"], b["guq"], b["gus"], B, In, b["w"], F, ax.SILU, b["dy2"], b["dw"], b["w1"], stream)
        ax.op_rmsnorm_bwd(b["dy2"], b["dy"], b["s"], b["gamma"], b["r"], B, In, b["dx"], b["dgamma"], b["w3"], stream)

    return b, go


RESULTS = ("s", "y", "yq", "h", "o", "dw", "dy2", "dx", "dgamma")


@pytest.mark.parametrize("B,In,F", [(1, 512, 1024), (40, 1024, 528), (333, 528, 1040)])
def test_block_together(ax, B, In, F):
    """Each stage against its formula on the values that the stage before it
    left."""
    b, go = _block(ax, 11, B, In, F)
    go()
    D = {k: v.double() for k, v in b.items() if hasattr(v, "double")}
    wy, wr = ff.norm_fwd(D["s"], D["gamma"], EPS)
    within(b["y"], wy, 100 * ff.U_F32 * wy.abs())
    want, g, u, dz, slack = ff.gated_fwd(D["y"], D["w"], 0)
    within(b["h"], want, slack)
    h8, w8 = ff.values(b["hq"], b["hs"]), ff.values(b["wq"], b["wsc"])
    within(b["o"], h8 @ w8.t(), ff.steps(F) * ff.ACC * (h8.abs() @ w8.abs().t()))
    wx, ww, ex, ew = ff.gated_bwd(D["dh"], ff.values(b["yq"], b["ys"]), ff.values(b["guq"][0], b["gus"][0]),
                                  ff.values(b["guq"][1], b["gus"][1]), D["w"], 0)
    within(b["dy2"], wx, ex)
    within(b["dw"], ww, ew)
    dx, dg = ff.norm_bwd(D["dy2"], D["dy"], D["s"], D["gamma"], D["r"])
    t = D["dy2"] * D["gamma"]
    mag = D["r"][:, None] * (t.abs() + D["s"].abs() * (D["r"] ** 2)[:, None] * (t * D["s"]).abs().mean(1, keepdim=True))
    within(b["dx"], dx, (In // 256 + 40) * ff.U_F32 * (mag + D["dy"].abs()))
    # the same calls give the same bits
    first = {k: b[k].clone() for k in RESULTS}
    go()
    import torch
    assert all(torch.equal(first[k], b[k]) for k in RESULTS)


def test_block_on_streams_at_once(ax):
    """Two blocks on two streams at the same time, each with its own buffers:
    the results of one stream alone."""
    import torch
    made = [_block(ax, 21, 70, 512, 784), _block(ax, 31, 1, 1024, 512)]
    alone = []
    for b, go in made:
        go()
        torch.cuda.synchronize()
        alone.append({k: b[k].clone() for k in RESULTS})
        for k in RESULTS:
            b[k].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(5):
        for (b, go), st in zip(made, streams):
            go(st)
    torch.cuda.synchronize()
    for (b, _), want in zip(made, alone):
        assert all(torch.equal(b[k], want[k]) for k in RESULTS)


@pytest.mark.parametrize("B,In,F", [(1, 512, 512), (300, 512, 784)])
def test_block_captured(ax, B, In, F):
    """A captured block, replayed on new inputs, gives what eager calls give;
    an eager call between the replays changes nothing."""
    import torch
    b, go = _block(ax, 41, B, In, F)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        go()
    for seed in (51, 61):
        other, go2 = _block(ax, seed, B, In, F)
        for k in ("x", "res", "gamma", "w", "dy", "dh", "wq", "wsc"):
            b[k].copy_(other[k])
        torch.cuda.synchronize()
        graph.replay()
        go2()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b[k], other[k]) for k in RESULTS)
    torch.cuda.synchronize()
    del graph


FIRST = """
import sys
import torch
sys.path.insert(0, %r)
from deep_cnn_image_b200 import alexnet as ax
from tests import test_gpu_ff as t
b, go = t._block(ax, 71, %d, 512, 1040)
st = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=st):
    go()
graph.replay()
torch.cuda.synchronize()
got = {k: b[k].clone() for k in t.RESULTS}
go()
torch.cuda.synchronize()
assert all(torch.equal(b[k], got[k]) for k in t.RESULTS)
print("the same")
"""


@pytest.mark.parametrize("B", [1, 300])
def test_first_calls_of_a_process_captured(ax, B):
    """No call needs an eager one before its capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % (root, B)], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "the same" in r.stdout, r.stdout + r.stderr


def test_block_from_threads(ax):
    """Host threads call at the same time, each on its own stream and buffers."""
    import threading
    import torch
    made = [_block(ax, 81 + 10 * i, B, 512, 784) for i, B in enumerate((1, 40, 300))]
    alone = []
    for b, go in made:
        go()
        torch.cuda.synchronize()
        alone.append({k: b[k].clone() for k in RESULTS})
    wrong = []

    def work_on(i):
        b, go = made[i]
        st = torch.cuda.Stream()
        for _ in range(20):
            go(st)
            st.synchronize()
            if not all(torch.equal(b[k], alone[i][k]) for k in RESULTS):
                wrong.append(i)

    threads = [threading.Thread(target=work_on, args=(i,)) for i in range(len(made))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong
