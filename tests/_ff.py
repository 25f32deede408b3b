"""The feed-forward operators in 64 bits, from their formulas, and the error
bounds that their tests state.  Works on torch tensors of any device.

Rounding: one rounding to a type is off by at most U[type] of the value.  The
tensor cores add exact products (bf16 x bf16 and 8-bit x 8-bit products have
at most 16 significant bits) 16 or 32 at a time into an fp32 accumulator; each
step is allowed one fp32 unit, 2^-23, of the running sum, which is at most
A = sum |x||w| (that covers truncating adders), so a sum of n products is off
by at most steps(n) * 2^-23 * A."""
import math

import torch

U_BF16 = 2.0 ** -8
U_E4M3, U_E5M2 = 2.0 ** -4, 2.0 ** -3
U_F32 = 2.0 ** -24
ACC = 2.0 ** -23
FMAX = {0: 448.0, 1: 57344.0}
MANT, LOW = {0: 3, 1: 2}, {0: -6, 1: -14}  # mantissa bits, lowest exponent of a normal code


def steps(n):
    """Accumulation steps of n products: 16 at a time, the join of at most 16
    partial sums and the last block's padding."""
    return n // 16 + 24


def pow2(e):
    """2^e from its bits (pow need not be exact), -1022 <= e <= 1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def blocks(v):
    """[R, C] -> [R, ceil(C / 128), 128], filled up with zeros."""
    R, C = v.shape
    K = -(-C // 128)
    out = torch.zeros(R, K * 128, dtype=v.dtype, device=v.device)
    out[:, :C] = v
    return out.view(R, K, 128)


def exponents(v, fmt=0):
    """The scale exponent of every block of v (64 bits, NaN and infinities
    left out): the smallest e with amax <= fmax 2^e."""
    b = blocks(torch.where(torch.isfinite(v), v, torch.zeros_like(v)).double())
    a = b.abs().amax(2)
    m, k = torch.frexp(a)  # a = m 2^k, m in [1/2, 1); fmax = 0.875 * 2^9 or 2^16
    e = k - (9 if fmt == 0 else 16) + (m > 0.875).int()
    return torch.where(a == 0, torch.full_like(e, -127), e.clamp(min=-127))


def tile_index(R, C, device):
    """Byte offsets [R, blocks] of the scales of a [R, C] matrix."""
    r = torch.arange(R, device=device)[:, None]
    b = torch.arange(-(-C // 128), device=device)[None, :]
    tiles = -(-C // 512)
    return (r // 128 * tiles + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4


def read_scales(s, R, C):
    """Exponents [R, blocks] of stored scales."""
    return s[tile_index(R, C, s.device)].int() - 127


def write_scales(e, C):
    R = e.shape[0]
    s = torch.full((-(-R // 128) * -(-C // 512) * 512,), 255, dtype=torch.uint8, device=e.device)
    s[tile_index(R, C, e.device)] = (e + 127).to(torch.uint8)
    return s


def code_values(q, fmt=0):
    """The codes' own values, from their bits."""
    v = q.long()
    mant = MANT[fmt]
    ex, m = (v & 127) >> mant, (v & ((1 << mant) - 1)).double() / (1 << mant)
    x = torch.where(ex > 0, (1 + m) * pow2(ex - 1 + LOW[fmt]), m * pow2(torch.full_like(ex, LOW[fmt])))
    nan = (v & 127) == 127 if fmt == 0 else (v & 127) > 124
    x = torch.where(nan, torch.full_like(x, math.nan), x)
    if fmt == 1:
        x = torch.where((v & 127) == 124, torch.full_like(x, math.inf), x)
    return torch.where(v > 127, -x, x)


def values(q, s, fmt=0):
    """What an 8-bit matrix stands for, in 64 bits."""
    R, C = q.shape
    return code_values(q, fmt) * pow2(read_scales(s, R, C)).repeat_interleave(128, 1)[:, :C]


def encode(v, fmt=0):
    """[R, C] -> (codes, scales): round to nearest even in 64 bits."""
    R, C = v.shape
    e = exponents(v, fmt)
    w = v.double() * pow2(-e).repeat_interleave(128, 1)[:, :C]
    _, k = torch.frexp(w)
    step = pow2((k - 1).clamp(min=LOW[fmt]) - MANT[fmt])
    w = torch.round(w / step) * step
    a = w.abs()
    _, k = torch.frexp(a)
    normal = a >= 2.0 ** LOW[fmt]
    ex = torch.where(normal, k - LOW[fmt], torch.zeros_like(k))
    m = torch.where(normal, a * pow2(1 - k) - 1, a * 2.0 ** -LOW[fmt]) * (1 << MANT[fmt])
    q = (ex.long() << MANT[fmt]) + m.long() + 128 * torch.signbit(w).long()
    return q.to(torch.uint8), write_scales(e, C)


def code_slack(e, C, fmt=0):
    """Half the distance of subnormal codes, as a value, for [R, blocks]
    exponents: what a rounding is off by near zero."""
    return 2.0 ** (LOW[fmt] - MANT[fmt] - 1) * pow2(e).repeat_interleave(128, 1)[:, :C]


def act(g, kind):
    """a(g) and a'(g)."""
    if kind == 0:
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    if kind == 2:
        return torch.clamp(g, min=0), (g > 0).double()
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


#: |a'| <= 1.13 for all three; the fast exp and quotient: |z| up to 80 makes
#: the exponent's argument off by 80 * 2^-23, the rest a few units
LIPSCHITZ, ACT_EPS = 1.13, 100 * ACC


def norm_fwd(s, gamma, eps):
    r = 1 / torch.sqrt((s * s).mean(1) + eps)
    return s * r[:, None] * gamma, r


def norm_bwd(dy, dsum, s, gamma, r):
    t = dy * gamma
    dx = r[:, None] * (t - s * (r * r)[:, None] * (t * s).mean(1, keepdim=True))
    return dx + (dsum if dsum is not None else 0), (dy * s * r[:, None]).sum(0)


def gated_fwd(x, w, kind):
    """h, g, u and the bound of g's and u's error."""
    F = w.shape[0] // 2
    z = x @ w.t()
    dz = steps(x.shape[1]) * ACC * (x.abs() @ w.abs().t())
    g, u = z[:, :F], z[:, F:]
    a = act(g, kind)[0]
    dg, du = dz[:, :F], dz[:, F:]
    slack = (u.abs() + du) * (LIPSCHITZ * dg + ACT_EPS * g.abs()) + a.abs() * du
    return a * u, g, u, dz, slack


def gated_bwd(dh, x, g, u, w, kind):
    """dx, dw and the bounds of their errors before the last rounding.  The
    products take the projections' gradients rounded to bf16, or, up to 32 rows,
    to two bf16 terms (2^-8 of 2^-8)."""
    unit = U_BF16 if dh.shape[0] > 32 else U_BF16 ** 2
    a, d = act(g, kind)
    dz = torch.cat([dh * u * d, dh * a], 1)
    # the product's own rounding to bf16, and the activation's evaluation:
    # a' is a sum of terms of at most 1 + |g|/4 in size
    ez = unit * dz.abs() + torch.cat([(dh * u).abs() * (1 + g.abs()), (dh * g).abs()], 1) * ACT_EPS
    za, wa, xa = dz.abs() + ez, w.abs(), x.abs()
    B, F2 = dz.shape
    B = 2 * B if B <= 32 else B  # two terms are two products
    return (dz @ w, dz.t() @ x, ez @ wa + steps(F2) * ACC * (za @ wa),
            ez.t() @ xa + steps(B) * ACC * (za.t() @ xa))
