"""The feed-forward operators' measured cases.

The operators are those of a pre-normalised gated feed-forward path with one
8-bit row format between them:

* ``norm`` / ``norm_grad``: root-mean-square norm of x + res with the sum
  stored, the output in 8 bits with a scale per 128 values; its gradient;
* ``f8``: matrix product of two 8-bit matrices with a scale per row and 128
  values of the reduction;
* ``gated`` / ``gated_train``: gated feed-forward block h = act(x Wg^T) *
  (x Wu^T), forward alone and forward with backward;
* ``ckpt8``: the same training step with every saved activation (the input,
  the gate and the up projection) held in 8 bits between the passes.

The 8-bit format: a row is cut in blocks of 128 values; a block's scale is
the smallest power of two 2^e (e in -127..127) for which the block's largest
magnitude is at most the type's largest value times 2^e, and the codes are
the values times 2^-e rounded to nearest even.  In memory a scale is the byte
e + 127; the bytes lie in tiles of 128 rows x 4 blocks of 512 bytes (row tile
slowest), byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of its tile.

`run` computes the plain forms out of elementary torch operations in 32 bits;
with `own` set it makes the library's calls.  `exact` computes the same
definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
#: largest value, exponent of the leading bit's carry point (fmax = 0.875 * 2^k), torch type
FORMATS = {"e4m3": (448.0, 9, torch.float8_e4m3fn), "e5m2": (57344.0, 16, torch.float8_e5m2)}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a single token through the norm of a served model: latency only
        {"name": "norm token", "op": "norm", "rows": 1, "cols": 4096},
        # the norm over a long prompt or a training batch: bandwidth
        {"name": "norm prompt", "op": "norm", "rows": 8192, "cols": 4096},
        # the norm's gradient over a ragged batch of sequences, an odd width
        {"name": "norm gradient", "op": "norm_grad", "rows": 4001, "cols": 4112},
        # a single token through an 8-bit projection: the weights' bytes
        {"name": "f8 token", "op": "f8", "B": 1, "In": 4096, "Out": 9216, "x": "e4m3", "w": "e4m3"},
        # a batch of tokens being decoded (the width of the widest FC layer)
        {"name": "f8 batch", "op": "f8", "B": 128, "In": 9216, "Out": 4096, "x": "e4m3", "w": "e4m3"},
        # a ragged prompt's gradient rows (wide-range type) against few outputs
        {"name": "f8 ragged", "op": "f8", "B": 777, "In": 2064, "Out": 1000, "x": "e5m2", "w": "e4m3"},
        # a long prompt through an 8-bit projection: the tensor cores' rate
        {"name": "f8 prompt", "op": "f8", "B": 8192, "In": 4096, "Out": 9216, "x": "e4m3", "w": "e4m3"},
        # a single token through the gated block
        {"name": "gated token", "op": "gated", "B": 1, "In": 4096, "F": 9216, "act": "silu"},
        # a prompt through the gated block
        {"name": "gated prompt", "op": "gated", "B": 2048, "In": 4096, "F": 9216, "act": "gelu"},
        # a training step's forward and backward of the block
        {"name": "gated train", "op": "gated_train", "B": 4096, "In": 4096, "F": 9216, "act": "silu"},
        # the same with the activations kept in 8 bits
        {"name": "ckpt8 train", "op": "ckpt8", "B": 4096, "In": 4096, "F": 9216, "act": "silu"},
        # a small ragged batch of a narrow block
        {"name": "ckpt8 ragged", "op": "ckpt8", "B": 333, "In": 1008, "F": 2320, "act": "gelu"},
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
        return max(lo, min(hi, int(v) // step * step))

    op = rng.choice(["norm", "norm_grad", "f8", "f8", "gated", "gated_train", "ckpt8"])
    if op in ("norm", "norm_grad"):
        return {"op": op, "rows": size(1, 8192), "cols": size(16, 8192, 16)}
    if op == "f8":
        return {"op": op, "B": size(1, 8192), "In": size(64, 9216, 16), "Out": size(64, 9216, 8),
                "x": rng.choice(["e4m3", "e5m2"]), "w": rng.choice(["e4m3", "e4m3", "e5m2"])}
    step = 16 if op == "ckpt8" else 8
    return {"op": op, "B": size(1, 2048 if op == "gated" else 4096), "In": size(64, 4096, step),
            "F": size(64, 9216, step), "act": rng.choice(["silu", "gelu", "relu"])}


def work(case):
    op = case["op"]
    if op == "norm":  # x, res read; sum and codes written
        n = case["rows"] * case["cols"]
        return {"bytes": n * 7 + n / 128 + 4 * case["cols"], "flops": 6 * n}
    if op == "norm_grad":  # dy, dsum, sum read; dx written
        n = case["rows"] * case["cols"]
        return {"bytes": n * 8 + 4 * case["rows"] + 8 * case["cols"], "flops": 10 * n}
    B, In = case["B"], case["In"]
    if op == "f8":
        Out = case["Out"]
        return {"bytes": (B * In + Out * In) * (1 + 1 / 128) + 2 * B * Out, "flops": 2 * B * In * Out}
    F = case["F"]
    fwd = {"bytes": 2 * (B * In + 2 * F * In + B * F), "flops": 4 * B * In * F}
    if op == "gated":
        return fwd
    # backward: dh read, dx and dw written (x and the weights are read once)
    return {"bytes": fwd["bytes"] + 2 * (B * F + B * In + 2 * F * In), "flops": 3 * fwd["flops"]}


# ---------------------------------------------------------------- inputs
def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _activations(g, rows, cols):
    """Normal values, one channel in 64 about eight times larger: the outlier
    channels that make 8-bit activations want a scale per block."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    big = torch.rand(cols, generator=g, device="cuda") < 1 / 64
    return torch.where(big, 8 * x, x).to(torch.bfloat16)


def _tiles(e):
    """Exponents [rows, blocks] -> the scale bytes in tiles."""
    R, K = e.shape
    t = torch.zeros(-(-R // 128) * 128, -(-K // 4) * 4, dtype=torch.uint8, device=e.device)
    t[:R, :K] = (e + 127).to(torch.uint8)
    t = t.view(t.shape[0] // 128, 4, 32, t.shape[1] // 4, 4)
    return t.permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untiles(s, R, C):
    K = -(-C // 128)
    t = s.view(-(-R // 128), -(-K // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(-(-R // 128) * 128, -1)[:R, :K].int() - 127


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    bf = {"dtype": torch.bfloat16, "device": "cuda"}
    if op in ("norm", "norm_grad"):
        R, C = case["rows"], case["cols"]
        s["gamma"] = 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
        if op == "norm":
            s.update(x=_normal(g, R, C), res=_activations(g, R, C), sum=torch.empty(R, C, **bf),
                     q=torch.empty(R, C, dtype=torch.uint8, device="cuda"), y=torch.empty(R, C, **bf),
                     scales=torch.empty(-(-R // 128) * -(-C // 512) * 512, dtype=torch.uint8, device="cuda"))
        else:
            s.update(dy=_normal(g, R, C), dsum=_normal(g, R, C), s=_activations(g, R, C), dx=torch.empty(R, C, **bf),
                     dgamma=torch.empty(C, device="cuda"))
            s["rstd"] = (s["s"].float().square().mean(1) + EPS).rsqrt()
        return s
    B, In = case["B"], case["In"]
    if op == "f8":
        Out = case["Out"]
        x, w = _activations(g, B, In), _normal(g, Out, In, scale=In ** -0.5)
        s["xq"], xe = _codes(x.float(), case["x"])
        s["wq"], we = _codes(w.float(), case["w"])
        s.update(xs=_tiles(xe), ws=_tiles(we), y=torch.empty(B, Out, **bf))
        return s
    F = case["F"]
    s.update(x=_activations(g, B, In), w=_normal(g, 2 * F, In, scale=In ** -0.5), h=torch.empty(B, F, **bf))
    if op != "gated":
        s.update(dh=_normal(g, B, F), dx=torch.empty(B, In, **bf), dw=torch.empty(2 * F, In, **bf))
    if op == "gated_train":
        s["gu"] = torch.empty(B, 2 * F, **bf)
    if op == "ckpt8":
        u8 = {"dtype": torch.uint8, "device": "cuda"}
        s.update(xq=torch.empty(B, In, **u8), xs=torch.empty(-(-B // 128) * -(-In // 512) * 512, **u8),
                 guq=torch.empty(2, B, F, **u8), gus=torch.empty(2, -(-B // 128) * -(-F // 512) * 512, **u8))
    return s


# ---------------------------------------------------------------- plain forms
def _pow2(e):
    """2^e in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _blocks(v):
    """[R, C] -> [R, blocks, 128], the last block filled up with zeros."""
    R, C = v.shape
    K = -(-C // 128)
    p = torch.zeros(R, K * 128, dtype=v.dtype, device=v.device)
    p[:, :C] = v
    return p.view(R, K, 128)


def _codes(v, fmt):
    """[R, C] in 32 bits -> the 8-bit codes (as bytes) and the exponents."""
    fmax, k, dtype = FORMATS[fmt]
    R, C = v.shape
    b = _blocks(v)
    m, ex = torch.frexp(b.abs().amax(2))
    e = torch.where(m == 0, -127, (ex - k + (m > 0.875).int()).clamp(-127, 127))
    q = (b.double() * _pow2(-e)[:, :, None]).float().to(dtype).view(torch.uint8)
    return q.view(R, -1)[:, :C].contiguous(), e


def _values(q, e, fmt):
    """The values that codes and exponents stand for, in 32 bits."""
    R, C = q.shape
    p = _pow2(e).float().repeat_interleave(128, 1)[:, :C]
    return q.view(FORMATS[fmt][2]).float() * p


def _through8(v):
    return _values(*_codes(v, "e4m3"), "e4m3")


def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    if act == "relu":
        return g.clamp_min(0), (g > 0).float()
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain(s):
    case = s["case"]
    op, bf = case["op"], torch.bfloat16
    if op == "norm":
        t = (s["x"].float() + s["res"].float()).to(bf)
        f = t.float()
        y = f * (f.square().mean(1, keepdim=True) + EPS).rsqrt() * s["gamma"]
        return t, _through8(y).to(bf)
    if op == "norm_grad":
        f, r, dy = s["s"].float(), s["rstd"][:, None], s["dy"].float()
        t = dy * s["gamma"]
        dx = r * (t - f * (r * r * (t * f).mean(1, keepdim=True))) + s["dsum"].float()
        return dx.to(bf), (dy * f * r).sum(0)
    if op == "f8":
        x = _values(s["xq"], _untiles(s["xs"], *s["xq"].shape), case["x"])
        w = _values(s["wq"], _untiles(s["ws"], *s["wq"].shape), case["w"])
        return (x @ w.t()).to(bf)
    F, x, w = case["F"], s["x"].float(), s["w"].float()
    z = x @ w.t()
    g, u = z[:, :F], z[:, F:]
    h = (_act(g, case["act"])[0] * u).to(bf)
    if op == "gated":
        return h
    if op == "ckpt8":
        x, g, u = _through8(x), _through8(g), _through8(u)
    a, d = _act(g, case["act"])
    dh = s["dh"].float()
    dz = torch.cat([dh * u * d, dh * a], 1)
    return h, (dz @ w).to(bf), (dz.t() @ x).to(bf)


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from deep_cnn_image_b200 import alexnet as ax

    case = s["case"]
    op = case["op"]
    if op == "norm":
        R, C = case["rows"], case["cols"]
        ax.op_rmsnorm_fwd(s["x"], s["res"], s["gamma"], R, C, EPS, s["sum"], None, None, s["q"], s["scales"])
        ax.op_f8_dequant(s["q"], s["scales"], R, C, ax.E4M3, s["y"])
        return s["sum"], s["y"]
    if op == "norm_grad":
        R, C = case["rows"], case["cols"]
        if "work" not in s:
            s["work"] = torch.empty(ax.rmsnorm_workspace_bytes(R, C), dtype=torch.uint8, device="cuda")
        ax.op_rmsnorm_bwd(s["dy"], s["dsum"], s["s"], s["gamma"], s["rstd"], R, C, s["dx"], s["dgamma"], s["work"])
        return s["dx"], s["dgamma"]
    B, In = case["B"], case["In"]
    if op == "f8":
        Out = case["Out"]
        if "work" not in s:
            s["work"] = torch.empty(ax.fc_f8_workspace_bytes(B, In, Out), dtype=torch.uint8, device="cuda")
        fmt = {"e4m3": ax.E4M3, "e5m2": ax.E5M2}
        ax.op_fc_f8_fwd(s["xq"], s["xs"], fmt[case["x"]], B, In, s["wq"], s["ws"], fmt[case["w"]], Out, ax.BF16, s["y"], s["work"])
        return s["y"]
    F = case["F"]
    act = {"silu": ax.SILU, "gelu": ax.GELU, "relu": ax.RELU}[case["act"]]
    if "work" not in s:
        s["work"] = torch.empty(ax.gated_workspace_bytes(B, In, F), dtype=torch.uint8, device="cuda")
    if op == "gated":
        ax.op_gated_fwd(s["x"], B, In, s["w"], F, act, s["h"], ax.FP32, None, s["work"])
        return s["h"]
    if op == "gated_train":
        if s["gu"].dtype != torch.float32:  # kept as summed: bf16 would add its rounding to the gradients
            s["gu"] = torch.empty(B, 2 * F, device="cuda")
        ax.op_gated_fwd(s["x"], B, In, s["w"], F, act, s["h"], ax.FP32, s["gu"], s["work"])
        ax.op_gated_bwd(s["dh"], s["x"], ax.FP32, s["gu"], B, In, s["w"], F, act, s["dx"], s["dw"], s["work"])
    else:
        ax.op_f8_quant(s["x"], B, In, ax.E4M3, s["xq"], s["xs"])
        ax.op_gated_fwd_ckpt8(s["x"], B, In, s["w"], F, act, s["h"], s["guq"], s["gus"], s["work"])
        ax.op_gated_bwd_ckpt8(s["dh"], s["xq"], s["xs"], s["guq"], s["gus"], B, In, s["w"], F, act, s["dx"], s["dw"], s["work"])
    return s["h"], s["dx"], s["dw"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _grid(v, mantissa, lowest):
    """v rounded to nearest even to `mantissa` bits after the leading one,
    exponents from `lowest` up."""
    _, ex = torch.frexp(v)
    step = _pow2(torch.clamp(ex.long() - 1, min=lowest) - mantissa)
    return torch.round(v / step) * step


def _eight(v):
    """What v's rows are worth after a round trip through e4m3 blocks."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], 128):
        b = v[:, c:c + 128]
        a = b.abs().amax(1, keepdim=True)
        e = torch.where(a > 0, torch.ceil(torch.log2(a / 448)), -127.0).clamp(-127, 127)
        e = torch.where(a > 448 * _pow2(e), e + 1, e)
        e = torch.where((a > 0) & (e > -127) & (a <= 448 * _pow2(e - 1)), e - 1, e)
        out[:, c:c + 128] = _grid(b / _pow2(e), 3, -6) * _pow2(e)
    return out


def _worth(q, s, fmt):
    """Codes and scale tiles -> values in 64 bits, bit by bit."""
    R, C = q.shape
    mantissa, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    v = q.long()
    ex, m = (v & 127) >> mantissa, (v & ((1 << mantissa) - 1)).double() / (1 << mantissa)
    x = torch.where(ex > 0, (1 + m) * _pow2(ex - bias), m * _pow2(torch.full_like(ex, 1 - bias)))
    x = torch.where(v > 127, -x, x)
    r = torch.arange(R, device=q.device)[:, None]
    b = (torch.arange(C, device=q.device) // 128)[None, :]
    tiles = (C + 511) // 512
    at = (r // 128 * tiles + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    return x * _pow2(s[at].long() - 127)


def _gate(g, act):
    if act == "silu":
        e = torch.exp(-g)
        return g / (1 + e), (1 + e + g * e) / (1 + e) ** 2
    if act == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g)), (g > 0).double()
    z = (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    dz = (2 / math.pi) ** 0.5 * (1 + 0.134145 * g ** 2)
    p = 1 / (1 + torch.exp(-2 * z))  # (1 + tanh z) / 2
    return g * p, p + 2 * g * p * (1 - p) * dz


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        t = (s["x"].double() + s["res"].double()).to(torch.bfloat16).double()
        r = 1 / torch.sqrt((t * t).sum(1) / case["cols"] + EPS)
        return t, _eight(t * r[:, None] * s["gamma"].double())
    if op == "norm_grad":
        v, r, dy = s["s"].double(), s["rstd"].double()[:, None], s["dy"].double()
        t = dy * s["gamma"].double()
        dot = (t * v).sum(1, keepdim=True)
        return r * t - r ** 3 * v * dot / case["cols"] + s["dsum"].double(), torch.einsum("rc,rc->c", dy, v * r)
    if op == "f8":
        return torch.einsum("bi,oi->bo", _worth(s["xq"], s["xs"], case["x"]), _worth(s["wq"], s["ws"], case["w"]))
    F, act, x, w = case["F"], case["act"], s["x"].double(), s["w"].double()
    wg, wu = w[:F], w[F:]
    g, u = torch.einsum("bi,fi->bf", x, wg), torch.einsum("bi,fi->bf", x, wu)
    h = _gate(g, act)[0] * u
    if op == "gated":
        return h
    if op == "ckpt8":
        x, g, u = _eight(x), _eight(g), _eight(u)
    a, d = _gate(g, act)
    dh = s["dh"].double()
    dg, du = dh * u * d, dh * a
    dw = torch.cat([torch.einsum("bf,bi->fi", dg, x), torch.einsum("bf,bi->fi", du, x)])
    return h, torch.einsum("bf,fi->bi", dg, wg) + torch.einsum("bf,fi->bi", du, wu), dw
