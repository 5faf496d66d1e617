"""Workloads of the int8 products, the gated feed-forward block and the norms around a block: inputs, plain forms and
64-bit definitions.

The operators are the feed-forward half of a decoder block.  The block before it ends in a norm, a gate per channel and
a residual scale, and the sum is normalised (b, residual -> s, h); h goes through the gate and up projections and the
product of the two, in bf16 or fp32 with gradients, or in 8-bit integers with a scale per token and per output channel
(the quantiser that quantisation-aware whitening calibrates for).  Sizes follow the library's workloads (hidden 4096,
FFN 11008, 32768 and 65536 calibration tokens) or are ragged on purpose.
"""
import math

import torch

own = False

BLOCK = 64                       # channels that share one exponent in an 8-bit checkpoint
ACTS = ("none", "relu", "gelu", "silu")
EPS = 1e-5


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one generated token through a quantised attention or FFN projection
        {"name": "int8_token", "op": "int8", "T": 1, "d_in": 4096, "d_out": 11008, "dtype": "bf16", "act": "none",
         "bias": False, "residual": False},
        # a ragged decoding batch through a quantised down projection onto the residual stream
        {"name": "int8_batch", "op": "int8", "T": 37, "d_in": 11008, "d_out": 4096, "dtype": "bf16", "act": "none",
         "bias": True, "residual": True},
        # a prompt block through a quantised up projection
        {"name": "int8_ffn", "op": "int8", "T": 8192, "d_in": 4096, "d_out": 11008, "dtype": "bf16", "act": "gelu",
         "bias": True, "residual": False},
        # a decoding batch through the quantised gate and up projections
        {"name": "int8_gated_batch", "op": "int8_gated", "T": 32, "d_in": 4096, "d_ff": 11008, "dtype": "bf16",
         "act": "silu"},
        # a prompt through the quantised gate and up projections
        {"name": "int8_gated_prompt", "op": "int8_gated", "T": 2048, "d_in": 4096, "d_ff": 11008, "dtype": "bf16",
         "act": "silu"},
        # one generated token through gate and up
        {"name": "gated_token", "op": "gated", "T": 1, "d_in": 4096, "d_ff": 11008, "dtype": "bf16", "act": "silu",
         "save": "none"},
        # a calibration block through gate and up, both kept in 8 bits for the backward pass
        {"name": "gated_ffn", "op": "gated", "T": 8192, "d_in": 4096, "d_ff": 11008, "dtype": "bf16", "act": "silu",
         "save": "checkpoint"},
        # gradients of a small block, no size a multiple of a tile
        {"name": "gated_grad_ragged", "op": "gated_grad", "T": 1000, "d_in": 521, "d_ff": 303, "dtype": "bf16",
         "act": "gelu", "checkpoint": False},
        # gradients of a calibration block from 8-bit activations
        {"name": "gated_grad_ffn", "op": "gated_grad", "T": 8192, "d_in": 4096, "d_ff": 11008, "dtype": "bf16",
         "act": "silu", "checkpoint": True},
        # one generated token between two blocks of an 8-bit model: what leaves is quantised
        {"name": "norm_token", "op": "norm", "T": 1, "d": 4096, "dtype": "bf16", "kind": "rms", "post": False,
         "gate": False, "quantize": True},
        # the calibration stream between two blocks, norms on both sides of the sum
        {"name": "norm_stream", "op": "norm", "T": 65536, "d": 4096, "dtype": "bf16", "kind": "rms", "post": True,
         "gate": True, "quantize": False},
        # gradients of that
        {"name": "norm_grad_stream", "op": "norm_grad", "T": 32768, "d": 4096, "dtype": "bf16", "kind": "rms",
         "post": True, "gate": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths are multiples of 64, as models have them; the others are whatever comes."""
    w = _log(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(["int8", "int8_gated", "gated", "gated_grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        T, d = _log(rng, 1, 65536), _width(rng, 16, 11008)
        T = min(T, max(1, (65536 if op == "norm" else 32768) * 4096 // d // (1 if dtype == "bf16" else 2)))
        c = {"op": op, "T": T, "d": d, "dtype": dtype, "kind": rng.choice(["rms", "layer"]),
             "post": rng.random() < 0.5, "gate": rng.random() < 0.5}
        if op == "norm":
            c["quantize"] = dtype == "bf16" and rng.random() < 0.3
        return c
    T, d_in, d_out = _log(rng, 1, 8192), _width(rng, 16, 11008), _width(rng, 16, 11008)
    most = 8192 * 4096 * 11008 // (8 if dtype == "f32" and op.startswith("gated") else 4 if op == "int8_gated" else 1)
    T = max(1, min(T, most // (d_in * d_out)))
    c = {"op": op, "T": T, "d_in": d_in, "d_out" if op == "int8" else "d_ff": d_out, "dtype": dtype}
    if op == "int8":
        c.update(act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    else:
        c["act"] = rng.choice(("silu", "silu", "gelu", "relu", "none"))
    if op == "gated":
        c["save"] = rng.choice(["none", "z", "checkpoint"])
    if op == "gated_grad":
        c["checkpoint"] = rng.random() < 0.5
    return c


def work(case):
    T, op = case["T"], case["op"]
    b = 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_grad"):
        d = case["d"]
        n, vectors = T * d, 4 * d * (2 + 2 * case["post"] + case["gate"])
        if op == "norm":                  # block and residual in, sum and normed sum out
            return {"bytes": 3 * n * b + (n + 4 * T if case["quantize"] else n * b) + vectors, "flops": 16 * n}
        return {"bytes": 6 * n * b + 16 * T + 2 * vectors, "flops": 30 * n}
    i = case["d_in"]
    if op == "int8":
        o = case["d_out"]
        return {"bytes": b * T * (i + o * (2 if case["residual"] else 1)) + o * i + 4 * o * (2 if case["bias"] else 1),
                "flops": 2 * T * i * o}
    o = case["d_ff"]
    if op == "int8_gated":
        return {"bytes": b * T * (i + o) + 2 * o * i + 8 * o, "flops": 4 * T * i * o}
    zpack = 2 * (T * o + T * -(-o // BLOCK))
    if op == "gated":
        save = {"none": 0, "z": 2 * T * o * b, "checkpoint": 2 * zpack + 4 * T * o}[case["save"]]
        return {"bytes": b * (T * i + 2 * o * i + T * o) + save, "flops": 4 * T * i * o}
    xin = T * i + T * -(-i // BLOCK) if case["checkpoint"] else b * T * i
    zin = zpack if case["checkpoint"] else 2 * b * T * o
    return {"bytes": xin + zin + b * (3 * T * o + 4 * o * i + T * i), "flops": 8 * T * i * o}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _stream(g, T, d, power, scale=1.0):
    """Token rows with a power-law spectrum over the channels and 1 % outlier channels 20 times as large; every
    64th token is padding (zeros)."""
    lam = torch.arange(1, d + 1, device="cuda", dtype=torch.float32) ** (-power / 2)
    lam = lam * (scale / lam.square().mean().sqrt())
    lam = lam[torch.randperm(d, generator=g, device="cuda")]
    lam[torch.randperm(d, generator=g, device="cuda")[:int(round(0.01 * d))]] *= 20
    x = _normal(g, T, d) * lam
    x[63::64] = 0
    return x


def _int8_weight(g, o, i):
    w = _normal(g, o, i) / math.sqrt(i)
    return _quantize(w)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, dt, op = case["T"], _dt(case), case["op"]
    s = dict(case)
    if op in ("norm", "norm_grad"):
        d = case["d"]
        s["b"] = _stream(g, T, d, 0.5).to(dt)
        s["residual"] = (_stream(g, T, d, 0.5, 3.0) + 0.1 * _normal(g, d)).to(dt)
        rms = case["kind"] == "rms"
        params = lambda: (1 + 0.2 * _normal(g, d), None if rms else 0.1 * _normal(g, d))   # noqa: E731
        s["pre"] = params()
        s["after"] = params() if case["post"] else None
        s["gates"] = 0.3 + 0.1 * _normal(g, d) if case["gate"] else None
        s["scale"] = 0.75
        if op == "norm_grad":        # what the forward pass left, and the two gradients that come in
            total, _, s["stats"] = _block_norm(s)
            s["s"] = total.to(dt)
            s["dh"], s["ds"] = _stream(g, T, d, 1.0, 1e-2).to(dt), _stream(g, T, d, 1.0, 1e-2).to(dt)
            del s["residual"]
        return s
    i = case["d_in"]
    x = _stream(g, T, i, 0.5).to(dt)
    if op == "int8":
        o = case["d_out"]
        s["x"], s["W"] = x, _int8_weight(g, o, i)
        s["b"] = 0.1 * _normal(g, o) if case["bias"] else None
        s["res"] = _normal(g, T, o).to(dt) if case["residual"] else None
        return s
    o = case["d_ff"]
    if op == "int8_gated":
        s["x"], s["Wg"], s["Wu"] = x, _int8_weight(g, o, i), _int8_weight(g, o, i)
        return s
    s["Wg"] = (_normal(g, o, i) / math.sqrt(i)).to(dt)
    s["Wu"] = (_normal(g, o, i) / math.sqrt(i)).to(dt)
    if op == "gated":
        s["x"] = x
        return s
    z = [_normal(g, T, o) * (0.5 + 1.5 * torch.rand(o, generator=g, device="cuda")) for _ in range(2)]
    s["dh"] = _stream(g, T, o, 1.0, 1e-2).to(dt)
    s["x"] = _pack(x.float()) if case["checkpoint"] else x
    s["g"], s["u"] = [_pack(v) if case["checkpoint"] else v.to(dt) for v in z]
    return s


# ---------------------------------------------------------------------------------------
# plain forms, in 32 bits, rounded once
# ---------------------------------------------------------------------------------------
def _blocks(x):
    T, d = x.shape
    nb = -(-d // BLOCK)
    if nb * BLOCK != d:
        x = torch.cat([x, x.new_zeros(T, nb * BLOCK - d)], 1)
    return x.reshape(T, nb, BLOCK)


def _pow2(e):
    """2^e of integers, as the fp32 number that has that exponent (torch.ldexp's power is not exact)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _pack(x):
    """8-bit codes and exponents of fp32 rows: per 64 channels the smallest e with max|x| <= 127 * 2^e."""
    xb = _blocks(x)
    frac, e2 = torch.frexp(xb.abs().amax(2))
    e = (e2 - 7 + (frac * 128 > 127).int()).clamp(-126, 121)
    e = torch.where(frac == 0, torch.full_like(e, -126), e)
    q = (xb * _pow2(-e)[..., None]).round().clamp(-127, 127)
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]].to(torch.int8), e.to(torch.int8)


def _unpack(codes, exps):
    v = _blocks(codes.float()) * _pow2(exps)[..., None]
    return v.reshape(codes.shape[0], -1)[:, :codes.shape[1]]


def _values(t):
    return _unpack(*t) if isinstance(t, tuple) else t.float()


def _quantize(x):
    """Codes and scales of fp32 rows: scale = max|x| / 127, code = x / scale to the nearest, ties to even."""
    scale = x.abs().amax(1) / 127
    q = (x / scale[:, None]).round().clamp(-127, 127)
    return torch.where(scale[:, None] > 0, q, torch.zeros_like(q)).to(torch.int8), scale


def _held(codes, scale, dt):
    return (codes.float() * scale[:, None]).to(dt)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _moments(x, kind):
    """(mean or zero, 1 / spread) of rows."""
    mean = x.mean(1) if kind == "layer" else x.new_zeros(x.shape[0])
    return mean, 1 / torch.sqrt((x - mean[:, None]).square().mean(1) + EPS)


def _normed(x, mean, rstd, params):
    y = (x - mean[:, None]) * rstd[:, None] * params[0]
    return y if params[1] is None else y + params[1]


def _block_norm(s):
    b, mean_b, rstd_b = s["b"].float(), None, None
    p = b
    if s["after"] is not None:
        mean_b, rstd_b = _moments(b, s["kind"])
        p = _normed(b, mean_b, rstd_b, s["after"])
    if s["gates"] is not None:
        p = p * s["gates"]
    total = s["residual"].float() + s["scale"] * p
    mean, rstd = _moments(total, s["kind"])
    return total, _normed(total, mean, rstd, s["pre"]), (mean_b, rstd_b, mean, rstd)


def _norm_grad(dy, x, mean, rstd, gamma, kind):
    """dx and what gamma's gradient sums."""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    inner = g - xh * (g * xh).mean(1, keepdim=True)
    if kind == "layer":
        inner = inner - g.mean(1, keepdim=True)
    return inner * rstd[:, None], dy * xh


def _plain(s):
    dt, op = _dt(s), s["op"]
    if op == "norm":
        total, h, _ = _block_norm(s)
        h = h.to(dt)
        return {"s": total.to(dt), "h": _held(*_quantize(h.float()), dt) if s["quantize"] else h}
    if op == "norm_grad":
        mean_b, rstd_b, mean, rstd = s["stats"]
        dh, b = s["dh"].float(), s["b"].float()
        through, gx = _norm_grad(dh, s["s"].float(), mean, rstd, s["pre"][0], s["kind"])
        ds = s["ds"].float() + through
        out = {"dresidual": ds.to(dt), "dgamma": gx.sum(0)}
        if s["pre"][1] is not None:
            out["dbeta"] = dh.sum(0)
        dp = ds * s["scale"]
        if s["gates"] is not None:
            p = b if s["after"] is None else _normed(b, mean_b, rstd_b, s["after"])
            out["dgate"] = (dp * p).sum(0)
            dp = dp * s["gates"]
        db = dp
        if s["after"] is not None:
            db, gx = _norm_grad(dp, b, mean_b, rstd_b, s["after"][0], s["kind"])
            out["dpost_gamma"] = gx.sum(0)
            if s["after"][1] is not None:
                out["dpost_beta"] = dp.sum(0)
        out["db"] = db.to(dt)
        return out
    if op in ("int8", "int8_gated"):
        codes, scale = _quantize(s["x"].float())
        product = lambda w: (codes.float() @ w[0].float().T) * scale[:, None] * w[1]   # noqa: E731
        if op == "int8_gated":
            return {"h": (_act(product(s["Wg"]), s["act"]) * product(s["Wu"])).to(dt)}
        z = product(s["W"])
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(z, s["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(dt)}
    if op == "gated":
        x = s["x"].float()
        g, u = x @ s["Wg"].float().T, x @ s["Wu"].float().T
        out = {"h": (_act(g, s["act"]) * u).to(dt)}
        if s["save"] == "z":
            out["g"], out["u"] = g.to(dt), u.to(dt)
        if s["save"] == "checkpoint":                        # the held values are exact in bf16
            out["g"], out["u"] = _unpack(*_pack(g)).to(torch.bfloat16), _unpack(*_pack(u)).to(torch.bfloat16)
        return out
    dh, g, u, x = s["dh"].float(), _values(s["g"]), _values(s["u"]), _values(s["x"])
    dg, du = dh * u * _act_grad(g, s["act"]), dh * _act(g, s["act"])
    dx = dg @ s["Wg"].float() + du @ s["Wu"].float()
    return {"dg": dg.to(dt), "du": du.to(dt), "dx": dx.to(dt), "dwg": (dg.T @ x).to(dt), "dwu": (du.T @ x).to(dt)}


def run(s):
    if not own:
        return _plain(s)
    import curvature_aware_rank_amd as lrc

    op = s["op"]
    if op == "norm":
        total, h, _, quantized, _ = lrc.lrc_block_norm(s["b"], s["residual"], kind=s["kind"], eps=EPS, post=s["after"],
                                                       gate=s["gates"], scale=s["scale"], pre=s["pre"],
                                                       quantize=s["quantize"])
        return {"s": total, "h": _held(*quantized, total.dtype) if s["quantize"] else h}
    if op == "norm_grad":
        dr, db, dgamma, dbeta, dpost_gamma, dpost_beta, dgate = lrc.lrc_block_norm_backward(
            s["dh"], s["ds"], s["s"], s["b"], s["stats"], kind=s["kind"], post=s["after"], gate=s["gates"],
            scale=s["scale"], pre=s["pre"])
        out = {"dresidual": dr, "dgamma": dgamma, "dbeta": dbeta, "dgate": dgate, "dpost_gamma": dpost_gamma,
               "dpost_beta": dpost_beta, "db": db}
        return {k: v for k, v in out.items() if v is not None}
    if op == "int8":
        y, _ = lrc.lrc_int8_linear(s["x"], s["W"], s["b"], act=s["act"], residual=s["res"])
        return {"y": y}
    if op == "int8_gated":
        h, _ = lrc.lrc_int8_gated_linear(s["x"], s["Wg"], s["Wu"], act=s["act"])
        return {"h": h}
    if op == "gated":
        h, saved, _ = lrc.lrc_gated_linear(s["x"], s["Wg"], s["Wu"], act=s["act"], save=s["save"])
        out = {"h": h}
        if s["save"] == "z":
            out["g"], out["u"] = saved
        if s["save"] == "checkpoint":
            out["g"], out["u"] = lrc.lrc_unpack_activations(*saved[0]), lrc.lrc_unpack_activations(*saved[1])
        return out
    dg, du, dx, dwg, dwu = lrc.lrc_gated_linear_backward(s["dh"], s["x"], s["Wg"], s["Wu"], s["g"], s["u"],
                                                         act=s["act"])
    return {"dg": dg, "du": du, "dx": dx, "dwg": dwg, "dwu": dwu}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _kept(v):
    """The values that 8 bits keep of double rows: column blocks one after the other."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], BLOCK):
        b = v[:, c:c + BLOCK]
        m = b.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(m / 127)).clamp(-126, 121)
        e = torch.where(m > 127 * _two_to(e), e + 1, e)
        e = torch.where(m <= 127 * _two_to(e - 1), e - 1, e).clamp(-126, 121)
        step = _two_to(e)
        out[:, c:c + BLOCK] = (b / step).round().clamp(-127, 127) * step
    return out


def _of_codes(t):
    if not isinstance(t, tuple):
        return t.double()
    codes, exps = t
    return codes.double() * _two_to(exps).repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _int8_rows(x):
    """Codes (as doubles) and steps of rows; the quantiser's two quotients are fp32 numbers by definition, which a
    double quotient rounded to fp32 gives."""
    step = (x.abs().max(1, keepdim=True).values / 127).float().double()
    q = torch.clamp((x / step).float().double().round(), -127, 127)
    return torch.nan_to_num(q, nan=0.0), step


def _curve(z, act):
    """An activation and its slope."""
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * (-z * z / 2).exp() * (2 * math.pi) ** -0.5
    return z, torch.ones_like(z)


def _standard(x, kind):
    """Rows centred (layer) and divided by their spread, and 1 / spread."""
    if kind == "layer":
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        x = x - mean
    else:
        var = x.pow(2).mean(1, keepdim=True)
    r = (var + EPS) ** -0.5
    return x * r, r


def _affine(xh, params):
    return xh * params[0].double() + (0 if params[1] is None else params[1].double())


def _back(dy, xh, r, kind):
    """Through a standardised row: dy already times gamma."""
    d = xh.shape[1]
    out = dy - xh * (torch.linalg.vecdot(dy, xh) / d)[:, None]
    if kind == "layer":
        out = out - dy.mean(1, keepdim=True)
    return out * r


def _through(x, mean, rstd):
    r = rstd.double()[:, None]
    return (x.double() - mean.double()[:, None]) * r, r


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        p = s["b"].double()
        if s["after"] is not None:
            p = _affine(_standard(p, s["kind"])[0], s["after"])
        weight = torch.full((case["d"],), s["scale"], dtype=torch.float64, device=p.device)
        if s["gates"] is not None:
            weight = weight * s["gates"].double()
        total = torch.addcmul(s["residual"].double(), p, weight)
        h = _affine(_standard(total, s["kind"])[0], s["pre"])
        if s["quantize"]:
            q, step = _int8_rows(h.to(_dt(case)).double())      # what is quantised is h in its own type
            h = q * step
        return {"s": total, "h": h}
    if op == "norm_grad":
        mean_b, rstd_b, mean, rstd = s["stats"]
        xh, r = _through(s["s"], mean, rstd)
        dh, kind = s["dh"].double(), s["kind"]
        ds = s["ds"].double() + _back(dh * s["pre"][0].double(), xh, r, kind)
        out = {"dresidual": ds, "dgamma": torch.einsum("td,td->d", dh, xh)}
        if s["pre"][1] is not None:
            out["dbeta"] = dh.sum(0)
        weight = s["scale"] * (1.0 if s["gates"] is None else s["gates"].double())
        if s["after"] is None:
            out["db"] = ds * weight
            if s["gates"] is not None:
                out["dgate"] = torch.einsum("td,td->d", ds, s["b"].double()) * s["scale"]
        else:
            bh, rb = _through(s["b"], mean_b, rstd_b)
            out["db"] = _back(ds * (weight * s["after"][0].double()), bh, rb, kind)
            along, plain = torch.einsum("td,td->d", ds, bh), ds.sum(0)
            if s["gates"] is not None:
                out["dgate"] = s["scale"] * (along * s["after"][0].double()
                                             + (0 if s["after"][1] is None else plain * s["after"][1].double()))
            out["dpost_gamma"] = along * weight
            if s["after"][1] is not None:
                out["dpost_beta"] = plain * weight
        order = ("dresidual", "dgamma", "dbeta", "dgate", "dpost_gamma", "dpost_beta", "db")
        return {k: out[k] for k in order if k in out}
    if op in ("int8", "int8_gated"):
        q, step = _int8_rows(s["x"].double())
        product = lambda w: torch.mm(q, w[0].double().t()) * (step * w[1].double())   # noqa: E731
        if op == "int8_gated":
            return {"h": _curve(product(s["Wg"]), case["act"])[0] * product(s["Wu"])}
        y = product(s["W"])
        if s["b"] is not None:
            y += s["b"].double()
        y = _curve(y, case["act"])[0]
        if s["res"] is not None:
            y = y + s["res"].double()
        return {"y": y}
    if op == "gated":
        x = s["x"].double()
        g, u = torch.mm(x, s["Wg"].double().t()), torch.mm(x, s["Wu"].double().t())
        out = {"h": _curve(g, case["act"])[0] * u}
        if case["save"] != "none":
            out["g"], out["u"] = (g, u) if case["save"] == "z" else (_kept(g), _kept(u))
        return out
    a, slope = _curve(_of_codes(s["g"]), case["act"])
    dh, x = s["dh"].double(), _of_codes(s["x"])
    du, dg = dh * a, dh * _of_codes(s["u"]) * slope
    dx = torch.addmm(torch.mm(dg, s["Wg"].double()), du, s["Wu"].double())
    return {"dg": dg, "du": du, "dx": dx, "dwg": torch.mm(dg.t(), x), "dwu": torch.mm(du.t(), x)}
