"""Workloads of the layer-norm, linear and 8-bit checkpoint operators: inputs, plain forms and 64-bit definitions.

The operators are those of a calibration or healing step of one normalised linear layer: a token block x (T, d) is
normalised, multiplied by a weight W (d_out, d_in) with bias, activation and residual, and differentiated from
activations that were kept in 8 bits.  Sizes follow the library's workloads (hidden 4096, FFN 11008, rank 1024,
32768 and 65536 calibration tokens) or are ragged on purpose.
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
        # one generated token through a norm: latency only
        {"name": "norm_token", "op": "norm", "T": 1, "d": 4096, "dtype": "bf16", "checkpoint": False},
        # the calibration stream of an attention projection, its input kept in 8 bits by the same pass
        {"name": "norm_calibration", "op": "norm", "T": 65536, "d": 4096, "dtype": "bf16", "checkpoint": True},
        # a small fp32 model's norm, widths that fit no vector
        {"name": "norm_grad_ragged", "op": "norm_grad", "T": 4099, "d": 301, "dtype": "f32", "checkpoint": False},
        # backward of the norm in a decoder layer from its 8-bit input
        {"name": "norm_grad_checkpoint", "op": "norm_grad", "T": 32768, "d": 4096, "dtype": "bf16",
         "checkpoint": True},
        # one generated token through an FFN gate
        {"name": "linear_token", "op": "linear", "T": 1, "d_in": 4096, "d_out": 11008, "dtype": "bf16",
         "act": "silu", "bias": False, "residual": False, "save": "none"},
        # a decoding batch through an FFN's down projection onto the residual stream
        {"name": "linear_batch", "op": "linear", "T": 24, "d_in": 11008, "d_out": 4096, "dtype": "bf16",
         "act": "none", "bias": True, "residual": True, "save": "none"},
        # a calibration block through an FFN's up projection, pre-activations kept in 8 bits
        {"name": "linear_ffn", "op": "linear", "T": 8192, "d_in": 4096, "d_out": 11008, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False, "save": "checkpoint"},
        # the left factor of a rank-1024 decomposition applied in fp32 (the factors' own type)
        {"name": "linear_factor_f32", "op": "linear", "T": 8192, "d_in": 1024, "d_out": 4096, "dtype": "f32",
         "act": "none", "bias": True, "residual": True, "save": "none"},
        # backward of a small layer, no size a multiple of a tile
        {"name": "linear_grad_ragged", "op": "linear_grad", "T": 1000, "d_in": 521, "d_out": 303, "dtype": "bf16",
         "act": "relu", "checkpoint": False},
        # backward of an FFN's up projection from 8-bit activations and pre-activations
        {"name": "linear_grad_ffn", "op": "linear_grad", "T": 8192, "d_in": 4096, "d_out": 11008, "dtype": "bf16",
         "act": "gelu", "checkpoint": True},
        # a small fp32 stream into and out of its checkpoint
        {"name": "checkpoint_small", "op": "checkpoint", "T": 4096, "d": 256, "dtype": "f32"},
        # the FFN's hidden activations of a calibration block
        {"name": "checkpoint_ffn", "op": "checkpoint", "T": 32768, "d": 11008, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths are multiples of 64, as models have them; the others are whatever comes."""
    w = _log(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "linear_grad", "linear_grad", "checkpoint"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad", "checkpoint"):
        T, d = _log(rng, 1, 65536), _width(rng, 16, 11008)
        T = min(T, max(1, 65536 * 4096 // d))
        c = {"op": op, "T": T, "d": d, "dtype": dtype}
        if op != "checkpoint":
            c["checkpoint"] = rng.random() < 0.5
        return c
    T, d_in, d_out = _log(rng, 1, 8192), _width(rng, 16, 11008), _width(rng, 16, 11008)
    most = 8192 * 4096 * 11008 // (1 if dtype == "bf16" else 8)
    T = max(1, min(T, most // (d_in * d_out)))
    c = {"op": op, "T": T, "d_in": d_in, "d_out": d_out, "dtype": dtype, "act": rng.choice(ACTS)}
    if op == "linear":
        c.update(bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                 save=rng.choice(["none", "none", "checkpoint", "z"]))
    else:
        c["checkpoint"] = rng.random() < 0.5
    return c


def work(case):
    T = case["T"]
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_grad", "checkpoint"):
        d = case["d"]
        n, packed = T * d, T * d + T * -(-d // BLOCK)
        if case["op"] == "norm":                      # x in, y out, statistics, parameters; the checkpoint out and in
            return {"bytes": 2 * n * b + 8 * T + 8 * d + (2 * packed + n * b if case["checkpoint"] else 0),
                    "flops": 8 * n}
        if case["op"] == "norm_grad":                 # dy and x in, dx out, statistics, gamma and both gradients
            return {"bytes": 2 * n * b + (packed if case["checkpoint"] else n * b) + 8 * T + 12 * d,
                    "flops": 14 * n}
        return {"bytes": 2 * n * b + 2 * packed, "flops": 4 * n}
    i, o = case["d_in"], case["d_out"]
    zpack = T * o + T * -(-o // BLOCK)
    if case["op"] == "linear":
        save = {"none": 0, "z": T * o * b, "checkpoint": 2 * zpack + 2 * T * o}[case["save"]]
        return {"bytes": b * (T * i + o * i + T * o * (2 if case["residual"] else 1)) + (4 * o if case["bias"] else 0)
                + save, "flops": 2 * T * i * o}
    xin = T * i + T * -(-i // BLOCK) if case["checkpoint"] else b * T * i
    zin = 0 if case["act"] == "none" else zpack if case["checkpoint"] else b * T * o
    dz = 0 if case["act"] == "none" else b * T * o
    return {"bytes": xin + zin + dz + b * (T * o + 2 * o * i + T * i) + 4 * o, "flops": 4 * T * i * o}


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, dt = case["T"], _dt(case)
    s = dict(case)
    if case["op"] in ("norm", "norm_grad", "checkpoint"):
        d = case["d"]
        x = (_stream(g, T, d, 0.5) + 0.1 * _normal(g, d)).to(dt)
        s["x"] = x
        if case["op"] != "checkpoint":
            s["gamma"] = 1 + 0.2 * _normal(g, d)
            s["beta"] = 0.1 * _normal(g, d)
        if case["op"] == "norm_grad":
            s["dy"] = _stream(g, T, d, 1.0, 1e-2).to(dt)
            xf = x.float()
            s["mean"] = xf.mean(1)
            s["rstd"] = 1 / torch.sqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
            if case["checkpoint"]:
                s["x"] = _pack(x.float())
        return s
    i, o = case["d_in"], case["d_out"]
    x = _stream(g, T, i, 0.5).to(dt)
    s["W"] = (_normal(g, o, i) / math.sqrt(i)).to(dt)
    if case["op"] == "linear":
        s["x"] = x
        s["b"] = 0.1 * _normal(g, o) if case["bias"] else None
        s["res"] = _normal(g, T, o).to(dt) if case["residual"] else None
        return s
    s["dy"] = _stream(g, T, o, 1.0, 1e-2).to(dt)
    z = _normal(g, T, o) * (0.5 + 1.5 * torch.rand(o, generator=g, device="cuda"))
    s["x"] = _pack(x.float()) if case["checkpoint"] else x
    s["z"] = None if case["act"] == "none" else _pack(z) if case["checkpoint"] else z.to(dt)
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


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _plain(s):
    dt = _dt(s)
    if s["op"] == "checkpoint":
        codes, exps = _pack(s["x"].float())
        return {"x": _unpack(codes, exps).to(dt), "exps": exps}
    if s["op"] == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1 / torch.sqrt(c.square().mean(1) + EPS)
        out = {"y": (c * rstd[:, None] * s["gamma"] + s["beta"]).to(dt), "mean": mean, "rstd": rstd}
        if s["checkpoint"]:
            out["x"] = _unpack(*_pack(x)).to(dt)
        return out
    if s["op"] == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (_values(s["x"]) - s["mean"][:, None]) * rstd
        g = dy * s["gamma"]
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    if s["op"] == "linear":
        z = s["x"].float() @ s["W"].float().T
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(z, s["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        out = {"y": y.to(dt)}
        if s["save"] == "z":
            out["z"] = z.to(dt)
        if s["save"] == "checkpoint":
            out["z"] = _unpack(*_pack(z)).to(torch.bfloat16)      # the held values are exact in bf16
        return out
    dz = s["dy"].float()
    if s["act"] != "none":
        dz = dz * _act_grad(_values(s["z"]), s["act"])
    return {"dz": dz.to(dt), "dx": (dz @ s["W"].float()).to(dt), "dw": (dz.T @ _values(s["x"])).to(dt),
            "db": dz.sum(0)}


def run(s):
    if not own:
        return _plain(s)
    import curvature_aware_rank_amd as lrc

    if s["op"] == "checkpoint":
        codes, exps, _ = lrc.lrc_pack_activations(s["x"])
        return {"x": lrc.lrc_unpack_activations(codes, exps, s["x"].dtype), "exps": exps}
    if s["op"] == "norm":
        y, mean, rstd, kept, _ = lrc.lrc_layer_norm(s["x"], s["gamma"], s["beta"], EPS, checkpoint=s["checkpoint"])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if s["checkpoint"]:
            out["x"] = lrc.lrc_unpack_activations(kept[0], kept[1], y.dtype)
        return out
    if s["op"] == "norm_grad":
        dx, dgamma, dbeta = lrc.lrc_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if s["op"] == "linear":
        y, z, _ = lrc.lrc_linear(s["x"], s["W"], s["b"], act=s["act"], residual=s["res"], save=s["save"])
        out = {"y": y}
        if s["save"] == "z":
            out["z"] = z
        if s["save"] == "checkpoint":
            out["z"] = lrc.lrc_unpack_activations(z[0], z[1])
        return out
    dz, dx, dw, db = lrc.lrc_linear_backward(s["dy"], s["x"], s["W"], act=s["act"], z=s["z"])
    return {"dz": dz, "dx": dx, "dw": dw, "db": db}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _held(v):
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


def _normal_cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        return {"x": _held(s["x"].double()), "exps": None}
    if op in ("norm", "norm_grad"):
        x = _of_codes(s["x"])
        gamma = s["gamma"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + EPS) ** -0.5
            y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], gamma)
            return {"y": y, "mean": mean, "rstd": rstd, **({"x": _held(x)} if case["checkpoint"] else {})}
        dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        xh, n = (x - mean) * rstd, case["d"]
        along = (dy * xh) @ gamma / n
        dx = (dy * gamma - ((dy @ gamma) / n)[:, None] - xh * along[:, None]) * rstd
        return {"dx": dx, "dgamma": torch.einsum("td,td->d", dy, xh), "dbeta": dy.sum(0)}
    W = s["W"].double()
    if op == "linear":
        z = torch.mm(s["x"].double(), W.t())
        if s["b"] is not None:
            z += s["b"].double()
        y = {"none": lambda: z.clone(), "relu": lambda: z.clamp_min(0), "gelu": lambda: z * _normal_cdf(z),
             "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
        if s["res"] is not None:
            y += s["res"].double()
        return {"y": y, **({"z": z} if case["save"] == "z" else {"z": _held(z)} if case["save"] == "checkpoint" else {})}
    dz = s["dy"].double()
    if case["act"] != "none":
        z = _of_codes(s["z"])
        sig = torch.sigmoid(z)
        dz *= {"relu": lambda: (z > 0).double(), "silu": lambda: sig + z * sig * (1 - sig),
               "gelu": lambda: _normal_cdf(z) + z * (-z * z / 2).exp() * (2 * math.pi) ** -0.5}[case["act"]]()
    return {"dz": dz, "dx": torch.mm(dz, W), "dw": torch.mm(dz.t(), _of_codes(s["x"])), "db": dz.sum(0)}
