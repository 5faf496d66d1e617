"""Layer norm, linear layer and 8-bit activation checkpoints on the GPU against their fp64 definitions.

Tolerances.  u = 2^-24.  A fp32 sum of K terms in any order is off by at most (K + c) u times the sum of the
terms' magnitudes; the matrix cores' internal adds are counted as two roundings each.  An output held in bf16
adds half a step, 2^-8 of its value.  Bounds are elementwise and computed in fp64 from the same inputs.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import train_oracle as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float32]
ACTS = ["none", "relu", "gelu", "silu"]
LIP = 1.13        # largest slope of the four activations (gelu 1.1289..., silu 1.0998...)
LAYOUTS = ["packed", "padded", "offset", "transposed"]


@pytest.fixture(scope="module")
def lrc():
    import curvature_aware_rank_amd as m
    return m


def dev():
    return torch.device("cuda:0")


def f64(t):
    return t.detach().double().cpu().numpy()


def lay(t, layout):
    """The CPU matrix `t` on the GPU in another layout; what lies between its rows is NaN."""
    n, d = t.shape
    if layout == "padded":
        b = torch.full((n, d + 24), float("nan"), dtype=t.dtype, device=dev())
        b[:, 8:8 + d] = t.to(dev())
        return b[:, 8:8 + d]
    if layout == "offset":       # an odd pitch and an odd start: no 16-byte piece is aligned
        b = torch.full((n * (d + 3) + 1,), float("nan"), dtype=t.dtype, device=dev())
        v = b[1:].view(n, d + 3)[:, :d]
        v.copy_(t)
        return v
    if layout == "transposed":
        return t.t().contiguous().to(dev()).t()
    return t.to(dev())


def stream(n, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g) * torch.exp(torch.randn(d, generator=g)) * scale + 0.1
    if n > 3:
        x[2] = 0          # a padding token
    return x.to(dtype)


def check(got, want, bound, what):
    """|got - want| <= bound elementwise."""
    got = f64(got)
    assert got.shape == want.shape, what
    over = np.abs(got - want) - bound
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert not over.size or over[i] <= 0, (what, i, got[i], want[i], bound[i] if np.ndim(bound) else bound)


# ----------------------------------------------------------------------------- 8-bit checkpoints
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 1), (3, 7), (5, 63), (1, 64), (7, 65), (4, 128), (33, 200), (2, 4096),
                                 (130, 1000), (3, 11008)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_pack_bit_exact(lrc, dtype, n, d, layout):
    x = stream(n, d, dtype, n * 31 + d)
    codes, exps, info = lrc.lrc_pack_activations(lay(x, layout))
    qc, qe = ref.pack(f64(x))
    assert np.array_equal(codes.cpu().numpy(), qc) and np.array_equal(exps.cpu().numpy(), qe)
    assert int(info.cpu()) == 0
    for dt in DTYPES:    # what is held is exact in both types
        v = lrc.lrc_unpack_activations(codes, exps, dt)
        assert v.dtype == dt and np.array_equal(f64(v), ref.unpack(qc, qe))


def test_pack_borders(lrc):
    """Ties, borders of the exponent, the ends of the range, subnormals and zeros."""
    big = float(np.finfo(np.float32).max)
    rows = [[127.0, 0.5, 1.5, -2.5, 126.5], [127.00001, 1.0, 3.0, -5.0, 0.0], [254.0, 1.0, 3.0, 5.0, 7.0],
            [128.0, 1.0, -1.0, 2.0, 3.0], [big, 1.0, -big, 0.0, big / 2], [127 * 2.0 ** 121, 2.0 ** 120, 0, 0, 0],
            [2.0 ** -149, -2.0 ** -140, 0, 0, 0], [2.0 ** -126, -2.0 ** -120, 2.0 ** -127, 0, 0], [0.0, -0.0, 0, 0, 0]]
    x = torch.tensor(rows, dtype=torch.float32)
    codes, exps, info = lrc.lrc_pack_activations(x.to(dev()))
    qc, qe = ref.pack(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), qc) and np.array_equal(exps.cpu().numpy(), qe)
    assert int(info.cpu()) == 0
    assert torch.isfinite(lrc.lrc_unpack_activations(codes, exps, torch.bfloat16)).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_pack_nonfinite(lrc, dtype):
    """NaN and infinities are flagged and do not spoil their block's exponent."""
    x = stream(6, 150, dtype, 3)
    x[1, 70], x[3, 0], x[4, 149] = float("nan"), float("inf"), float("-inf")
    codes, exps, info = lrc.lrc_pack_activations(x.to(dev()))
    qc, qe = ref.pack(f64(x))
    assert np.array_equal(codes.cpu().numpy(), qc) and np.array_equal(exps.cpu().numpy(), qe)
    assert qc[1, 70] == 0 and qc[3, 0] == 127 and qc[4, 149] == -127
    assert int(info.cpu()) == lrc.LRC_ENONFINITE
    # the flag is sticky
    _, _, again = lrc.lrc_pack_activations(stream(2, 9, dtype, 4).to(dev()), info=info)
    assert again is info and int(info.cpu()) == lrc.LRC_ENONFINITE


# ----------------------------------------------------------------------------- layer norm
NORM_SHAPES = [(1, 1), (5, 2), (3, 7), (2, 64), (65, 65), (1, 4096), (300, 300), (9, 1000), (70, 1024), (3, 8200),
               (4, 11008), (2, 20000)]


def norm_bounds(x, mean, rstd, gamma, beta, half):
    """Forward: sums of d terms over per-thread runs and a tree, at most d / 64 + 24 deep."""
    d = x.shape[1]
    k = (d / 64 + 24) * U
    e_mean = k * np.abs(x).mean(1) + U * np.abs(mean)
    c = x - mean[:, None]
    e_c = e_mean[:, None] + 2 * U * (np.abs(c) + np.abs(mean)[:, None])
    var = (c * c).mean(1)
    e_var = 2 * (np.abs(c) * e_c).mean(1) + (e_c * e_c).mean(1) + (k + 2 * U) * var
    rel = 0.5 * e_var * rstd ** 2 / np.maximum(1 - e_var * rstd ** 2, 0.5) + 4 * U
    xh = c * rstd[:, None]
    e_xh = (e_c * rstd[:, None] + np.abs(xh) * (rel[:, None] + 2 * U)) * 1.01
    y = xh * gamma + beta
    e_y = e_xh * np.abs(gamma) + 2 * U * (np.abs(xh * gamma) + np.abs(beta))
    return e_mean + 1e-37, rel * rstd, e_y + half * (np.abs(y) + e_y) + 1e-37


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", NORM_SHAPES)
def test_layer_norm(lrc, dtype, n, d):
    g = torch.Generator().manual_seed(d)
    x = stream(n, d, dtype, n + d)
    gamma, beta = 1 + 0.2 * torch.randn(d, generator=g), 0.1 * torch.randn(d, generator=g)
    for layout in LAYOUTS if d < 2000 else ["packed", "offset"]:
        for affine in (True, False):
            xl = lay(x, layout)
            ga, be = (gamma.to(dev()), beta.to(dev())) if affine else (None, None)
            y, mean, rstd, kept, info = lrc.lrc_layer_norm(xl, ga, be, 1e-5, checkpoint=affine)
            gn, bn = (f64(gamma), f64(beta)) if affine else (np.ones(d), np.zeros(d))
            wy, wm, wr = ref.layer_norm(f64(x), gn, bn, float(np.float32(1e-5)))
            bm, br, by = norm_bounds(f64(x), wm, wr, gn, bn, HALF[dtype])
            check(mean, wm, bm, "mean")
            check(rstd, wr, br, "rstd")
            check(y, wy, by, "y")
            if affine:   # the checkpoint written by the same pass is the packed input, bit for bit
                codes, exps, _ = lrc.lrc_pack_activations(xl)
                assert torch.equal(kept[0], codes) and torch.equal(kept[1], exps) and int(info.cpu()) == 0
            else:
                assert kept is None and info is None


def norm_grad_bounds(dy, x, mean, rstd, gamma, half):
    d = x.shape[1]
    k = (d / 64 + 24) * U
    m, r = mean[:, None], rstd[:, None]
    xh = (x - m) * r
    e_xh = U * (np.abs(x) + np.abs(m)) * r + 2 * U * np.abs(xh)
    g = dy * gamma
    e_c1 = (k + 2 * U) * np.abs(g).mean(1)[:, None]
    e_c2 = (k + 4 * U) * np.abs(g * xh).mean(1)[:, None] + (np.abs(g) * e_xh).mean(1)[:, None]
    c1, c2 = g.mean(1)[:, None], (g * xh).mean(1)[:, None]
    inner = np.abs(g) + np.abs(c1) + np.abs(xh * c2)
    e = r * (4 * U * inner + e_c1 + np.abs(xh) * e_c2 + e_xh * np.abs(c2)) * 1.01
    dx = r * (g - c1 - xh * c2)
    n = x.shape[0]
    e_dg = (n + 8) * U * np.abs(dy * xh).sum(0) + (np.abs(dy) * e_xh).sum(0)
    return e + half * (np.abs(dx) + e) + 1e-37, e_dg + 1e-37, (n + 8) * U * np.abs(dy).sum(0) + 1e-37


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", NORM_SHAPES + [(1300, 40), (700, 512)])
@pytest.mark.parametrize("held", [False, True])
def test_layer_norm_backward(lrc, dtype, n, d, held):
    g = torch.Generator().manual_seed(d + 1)
    x, dy = stream(n, d, dtype, n + d), stream(n, d, dtype, n + d + 7, 0.01)
    gamma = 1 + 0.2 * torch.randn(d, generator=g)
    for layout in ["packed", "padded", "offset"] if d < 2000 else ["packed", "offset"]:
        xl = lay(x, layout)
        _, mean, rstd, kept, _ = lrc.lrc_layer_norm(xl, None, None, 1e-5, checkpoint=held)
        for affine in (True, False):
            ga = gamma.to(dev()) if affine else None
            dx, dgamma, dbeta = lrc.lrc_layer_norm_backward(lay(dy, layout), kept if held else xl, mean, rstd, ga)
            xin = ref.unpack(f64(kept[0]).astype(np.int8), f64(kept[1]).astype(np.int8)) if held else f64(x)
            gn = f64(gamma) if affine else np.ones(d)
            args = (f64(dy), xin, f64(mean), f64(rstd), gn)
            wx, wg, wb = ref.layer_norm_backward(*args)
            bx, bg, bb = norm_grad_bounds(*args, HALF[dtype])
            check(dx, wx, bx, "dx")
            check(dgamma, wg, bg, "dgamma")
            check(dbeta, wb, bb, "dbeta")


def test_layer_norm_backward_parts_and_differences(lrc):
    """Each output alone equals the joint call; the gradient against central differences of the fp64 forward."""
    n, d = 6, 37
    x, dy = stream(n, d, torch.float32, 1), stream(n, d, torch.float32, 2)
    gamma = 1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(3))
    _, mean, rstd, _, _ = lrc.lrc_layer_norm(x.to(dev()), gamma.to(dev()))
    a = (dy.to(dev()), x.to(dev()), mean, rstd, gamma.to(dev()))
    dx, dgamma, dbeta = lrc.lrc_layer_norm_backward(*a)
    only, none1, none2 = lrc.lrc_layer_norm_backward(*a, need_dparams=False)
    assert torch.equal(only, dx) and none1 is None and none2 is None
    none, dg, db = lrc.lrc_layer_norm_backward(*a, need_dx=False)
    assert none is None and torch.equal(dg, dgamma) and torch.equal(db, dbeta)
    loss = lambda xx, gg: (ref.layer_norm(xx, gg, 0.0, 1e-5)[0] * f64(dy)).sum()   # noqa: E731
    h = 1e-5
    # rows with a spread of about one: the third derivative is of order |dy| / spread^3, so the
    # differences are good to h^2 d * max|dy| ~ 1e-7, the GPU's fp32 to about 1e-5
    for t, j in [(0, 0), (1, 17), (4, 36), (5, 20)]:
        e = np.zeros((n, d))
        e[t, j] = h
        want = (loss(f64(x) + e, f64(gamma)) - loss(f64(x) - e, f64(gamma))) / (2 * h)
        assert abs(float(dx[t, j]) - want) < 1e-4 * max(1.0, abs(want))
    e = np.zeros(d)
    e[11] = h
    want = (loss(f64(x), f64(gamma) + e) - loss(f64(x), f64(gamma) - e)) / (2 * h)
    assert abs(float(dgamma[11]) - want) < 1e-4 * max(1.0, abs(want))


# ----------------------------------------------------------------------------- linear
LINEAR_SHAPES = [(1, 1, 1), (3, 5, 7), (1, 64, 96), (2, 512, 130), (16, 96, 64), (17, 257, 33), (33, 128, 200),
                 (64, 1000, 48), (65, 64, 65), (100, 300, 520), (130, 72, 256), (257, 136, 264), (600, 520, 136)]


def linear_bounds(x, w, b, res, z, y, name, half):
    k = (x.shape[1] + 8) * 2 * U
    e_z = k * (np.abs(x) @ np.abs(w).T) + 2 * U * (np.abs(b) + np.abs(z))
    e_y = LIP * e_z + 8 * U * (np.abs(z) + np.abs(res)) + 8 * U * np.abs(y)
    return e_z + half * (np.abs(z) + e_z) + 1e-37, e_y + half * (np.abs(y) + e_y) + 1e-37


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_out", LINEAR_SHAPES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_linear(lrc, dtype, n, d_in, d_out, layout):
    g = torch.Generator().manual_seed(n + d_in)
    x = stream(n, d_in, dtype, n + d_in)
    w = (torch.randn(d_out, d_in, generator=g) / math.sqrt(d_in)).to(dtype)
    b = torch.randn(d_out, generator=g)
    res = stream(n, d_out, dtype, 5)
    for i, name in enumerate(ACTS):
        with_b, with_r = i != 1, i % 2 == 0
        for save in ["none", "z", "checkpoint"]:
            y, kept, info = lrc.lrc_linear(lay(x, layout), lay(w, layout), b.to(dev()) if with_b else None, act=name,
                                           residual=lay(res, layout) if with_r else None, save=save)
            bn = f64(b) if with_b else np.zeros(d_out)
            rn = f64(res) if with_r else np.zeros((n, d_out))
            wy, wz = ref.linear(f64(x), f64(w), bn, name, rn)
            bz, by = linear_bounds(f64(x), f64(w), bn, rn, wz, wy, name, HALF[dtype])
            check(y, wy, by, ("y", name, save))
            if save == "z":
                check(kept, wz, bz, ("z", name))
            elif save == "checkpoint":
                # within one half step of the block's exponent (and the fp32 error of z); the exponent
                # is the one of a z within that error
                held = f64(lrc.lrc_unpack_activations(*kept))
                bz, _ = linear_bounds(f64(x), f64(w), bn, rn, wz, wy, name, 0.0)
                step = np.repeat(2.0 ** f64(kept[1]), 64, 1)[:, :d_out]
                assert (np.abs(held - wz) <= 0.5 * step + bz).all(), name
                lo, hi = (ref.pack(np.abs(wz) + s * bz)[1] for s in (-1, 1))
                e = kept[1].cpu().numpy()
                assert (e <= np.maximum(lo, hi)).all() and int(info.cpu()) == 0
            else:
                assert kept is None and info is None


@pytest.mark.parametrize("n,d_in,d_out", [(1, 4096, 1000), (7, 11008, 256), (40, 2048, 520), (96, 4096, 512),
                                          (300, 4096, 1032), (1500, 264, 2056), (520, 1032, 4104), (2100, 96, 520)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_exact_on_small_integers(lrc, dtype, n, d_in, d_out):
    """Small integers: every product and partial sum is an integer below 2^24, so the fp32 sums are exact in any
    order and y is the rounded integer.  Catches a dropped, repeated or misplaced tile, step or split."""
    g = torch.Generator().manual_seed(n)
    x = torch.randint(-3, 4, (n, d_in), generator=g).to(dtype).to(dev())
    w = torch.randint(-3, 4, (d_out, d_in), generator=g).to(dtype).to(dev())
    b = torch.randint(-9, 10, (d_out,), generator=g).float().to(dev())
    want = (x.double() @ w.double().T + b.double())
    y, z, _ = lrc.lrc_linear(x, w, b, act="relu", save="z")
    assert torch.equal(z, want.to(dtype)) and torch.equal(y, want.clamp_min(0).to(dtype))
    y, kept, _ = lrc.lrc_linear(x, w, b, save="checkpoint")
    codes, exps, _ = lrc.lrc_pack_activations(want.float())
    assert torch.equal(y, want.to(dtype)) and torch.equal(kept[0], codes) and torch.equal(kept[1], exps)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_out", [(4096, 160, 4104), (3900, 2100, 2500), (5001, 1500, 5011)])
def test_linear_large_tiles_exact(lrc, dtype, n, d_in, d_out):
    """As the tests on small integers, at sizes that fill the chip with large tiles; ragged ones among them."""
    g = torch.Generator().manual_seed(n)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).to(dtype).to(dev())   # noqa: E731
    x, w, dy = ints(n, d_in), ints(d_out, d_in), ints(n, d_out)
    b = torch.randint(-9, 10, (d_out,), generator=g).float().to(dev())
    y, kept, _ = lrc.lrc_linear(x, w, b, act="relu", residual=dy, save="checkpoint")
    z = x.double() @ w.double().T + b.double()
    codes, exps, _ = lrc.lrc_pack_activations(z.float())
    assert torch.equal(y, (z.clamp_min(0) + dy.double()).to(dtype))
    assert torch.equal(kept[0], codes) and torch.equal(kept[1], exps)
    for held in (False, True):
        xa = lrc.lrc_pack_activations(x)[:2] if held else x
        _, dx, dw, db = lrc.lrc_linear_backward(dy, xa, w, dw_dtype=torch.float32)
        assert torch.equal(dx, (dy.double() @ w.double()).to(dtype))
        assert torch.equal(dw.double(), dy.double().T.contiguous() @ x.double())
        assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_out", [(1, 3000, 600), (70, 1024, 1500), (1100, 1100, 1100)])
def test_linear_accuracy_at_long_sums(lrc, dtype, n, d_in, d_out):
    """Against fp64 within the norm-wise accuracy of fp32 sums: with random signs the error of a K-term fp32 sum is
    about sqrt(K) u of the terms' root mean square, i.e. about u sqrt(K) / sqrt(K) = u of the result per add; 24 u
    of the 2-norm leaves room for the adds inside a matrix instruction and a biased rounding.  bf16 results add
    2^-8 / sqrt(3)."""
    g = torch.Generator().manual_seed(d_in)
    x, dy = stream(n, d_in, dtype, 1).to(dev()), stream(n, d_out, dtype, 2).to(dev())
    w = (torch.randn(d_out, d_in, generator=g) / math.sqrt(d_in)).to(dtype).to(dev())
    bound = 24 * U + (2.0 ** -8 / math.sqrt(3) if dtype == torch.bfloat16 else 0)
    off = lambda got, want: float((got.double() - want).norm() / want.norm())   # noqa: E731
    assert off(lrc.lrc_linear(x, w)[0], x.double() @ w.double().T) < bound
    _, dx, dw, _ = lrc.lrc_linear_backward(dy, x, w, dw_dtype=torch.float32)
    assert off(dx, dy.double() @ w.double()) < bound
    assert off(dw, dy.double().T.contiguous() @ x.double()) < 24 * U


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("n,d_in,d_out", [(5, 17, 9), (300, 136, 264), (1000, 521, 303), (2500, 1032, 2056)])
@pytest.mark.parametrize("held", [False, True])
def test_weight_gradient_keeps_the_bits_of_dz(lrc, act, n, d_in, d_out, held):
    """dW of a bf16 layer with a smooth activation takes dz to 11 bits: a rounding of at most 2^-11 relative (2^-12
    half steps, uniform: 2^-12 / sqrt(3) in the 2-norm, the slope's 16 u besides), whatever the channels' scales."""
    g = torch.Generator().manual_seed(n)
    x, dy = stream(n, d_in, torch.bfloat16, 1), stream(n, d_out, torch.bfloat16, 2)
    x = (x.float() * 2.0 ** torch.randint(-30, 31, (d_in,), generator=g)).bfloat16()
    dy = (dy.float() * 2.0 ** torch.randint(-40, 41, (d_out,), generator=g)).bfloat16()
    dy[:, 0], x[:, 1] = 0, 0
    z = torch.randn(n, d_out, generator=g).bfloat16()
    w = torch.zeros(d_out, d_in, dtype=torch.bfloat16, device=dev())
    xa, xn = x.to(dev()), f64(x)
    if held:
        xa = lrc.lrc_pack_activations(xa)[:2]
        xn = ref.unpack(xa[0].cpu().numpy(), xa[1].cpu().numpy())
    _, _, dw, _ = lrc.lrc_linear_backward(dy.to(dev()), xa, w, act=act, z=z.to(dev()), dw_dtype=torch.float32)
    dz = f64(dy) * ref.act_slope(f64(z), act)
    want, got = dz.T @ xn, f64(dw)
    rows = np.linalg.norm(dz, axis=0)[:, None] * np.linalg.norm(xn, axis=0)[None]   # by channel, so that each counts
    ok = rows > 0
    assert not got[~ok].any()
    err = ((got - want)[ok] / rows[ok])
    assert np.abs(err).max() < 2.0 ** -11 and math.sqrt((err ** 2).mean()) < 2.0 ** -12


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_weight_gradient_of_channels_that_are_shut(lrc, act):
    """Channels whose slopes are all tiny (z near -9: 1e-17 for gelu, 1e-3 for silu) keep their gradients' bits: the
    exponential's argument, 58 in powers of two, is off by at most 58 u twice, 5e-6 of the slope."""
    n, d = 100, 80
    g = torch.Generator().manual_seed(7)
    x, dy = stream(n, d, torch.bfloat16, 1), stream(n, d, torch.bfloat16, 2, 0.01)
    z = (torch.randn(n, d, generator=g) * 0.25 - 9 * (torch.arange(d) % 2)).bfloat16()
    w = torch.zeros(d, d, dtype=torch.bfloat16, device=dev())
    zk = lrc.lrc_pack_activations(z.to(dev()))[:2]
    for za, zn in ((z.to(dev()), f64(z)), (zk, ref.unpack(zk[0].cpu().numpy(), zk[1].cpu().numpy()))):
        _, _, dw, _ = lrc.lrc_linear_backward(dy.to(dev()), x.to(dev()), w, act=act, z=za, dw_dtype=torch.float32)
        dz = f64(dy) * ref.act_slope(zn, act)
        err = (f64(dw) - dz.T @ f64(x)) / (np.linalg.norm(dz, axis=0)[:, None] * np.linalg.norm(f64(x), axis=0)[None])
        assert np.abs(err).max() < 2.0 ** -11


def test_weight_gradient_with_nonfinite_entries(lrc):
    n, d = 200, 72
    ones = lambda *s: torch.ones(*s, dtype=torch.bfloat16)   # noqa: E731
    x, dy, z = ones(n, d), ones(n, d), ones(n, d)
    dy[3, 5], dy[4, 6], x[7, 8], z[9, 10] = float("inf"), float("nan"), float("-inf"), float("nan")
    args = [t.to(dev()) for t in (dy, x, ones(d, d))]
    _, _, dw, _ = lrc.lrc_linear_backward(*args, act="silu", z=z.to(dev()))
    dz = dy.double() * torch.from_numpy(ref.act_slope(f64(z), "silu"))
    want = (dz.T @ x.double()).to(dev())
    assert torch.equal(torch.isnan(dw), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(dw.double()[inf], want[inf])
    fine = torch.isfinite(want)
    # sums of 200 equal terms: half a bf16 step and the slope's error
    assert ((dw.double() - want)[fine].abs() <= (2.0 ** -8 + 2.0 ** -11) * want[fine].abs()).all()


@pytest.mark.parametrize("n,d_in,d_out", [(520, 264, 392), (1300, 904, 1101)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("where", ["x", "w", "dy"])
def test_nonfinite_entries_in_a_large_product(lrc, dtype, where, n, d_in, d_out):
    """Infinities and NaN at sizes that go to the large tiles (the larger one in fp32 too): what the plain products
    give."""
    ones = lambda *s: torch.ones(*s, dtype=dtype)   # noqa: E731
    t = {"x": ones(n, d_in), "w": ones(d_out, d_in), "dy": ones(n, d_out)}
    t[where][3, 5], t[where][40, 77], t[where][41, 77] = float("inf"), float("-inf"), float("nan")
    x, w, dy = (t[k].to(dev()) for k in ("x", "w", "dy"))
    res = ones(n, d_out).to(dev())
    same = lambda p, q: torch.equal(torch.nan_to_num(p.double(), 9e9, 8e8, 7e7),   # noqa: E731
                                    torch.nan_to_num(q.to(p.dtype).double(), 9e9, 8e8, 7e7))
    assert same(lrc.lrc_linear(x, w, residual=res)[0], x.double() @ w.double().T + 1)
    _, dx, dw, _ = lrc.lrc_linear_backward(dy, x, w)
    assert same(dx, dy.double() @ w.double()) and same(dw, dy.double().T.contiguous() @ x.double())


F32_SHAPES = [(700, 516, 1300), (701, 517, 1301), (513, 2047, 900), (130, 4100, 1000), (900, 100, 3500), (67, 3001, 777),
              (3000, 260, 514), (2048, 2048, 1024), (6912, 1080, 1984), (6913, 1075, 1981)]


@pytest.mark.parametrize("n,d_in,d_out", F32_SHAPES)
def test_fp32_products_of_every_kind_exact(lrc, n, d_in, d_out):
    """Small integers, whose products and sums are exact: sizes on either side of every choice between the kernels
    of an fp32 product, whole pieces and ragged rows, split k and not."""
    g = torch.Generator().manual_seed(n)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).float().to(dev())   # noqa: E731
    x, w, dy, z, res = ints(n, d_in), ints(d_out, d_in), ints(n, d_out), ints(n, d_out), ints(n, d_out)
    b = ints(d_out)
    want = x.double() @ w.double().T + b.double()
    y, kept, _ = lrc.lrc_linear(x, w, b, act="relu", residual=res, save="z")
    assert torch.equal(kept.double(), want) and torch.equal(y.double(), want.clamp(min=0) + res.double())
    y, kept, info = lrc.lrc_linear(x, w, b, save="checkpoint")
    assert torch.equal(y.double(), want) and int(info.cpu()) == 0
    for a, c in zip(kept, lrc.lrc_pack_activations(want.float())[:2]):
        assert torch.equal(a, c)
    dz = dy.double() * (z.double() > 0)
    for held in (False, True):
        xa, za = (lrc.lrc_pack_activations(x)[:2], lrc.lrc_pack_activations(z)[:2]) if held else (x, z)
        got = lrc.lrc_linear_backward(dy, xa, w, act="relu", z=za)
        assert torch.equal(got[0].double(), dz) and torch.equal(got[1].double(), dz @ w.double())
        assert torch.equal(got[2].double(), dz.T.contiguous() @ x.double())
        for only in ("need_dx", "need_dw"):
            some = lrc.lrc_linear_backward(dy, xa, w, act="relu", z=za, **{only: False})
            k = 2 if only == "need_dx" else 1
            assert torch.equal(some[k], got[k])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [8, 9, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("d_in,d_out", [(4096, 520), (4100, 1000), (8192, 640), (2047, 333), (1024, 4096), (5000, 1)])
def test_few_tokens_exact(lrc, dtype, n, d_in, d_out):
    """On either side of the choices between streaming the weight and tiles with split k; entries of one keep the
    sums below 2^24."""
    g = torch.Generator().manual_seed(n)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g).to(dtype).to(dev())   # noqa: E731
    x, w, dy, res = ints(n, d_in), ints(d_out, d_in), ints(n, d_out), ints(n, d_out)
    want = x.double() @ w.double().T
    y, z, _ = lrc.lrc_linear(x, w, act="relu", residual=res, save="z")
    assert torch.equal(z, want.to(dtype)) and torch.equal(y, (want.clamp_min(0) + res.double()).to(dtype))
    _, dx, dw, db = lrc.lrc_linear_backward(dy, x, w)
    assert torch.equal(dx, (dy.double() @ w.double()).to(dtype))
    assert torch.equal(dw, (dy.double().T.contiguous() @ x.double()).to(dtype))
    assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("n,d_in,d_out", F32_SHAPES)
@pytest.mark.parametrize("where", ["x", "w", "dy"])
def test_fp32_products_of_every_kind_with_nonfinite_entries(lrc, n, d_in, d_out, where):
    """What the plain products give, on every kernel of an fp32 product."""
    t = {"x": torch.ones(n, d_in), "w": torch.ones(d_out, d_in), "dy": torch.ones(n, d_out)}
    t[where][3, 5], t[where][40, -1], t[where][-1, -2] = float("inf"), float("-inf"), float("nan")
    x, w, dy = (t[k].to(dev()) for k in ("x", "w", "dy"))
    same = lambda p, q: torch.equal(torch.nan_to_num(p.double(), 9e9, 8e8, 7e7),   # noqa: E731
                                    torch.nan_to_num(q.float().double(), 9e9, 8e8, 7e7))
    assert same(lrc.lrc_linear(x, w)[0], x.double() @ w.double().T)
    _, dx, dw, _ = lrc.lrc_linear_backward(dy, x, w)
    assert same(dx, dy.double() @ w.double()) and same(dw, dy.double().T.contiguous() @ x.double())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_out", LINEAR_SHAPES)
@pytest.mark.parametrize("held", [False, True])
def test_linear_backward(lrc, dtype, n, d_in, d_out, held):
    g = torch.Generator().manual_seed(n + d_out)
    x, dy = stream(n, d_in, dtype, n + d_in), stream(n, d_out, dtype, n + d_out, 0.01)
    w = (torch.randn(d_out, d_in, generator=g) / math.sqrt(d_in)).to(dtype)
    z = (2 * torch.randn(n, d_out, generator=g)).to(dtype)
    for i, name in enumerate(ACTS):
        layout = LAYOUTS[i % 3]
        xl, zl = lay(x, layout), lay(z, layout)
        xn, zn = f64(x), f64(z)
        if held:
            xl, zl = lrc.lrc_pack_activations(xl)[:2], lrc.lrc_pack_activations(zl)[:2]
            xn, zn = (ref.unpack(p[0].cpu().numpy(), p[1].cpu().numpy()) for p in (xl, zl))
        dwt = torch.float32 if i % 2 else None
        dz, dx, dw, db = lrc.lrc_linear_backward(lay(dy, layout), xl, lay(w, layout), act=name, z=zl, dw_dtype=dwt)
        wz, wx, ww, wb = ref.linear_backward(f64(dy), xn, f64(w), name, zn)
        # slopes are good to 16 u absolutely (erf, exp and the products around them, |z| < 12)
        e_z = 16 * U * np.abs(f64(dy)) + 2 * U * np.abs(wz) if name != "none" else 0 * wz
        e_db = (n + 8) * U * np.abs(wz).sum(0) + e_z.sum(0)
        half = HALF[dtype]
        if name != "none":
            e_z = e_z + half * (np.abs(wz) + e_z) + 1e-37
        check(dz, wz, e_z, ("dz", name))
        aw, ax = np.abs(f64(w)), np.abs(xn)
        e_x = (d_out + 8) * 2 * U * (np.abs(wz) @ aw) + e_z @ aw
        e_w = (n + 8) * 2 * U * (np.abs(wz).T @ ax) + e_z.T @ ax
        hw = HALF[dw.dtype]
        assert dw.dtype == (dwt or dtype)
        check(dx, wx, e_x * 1.01 + half * (np.abs(wx) + e_x) + 1e-37, ("dx", name))
        check(dw, ww, e_w * 1.01 + hw * (np.abs(ww) + e_w) + 1e-37, ("dw", name))
        check(db, wb, e_db + 1e-37, ("db", name))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_out", [(7, 520, 264), (3000, 264, 520), (300, 1032, 2056), (1111, 520, 303),
                                          (5000, 72, 136), (130, 4096, 512)])
@pytest.mark.parametrize("held", [False, True])
def test_linear_backward_exact_on_small_integers(lrc, dtype, n, d_in, d_out, held):
    """As the forward test; relu keeps dz an integer, and small integers are held exactly in 8 bits."""
    g = torch.Generator().manual_seed(n)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).to(dtype).to(dev())   # noqa: E731
    x, w, dy, z = ints(n, d_in), ints(d_out, d_in), ints(n, d_out), ints(n, d_out)
    dz = dy.double() * (z.double() > 0)
    xa, za = (lrc.lrc_pack_activations(x)[:2], lrc.lrc_pack_activations(z)[:2]) if held else (x, z)
    got = lrc.lrc_linear_backward(dy, xa, w, act="relu", z=za, dw_dtype=torch.float32)
    assert torch.equal(got[0].double(), dz)
    assert torch.equal(got[1], (dz @ w.double()).to(dtype))
    assert torch.equal(got[2].double(), dz.T.contiguous() @ x.double())
    assert torch.equal(got[3].double(), dz.sum(0))
    plain = lrc.lrc_linear_backward(dy, xa, w)     # no activation: dz is dy
    assert plain[0] is dy
    assert torch.equal(plain[1], (dy.double() @ w.double()).to(dtype))
    assert torch.equal(plain[2], (dy.double().T.contiguous() @ x.double()).to(dtype))


def test_linear_backward_parts_and_differences(lrc):
    n, d_in, d_out = 5, 19, 11
    g = torch.Generator().manual_seed(1)
    x, w, dy = (torch.randn(*s, generator=g) for s in ((n, d_in), (d_out, d_in), (n, d_out)))
    b = torch.randn(d_out, generator=g)
    for name in ACTS[2:]:
        _, z, _ = lrc.lrc_linear(x.to(dev()), w.to(dev()), b.to(dev()), act=name, save="z")
        a = (dy.to(dev()), x.to(dev()), w.to(dev()))
        dz, dx, dw, db = lrc.lrc_linear_backward(*a, act=name, z=z)
        for need in ("need_dx", "need_dw", "need_db"):
            some = lrc.lrc_linear_backward(*a, act=name, z=z, **{need: False})
            for k, (p, q) in enumerate(zip(some, (dz, dx, dw, db))):
                assert (p is None) == (k == ("need_dx", "need_dw", "need_db").index(need) + 1)
                assert p is None or torch.equal(p, q)
        loss = lambda xx, ww, bb: (ref.linear(xx, ww, bb, name, 0.0)[0] * f64(dy)).sum()   # noqa: E731
        h, args = 1e-5, [f64(x), f64(w), f64(b)]
        for k, got in enumerate((dx, dw, db)):
            for at in [(0,) * got.dim(), tuple(s - 1 for s in got.shape)]:
                e = np.zeros(got.shape)
                e[at] = h
                hi, lo = ([v + s * e if i == k else v for i, v in enumerate(args)] for s in (1, -1))
                want = (loss(*hi) - loss(*lo)) / (2 * h)
                # fp32 products of ten to twenty terms of order one, differences good to 1e-8
                assert abs(float(got[at]) - want) < 2e-5 * max(1.0, abs(want)), (name, k)


# ----------------------------------------------------------------------------- the operators together
def test_step_of_a_layer_feeds_the_compression(lrc):
    """norm -> up projection (gelu, 8-bit checkpoints) -> down projection onto the residual stream; backward; then
    the layer's input and gradient streams go into the covariances, the decomposition and the Fisher scores."""
    n, d, h = 600, 96, 160
    g = torch.Generator().manual_seed(0)
    x = stream(n, d, torch.bfloat16, 1).to(dev())
    w1 = (torch.randn(h, d, generator=g) / math.sqrt(d)).bfloat16().to(dev())
    w2 = (torch.randn(d, h, generator=g) / math.sqrt(h)).bfloat16().to(dev())
    gamma, b1 = torch.ones(d, device=dev()), torch.zeros(h, device=dev())
    a, mean, rstd, xk, _ = lrc.lrc_layer_norm(x, gamma, None, checkpoint=True)
    ak = lrc.lrc_pack_activations(a)[:2]
    u, zk, _ = lrc.lrc_linear(a, w1, b1, act="gelu", save="checkpoint")
    uk = lrc.lrc_pack_activations(u)[:2]
    y, _, _ = lrc.lrc_linear(u, w2, residual=x)
    dy = stream(n, d, torch.bfloat16, 2, 0.01).to(dev())
    _, du, dw2, _ = lrc.lrc_linear_backward(dy, uk, w2)
    dz, da, dw1, db1 = lrc.lrc_linear_backward(du, ak, w1, act="gelu", z=zk)
    dxn, dgamma, dbeta = lrc.lrc_layer_norm_backward(da, xk, mean, rstd, gamma)
    # the same step in fp64 with full activations
    xd = x.double().requires_grad_()
    p = [t.double().requires_grad_() for t in (w1, w2, gamma, b1)]
    c = xd - xd.mean(1, keepdim=True)
    ad = c / torch.sqrt(c.square().mean(1, keepdim=True) + 1e-5) * p[2]
    zd = ad @ p[0].T + p[3]
    yd = (0.5 * zd * (1 + torch.erf(zd / math.sqrt(2)))) @ p[1].T + xd
    (yd * dy.double()).sum().backward()

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())

    # 8-bit checkpoints: a block's step is at most max / 63.5, so a value is held to max / 127 / sqrt(3) rms
    # at worst, about 1.3 % of the block's largest value; with bf16 streams in between 5 % is far outside
    assert off(y, yd.detach()) < 0.01
    assert off(dxn + dy.float(), xd.grad) < 0.05
    for got, leaf in ((dw1, p[0]), (dw2, p[1]), (dgamma, p[2]), (db1, p[3])):
        assert off(got, leaf.grad) < 0.05
    # what the compression takes: A held in 8 bits (exact in bf16) and B = dz
    A = lrc.lrc_unpack_activations(*ak)
    xs, gs = torch.zeros(d, d, device=dev()), torch.zeros(h, h, device=dev())
    lrc.lrc_accumulate_cov(A, xs)
    lrc.lrc_accumulate_cov(dz, gs)
    assert off(xs.tril(), (A.double().T.contiguous() @ A.double()).tril()) < 1e-5
    sig, left, right, info = lrc.lrc_whiten_decompose(w1.float(), d, xs, n, None, 0, damping=1e-3)
    scores, sinfo = lrc.lrc_score_components(left, right, A=A, B=dz)
    assert int(info.cpu()) == 0 and int(sinfo.cpu()) == 0 and (scores >= 0).all() and scores.max() > 0
    # the full-rank factors as two linear calls give the layer back
    z2 = lrc.lrc_linear(lrc.lrc_linear(a.float(), right)[0], left, b1)[0]
    assert off(z2, zd.detach()) < 0.02


# ----------------------------------------------------------------------------- how they run
def _ops(lrc, dtype, n, d_in, d_out):
    """Calls of every operator on one set of inputs, each returning a tuple of tensors."""
    g = torch.Generator().manual_seed(n)
    x, dy = stream(n, d_in, dtype, 1).to(dev()), stream(n, d_out, dtype, 2, 0.01).to(dev())
    w = (torch.randn(d_out, d_in, generator=g) / math.sqrt(d_in)).to(dtype).to(dev())
    b = torch.randn(d_out, generator=g).to(dev())
    gamma = (1 + 0.1 * torch.randn(d_in, generator=g)).to(dev())
    _, mean, rstd, xk, _ = lrc.lrc_layer_norm(x, gamma, checkpoint=True)
    _, zk, _ = lrc.lrc_linear(x, w, b, save="checkpoint")
    return [lambda: lrc.lrc_pack_activations(x)[:2],
            lambda: (lrc.lrc_unpack_activations(*xk, dtype),),
            lambda: lrc.lrc_layer_norm(x, gamma)[:3],
            lambda: lrc.lrc_layer_norm_backward(x, xk, mean, rstd, gamma),
            lambda: lrc.lrc_linear(x, w, b, act="silu", residual=dy)[:1],
            lambda: lrc.lrc_linear_backward(dy, xk, w, act="gelu", z=zk)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_out", [(5, 512, 256), (200, 136, 520), (1200, 320, 264)])
def test_equal_inputs_give_equal_bits_and_graphs_replay(lrc, dtype, n, d_in, d_out):
    """Two calls agree bit for bit; a captured call replays to the same bits, also with other work in between."""
    for call in _ops(lrc, dtype, n, d_in, d_out):
        want = [t.clone() for t in call()]
        assert all(torch.equal(p, q) for p, q in zip(call(), want))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = call()
        for _ in range(3):
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, want))
            assert all(torch.equal(p, q) for p, q in zip(call(), want))


def test_two_streams(lrc):
    """Calls on two streams at once, each on its own data, give the bits of calls one after the other."""
    sets = [_ops(lrc, torch.bfloat16, n, 264, 520) for n in (700, 900)]
    want = [[[t.clone() for t in call()] for call in ops] for ops in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = [call() for call in sets[k]]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for p, q in zip(g, w):
            assert all(torch.equal(a, b) for a, b in zip(p, q))


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_tokens(lrc, dtype):
    x, w = torch.empty(0, 48, dtype=dtype, device=dev()), torch.ones(32, 48, dtype=dtype, device=dev())
    codes, exps, info = lrc.lrc_pack_activations(x)
    assert codes.shape == (0, 48) and exps.shape == (0, 1) and int(info.cpu()) == 0
    assert lrc.lrc_unpack_activations(codes, exps).shape == (0, 48)
    y, mean, rstd, kept, _ = lrc.lrc_layer_norm(x, checkpoint=True)
    assert y.shape == (0, 48) and mean.shape == (0,) and kept[0].shape == (0, 48)
    dx, dg, db = lrc.lrc_layer_norm_backward(x, kept, mean, rstd)
    assert dx.shape == (0, 48) and not dg.any() and not db.any()
    y, z, _ = lrc.lrc_linear(x, w, act="gelu", save="checkpoint")
    assert y.shape == (0, 32)
    for dwt in (dtype, torch.float32):
        dz, dx, dw, db = lrc.lrc_linear_backward(y, x, w, act="gelu", z=z, dw_dtype=dwt)
        assert dz.shape == (0, 32) and dx.shape == (0, 48) and dw.dtype == dwt and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_outputs_stay_inside_their_rows(lrc, dtype):
    """Outputs with a pitch through the C interface: what lies between and behind the rows is left as it was."""
    n, d_in, d_out, gap = 37, 72, 104, 8
    code = 1 if dtype == torch.bfloat16 else 0
    x, dy = stream(n, d_in, dtype, 1).to(dev()), stream(n, d_out, dtype, 2).to(dev())
    w = stream(d_out, d_in, dtype, 3).to(dev())
    p = lambda t: ctypes.c_void_p(t.data_ptr())   # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    box = lambda rows, cols: torch.full((rows + 2, cols + gap), 7.0, dtype=dtype, device=dev())   # noqa: E731
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=dev())
    y, z, dx, dw, o, dxn = box(n, d_out), box(n, d_out), box(n, d_in), box(d_out, d_in), box(n, d_in), box(n, d_in)
    L = lrc.lib
    assert L.lrc_linear(p(x), code, n, d_in, d_out, d_in, p(w), d_in, None, 0, None, 0, p(y), d_out + gap, p(z),
                        d_out + gap, None, None, None, p(ws), ws.numel(), st) == 0
    assert L.lrc_linear_backward(p(dy), code, n, d_in, d_out, d_out, p(w), d_in, p(x), d_in, None, None, 0, None, 0,
                                 None, None, None, 0, p(dx), d_in + gap, p(dw), code, d_in + gap, None, p(ws),
                                 ws.numel(), st) == 0
    stat = torch.empty(2, n, device=dev())
    assert L.lrc_layer_norm(p(x), code, n, d_in, d_in, None, None, 1e-5, p(o), d_in + gap, p(stat[0]), p(stat[1]),
                            None, None, None, st) == 0
    assert L.lrc_layer_norm_backward(p(o), code, n, d_in, d_in + gap, p(x), d_in, None, None, p(stat[0]), p(stat[1]),
                                     None, p(dxn), d_in + gap, None, None, p(ws), ws.numel(), st) == 0
    for t, rows, cols in ((y, n, d_out), (z, n, d_out), (dx, n, d_in), (dw, d_out, d_in), (o, n, d_in),
                          (dxn, n, d_in)):
        assert (t[rows:] == 7).all() and (t[:, cols:] == 7).all() and not (t[:rows, :cols] == 7).all()
    assert torch.equal(y[:n, :d_out], lrc.lrc_linear(x, w)[0]) and torch.equal(z, y)


def test_offsets_past_32_bits(lrc):
    """Rows whose offsets pass 2^32 elements: the same results as rows that lie together."""
    n, d, ld = 5, 72, (1 << 30) + 64
    big = torch.empty((n - 1) * ld + d, dtype=torch.bfloat16, device=dev())
    far = big.as_strided((n, d), (ld, 1))
    x = stream(n, d, torch.bfloat16, 1).to(dev())
    far.copy_(x)
    w = stream(40, d, torch.bfloat16, 2).to(dev())
    dy = stream(n, 40, torch.bfloat16, 3).to(dev())
    for a, b in zip(lrc.lrc_layer_norm(far, checkpoint=True)[:3], lrc.lrc_layer_norm(x, checkpoint=True)[:3]):
        assert torch.equal(a, b)
    for a, b in zip(lrc.lrc_pack_activations(far)[:2], lrc.lrc_pack_activations(x)[:2]):
        assert torch.equal(a, b)
    assert torch.equal(lrc.lrc_linear(far, w)[0], lrc.lrc_linear(x, w)[0])
    for a, b in zip(lrc.lrc_linear_backward(dy, far, w), lrc.lrc_linear_backward(dy, x, w)):
        assert torch.equal(a, b)
    _, mean, rstd, _, _ = lrc.lrc_layer_norm(x)
    for a, b in zip(lrc.lrc_layer_norm_backward(far, far, mean, rstd), lrc.lrc_layer_norm_backward(x, x, mean, rstd)):
        assert torch.equal(a, b)


def test_more_blocks_than_a_launch_has_threads_for(lrc):
    """2^29 + 4096 rows of one channel, eight lanes a row: the rows repeat a pattern and so do codes and values."""
    p = stream(4096, 1, torch.bfloat16, 1).to(dev())
    p[7], p[9] = 0.0, 300.0
    want = lrc.lrc_pack_activations(p)
    x = p.repeat((1 << 17) + 1, 1)
    got = lrc.lrc_pack_activations(x)
    for a, b in zip(got[:2], want[:2]):
        assert (a.view(-1, 4096) == b.view(4096)).all()
    back = lrc.lrc_unpack_activations(*got[:2])
    assert (back.view(-1, 4096) == lrc.lrc_unpack_activations(*want[:2]).view(4096)).all()
    x[-3] = float("inf")
    assert int(lrc.lrc_pack_activations(x)[2].cpu()) == lrc.LRC_ENONFINITE and int(got[2].cpu()) == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_products_of_unaligned_rows(lrc, dtype):
    """Rows that start on no 16 bytes give the bits of rows that do (2^30 products: the operands are laid out
    first)."""
    n, d_in, d_out = 1030, 1024, 1032
    x, w = stream(n, d_in, dtype, 1), stream(d_out, d_in, dtype, 2)
    dy, z = stream(n, d_out, dtype, 3), stream(n, d_out, dtype, 4)
    for layout in LAYOUTS[1:]:
        xl, wl, dl, zl = (lay(t, layout) for t in (x, w, dy, z))
        xp, wp, dp, zp = (t.to(dev()) for t in (x, w, dy, z))
        assert torch.equal(lrc.lrc_linear(xl, wl, residual=dl)[0], lrc.lrc_linear(xp, wp, residual=dp)[0])
        for act in ("none", "relu", "silu"):
            got = lrc.lrc_linear_backward(dl, xl, wl, act=act, z=zl)
            for a, b in zip(got, lrc.lrc_linear_backward(dp, xp, wp, act=act, z=zp)):
                assert torch.equal(a, b)
        assert lrc.lrc_linear_backward(dp[:, 8:], xp, wp[8:])[0].stride(0) == d_out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_out", [(5, 512, 256), (70, 100, 90), (200, 1000, 520), (1100, 1032, 1024)])
def test_residual_in_the_output(lrc, dtype, n, d_in, d_out):
    """The residual may be y itself: few tokens, split k, and tiles of either kind."""
    x, w = stream(n, d_in, dtype, 1).to(dev()), stream(d_out, d_in, dtype, 2).to(dev())
    res = stream(n, d_out, dtype, 3).to(dev())
    want = lrc.lrc_linear(x, w, act="silu", residual=res)[0]
    code = lrc.LRC_BF16 if dtype == torch.bfloat16 else lrc.LRC_F32
    size = lrc.lib.lrc_linear_workspace(code, n, d_in, d_out)
    ws = torch.empty(max(1, size), dtype=torch.uint8, device=dev())
    st = torch.cuda.current_stream().cuda_stream
    assert lrc.lib.lrc_linear(x.data_ptr(), code, n, d_in, d_out, d_in, w.data_ptr(), d_in, None, 3, res.data_ptr(),
                              d_out, res.data_ptr(), d_out, None, 0, None, None, None, ws.data_ptr(), size, st) == 0
    assert torch.equal(res, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nonfinite_values_stay_in_their_rows(lrc, dtype):
    """A token with NaN or an infinity spoils its own row and the token sums, nothing else, and y of an infinite
    entry is what arithmetic gives."""
    n, d_in, d_out = 150, 136, 72
    x, w = stream(n, d_in, dtype, 1), stream(d_out, d_in, dtype, 2)
    clean, _, _ = lrc.lrc_linear(x.to(dev()), w.to(dev()))
    cn = lrc.lrc_layer_norm(x.to(dev()))[0]
    bad = x.clone()
    bad[5, 3], bad[77, 40] = float("nan"), float("inf")
    y, kept, info = lrc.lrc_linear(bad.to(dev()), w.to(dev()), save="checkpoint")
    rows = [t for t in range(n) if t not in (5, 77)]
    assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[5]).all() and int(info.cpu()) == lrc.LRC_ENONFINITE
    want = (float("inf") * w[:, 40].float()).to(dev())   # the weight row of zeros gives NaN
    assert torch.allclose(y[77].float(), want, equal_nan=True)
    yn = lrc.lrc_layer_norm(bad.to(dev()))[0]
    assert torch.equal(yn[rows], cn[rows]) and torch.isnan(yn[5]).all() and torch.isnan(yn[77]).all()


def test_refusals(lrc):
    x = torch.zeros(4, 64, device=dev())
    w = torch.zeros(8, 64, device=dev())
    bad = [lambda: lrc.lrc_pack_activations(x.cpu()), lambda: lrc.lrc_pack_activations(x.half()),
           lambda: lrc.lrc_pack_activations(x[0]), lambda: lrc.lrc_pack_activations(x, info=torch.zeros(1)),
           lambda: lrc.lrc_unpack_activations(x, x), lambda: lrc.lrc_layer_norm(x, gamma=torch.zeros(63, device=dev())),
           lambda: lrc.lrc_unpack_activations(x.to(torch.int8), torch.zeros(4, 2, dtype=torch.int8, device=dev())),
           lambda: lrc.lrc_unpack_activations(x.to(torch.int8), torch.zeros(4, 1, dtype=torch.int8, device=dev()),
                                              torch.float16),
           lambda: lrc.lrc_layer_norm(x, gamma=torch.zeros(64, device=dev()).bfloat16()),
           lambda: lrc.lrc_layer_norm_backward(x, x[:3], x[:, 0], x[:, 0]),
           lambda: lrc.lrc_layer_norm_backward(x, None, x[:, 0], x[:, 0]),
           lambda: lrc.lrc_linear(x, w.bfloat16()), lambda: lrc.lrc_linear(x, w[:, :63]),
           lambda: lrc.lrc_linear(x, w, act="tanh"), lambda: lrc.lrc_linear(x, w, save="all"),
           lambda: lrc.lrc_linear(x, w, residual=x), lambda: lrc.lrc_linear(x, w, bias=x[:, 0]),
           lambda: lrc.lrc_linear_backward(x[:, :8], None, w), lambda: lrc.lrc_linear_backward(x, x, w),
           lambda: lrc.lrc_linear_backward(x[:, :8], x, w, act="relu"),
           lambda: lrc.lrc_linear_backward(x[:, :8], x, w, dw_dtype=torch.bfloat16)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(lrc.LrcError):
        lrc.lrc_layer_norm(x, eps=-1.0)
    with pytest.raises(lrc.LrcError):
        lrc.lrc_layer_norm(x, eps=float("nan"))
