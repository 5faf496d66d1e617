"""The gated feed-forward block, the products in 8-bit integers and the norms around a block on the GPU against their
fp64 definitions.

Tolerances.  u = 2^-24.  A fp32 sum of K terms in any order is off by at most (K + c) u times the sum of the
terms' magnitudes; the matrix cores' internal adds are counted as two roundings each.  An output held in bf16
adds half a step, 2^-8 of its value.  Integer sums are exact.  Bounds are elementwise and computed in fp64 from the
same inputs.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as ref
from oracle import train_oracle as base
from tests.test_gpu_train_ops import DTYPES, HALF, LAYOUTS, LIP, U, check, dev, f64, lay, stream

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "relu", "none"]
TINY = 1e-37


@pytest.fixture(scope="module")
def lrc():
    import curvature_aware_rank_amd as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weight(o, i, dtype, seed):
    return (torch.randn(o, i, generator=gen(seed)) / math.sqrt(i)).to(dtype)


def codes_of(o, i, seed):
    """Codes and scales of a weight, as the rows' quantiser writes them."""
    q, s = ref.quantize(weight(o, i, torch.float32, seed).numpy())
    return torch.from_numpy(q), torch.from_numpy(s)


def lay8(t, layout):
    """int8 rows on the GPU in another layout."""
    n, d = t.shape
    if layout == "padded":
        b = torch.full((n, d + 48), 77, dtype=torch.int8, device=dev())
        b[:, 16:16 + d] = t.to(dev())
        return b[:, 16:16 + d]
    if layout == "offset":
        b = torch.full((n * (d + 3) + 1,), 77, dtype=torch.int8, device=dev())
        v = b[1:].view(n, d + 3)[:, :d]
        v.copy_(t)
        return v
    if layout == "transposed":
        return t.t().contiguous().to(dev()).t()
    return t.to(dev())


def flag():
    return torch.zeros(1, dtype=torch.int32, device=dev())


def on(*ts):
    return [None if t is None else t.to(dev()) for t in ts]


# ----------------------------------------------------------------------------- the quantiser
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 1), (3, 7), (5, 63), (1, 64), (70, 65), (33, 520), (9, 1000), (300, 1024), (3, 4096),
                                 (4, 8200), (5, 11008), (2, 16384), (2, 20001)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_quantize_tokens_bit_exact(lrc, dtype, n, d, layout):
    x = stream(n, d, dtype, n * 31 + d)
    q, s, info = lrc.lrc_quantize_tokens(lay(x, layout))
    wq, ws = ref.quantize(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws) and int(info.cpu()) == 0
    if dtype == torch.float32:
        rq, rs = lrc.lrc_quantize_rows(x.to(dev()))
        assert torch.equal(rq, q) and torch.equal(rs, s)


def test_quantize_tokens_borders(lrc):
    """Ties, the ends of the range, subnormals, zeros, NaN and infinities."""
    big = float(np.finfo(np.float32).max)
    rows = [[127.0, 0.5, 1.5, -2.5, 126.5], [254.0, 1.0, 3.0, -5.0, 0.0], [big, 1.0, -big, 0.0, big / 2],
            [2.0 ** -149, -2.0 ** -149, 0, 0, 0], [2.0 ** -126, -2.0 ** -130, 2.0 ** -127, 0, 0], [0.0, -0.0, 0, 0, 0],
            [190 * 2.0 ** -149, 3 * 2.0 ** -149, -95 * 2.0 ** -149, 0, 0]]
    x = torch.tensor(rows, dtype=torch.float32)
    q, s, info = lrc.lrc_quantize_tokens(x.to(dev()))
    wq, ws = ref.quantize(x.numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws) and int(info.cpu()) == 0
    for dtype in DTYPES:
        x = stream(6, 150, dtype, 3)
        x[1, 70], x[3, 0], x[4, 149], x[5, :] = float("nan"), float("inf"), float("-inf"), float("nan")
        q, s, info = lrc.lrc_quantize_tokens(x.to(dev()))
        wq, ws = ref.quantize(x.float().numpy())
        assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
        assert wq[1, 70] == 0 and wq[3, 0] == 127 and wq[4, 149] == -127 and not wq[5].any()
        assert int(info.cpu()) == lrc.LRC_ENONFINITE
        assert lrc.lrc_quantize_tokens(stream(2, 9, dtype, 4).to(dev()), info=info)[2] is info
        assert int(info.cpu()) == lrc.LRC_ENONFINITE


# ----------------------------------------------------------------------------- 8-bit products
INT8_SHAPES = [(1, 1, 1), (3, 5, 7), (1, 64, 96), (2, 512, 130), (16, 96, 64), (17, 257, 33), (33, 128, 200),
               (64, 1000, 48), (65, 64, 65), (100, 300, 520), (130, 80, 256), (257, 144, 264), (600, 528, 136)]


def int8_bounds(z, b, res, y, half):
    """z: the integer as a number, two products and the bias' sum round."""
    e_z = 4 * U * (np.abs(z - b) + np.abs(b)) + U * np.abs(z)
    e_y = LIP * e_z + 8 * U * (np.abs(z) + np.abs(res)) + 8 * U * np.abs(y)
    return e_y + half * (np.abs(y) + e_y) + TINY


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_out", INT8_SHAPES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_int8_linear(lrc, dtype, n, d_in, d_out, layout):
    x = stream(n, d_in, dtype, n + d_in)
    wq, ws = codes_of(d_out, d_in, d_in)
    b, res = torch.randn(d_out, generator=gen(1)), stream(n, d_out, dtype, 5)
    xq, xs = ref.quantize(x.float().numpy())
    W = (lay8(wq, layout), ws.to(dev()))
    for i, name in enumerate(ACTS):
        with_b, with_r = i != 1, i % 2 == 0
        bias, r = b.to(dev()) if with_b else None, lay(res, layout) if with_r else None
        y, info = lrc.lrc_int8_linear(lay(x, layout), W, bias, act=name, residual=r)
        bn, rn = f64(b) if with_b else np.zeros(d_out), f64(res) if with_r else np.zeros((n, d_out))
        wy, wz = ref.int8_linear(xq, xs, wq.numpy(), ws.numpy(), bn, name, rn)
        check(y, wy, int8_bounds(wz, bn, rn, wy, HALF[dtype]), ("y", name))
        assert y.dtype == dtype and info is None
        # tokens quantised before the call: the same bits
        pair = (lay8(torch.from_numpy(xq), layout), torch.from_numpy(xs).to(dev()))
        again, _ = lrc.lrc_int8_linear(pair, W, bias, act=name, residual=r, dtype=dtype)
        assert torch.equal(again, y)


EXACT_SHAPES = [(1, 4096, 1000), (7, 11008, 256), (16, 4096, 4104), (17, 4096, 4104), (40, 2048, 520), (96, 4096, 512),
                (300, 4096, 1032), (1500, 264, 2056), (520, 1032, 4104), (2100, 96, 520), (4096, 160, 4104),
                (3900, 2100, 2500), (5001, 1500, 5011)]


@pytest.mark.parametrize("n,d_in,d_out", EXACT_SHAPES)
def test_int8_products_exact(lrc, n, d_in, d_out):
    """Scales of one: y is the integer itself (below 2^24).  Catches a dropped, repeated or misplaced tile, step or
    split, of each of the two weights of a gated product."""
    g = gen(n)
    codes = lambda *s: torch.randint(-9, 10, s, generator=g, dtype=torch.int8).to(dev())   # noqa: E731
    xq, wq, uq = codes(n, d_in), codes(d_out, d_in), codes(d_out, d_in)
    wq[-1], xq[-1] = -128, 127
    one = lambda k: torch.ones(k, device=dev())   # noqa: E731
    want, up = xq.double() @ wq.double().T, xq.double() @ uq.double().T
    y, _ = lrc.lrc_int8_linear((xq, one(n)), (wq, one(d_out)), dtype=torch.float32)
    assert torch.equal(y.double(), want.float().double())
    y, _ = lrc.lrc_int8_linear((xq, one(n)), (wq, one(d_out)), act="relu")
    assert torch.equal(y, want.float().clamp_min(0).bfloat16())
    h, _ = lrc.lrc_int8_gated_linear((xq, one(n)), (wq, one(d_out)), (uq, one(d_out)), act="relu", dtype=torch.float32)
    assert torch.equal(h, want.float().clamp_min(0) * up.float())


def test_int8_longest_sums(lrc):
    """The largest magnitude an exact int32 sum may reach, through every kernel and over split k."""
    d = (1 << 17) - 1
    for n in (2, 20, 130):
        xq = torch.full((n, d), -128, dtype=torch.int8, device=dev())
        wq = torch.full((33, d), -128, dtype=torch.int8, device=dev())
        wq[1], wq[2] = 127, 1
        want = torch.tensor([128 * 128 * d, -127 * 128 * d, -128 * d], dtype=torch.float64).float()
        y, _ = lrc.lrc_int8_linear((xq, torch.ones(n, device=dev())), (wq, torch.ones(33, device=dev())),
                                   dtype=torch.float32)
        assert torch.equal(y[:, :3].cpu(), want.expand(n, 3)) and torch.equal(y[:, 3:], y[:, :1].expand(n, 30))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_ff", INT8_SHAPES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_int8_gated(lrc, dtype, n, d_in, d_ff, layout):
    x = stream(n, d_in, dtype, n + d_in)
    (gq, gs), (uq, us) = codes_of(d_ff, d_in, 1), codes_of(d_ff, d_in, 2)
    xq, xs = ref.quantize(x.float().numpy())
    zero = np.zeros(d_ff), "none", np.zeros((n, d_ff))
    _, g = ref.int8_linear(xq, xs, gq.numpy(), gs.numpy(), *zero)
    _, u = ref.int8_linear(xq, xs, uq.numpy(), us.numpy(), *zero)
    Wg, Wu = (lay8(gq, layout), gs.to(dev())), (lay8(uq, "packed"), us.to(dev()))
    for name in ACTS:
        h, _ = lrc.lrc_int8_gated_linear(lay(x, layout), Wg, Wu, act=name)
        a = base.act(g, name)
        e = (LIP * 5 * U + 8 * U) * np.abs(g) * np.abs(u) + np.abs(a * u) * 8 * U
        want = a * u
        check(h, want, e * 1.01 + HALF[dtype] * (np.abs(want) + e) + TINY, ("h", name))
        pair = (lay8(torch.from_numpy(xq), layout), torch.from_numpy(xs).to(dev()))
        assert torch.equal(lrc.lrc_int8_gated_linear(pair, Wg, Wu, act=name, dtype=dtype)[0], h)


def test_int8_nonfinite_tokens_are_flagged(lrc):
    x = stream(40, 96, torch.bfloat16, 1)
    w = [t.to(dev()) for t in codes_of(24, 96, 2)]
    info = torch.zeros(1, dtype=torch.int32, device=dev())
    clean, _ = lrc.lrc_int8_linear(x.to(dev()), w, info=info)
    assert int(info.cpu()) == 0
    x[5, 3], x[7, 9] = float("nan"), float("inf")
    for n in (8, 40):
        info.zero_()
        y, same = lrc.lrc_int8_linear(x[:n].to(dev()), w, info=info)
        assert same is info and int(info.cpu()) == lrc.LRC_ENONFINITE and torch.isfinite(y).all()
        keep = [t for t in range(n) if t not in (5, 7)]
        assert torch.equal(y[keep], clean[keep])
        info.zero_()
        lrc.lrc_int8_gated_linear(x[:n].to(dev()), w, w, info=info)
        assert int(info.cpu()) == lrc.LRC_ENONFINITE


# ----------------------------------------------------------------------------- gated block
GATED_SHAPES = [(1, 1, 1), (3, 5, 7), (1, 64, 96), (2, 512, 130), (8, 96, 64), (9, 96, 72), (17, 257, 33), (64, 1000, 48),
                (65, 64, 65), (100, 300, 520), (130, 72, 256), (257, 136, 264), (600, 520, 136)]


def product_bound(a, b, z):
    return (a.shape[1] + 8) * 2 * U * (np.abs(a) @ np.abs(b).T) + 2 * U * np.abs(z)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_ff", GATED_SHAPES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_gated(lrc, dtype, n, d_in, d_ff, layout):
    x, wg, wu = stream(n, d_in, dtype, n + d_in), weight(d_ff, d_in, dtype, 1), weight(d_ff, d_in, dtype, 2)
    half = HALF[dtype]
    _, g, u = ref.gated(f64(x), f64(wg), f64(wu), "none")
    e_g, e_u = product_bound(f64(x), f64(wg), g), product_bound(f64(x), f64(wu), u)
    first = None
    for name in ACTS:
        a = base.act(g, name)
        e = (LIP * e_g + 8 * U * np.abs(g)) * (np.abs(u) + e_u) + np.abs(a) * e_u + 4 * U * np.abs(a * u)
        for save in ["none", "z", "checkpoint"]:
            f = flag() if save == "checkpoint" else None
            h, kept, info = lrc.lrc_gated_linear(lay(x, layout), lay(wg, layout), lay(wu, "packed"), act=name, save=save,
                                                 info=f)
            check(h, a * u, e + half * (np.abs(a * u) + e) + TINY, ("h", name, save))
            if save == "z":
                check(kept[0], g, e_g + half * (np.abs(g) + e_g) + TINY, "g")
                check(kept[1], u, e_u + half * (np.abs(u) + e_u) + TINY, "u")
                assert info is None
                first = first or kept
                assert torch.equal(kept[0], first[0]) and torch.equal(kept[1], first[1])
            elif save == "checkpoint":
                # within half a step of the block's exponent, which is that of a value within the fp32 error
                for held, z, e_z in ((kept[0], g, e_g), (kept[1], u, e_u)):
                    step = np.repeat(2.0 ** f64(held[1]), 64, 1)[:, :d_ff]
                    assert (np.abs(f64(lrc.lrc_unpack_activations(*held)) - z) <= 0.5 * step + e_z).all()
                    lo, hi = (base.pack(np.abs(z) + s * e_z)[1] for s in (-1, 1))
                    assert (held[1].cpu().numpy() <= np.maximum(lo, hi)).all()
                assert int(info.cpu()) == 0
            else:
                assert kept is None and info is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_ff", [(1, 3000, 500), (8, 4096, 640), (9, 4096, 640), (33, 2048, 520), (96, 2040, 1032),
                                         (300, 1500, 1032), (1500, 264, 1030), (4096, 160, 2056), (3900, 1100, 1500),
                                         (12, 9000, 2056), (29, 4096, 2051), (64, 3999, 40)])
def test_gated_exact_on_small_integers(lrc, dtype, n, d_in, d_ff):
    """Small integers: g, u and their product are integers below 2^24, exact in any order; h is the rounded integer."""
    r = gen(n)
    ints = lambda *s: torch.randint(-1, 2, s, generator=r).to(dtype).to(dev())   # noqa: E731
    x, wg, wu = ints(n, d_in), ints(d_ff, d_in), ints(d_ff, d_in)
    g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
    h, kept, _ = lrc.lrc_gated_linear(x, wg, wu, act="relu", save="z")
    assert torch.equal(h, (g.clamp_min(0) * u).to(dtype))
    assert torch.equal(kept[0], g.to(dtype)) and torch.equal(kept[1], u.to(dtype))
    h, kept, info = lrc.lrc_gated_linear(x, wg, wu, act="none", save="checkpoint", info=flag())
    assert torch.equal(h, (g * u).to(dtype)) and int(info.cpu()) == 0
    for held, z in zip(kept, (g, u)):
        for p, q in zip(held, lrc.lrc_pack_activations(z.float())[:2]):
            assert torch.equal(p, q)


SLOPE = 24 * U      # of the slopes' fp32 evaluation, relative to 1 + |z|: an exponential, a reciprocal, a fit


def slope_errors(g, name):
    """Absolute errors of act(g) and act'(g) in fp32 (none, relu: exact)."""
    if name in ("none", "relu"):
        return 0 * g, 0 * g
    return 8 * U * np.abs(g), SLOPE * (1 + np.abs(g))


def held_or_not(lrc, t, held):
    """(what the call takes, its values in fp64)."""
    if not held:
        return t, f64(t)
    codes, exps, _ = lrc.lrc_pack_activations(t)
    return (codes, exps), base.unpack(codes.cpu().numpy(), exps.cpu().numpy())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_ff", GATED_SHAPES + [(300, 24, 1000)])
@pytest.mark.parametrize("held", [False, True])
def test_gated_backward(lrc, dtype, n, d_in, d_ff, held):
    x, dh = stream(n, d_in, dtype, n + d_in), stream(n, d_ff, dtype, 9, 0.01)
    wg, wu = weight(d_ff, d_in, dtype, 1), weight(d_ff, d_in, dtype, 2)
    z = [(1.5 * torch.randn(n, d_ff, generator=gen(k))).to(dtype) for k in (3, 4)]
    half = HALF[dtype]
    for k, layout in enumerate(LAYOUTS):
        name = ACTS[(n + k) % 4]
        (xa, xn), (ga, gn), (ua, un) = (held_or_not(lrc, lay(t, layout), held) for t in (x, *z))
        dg, du, dx, dwg, dwu = lrc.lrc_gated_linear_backward(lay(dh, layout), xa, lay(wg, layout), lay(wu, layout), ga,
                                                             ua, act=name)
        d = f64(dh)
        wdg, wdu, wdx, wwg, wwu = ref.gated_backward(d, xn, f64(wg), f64(wu), name, gn, un)
        ea, es = slope_errors(gn, name)
        e_g = np.abs(d * un) * es + 4 * U * np.abs(wdg)
        e_u = np.abs(d) * ea + 4 * U * np.abs(wdu)
        check(dg, wdg, e_g + half * (np.abs(wdg) + e_g) + TINY, ("dg", name))
        check(du, wdu, e_u + half * (np.abs(wdu) + e_u) + TINY, ("du", name))
        # dx: of the streams as they are held, one fp32 sum (fp32: two, added)
        sg, su = f64(dg), f64(du)
        want = sg @ f64(wg) + su @ f64(wu)
        e = (2 * d_ff + 12) * 2 * U * (np.abs(sg) @ np.abs(f64(wg)) + np.abs(su) @ np.abs(f64(wu)))
        check(dx, want, e + half * (np.abs(want) + e) + TINY, ("dx", name))
        assert np.abs(want - wdx).max() <= (2 * half * (np.abs(wdg) @ np.abs(f64(wg)) + np.abs(wdu) @ np.abs(f64(wu)))
                                            + e_g @ np.abs(f64(wg)) + e_u @ np.abs(f64(wu)) + 1e-30).max()
        # dW: bf16 carries two pieces of dz, 2^-8 of 2^-8 of an entry is left out
        left = 2.0 ** -16 if dtype == torch.bfloat16 else 0.0
        for got, w, dz, e_z in ((dwg, wwg, wdg, e_g), (dwu, wwu, wdu, e_u)):
            e = (e_z + left * np.abs(dz)).T @ np.abs(xn) + (2 * n + 12) * 2 * U * (np.abs(dz).T @ np.abs(xn))
            e = 1.02 * e
            check(got, w, e + half * (np.abs(w) + e) + TINY, ("dw", name))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d_in,d_ff", [(7, 520, 264), (1000, 264, 520), (300, 1032, 1030), (1111, 519, 303),
                                         (2500, 1032, 2056), (4100, 2064, 1504)])
@pytest.mark.parametrize("held", [False, True])
def test_gated_backward_exact_on_small_integers(lrc, dtype, n, d_in, d_ff, held):
    """Small integers: dg and du are exact in bf16, every sum is an integer below 2^24."""
    r = gen(n)
    ints = lambda *s: torch.randint(-2, 3, s, generator=r).to(dtype).to(dev())   # noqa: E731
    x, dh, g, u, wg, wu = ints(n, d_in), ints(n, d_ff), ints(n, d_ff), ints(n, d_ff), ints(d_ff, d_in), ints(d_ff, d_in)
    wdg, wdu = dh.double() * u.double() * (g.double() > 0), dh.double() * g.double().clamp_min(0)
    args = [held_or_not(lrc, t, held)[0] for t in (x, g, u)]
    call = lambda **k: lrc.lrc_gated_linear_backward(dh, args[0], wg, wu, args[1], args[2], act="relu", **k)   # noqa: E731
    got = call()
    assert torch.equal(got[0].double(), wdg) and torch.equal(got[1].double(), wdu)
    assert torch.equal(got[2], (wdg @ wg.double() + wdu @ wu.double()).to(dtype))
    assert torch.equal(got[3], (wdg.T.contiguous() @ x.double()).to(dtype))
    assert torch.equal(got[4], (wdu.T.contiguous() @ x.double()).to(dtype))
    wide = call(dw_dtype=torch.float32, need_dx=False)
    assert wide[2] is None and torch.equal(wide[3].double(), wdg.T.contiguous() @ x.double())
    some = call(need_dw=False)
    assert some[3] is None and some[4] is None and all(torch.equal(p, q) for p, q in zip(some[:3], got[:3]))
    some = call(need_dx=False)
    assert some[2] is None and all(torch.equal(some[k], got[k]) for k in (0, 1, 3, 4))


@pytest.mark.parametrize("n,d_in,d_ff", [(300, 200, 136), (64, 1000, 72), (1, 8, 8), (4096, 1536, 1024), (8192, 512, 4096),
                                         (4100, 1540, 1030), (2048, 5632, 1024), (2050, 5637, 1026), (4096, 256, 1024),
                                         (4147, 80, 8464)])
def test_gated_backward_joined_products(lrc, n, d_in, d_ff):
    """All products of a bf16 block in one launch or two, on each kind of tile, with and without splits: the bits of each
    gradient asked for alone, and its own formula's value from the streams."""
    r = gen(n + d_in)
    make = lambda *s: torch.randn(*s, generator=r).bfloat16().to(dev())   # noqa: E731
    dh, g, u, x, wg, wu = make(n, d_ff), make(n, d_ff), make(n, d_ff), make(n, d_in), make(d_ff, d_in), make(d_ff, d_in)
    for dw_dtype in (torch.bfloat16, torch.float32):
        call = lambda **k: lrc.lrc_gated_linear_backward(dh, x, wg, wu, g, u, dw_dtype=dw_dtype, **k)   # noqa: E731
        full, only_w, only_x = call(), call(need_dx=False), call(need_dw=False)
        assert all(torch.isfinite(t).all() for t in full)
        assert all(torch.equal(full[k], only_w[k]) for k in (0, 1, 3, 4))
        assert all(torch.equal(full[k], only_x[k]) for k in (0, 1, 2))
    # fp32 sums of k terms in any order: k 2^-24 of the terms' magnitudes (two reductions), and the result's rounding;
    # a weight gradient may differ from the streams' product by what their rounding left out, 2^-8 of each term
    f = lambda t: t.float()   # noqa: E731
    dg, du, dx, dwg, dwu = full
    want = f(dg) @ f(wg) + f(du) @ f(wu)
    size = f(dg).abs() @ f(wg).abs() + f(du).abs() @ f(wu).abs()
    assert ((f(dx) - want).abs() <= 2**-8 * want.abs() + 6 * d_ff * 2**-24 * size).all()
    for got, dz in ((dwg, dg), (dwu, du)):
        size = f(dz).abs().T.contiguous() @ f(x).abs()
        err = (got - f(dz).T.contiguous() @ f(x)).abs()
        assert (err <= (2**-8 * 1.01 + 6 * n * 2**-24) * size).all()


def test_gated_backward_against_differences(lrc):
    n, d, f = 5, 24, 40
    x, dh = stream(n, d, torch.float32, 1), stream(n, f, torch.float32, 2)
    wg, wu = weight(f, d, torch.float32, 3), weight(f, d, torch.float32, 4)
    h = 1e-5
    for name in ("silu", "gelu"):
        _, (g, u), _ = lrc.lrc_gated_linear(*on(x, wg, wu), act=name, save="z")
        _, _, dx, dwg, dwu = lrc.lrc_gated_linear_backward(*on(dh, x, wg, wu), g, u, act=name)
        loss = lambda a, b, c: (ref.gated(a, b, c, name)[0] * f64(dh)).sum()   # noqa: E731
        args = [f64(x), f64(wg), f64(wu)]
        for k, got in enumerate((dx, dwg, dwu)):
            for at in ((0, 0), (3, 17), (4, 23)):
                lo, hi = [a.copy() for a in args], [a.copy() for a in args]
                lo[k][at] -= h
                hi[k][at] += h
                want = (loss(*hi) - loss(*lo)) / (2 * h)
                assert abs(float(got[at]) - want) < 1e-4 * max(1.0, abs(want))


@pytest.mark.parametrize("n,d_in,d_ff", [(300, 136, 264), (1000, 521, 303), (2500, 1032, 2056)])
@pytest.mark.parametrize("act", ["silu", "gelu", "none"])
def test_gated_weight_gradient_keeps_the_bits_of_dz(lrc, act, n, d_in, d_ff):
    """fp32 dW of bf16 streams: within 2^-11 of the channels' norms, with magnitudes from 2^-40 to 2^40 among them."""
    r = gen(n)
    x = (torch.randn(n, d_in, generator=r) * 2.0 ** torch.randint(-30, 31, (d_in,), generator=r)).bfloat16()
    dh = (torch.randn(n, d_ff, generator=r) * 2.0 ** torch.randint(-40, 41, (d_ff,), generator=r)).bfloat16()
    g, u = (torch.randn(n, d_ff, generator=r).bfloat16() for _ in range(2))
    w = torch.zeros(d_ff, d_in, dtype=torch.bfloat16, device=dev())
    got = lrc.lrc_gated_linear_backward(*on(dh, x), w, w, *on(g, u), act=act, dw_dtype=torch.float32)
    dg, du, _, wwg, wwu = ref.gated_backward(f64(dh), f64(x), np.zeros((d_ff, d_in)), np.zeros((d_ff, d_in)), act, f64(g),
                                             f64(u))
    for dw, want, dz in ((got[3], wwg, dg), (got[4], wwu, du)):
        err = (f64(dw) - want) / (np.linalg.norm(dz, axis=0)[:, None] * np.linalg.norm(f64(x), axis=0)[None])
        assert np.abs(err).max() < 2.0 ** -11


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(200, 72), (1300, 904), (4100, 2104)])
def test_gated_nonfinite_entries(lrc, dtype, n, d):
    """NaN and infinities give what the plain products give, and stay in their rows."""
    ones = lambda *s: torch.ones(*s, dtype=dtype)   # noqa: E731
    same = lambda p, q: torch.equal(torch.nan_to_num(p.double(), 9e9, 8e8, 7e7),   # noqa: E731
                                    torch.nan_to_num(q.to(p.dtype).double(), 9e9, 8e8, 7e7))
    x, dh, w = ones(n, d), ones(n, d), ones(d, d).to(dev())
    x[7, 8], x[9, 20], dh[3, 5], dh[4, 6] = float("-inf"), float("nan"), float("inf"), float("nan")
    g, u = 2 * ones(n, d), 3 * ones(n, d)
    x, dh, g, u = on(x, dh, g, u)
    got = lrc.lrc_gated_linear_backward(dh, x, w, w, g, u, act="none")
    dg, du = dh.double() * 3, dh.double() * 2
    assert same(got[0], dg) and same(got[1], du) and same(got[2], dg @ w.double() + du @ w.double())
    assert same(got[3], dg.T.contiguous() @ x.double()) and same(got[4], du.T.contiguous() @ x.double())
    h, kept, info = lrc.lrc_gated_linear(x, w, w, act="none", save="checkpoint", info=flag())
    z = x.double() @ w.double().T
    assert same(h, z * z) and int(info.cpu()) == lrc.LRC_ENONFINITE
    clean = [t for t in range(n) if t not in (7, 9)]
    assert torch.equal(h[clean], lrc.lrc_gated_linear(ones(n, d).to(dev()), w, w, act="none")[0][clean])


def test_lowest_values_in_tokens_that_count_for_nothing(lrc):
    """Rows that a mask filled with the type's lowest value, their gradients zero: the other rows and the weights'
    gradients are as without them."""
    n, d, f = 130, 72, 136
    x, dh = stream(n, d, torch.bfloat16, 1), stream(n, f, torch.bfloat16, 2)
    g, u = stream(n, f, torch.bfloat16, 3), stream(n, f, torch.bfloat16, 4)
    wg, wu = weight(f, d, torch.bfloat16, 5), weight(f, d, torch.bfloat16, 6)
    dh[60:70] = 0
    want = lrc.lrc_gated_linear_backward(*on(dh, x, wg, wu, g, u))
    low = float(torch.finfo(torch.bfloat16).min)
    x[60:70], g[60:70], u[60:70] = low, low, low
    got = lrc.lrc_gated_linear_backward(*on(dh, x, wg, wu, g, u))
    for p, q in zip(got, want):
        assert torch.equal(p, q)


# ----------------------------------------------------------------------------- norms around a block
NORM_SHAPES = [(1, 1), (5, 2), (3, 7), (2, 64), (65, 65), (1, 4096), (300, 300), (9, 1000), (70, 1024), (5, 2050),
               (3, 8200), (4, 11008), (2, 16384)]
KINDS = ["rms", "layer"]


def standardise(x, e_x, kind, eps):
    """x^ and its error, the mean's and 1 / spread's, of rows known to within e_x: sums of d terms over per-thread
    runs and a tree, at most d / 64 + 24 deep."""
    d = x.shape[1]
    k = (d / 64 + 24) * U
    mean = x.mean(1) if kind == "layer" else np.zeros(len(x))
    e_mean = (k * np.abs(x).mean(1) + U * np.abs(mean) + e_x.mean(1)) * (kind == "layer")
    c = x - mean[:, None]
    e_c = e_x + e_mean[:, None] + 2 * U * (np.abs(c) + np.abs(mean)[:, None]) * (kind == "layer")
    var = (c * c).mean(1)
    r = 1 / np.sqrt(var + eps)
    e_var = 2 * (np.abs(c) * e_c).mean(1) + (e_c * e_c).mean(1) + (k + 2 * U) * var
    rel = 0.5 * e_var * r ** 2 / np.maximum(1 - e_var * r ** 2, 0.5) + 4 * U
    xh = c * r[:, None]
    return xh, (e_c * r[:, None] + np.abs(xh) * (rel[:, None] + 2 * U)) * 1.01, e_mean, rel * r


def norm_inputs(n, d, dtype, kind, seed):
    r = gen(seed)
    vec = lambda c, s: (c + s * torch.randn(d, generator=r))   # noqa: E731
    beta = (lambda: vec(0, 0.1)) if kind == "layer" else lambda: None
    return (stream(n, d, dtype, seed), stream(n, d, dtype, seed + 1, 3.0), (vec(1, 0.2), beta()), vec(0.4, 0.2),
            (vec(1, 0.2), beta()))


def params(p, d):
    """fp64 (gamma, beta) of a pair, absent ones 1 and 0."""
    g, b = p if p is not None else (None, None)
    return np.ones(d) if g is None else f64(g), np.zeros(d) if b is None else f64(b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", NORM_SHAPES)
@pytest.mark.parametrize("kind", KINDS)
def test_block_norm(lrc, dtype, n, d, kind):
    b, res, post, gate, pre = norm_inputs(n, d, dtype, kind, n + d)
    eps, half = 1e-5, HALF[dtype]
    e32 = float(np.float32(eps))
    for i, layout in enumerate(LAYOUTS if d < 2000 else ["packed", "offset"]):
        for with_post in (True, False):
            use_gate, use_res, scale = (i + with_post) % 2 == 0, i != 1, (0.75, 1.0, -2.5, 0.0)[i]
            po = tuple(on(*post)) if with_post else None
            s, h, stats, q, info = lrc.lrc_block_norm(
                lay(b, layout), lay(res, layout) if use_res else None, kind=kind, eps=eps, post=po,
                gate=gate.to(dev()) if use_gate else None, scale=scale, pre=tuple(on(*pre)) if i != 2 else None)
            assert q is None and info is None
            bn, p, e_p = f64(b), f64(b), np.zeros((n, d))
            if with_post:
                xh, e_xh, e_m, e_r = standardise(bn, 0 * bn, kind, e32)
                pg, pb = params(post, d)
                p, e_p = xh * pg + pb, e_xh * np.abs(pg) + 4 * U * (np.abs(xh * pg) + np.abs(pb))
            gn, rn = f64(gate) if use_gate else np.ones(d), f64(res) if use_res else np.zeros((n, d))
            add = scale * gn * p
            spread = np.abs(scale * gn) * (np.abs(p) + (2 * np.abs(params(post, d)[1]) if with_post else 0))
            e_s = np.abs(scale * gn) * e_p + 6 * U * spread + 2 * U * (np.abs(rn) + np.abs(add))
            ga, be = params(pre if i != 2 else None, d)
            ws, wh, wst = ref.block_norm(bn, rn, kind, e32, params(post, d) if with_post else None, gn, scale, ga, be)
            check(s, ws, e_s + half * (np.abs(ws) + e_s) + TINY, "s")
            xh, e_xh, e_m, e_r = standardise(ws, e_s, kind, e32)
            e_h = e_xh * np.abs(ga) + 4 * U * (np.abs(xh * ga) + np.abs(be))
            check(h, wh, e_h + half * (np.abs(wh) + e_h) + TINY, "h")
            check(stats[3], wst[3], e_r + TINY, "rstd_s")
            assert (stats[0] is None) == (not with_post or kind == "rms") and (stats[1] is None) == (not with_post)
            if kind == "layer":
                check(stats[2], wst[2], e_m + TINY, "mean_s")
            # codes: those of the written h
            out = lrc.lrc_block_norm(lay(b, layout), lay(res, layout) if use_res else None, kind=kind, eps=eps, post=po,
                                     gate=gate.to(dev()) if use_gate else None, scale=scale,
                                     pre=tuple(on(*pre)) if i != 2 else None, need_s=False, quantize=True, info=flag())
            wq, wqs, _ = lrc.lrc_quantize_tokens(h)
            assert out[0] is None and out[1] is None and torch.equal(out[3][0], wq) and torch.equal(out[3][1], wqs)
            assert int(out[4].cpu()) == 0 and out[2] is None


def through(v, e_v, xh, e_xh, r, kind):
    """Gradient of a standardised row and its error."""
    d = v.shape[1]
    k = (d / 64 + 24) * U
    c2 = (v * xh).mean(1)[:, None]
    e_c2 = (k + 4 * U) * np.abs(v * xh).mean(1)[:, None] + (e_v * np.abs(xh) + (np.abs(v) + e_v) * e_xh).mean(1)[:, None]
    c1 = e_c1 = np.zeros((len(v), 1))
    if kind == "layer":
        c1, e_c1 = v.mean(1)[:, None], (k + 2 * U) * np.abs(v).mean(1)[:, None] + e_v.mean(1)[:, None]
    out = r[:, None] * (v - c1 - xh * c2)
    e = e_v + 4 * U * (np.abs(v) + np.abs(c1) + np.abs(xh * c2)) + e_c1 + np.abs(xh) * e_c2 + e_xh * (np.abs(c2) + e_c2)
    return out, r[:, None] * e * 1.01


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", NORM_SHAPES + [(1300, 40), (700, 512), (2300, 136)])
@pytest.mark.parametrize("kind", KINDS)
def test_block_norm_backward(lrc, dtype, n, d, kind):
    b, res, post, gate, pre = norm_inputs(n, d, dtype, kind, n + d)
    dh, ds = stream(n, d, dtype, 7, 0.01), stream(n, d, dtype, 8, 0.01)
    half, layer = HALF[dtype], kind == "layer"
    for i, layout in enumerate(["packed", "padded", "offset"] if d < 2000 else ["packed", "offset"]):
        for with_post in (True, False):
            use_gate, use_ds, scale = (i + with_post) % 2 == 0, i != 1, (0.75, -2.0, 1.0)[i]
            opt = dict(kind=kind, post=tuple(on(*post)) if with_post else None,
                       gate=gate.to(dev()) if use_gate else None, scale=scale, pre=tuple(on(*pre)))
            s, _, stats, _, _ = lrc.lrc_block_norm(lay(b, layout), lay(res, layout), **opt)
            got = lrc.lrc_block_norm_backward(lay(dh, layout), lay(ds, layout) if use_ds else None, s, lay(b, layout),
                                              stats, **opt)
            zero = np.zeros(n)
            st = [zero if v is None else f64(v) for v in stats]
            norm = lambda x, m, r: ((x - m[:, None]) * r[:, None],   # noqa: E731
                                    U * (np.abs(x) + np.abs(m)[:, None]) * r[:, None] * layer
                                    + 2 * U * np.abs((x - m[:, None]) * r[:, None]))
            sh, e_sh = norm(f64(s), st[2], st[3])
            ga, gn = f64(pre[0]), f64(gate) if use_gate else np.ones(d)
            dn, dsn = f64(dh), f64(ds) if use_ds else np.zeros((n, d))
            v, e_v = through(dn * ga, 2 * U * np.abs(dn * ga), sh, e_sh, st[3], kind)
            t = dsn + v
            e_t = e_v + 2 * U * (np.abs(dsn) + np.abs(v))
            pg, pb = params(post, d) if with_post else (np.ones(d), np.zeros(d))
            bh, e_bh = norm(f64(b), st[0], st[1]) if with_post else (f64(b), 0 * f64(b))
            dp = scale * gn * t * pg
            e_p = np.abs(scale * gn * pg) * e_t + 4 * U * np.abs(dp)
            db, e_db = through(dp, e_p, bh, e_bh, st[1], kind) if with_post else (dp, e_p)
            want = ref.block_norm_backward(dn, dsn, f64(s), f64(b), st, kind, (pg, pb) if with_post else None, gn, scale,
                                           ga)
            assert np.allclose(want[0], t, rtol=1e-9, atol=1e-12) and np.allclose(want[1], db, rtol=1e-7, atol=1e-10)
            check(got[0], want[0], e_t + half * (np.abs(t) + e_t) + TINY, "dresidual")
            check(got[1], want[1], e_db + half * (np.abs(db) + e_db) + TINY, "db")
            sums = (n + 12) * U
            check(got[2], want[2], sums * np.abs(dn * sh).sum(0) + (np.abs(dn) * e_sh).sum(0) + TINY, "dgamma")
            e_C = sums * np.abs(t * bh).sum(0) + (e_t * np.abs(bh) + (np.abs(t) + e_t) * e_bh).sum(0)
            e_D = sums * np.abs(t).sum(0) + e_t.sum(0)
            C, D = np.abs((t * bh).sum(0)), np.abs(t.sum(0))
            w = np.abs(scale * gn)
            assert (got[3] is not None) == layer and (got[4] is not None) == with_post
            assert (got[5] is not None) == (with_post and layer) and (got[6] is not None) == use_gate
            if layer:
                check(got[3], want[3], sums * np.abs(dn).sum(0) + TINY, "dbeta")
            if with_post:
                check(got[4], want[4], w * (e_C + 3 * U * C) + TINY, "dpost_gamma")
            if with_post and layer:
                check(got[5], want[5], w * (e_D + 3 * U * D) + TINY, "dpost_beta")
            if use_gate:
                e = np.abs(pg) * (e_C + 4 * U * C) + np.abs(pb) * (e_D + 4 * U * D)
                check(got[6], want[6], abs(scale) * e * 1.01 + TINY, "dgate")


def test_block_norm_backward_parts_and_differences(lrc):
    """Each output alone equals the joint call; the gradients against central differences of the fp64 forward."""
    n, d, h = 6, 37, 1e-5
    for kind in KINDS:
        b, res, post, gate, pre = norm_inputs(n, d, torch.float32, kind, 5)
        dh, ds = stream(n, d, torch.float32, 7), stream(n, d, torch.float32, 8)
        b[2], res[2] = torch.randn(d, generator=gen(1)), torch.randn(d, generator=gen(2))   # no row without a spread
        opt = dict(kind=kind, post=tuple(on(*post)), gate=gate.to(dev()), scale=0.75, pre=tuple(on(*pre)))
        s, _, stats, _, _ = lrc.lrc_block_norm(*on(b, res), **opt)
        a = (*on(dh, ds), s, b.to(dev()), stats)
        full = lrc.lrc_block_norm_backward(*a, **opt)
        for only in ("need_dresidual", "need_db", "need_dparams"):
            some = lrc.lrc_block_norm_backward(*a, **opt, **{only: False})
            assert all(q is None or torch.equal(p, q) for p, q in zip(full, some))
            assert (some[0] is None, some[1] is None, some[2] is None) == tuple(
                only == k for k in ("need_dresidual", "need_db", "need_dparams"))

        def loss(bb, rr, g):
            pg, pb = params(post, d)
            ga, be = params(pre, d)
            ss, hh, _ = ref.block_norm(bb, rr, kind, 1e-5, (pg, pb), g, 0.75, ga, be)
            return (hh * f64(dh)).sum() + (ss * f64(ds)).sum()

        args = [f64(b), f64(res), f64(gate)]
        for k, got in ((0, full[1]), (1, full[0]), (2, full[6])):
            for at in ((0, 0), (4, 36), (5, 20)):
                at = at if k < 2 else at[1:]
                lo, hi = [v.copy() for v in args], [v.copy() for v in args]
                lo[k][at] -= h
                hi[k][at] += h
                want = (loss(*hi) - loss(*lo)) / (2 * h)
                assert abs(float(got[at]) - want) < 2e-4 * max(1.0, abs(want)), (kind, k, at)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_block_norm_ends(lrc, dtype, kind):
    """The last block (no h), a gradient from one side only, a plain norm (no residual, s not written), s in place."""
    n, d = 70, 264
    b, res, post, gate, pre = norm_inputs(n, d, dtype, kind, 3)
    bd, rd = on(b, res)
    po, pr, ga = tuple(on(*post)), tuple(on(*pre)), gate.to(dev())
    opt = dict(kind=kind, post=po, gate=ga, scale=0.5)
    s, h, stats, _, _ = lrc.lrc_block_norm(bd, rd, pre=pr, **opt)
    s2, h2, st2, _, _ = lrc.lrc_block_norm(bd, rd, need_h=False, **opt)
    assert torch.equal(s, s2) and h2 is None and st2[3] is None and torch.equal(st2[1], stats[1])
    ds, dh = stream(n, d, dtype, 5).to(dev()), stream(n, d, dtype, 6).to(dev())
    got = lrc.lrc_block_norm_backward(None, ds, None, bd, st2, **opt)
    zero = lrc.lrc_block_norm_backward(torch.zeros_like(ds), ds, s, bd, stats, **opt)
    assert torch.equal(got[0], ds) and all(torch.equal(p, q) for p, q in zip(got, zero) if p is not None)
    assert got[2] is None
    one = lrc.lrc_block_norm_backward(dh, None, s, bd, stats, pre=pr, **opt)
    two = lrc.lrc_block_norm_backward(dh, torch.zeros_like(ds), s, bd, stats, pre=pr, **opt)
    assert all(torch.equal(p, q) for p, q in zip(one, two) if p is not None)
    # a plain norm
    none, y, st, _, _ = lrc.lrc_block_norm(bd, kind=kind, pre=pr, need_s=False)
    copy, y2, _, _, _ = lrc.lrc_block_norm(bd, torch.zeros_like(bd), kind=kind, pre=pr)
    assert none is None and torch.equal(y, y2) and torch.equal(copy, bd)
    if kind == "layer":
        ln, mean, rstd, _, _ = lrc.lrc_layer_norm(bd, *pr)
        assert torch.equal(ln, y) and torch.equal(st[2], mean) and torch.equal(st[3], rstd)
    # s in the residual's place
    code = 1 if dtype == torch.bfloat16 else 0
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())   # noqa: E731
    stm = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    out = torch.empty_like(h)
    r2 = rd.clone()
    assert lrc.lib.lrc_block_norm(p(bd), code, n, d, d, p(r2), d, lrc._NORMS[kind], 1e-5, 1, p(po[0]), p(po[1]), p(ga), 0.5,
                                  p(pr[0]), p(pr[1]), p(r2), d, p(out), d, None, None, None, None, None, 0, None, None,
                                  stm) == 0
    assert torch.equal(r2, s) and torch.equal(out, h)


@pytest.mark.parametrize("kind", KINDS)
def test_block_norm_extremes(lrc, kind):
    """Rows of zeros, of the lowest value, past the range of the squares, with NaN and infinities: the formula's
    result, in their own rows."""
    n, d = 12, 96
    for dtype in DTYPES:
        low = float(torch.finfo(dtype).min)
        x = stream(n, d, dtype, 1)
        clean = lrc.lrc_block_norm(x.to(dev()), kind=kind)[1]
        y = x.clone()
        y[3], y[4], y[5, 7], y[6, 8] = 0, low, float("nan"), float("inf")
        y[7] = low
        y[7, ::2] = -low
        s, h, stats, q, info = lrc.lrc_block_norm(y.to(dev()), kind=kind)
        keep = [t for t in range(n) if t not in (3, 4, 5, 6, 7)]
        assert torch.equal(h[keep], clean[keep]) and not h[3].any() and not h[4].any() and not h[7].any()
        assert torch.isnan(h[5]).all() and torch.isnan(h[6]).any()
        out = lrc.lrc_block_norm(y.to(dev()), kind=kind, quantize=True, info=flag())
        assert int(out[4].cpu()) == lrc.LRC_ENONFINITE
        wq, ws, _ = lrc.lrc_quantize_tokens(h)
        assert torch.equal(out[3][0], wq) and torch.equal(out[3][1], ws)


# ----------------------------------------------------------------------------- the operators together
def test_step_of_a_block(lrc):
    """Norm of the sum -> gated projections (8-bit checkpoints) -> down projection -> norm of the next sum; backward;
    the two output-gradient streams go into a covariance."""
    n, d, f = 600, 96, 160
    bf = torch.bfloat16
    b, res = stream(n, d, bf, 1).to(dev()), stream(n, d, bf, 2).to(dev())
    wg, wu, wd = weight(f, d, bf, 3).to(dev()), weight(f, d, bf, 4).to(dev()), weight(d, f, bf, 5).to(dev())
    r = gen(6)
    vec = lambda: (1 + 0.1 * torch.randn(d, generator=r)).to(dev())   # noqa: E731
    g1, g2, g3, gate = vec(), vec(), vec(), 0.5 * vec()
    s1, h1, st1, _, _ = lrc.lrc_block_norm(b, res, gate=gate, pre=(g1, None))
    h1k = lrc.lrc_pack_activations(h1)[:2]
    a, kept, info = lrc.lrc_gated_linear(h1, wg, wu, save="checkpoint", info=flag())
    ak = lrc.lrc_pack_activations(a)[:2]
    y, _, _ = lrc.lrc_linear(a, wd)
    s2, h2, st2, _, _ = lrc.lrc_block_norm(y, s1, post=(g2, None), scale=0.7, pre=(g3, None))
    assert int(info.cpu()) == 0
    dh2, ds2 = stream(n, d, bf, 7, 0.01).to(dev()), stream(n, d, bf, 8, 0.01).to(dev())
    ds1, dy, dg3, _, dg2, _, _ = lrc.lrc_block_norm_backward(dh2, ds2, s2, y, st2, post=(g2, None), scale=0.7,
                                                             pre=(g3, None))
    _, da, dwd, _ = lrc.lrc_linear_backward(dy, ak, wd)
    dg, du, dh1, dwg, dwu = lrc.lrc_gated_linear_backward(da, h1k, wg, wu, *kept)
    dres, db, dg1, _, _, _, dgate = lrc.lrc_block_norm_backward(dh1, ds1, s1, b, st1, gate=gate, pre=(g1, None))
    # the same step in fp64
    leaves = [t.double().requires_grad_() for t in (b, res, wg, wu, wd, g1, g2, g3, gate)]
    B, R, WG, WU, WD, G1, G2, G3, GT = leaves
    rms = lambda v: v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5)   # noqa: E731
    S1 = R + GT * B
    H1 = rms(S1) * G1
    z = H1 @ WG.T
    Y = ((z * torch.sigmoid(z)) * (H1 @ WU.T)) @ WD.T
    S2 = S1 + 0.7 * rms(Y) * G2
    H2 = rms(S2) * G3
    ((H2 * dh2.double()).sum() + (S2 * ds2.double()).sum()).backward()
    off = lambda got, want: float((got.double() - want).norm() / want.norm())   # noqa: E731
    # 8-bit checkpoints hold a value to about 1.3 % of its block's largest; with bf16 streams in between 6 % is far
    # outside
    assert off(s2, S2.detach()) < 0.01 and off(h2, H2.detach()) < 0.01
    for got, leaf in zip((db, dres, dwg, dwu, dwd, dg1, dg2, dg3, dgate), leaves):
        assert off(got, leaf.grad) < 0.06
    for t in (dg, du):
        c = torch.zeros(f, f, device=dev())
        lrc.lrc_accumulate_cov(t, c)
        assert off(c.tril(), (t.double().T.contiguous() @ t.double()).tril()) < 1e-5


def test_block_in_8_bits(lrc):
    """Norm with codes -> gated product -> down product onto the stream, all in 8-bit integers, one token and many:
    the bits of the operators apart, and near the bf16 block."""
    d, f = 96, 160
    r = gen(1)
    w = [(torch.randn(*s, generator=r) / math.sqrt(s[1])).to(dev()) for s in ((f, d), (f, d), (d, f))]
    wg, wu, wd = (lrc.lrc_quantize_rows(t) for t in w)
    gamma = (1 + 0.1 * torch.randn(d, generator=r)).to(dev())
    for n in (1, 8, 40, 300):
        b, res = stream(n, d, torch.bfloat16, 2).to(dev()), stream(n, d, torch.bfloat16, 3).to(dev())
        s, _, _, q, info = lrc.lrc_block_norm(b, res, pre=(gamma, None), quantize=True, info=flag())
        a, _ = lrc.lrc_int8_gated_linear(q, wg, wu)
        y, _ = lrc.lrc_int8_linear(a, wd, residual=s, info=info)
        assert int(info.cpu()) == 0
        s2, h, _, _, _ = lrc.lrc_block_norm(b, res, pre=(gamma, None))
        a2, _ = lrc.lrc_int8_gated_linear(h, wg, wu)
        assert torch.equal(s, s2) and torch.equal(a, a2)
        assert torch.equal(y, lrc.lrc_int8_linear(lrc.lrc_quantize_tokens(a)[:2], wd, residual=s)[0])
        plain = lrc.lrc_linear(lrc.lrc_gated_linear(h, w[0].bfloat16(), w[1].bfloat16())[0], w[2].bfloat16())[0].double()
        # steps of 1 / 127 of the largest of about 100 values: about 1 % of their root mean square for each operand
        assert float(((y.double() - s.double()) - plain).norm() / plain.norm()) < 0.1


# ----------------------------------------------------------------------------- how they run
def _ops(lrc, dtype, n, d, f):
    """Calls of every operator on one set of inputs, each returning a tuple of tensors."""
    x, dh = stream(n, d, dtype, 1).to(dev()), stream(n, f, dtype, 2, 0.01).to(dev())
    res, dx = stream(n, d, dtype, 3).to(dev()), stream(n, d, dtype, 4).to(dev())
    wg, wu = weight(f, d, dtype, 5).to(dev()), weight(f, d, dtype, 6).to(dev())
    g8, u8 = (tuple(on(*codes_of(f, d, k))) for k in (7, 8))
    _, kept, _ = lrc.lrc_gated_linear(x, wg, wu, save="checkpoint")
    gamma = (1 + 0.1 * torch.randn(d, generator=gen(9))).to(dev())
    opt = dict(kind="layer", post=(gamma, gamma), gate=gamma, scale=0.5, pre=(gamma, gamma))
    s, _, st, _, _ = lrc.lrc_block_norm(x, res, **opt)
    return [lambda: lrc.lrc_quantize_tokens(x)[:2],
            lambda: lrc.lrc_int8_linear(x, g8, act="gelu", residual=dh)[:1],
            lambda: lrc.lrc_int8_gated_linear(x, g8, u8)[:1],
            lambda: lrc.lrc_gated_linear(x, wg, wu)[:1],
            lambda: sum(lrc.lrc_gated_linear(x, wg, wu, save="checkpoint")[1], ()),
            lambda: lrc.lrc_gated_linear_backward(dh, x, wg, wu, *kept),
            lambda: lrc.lrc_block_norm(x, res, **opt)[:2],
            lambda: lrc.lrc_block_norm(x, res, **opt, quantize=True)[3],
            lambda: lrc.lrc_block_norm_backward(dx, res, s, x, st, **opt)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d,f", [(5, 512, 256), (20, 136, 520), (200, 136, 520), (1200, 321, 264)])
def test_equal_inputs_give_equal_bits_and_graphs_replay(lrc, dtype, n, d, f):
    """Two calls agree bit for bit; a captured call replays to the same bits, also with other work in between."""
    for call in _ops(lrc, dtype, n, d, f):
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
    w8 = (torch.ones(32, 48, dtype=torch.int8, device=dev()), torch.ones(32, device=dev()))
    q, s, _ = lrc.lrc_quantize_tokens(x)
    assert q.shape == (0, 48) and s.shape == (0,)
    assert lrc.lrc_int8_linear(x, w8)[0].shape == (0, 32) and lrc.lrc_int8_linear((q, s), w8)[0].shape == (0, 32)
    assert lrc.lrc_int8_gated_linear(x, w8, w8)[0].shape == (0, 32)
    h, kept, _ = lrc.lrc_gated_linear(x, w, w, save="checkpoint")
    assert h.shape == (0, 32) and kept[1][0].shape == (0, 32)
    for dwt in (dtype, torch.float32):
        dg, du, dx, dwg, dwu = lrc.lrc_gated_linear_backward(h, x, w, w, *kept, dw_dtype=dwt)
        assert dg.shape == (0, 32) and dx.shape == (0, 48) and dwg.dtype == dwt and not dwg.any() and not dwu.any()
    one = torch.ones(48, device=dev())
    opt = dict(kind="layer", post=(one, one), gate=one, pre=(one, one))
    s, h, st, _, _ = lrc.lrc_block_norm(x, x, **opt)
    assert s.shape == h.shape == (0, 48)
    got = lrc.lrc_block_norm_backward(x, x, s, x, st, **opt)
    assert got[0].shape == (0, 48) and not any(v.any() for v in got[2:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [5, 37])
def test_outputs_stay_inside_their_rows(lrc, dtype, n):
    """Outputs with a pitch through the C interface: what lies between and behind the rows is left as it was."""
    d, f, gap = 80, 104, 8
    code, L = (1 if dtype == torch.bfloat16 else 0), lrc.lib
    x, dh = stream(n, d, dtype, 1).to(dev()), stream(n, f, dtype, 2).to(dev())
    w, w2 = weight(f, d, dtype, 3).to(dev()), weight(f, d, dtype, 4).to(dev())
    q8, s8 = on(*codes_of(f, d, 5))
    p = lambda t: ctypes.c_void_p(t.data_ptr())   # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    box = lambda rows, cols, dt=dtype: torch.full((rows + 2, cols + gap), 7, dtype=dt, device=dev())   # noqa: E731
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=dev())
    tail = (p(ws), ws.numel(), st)
    h, g, u, y, hg = (box(n, f) for _ in range(5))
    dx, dwg, dwu, s, hn, dr, db = box(n, d), box(f, d), box(f, d), box(n, d), box(n, d), box(n, d), box(n, d)
    q, flat = box(n, d, torch.int8), torch.empty(3, n, f, dtype=dtype, device=dev())
    vec = torch.empty(4, n, device=dev())
    assert L.lrc_gated_linear(p(x), code, n, d, f, d, p(w), p(w2), d, 3, p(h), f + gap, p(g), p(u), f + gap, None, None,
                              None, None, None, *tail) == 0
    assert L.lrc_gated_linear_backward(p(dh), code, n, d, f, f, p(w), p(w2), d, p(x), d, None, None, 3, p(g), p(u), f + gap,
                                       None, None, None, None, p(flat[0]), p(flat[1]), p(dx), d + gap, p(dwg), p(dwu),
                                       code, d + gap, *tail) == 0
    assert L.lrc_int8_linear(p(x), code, n, d, f, d, None, 0, None, p(q8), d, p(s8), None, 0, None, 0, p(y), f + gap, None,
                             *tail) == 0
    assert L.lrc_int8_gated_linear(p(x), code, n, d, f, d, None, 0, None, p(q8), d, p(s8), p(q8), d, p(s8), 0, p(hg),
                                   f + gap, None, *tail) == 0
    assert L.lrc_quantize_tokens(p(x), code, n, d, d, p(q), d + gap, p(vec[0]), None, st) == 0
    assert L.lrc_block_norm(p(x), code, n, d, d, p(x), d, 1, 1e-5, 1, None, None, None, 0.5, None, None, p(s), d + gap,
                            p(hn), d + gap, None, p(vec[1]), None, p(vec[2]), None, 0, None, None, st) == 0
    assert L.lrc_block_norm_backward(p(x), code, n, d, d, None, 0, p(s), d + gap, p(x), d, None, p(vec[1]), None, p(vec[2]),
                                     1, 1, None, None, None, 0.5, None, p(dr), d + gap, p(db), d + gap, None, None, None,
                                     None, None, *tail) == 0
    for t, rows, cols in ((h, n, f), (g, n, f), (u, n, f), (y, n, f), (hg, n, f), (dx, n, d), (dwg, f, d), (dwu, f, d),
                          (s, n, d), (hn, n, d), (dr, n, d), (db, n, d), (q, n, d)):
        assert (t[rows:] == 7).all() and (t[:, cols:] == 7).all() and not (t[:rows, :cols] == 7).all()
    hh, (gg, uu), _ = lrc.lrc_gated_linear(x, w, w2, save="z")
    assert torch.equal(h[:n, :f], hh) and torch.equal(g[:n, :f], gg) and torch.equal(u[:n, :f], uu)
    assert torch.equal(y[:n, :f], lrc.lrc_int8_linear(x, (q8, s8))[0])


def test_offsets_past_32_bits(lrc):
    """Rows whose offsets pass 2^32 elements: the same results as rows that lie together."""
    n, d, ld = 5, 80, (1 << 30) + 64
    big = torch.empty((n - 1) * ld + d, dtype=torch.bfloat16, device=dev())
    far = big.as_strided((n, d), (ld, 1))
    x = stream(n, d, torch.bfloat16, 1).to(dev())
    far.copy_(x)
    w, w2, w8 = weight(40, d, torch.bfloat16, 2).to(dev()), weight(40, d, torch.bfloat16, 3).to(dev()), on(*codes_of(40, d, 4))
    dh = stream(n, 40, torch.bfloat16, 5).to(dev())
    for a, b in zip(lrc.lrc_quantize_tokens(far)[:2], lrc.lrc_quantize_tokens(x)[:2]):
        assert torch.equal(a, b)
    assert torch.equal(lrc.lrc_int8_linear(far, w8, residual=None)[0], lrc.lrc_int8_linear(x, w8)[0])
    h, (g, u), _ = lrc.lrc_gated_linear(x, w, w2, save="z")
    assert torch.equal(lrc.lrc_gated_linear(far, w, w2)[0], h)
    for a, b in zip(lrc.lrc_gated_linear_backward(dh, far, w, w2, g, u), lrc.lrc_gated_linear_backward(dh, x, w, w2, g, u)):
        assert torch.equal(a, b)
    s, hn, st, _, _ = lrc.lrc_block_norm(far, far, post=(None, None))
    s2, h2, _, _, _ = lrc.lrc_block_norm(x, x, post=(None, None))
    assert torch.equal(s, s2) and torch.equal(hn, h2)
    for a, b in zip(lrc.lrc_block_norm_backward(far, far, far, far, st, post=(None, None)),
                    lrc.lrc_block_norm_backward(x, x, x, x, st, post=(None, None))):
        assert a is b is None or torch.equal(a, b)


def test_refusals(lrc):
    x, w = torch.zeros(4, 64, device=dev()), torch.zeros(8, 64, device=dev())
    q, s = torch.zeros(8, 64, dtype=torch.int8, device=dev()), torch.zeros(8, device=dev())
    h, v = x[:, :8], torch.zeros(64, device=dev())
    st = (None, None, None, torch.ones(4, device=dev()))
    bad = [lambda: lrc.lrc_quantize_tokens(x.half()), lambda: lrc.lrc_quantize_tokens(x.cpu()),
           lambda: lrc.lrc_int8_linear(x, q), lambda: lrc.lrc_int8_linear(x, (w, s)),
           lambda: lrc.lrc_int8_linear(x, (q[:, :63], s)), lambda: lrc.lrc_int8_linear(x, (q, s[:7])),
           lambda: lrc.lrc_int8_linear(x, (q, None)), lambda: lrc.lrc_int8_linear((q, None), (q, s)),
           lambda: lrc.lrc_int8_linear((q, s, s), (q, s)), lambda: lrc.lrc_int8_linear(x, (q, s), dtype=torch.bfloat16),
           lambda: lrc.lrc_int8_linear((q, s), (q, s), dtype=torch.float16),
           lambda: lrc.lrc_int8_linear(x, (q, s), act="tanh"), lambda: lrc.lrc_int8_linear(x, (q, s), residual=x),
           lambda: lrc.lrc_int8_gated_linear(x, (q, s), (q[:7], s[:7])),
           lambda: lrc.lrc_gated_linear(x, w, w[:7]), lambda: lrc.lrc_gated_linear(x, w, w.bfloat16()),
           lambda: lrc.lrc_gated_linear(x, w[:, :63], w), lambda: lrc.lrc_gated_linear(x, w, w, save="all"),
           lambda: lrc.lrc_gated_linear(x, w, w, act="tanh"),
           lambda: lrc.lrc_gated_linear_backward(h, None, w, w, h, h), lambda: lrc.lrc_gated_linear_backward(h, x, w, w, h, None),
           lambda: lrc.lrc_gated_linear_backward(h, x, w, w, h, (q, q)), lambda: lrc.lrc_gated_linear_backward(x, x, w, w, h, h),
           lambda: lrc.lrc_gated_linear_backward(h, x, w, w, h, h, dw_dtype=torch.bfloat16),
           lambda: lrc.lrc_block_norm(x, kind="batch"), lambda: lrc.lrc_block_norm(x, x[:3]),
           lambda: lrc.lrc_block_norm(x, pre=(v, v)), lambda: lrc.lrc_block_norm(x, post=(v,)),
           lambda: lrc.lrc_block_norm(x, gate=v[:63]), lambda: lrc.lrc_block_norm(x, need_s=False, need_h=False),
           lambda: lrc.lrc_block_norm(x, x.bfloat16()),
           lambda: lrc.lrc_block_norm_backward(None, None, x, x, st), lambda: lrc.lrc_block_norm_backward(x, None, None, x, st),
           lambda: lrc.lrc_block_norm_backward(x, None, x, x, st[:3]), lambda: lrc.lrc_block_norm_backward(x, x, x, x, None),
           lambda: lrc.lrc_block_norm_backward(x, None, x, x, st, kind="layer"),
           lambda: lrc.lrc_block_norm_backward(x, None, x, None, st, gate=v)]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was taken")
    for call in (lambda: lrc.lrc_block_norm(x, eps=-1.0), lambda: lrc.lrc_block_norm(x, eps=float("nan")),
                 lambda: lrc.lrc_block_norm(torch.zeros(2, 16385, device=dev())),
                 lambda: lrc.lrc_int8_linear(torch.zeros(2, 1 << 17, device=dev()),
                                             (torch.zeros(2, 1 << 17, dtype=torch.int8, device=dev()), s[:2]))):
        with pytest.raises(lrc.LrcError):
            call()
