"""Block operators over the ranges of their kernels: every shape of a row, every kind of tile and split of the weight
gradients, the ends of the norms' epsilon.

Tolerances as in test_gpu_block_ops.py: u = 2^-24, a fp32 sum of K terms is off by at most (K + c) u times the sum of
the terms' magnitudes, the matrix cores' internal adds counted as two roundings each.
"""
import pytest
import torch

import tests.test_gpu_block_ops as ops
from tests.test_gpu_train_ops import DTYPES, dev, stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lrc():
    import curvature_aware_rank_amd as m
    return m


# ----------------------------------------------------------------------------- norms around a block
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ops.KINDS)
@pytest.mark.parametrize("d", [24, 200, 300, 1000, 2000, 4100])
def test_block_norm_codes_without_an_epsilon(lrc, dtype, kind, d):
    """eps = 0, tokens that do not fill a workgroup: only the tokens that exist count for `info`."""
    for n in (1, 5, 18):
        x = torch.randn(n, d, generator=ops.gen(n + d)).to(dtype).to(dev())
        one = torch.ones(d, device=dev())
        for post in (None, (one, None)):
            opt = dict(kind=kind, eps=0.0, post=post)
            h = lrc.lrc_block_norm(x, **opt)[1]
            assert torch.isfinite(h).all()
            _, _, _, (q, scale), info = lrc.lrc_block_norm(x, quantize=True, info=ops.flag(), **opt)
            wq, ws, _ = lrc.lrc_quantize_tokens(h)
            assert torch.equal(q, wq) and torch.equal(scale, ws)
            assert int(info.cpu()) == 0
    x[0] = 0   # a token of zeros has no spread: 0 / 0
    info = lrc.lrc_block_norm(x, kind=kind, eps=0.0, quantize=True, info=ops.flag())[4]
    assert int(info.cpu()) == lrc.LRC_ENONFINITE


# ----------------------------------------------------------------------------- gradients of the gated block
def _left_out_products(sign):
    """(m, m', how many): bf16 factors m / 128, m' / 128 whose product lies in [1, 2) and rounds to bf16 with a remainder
    of `sign` that is 0.31 to 0.48 of a step (2^-7): 2^-8.7 of the product at least, and exact in bf16.  A row of m' for
    each m."""
    lo, hi = (40, 62) if sign > 0 else (66, 88)
    rows = {m: [k for k in range(128, 256) if 1 << 14 <= m * k < 1 << 15 and lo <= m * k % 128 <= hi]
            for m in range(128, 182)}
    rows = {m: r for m, r in rows.items() if r}
    longest = max(len(r) for r in rows.values())
    return (torch.tensor(list(rows)), torch.tensor([r + r[:1] * (longest - len(r)) for r in rows.values()]),
            torch.tensor([len(r) for r in rows.values()]))


def _left_out_inputs(n, d_in, d_ff, seed, sign):
    """dh, g, u and x of a block without an activation whose dg and du all round with a remainder of one sign, and whose
    products with x all have the sign of the channel: no term of a weight gradient cancels another."""
    r = ops.gen(seed)
    first, second, count = _left_out_products(sign)
    m = torch.randint(0, len(first), (n, d_ff), generator=r)
    pick = lambda: second[m, (torch.rand(n, d_ff, generator=r) * count[m]).long()] / 128   # noqa: E731
    token = torch.randint(0, 2, (n, 1), generator=r) * 2 - 1
    channel = 2.0 ** torch.randint(-3, 4, (1, d_ff), generator=r) * (torch.randint(0, 2, (1, d_ff), generator=r) * 2 - 1)
    dh = first[m] / 128 * token * channel
    x = torch.randint(1, 4, (n, d_in), generator=r) * token
    return [t.bfloat16() for t in (dh, pick(), pick(), x)]


def _left_out_bound(n):
    """Of a weight gradient, relative: dz is exact in two bf16, the left-out pieces are multiples of 2^-14 whose sums (at
    most 3 n 62 of them) are exact, so only the sum of the streams' n terms rounds, two roundings each."""
    assert 3 * 62 * n < 1 << 24
    return (n + 12) * 2 * ops.U


# weight gradients on the smallest tiles, on 128 x 128 and on 256 x 256 ones, not split; split in two and in four;
# split in three, so that one split ends the first segment and begins the second, in a launch apart from dx
LEFT_OUT_SHAPES = [(300, 136, 264), (2500, 1032, 2056), (2048, 5632, 1024), (4096, 1536, 1024), (4096, 256, 1024),
                   (4147, 80, 8464)]


@pytest.mark.parametrize("n,d_in,d_ff", LEFT_OUT_SHAPES)
def test_gated_weight_gradient_has_what_rounding_left_out(lrc, n, d_in, d_ff):
    """bf16 streams, fp32 weight gradients, elementwise: every entry would be 2^-8.7 of itself off without the left-out
    pieces, and as much if they counted twice or the streams came in their place."""
    dh, g, u, x = _left_out_inputs(n, d_in, d_ff, n, 1)
    w = torch.zeros(d_ff, d_in, dtype=torch.bfloat16, device=dev())
    got = lrc.lrc_gated_linear_backward(*ops.on(dh, x), w, w, *ops.on(g, u), act="none", dw_dtype=torch.float32)
    rel = _left_out_bound(n)
    for dw, stream_out, factor in ((got[3], got[0], u), (got[4], got[1], g)):
        dz = dh.double() * factor.double()
        rounded = dz.bfloat16().double()
        assert torch.equal(stream_out.cpu().double(), rounded)
        want, without = dz.T @ x.double(), rounded.T @ x.double()
        bound = rel * want.abs()
        # the oracle with the mistake is off by more than three times the bound everywhere
        assert ((want - without).abs() > 3 * bound).all()
        assert ((dw.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("n,d_in,d_ff", LEFT_OUT_SHAPES)
@pytest.mark.parametrize("dw_dtype", DTYPES)
def test_gated_weight_gradient_of_nonfinite_inputs(lrc, n, d_in, d_ff, dw_dtype):
    """Infinities and NaN in x: where a channel has one the stream alone counts, whose pieces have the other sign here,
    and the other channels keep their left-out pieces; on every kind of tile and split."""
    dh, g, u, x = _left_out_inputs(n, d_in, d_ff, n + 1, -1)
    token = x[:, :1].sign()
    inf = float("inf")
    for c, t in ((3, 5), (10, n // 4), (20, n // 2), (31, n - 3)):
        x[t, c] = inf * token[t, 0]
    x[n // 3, 40], x[7, 50], x[n - 7, 50] = float("nan"), inf * token[7, 0], -inf * token[n - 7, 0]
    x[n // 2, 60] = -inf * token[n // 2, 0]
    w = torch.zeros(d_ff, d_in, dtype=torch.bfloat16, device=dev())
    got = lrc.lrc_gated_linear_backward(*ops.on(dh, x), w, w, *ops.on(g, u), act="none", dw_dtype=dw_dtype)
    rel = _left_out_bound(n)
    if dw_dtype == torch.bfloat16:   # the result's rounding: values of [1, 2) lie 2^-7 apart, half of that is 2^-8
        rel += (1 + rel) * ops.HALF[dw_dtype]
    clean = torch.isfinite(x).all(0)
    assert int((~clean).sum()) == 7
    for dw, factor in ((got[3], u), (got[4], g)):
        dz = dh.double() * factor.double()
        dw = dw.cpu().double()
        plain = dz.bfloat16().double().T @ x[:, ~clean].double()
        assert not torch.isfinite(plain).any()
        assert torch.equal(torch.nan_to_num(dw[:, ~clean], 9.0, 8.0, 7.0), torch.nan_to_num(plain, 9.0, 8.0, 7.0))
        want = dz.T @ x[:, clean].double()
        assert ((dw[:, clean] - want).abs() <= rel * want.abs()).all()


# ----------------------------------------------------------------------------- every shape of a row
# a ragged and a full width of the shapes that a token may have in registers: 32 lanes, 2 waves (backward 3 and 4), 8 waves
ROW_WIDTHS = [200, 256, 1030, 1536, 1540, 2048, 4100, 5120, 8192]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", ROW_WIDTHS)
@pytest.mark.parametrize("layout", ["packed", "offset"])
def test_quantize_tokens_row_shapes(lrc, dtype, d, layout):
    ops.test_quantize_tokens_bit_exact(lrc, dtype, 5, d, layout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", ROW_WIDTHS)
@pytest.mark.parametrize("kind", ops.KINDS)
def test_block_norm_row_shapes(lrc, dtype, d, kind):
    ops.test_block_norm(lrc, dtype, 5, d, kind)


# the widths, and several workgroups of uneven counts of tokens (rows past 8192 channels keep two of the sums in LDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [*((5, d) for d in ROW_WIDTHS), (70, 1536), (45, 2048), (30, 5120), (41, 8200), (37, 11008),
                                 (18, 16384)])
@pytest.mark.parametrize("kind", ops.KINDS)
def test_block_norm_backward_row_shapes(lrc, dtype, n, d, kind):
    ops.test_block_norm_backward(lrc, dtype, n, d, kind)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 1), (5, 2), (65, 65), (300, 300), (9, 1000), (70, 1024), (5, 2050), (3, 4096), (3, 8200),
                                 (4, 11008), (2, 16384), *((6, d) for d in ROW_WIDTHS)])
@pytest.mark.parametrize("kind", ops.KINDS)
def test_block_norm_statistics_of_the_block(lrc, dtype, n, d, kind):
    """The post-norm's mean and 1 / spread as values, also where h is not asked for."""
    b, res, post, gate, _ = ops.norm_inputs(n, d, dtype, kind, n + d)
    eps = float(torch.tensor(1e-5))
    _, _, e_mean, e_rstd = ops.standardise(ops.f64(b), 0 * ops.f64(b), kind, eps)
    mean, rstd = ops.ref._moments(ops.f64(b), kind, eps)
    post = tuple(ops.on(*post))
    for need_h in (True, False):
        stats = lrc.lrc_block_norm(*ops.on(b, res), kind=kind, eps=1e-5, post=post, gate=gate.to(dev()), need_h=need_h)[2]
        ops.check(stats[1], rstd, e_rstd + ops.TINY, "rstd_b")
        if kind == "layer":
            ops.check(stats[0], mean, e_mean + ops.TINY, "mean_b")


# More tokens than the widest launch holds at once, for every shape: a workgroup takes several, its loads a token ahead.
LONG = [(33000, 24), (16700, 200), (8300, 300), (8200, 1000), (2100, 1030), (4200, 1536), (4200, 2048), (2100, 4096),
        (1100, 4100), (1050, 8200), (1030, 16384)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", LONG)
@pytest.mark.parametrize("kind", ops.KINDS)
def test_block_norm_many_tokens(lrc, dtype, n, d, kind):
    """A token's results do not depend on the others: the bits of calls on a few tokens each."""
    b, res, post, gate, pre = ops.norm_inputs(n, d, dtype, kind, n + d)
    b, res, dh, ds = ops.on(b, res, stream(n, d, dtype, 7, 0.01), stream(n, d, dtype, 8, 0.01))
    opt = dict(kind=kind, post=tuple(ops.on(*post)), gate=gate.to(dev()), scale=0.75, pre=tuple(ops.on(*pre)))
    s, h, stats, _, _ = lrc.lrc_block_norm(b, res, **opt)
    _, _, _, q, info = lrc.lrc_block_norm(b, res, quantize=True, info=ops.flag(), **opt)
    wq, ws, _ = lrc.lrc_quantize_tokens(h)
    assert torch.equal(q[0], wq) and torch.equal(q[1], ws) and int(info.cpu()) == 0
    dr, db, *_ = lrc.lrc_block_norm_backward(dh, ds, s, b, stats, **opt)
    some = slice(0, None, 97)
    few = lambda t: None if t is None else t[some].contiguous()   # noqa: E731
    s2, h2, stats2, _, _ = lrc.lrc_block_norm(few(b), few(res), **opt)
    for p, w in zip((s, h, *stats), (s2, h2, *stats2)):
        assert p is w is None or torch.equal(few(p), w)
    dr2, db2, *_ = lrc.lrc_block_norm_backward(few(dh), few(ds), s2, few(b), stats2, **opt)
    assert torch.equal(few(dr), dr2) and torch.equal(few(db), db2)
    p2, s2, _ = lrc.lrc_quantize_tokens(few(h))
    assert torch.equal(few(wq), p2) and torch.equal(few(ws), s2)
    # and all the others: every token again in the opposite order, where it meets another workgroup
    flip = lambda t: t.flip(0).contiguous()   # noqa: E731
    s2, h2, _, _, _ = lrc.lrc_block_norm(flip(b), flip(res), **opt)
    assert torch.equal(s2, flip(s)) and torch.equal(h2, flip(h))
    dr2, db2, *_ = lrc.lrc_block_norm_backward(flip(dh), flip(ds), flip(s), flip(b),
                                               tuple(None if t is None else flip(t) for t in stats), **opt)
    assert torch.equal(dr2, flip(dr)) and torch.equal(db2, flip(db))


@pytest.mark.parametrize("n,d", LONG)
@pytest.mark.parametrize("kind", ops.KINDS)
def test_block_norm_many_tokens_sums(lrc, n, d, kind):
    """The parameters' gradients over many workgroups, each with several tokens, fp32, from the call's own total
    gradient.  Sums of n terms (n + 12) u, and three roundings a term."""
    b, res, post, gate, pre = ops.norm_inputs(n, d, torch.float32, kind, n + d)
    b, res, dh, ds = ops.on(b, res, stream(n, d, torch.float32, 7, 0.01), stream(n, d, torch.float32, 8, 0.01))
    post, pre, gate = tuple(ops.on(*post)), tuple(ops.on(*pre)), gate.to(dev())
    opt = dict(kind=kind, post=post, gate=gate, scale=0.75, pre=pre)
    s, _, stats, _, _ = lrc.lrc_block_norm(b, res, **opt)
    t, _, dgamma, dbeta, dpost_gamma, dpost_beta, dgate = lrc.lrc_block_norm_backward(dh, ds, s, b, stats, **opt)
    mb, rb, ms, rs = (torch.zeros(n, device=dev()) if v is None else v for v in stats)
    hat = lambda v, m, r: (v.double() - m.double()[:, None]) * r.double()[:, None]   # noqa: E731
    # normalised values, two roundings of a difference whose terms may be larger than it, one of the product
    size = lambda v, m, r: (v.double().abs() + m.double().abs()[:, None]) * r.double()[:, None]   # noqa: E731
    w = (0.75 * gate).double()
    cases = [(dgamma, dh.double() * hat(s, ms, rs), dh.double().abs() * size(s, ms, rs), 1.0)]
    C = t.double() * hat(b, mb, rb), t.double().abs() * size(b, mb, rb)
    cases.append((dpost_gamma, *C, w))
    along = post[0].double() * C[0]
    if kind == "layer":
        cases += [(dbeta, dh.double(), dh.double().abs(), 1.0), (dpost_beta, t.double(), t.double().abs(), w)]
        along = along + post[1].double() * t.double()
    cases.append((dgate, along, post[0].double().abs() * C[1]
                  + (post[1].double().abs() * t.double().abs() if kind == "layer" else 0), torch.tensor(0.75).double()))
    for got, terms, sizes, scale in cases:
        want = terms.sum(0) * scale
        bound = ((n + 12) * terms.abs().sum(0) + 4 * sizes.sum(0)) * ops.U * abs(scale) + 4 * ops.U * want.abs() + ops.TINY
        assert ((got.double() - want).abs() <= bound).all()


def test_gated_backward_does_not_copy_weights_it_does_not_read(lrc):
    """Without dx the two weights only say how many input channels there are, whatever their pitches."""
    n, d_in, d_ff = 8, 4096, 8192
    bf = dict(dtype=torch.bfloat16, device=dev())
    wg, wu = torch.ones(d_ff, d_in, **bf), torch.ones(d_ff, d_in + 8, **bf)[:, :d_in]
    dh, g, u, x = (torch.ones(n, d, **bf) for d in (d_ff, d_ff, d_ff, d_in))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    dg, du, dx, dwg, _ = lrc.lrc_gated_linear_backward(dh, x, wg, wu, g, u, act="none", need_dx=False, need_dw=False)
    assert dx is None and dwg is None and (dg == 1).all() and (du == 1).all()
    assert torch.cuda.max_memory_allocated() - before < wu.numel()      # half of what a copy of one takes
