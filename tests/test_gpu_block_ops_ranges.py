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
