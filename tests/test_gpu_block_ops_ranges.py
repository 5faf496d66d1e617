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
