"""Layer norm, linear layer and 8-bit checkpoints on the GPU: values at the ends of their range, entries that meet
only zeros, operands past 2^31 elements, and the bits of one output with and without the others.

Tolerances.  u = 2^-24.  A fp32 sum of K terms is off by at most (K + 8) 2 u times the sum of the terms'
magnitudes, the adds inside a matrix instruction counted as two roundings each.
"""
import math

import numpy as np
import pytest
import torch

from oracle import train_oracle as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16_LOWEST = float(torch.finfo(torch.bfloat16).min)


@pytest.fixture(scope="module")
def lrc():
    import curvature_aware_rank_amd as m
    return m


def dev():
    return torch.device("cuda:0")


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device=dev()) * scale)


# ----------------------------------------------------------------------------- one output without the others
@pytest.mark.parametrize("n,d_in,d_out", [(6912, 1080, 1984), (3000, 260, 514), (512, 4096, 4096), (1024, 2048, 4096)])
@pytest.mark.parametrize("held", [False, True])
def test_fp32_gradients_alone_have_the_bits_of_the_joint_call(lrc, n, d_in, d_out, held):
    """The kernels of an fp32 backward pass go by the sizes, not by which gradients are asked for."""
    x, dy, w = normal(1, n, d_in), normal(2, n, d_out), normal(3, d_out, d_in, scale=1 / math.sqrt(d_in))
    z = normal(4, n, d_out)
    xa, za = (lrc.lrc_pack_activations(t)[:2] if held else t for t in (x, z))
    for act in ("none", "silu"):
        joint = lrc.lrc_linear_backward(dy, xa, w, act=act, z=za)
        for need in (("need_dx",), ("need_dw",), ("need_db",), ("need_dx", "need_db"), ("need_dw", "need_db")):
            some = lrc.lrc_linear_backward(dy, xa, w, act=act, z=za, **{k: False for k in need})
            for name, p, q in zip(("dz", "dx", "dw", "db"), some, joint):
                assert (p is None) == (f"need_{name}" in need)
                assert p is None or torch.equal(p, q), (act, need, name)
