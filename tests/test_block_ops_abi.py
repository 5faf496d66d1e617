"""Gated block, 8-bit products and norms around a block without a GPU: bad arguments are refused on the host before any
HIP call, workspace queries answer over the range, and the fp64 definitions the GPU tests compare with are pinned."""
import ctypes
import os

import numpy as np
import pytest

from oracle import block_oracle as ref
from oracle import train_oracle as base

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "curvature_aware_rank_amd", "liblrc.so")
needs_lib = pytest.mark.skipif(not os.path.exists(LIB), reason="liblrc.so not built")

EINVAL, EDTYPE, EWORKSPACE = 1, 2, 3
P = ctypes.c_void_p(0x1000)     # never dereferenced: validation returns first
ODD = ctypes.c_void_p(0x1002)   # starts on no 16 bytes


@pytest.fixture(scope="module")
def lib():
    import curvature_aware_rank_amd as m
    return m.lib


def caller(f, ok):
    def call(**over):
        a = list(ok)
        for i, v in over.items():
            a[int(i[1:])] = v
        return f(*a)
    return call


@needs_lib
def test_quantize_tokens_validation(lib):
    # x, dt, n, d, ldx, q, ldq, scale, info, stream
    call = caller(lib.lrc_quantize_tokens, [P, 1, 4, 64, 64, P, 64, P, None, None])
    assert call(a1=2) == EDTYPE and call(a2=-1) == EINVAL and call(a2=1 << 31) == EINVAL and call(a3=0) == EINVAL
    assert call(a4=63) == EINVAL and call(a6=63) == EINVAL and call(a3=(1 << 24) + 1, a4=1 << 25, a6=1 << 25) == EINVAL
    for k in (0, 5, 7):
        assert call(**{f"a{k}": None}) == EINVAL
    assert call(a2=0, a0=None, a5=None, a7=None) == 0


@needs_lib
def test_int8_linear_validation(lib):
    # 0 x, dt, n, di, do, 5 ldx, xcodes, ldxc, xscale, 9 W, ldw, wscale, 12 bias, act, 14 res, ldr, 16 y, ldy, info,
    # 19 ws, ws_bytes, stream
    call = caller(lib.lrc_int8_linear, [P, 1, 40, 64, 32, 64, None, 0, None, P, 64, P, None, 0, None, 0, P, 32, None, P,
                                        1 << 40, None])
    assert call(a1=5) == EDTYPE and call(a13=4) == EDTYPE and call(a13=-1) == EDTYPE
    for k, v in ((3, 0), (4, 0), (5, 63), (10, 63), (17, 31), (2, -1), (2, 1 << 31)):
        assert call(**{f"a{k}": v}) == EINVAL, k
    assert call(a3=1 << 17, a5=1 << 17, a10=1 << 17) == EINVAL
    assert call(a14=P, a15=31) == EINVAL
    for k in (0, 9, 11, 16):
        assert call(**{f"a{k}": None}) == EINVAL, k
    # tokens given twice, or half a pair
    assert call(a6=P, a7=64, a8=P) == EINVAL and call(a0=None, a6=P, a7=64) == EINVAL and call(a0=None, a8=P) == EINVAL
    assert call(a0=None, a6=P, a7=63, a8=P) == EINVAL
    # codes that the products cannot read where they lie
    assert call(a9=ODD) == EINVAL and call(a10=72) == EINVAL and call(a10=(1 << 22) + 16) == EINVAL
    assert call(a0=None, a6=ODD, a7=64, a8=P) == EINVAL
    assert call(a2=0, a0=None, a16=None) == 0
    need = lib.lrc_int8_linear_workspace(40, 64, 32)
    assert need > 0 and call(a20=need - 1) == EWORKSPACE and call(a19=None) == EWORKSPACE
    assert lib.lrc_int8_linear_workspace(40, 1 << 17, 32) == lib.lrc_int8_linear_workspace(40, 64, 0) == 0


@needs_lib
def test_int8_gated_linear_validation(lib):
    # 0 x, dt, n, di, df, 5 ldx, xcodes, ldxc, xscale, 9 Wg, ldwg, gscale, 12 Wu, ldwu, uscale, 15 act, h, ldh, info,
    # 19 ws, ws_bytes, stream
    call = caller(lib.lrc_int8_gated_linear, [P, 0, 40, 64, 32, 64, None, 0, None, P, 64, P, P, 64, P, 3, P, 32, None, P,
                                              1 << 40, None])
    assert call(a1=5) == EDTYPE and call(a15=4) == EDTYPE
    for k, v in ((3, 0), (4, 0), (5, 63), (10, 63), (13, 63), (17, 31), (2, -1)):
        assert call(**{f"a{k}": v}) == EINVAL, k
    for k in (0, 9, 11, 12, 14, 16):
        assert call(**{f"a{k}": None}) == EINVAL, k
    assert call(a12=ODD) == EINVAL and call(a13=72) == EINVAL and call(a2=0, a0=None, a16=None) == 0
    need = lib.lrc_int8_gated_linear_workspace(40, 64, 32)
    assert need > 0 and call(a20=need - 1) == EWORKSPACE and call(a19=None) == EWORKSPACE


@needs_lib
def test_gated_linear_validation(lib):
    # 0 x, dt, n, di, df, 5 ldx, Wg, Wu, ldw, 9 act, h, ldh, 12 g, u, ldz, 15 gcodes, gexps, ucodes, uexps, info, 20 ws,
    # ws_bytes, stream
    call = caller(lib.lrc_gated_linear, [P, 1, 300, 64, 32, 64, P, P, 64, 3, P, 32, None, None, 0, None, None, None, None,
                                         None, P, 1 << 40, None])
    assert call(a1=5) == EDTYPE and call(a9=4) == EDTYPE and call(a9=-1) == EDTYPE
    for k, v in ((3, 0), (4, 0), (5, 63), (8, 63), (11, 31), (2, -1), (2, 1 << 27)):
        assert call(**{f"a{k}": v}) == EINVAL, k
    assert call(a3=(1 << 20) + 8, a5=1 << 21, a8=1 << 21) == EINVAL and call(a4=(1 << 20) + 1, a11=1 << 21) == EINVAL
    assert call(a12=P, a14=32) == EINVAL and call(a13=P, a14=32) == EINVAL and call(a12=P, a13=P, a14=31) == EINVAL
    for k in (15, 16, 17, 18):                                        # a part of a checkpoint
        assert call(**{f"a{k}": P}) == EINVAL, k
    assert call(a12=P, a13=P, a14=32, a15=P, a16=P, a17=P, a18=P) == EINVAL
    for k in (0, 6, 7, 10):
        assert call(**{f"a{k}": None}) == EINVAL, k
    for k in (0, 6, 7):                                               # bf16 rows that could be whole pieces
        assert call(**{f"a{k}": ODD}) == EINVAL, k
    assert call(a5=68) == EINVAL and call(a8=68) == EINVAL and call(a5=(1 << 21) + 8) == EINVAL
    assert call(a2=0, a0=None, a10=None) == 0
    for dt in (0, 1):
        for over in ({}, {"a15": P, "a16": P, "a17": P, "a18": P}):
            need = lib.lrc_gated_linear_workspace(dt, 300, 60, 32)
            assert need > 0 and call(a1=dt, a3=60, a21=need - 1, **over) == EWORKSPACE
            assert call(a1=dt, a3=60, a20=None, **over) == EWORKSPACE


@needs_lib
def test_gated_linear_backward_validation(lib):
    # 0 dh, dt, n, di, df, 5 lddh, Wg, Wu, ldw, 9 x, ldx, xcodes, xexps, 13 act, g, u, ldz, 17 gcodes, gexps, ucodes,
    # uexps, 21 dg, du, dx, lddx, 25 dWg, dWu, dw_dt, lddw, 29 ws, ws_bytes, stream
    call = caller(lib.lrc_gated_linear_backward,
                  [P, 1, 4, 64, 32, 32, P, P, 64, P, 64, None, None, 3, P, P, 32, None, None, None, None, P, P, P, 64, P, P,
                   1, 64, P, 1 << 40, None])
    assert call(a1=5) == EDTYPE and call(a13=7) == EDTYPE and call(a27=2) == EDTYPE and call(a1=0, a27=1) == EDTYPE
    for k, v in ((3, 0), (4, 0), (5, 31), (8, 63), (10, 63), (16, 31), (24, 63), (28, 63), (2, -1), (2, 1 << 27)):
        assert call(**{f"a{k}": v}) == EINVAL, k
    for k in (0, 6, 7, 9, 14, 15, 21, 22, 25, 26):
        assert call(**{f"a{k}": None}) == EINVAL, k
    assert call(a9=None, a11=P) == EINVAL and call(a14=None, a15=None, a17=P, a18=P, a19=P) == EINVAL
    for k in (6, 7, 9, 21, 22):
        assert call(**{f"a{k}": ODD}) == EINVAL, k
    for dt, dw in ((0, 0), (1, 1), (1, 0)):
        need = lib.lrc_gated_linear_backward_workspace(dt, 4, 64, 32)
        assert need > 0 and call(a1=dt, a27=dw, a30=need - 1) == EWORKSPACE
        assert call(a1=dt, a27=dw, a29=None) == EWORKSPACE
    assert call(a2=0, a25=None, a26=None, a0=None) == 0


@needs_lib
def test_block_norm_validation(lib):
    # 0 b, dt, n, d, ldb, 5 res, ldr, kind, eps, post, 10 post_gamma, post_beta, gate, scale, 14 gamma, beta, 16 s, lds, h,
    # ldh, 20 mean_b, rstd_b, mean_s, rstd_s, 24 q, ldq, qscale, info, stream
    call = caller(lib.lrc_block_norm, [P, 1, 4, 64, 64, P, 64, 0, 1e-5, 1, P, P, P, 0.5, P, P, P, 64, P, 64, P, P, P, P, P,
                                       64, P, None, None])
    assert call(a1=3) == EDTYPE and call(a7=2) == EDTYPE and call(a7=-1) == EDTYPE
    for k, v in ((3, 0), (3, 16385), (4, 63), (6, 63), (17, 63), (19, 63), (25, 63), (2, -1), (2, 1 << 31)):
        assert call(**{f"a{k}": v}) == EINVAL, k
    assert call(a8=-1e-5) == EINVAL and call(a8=float("nan")) == EINVAL
    assert call(a24=None) == EINVAL and call(a26=None) == EINVAL and call(a9=0) == EINVAL      # post vectors without post
    assert call(a7=1) == EINVAL and call(a7=1, a11=None) == EINVAL                             # a beta of an RMS norm
    assert call(a7=1, a15=None) == EINVAL
    assert call(a0=None) == EINVAL and call(a16=None, a18=None, a24=None, a26=None) == EINVAL
    assert call(a2=0, a0=None) == 0


@needs_lib
def test_block_norm_backward_validation(lib):
    # 0 dh, dt, n, d, lddh, 5 ds, ldds, s, lds, 9 b, ldb, 11 mean_b, rstd_b, mean_s, rstd_s, 15 kind, post, post_gamma,
    # post_beta, gate, 20 scale, gamma, 22 dres, lddr, db, lddb, 26 dgamma, dbeta, dpost_gamma, dpost_beta, dgate, 31 ws,
    # ws_bytes, stream
    ws = lib.lrc_block_norm_backward_workspace(4, 64)
    assert ws > 0 and lib.lrc_block_norm_backward_workspace(4, 16385) == 0
    call = caller(lib.lrc_block_norm_backward,
                  [P, 1, 4, 64, 64, P, 64, P, 64, P, 64, P, P, P, P, 0, 1, P, P, P, 0.5, P, P, 64, P, 64, P, P, P, P, P, P,
                   ws, None])
    assert call(a1=9) == EDTYPE and call(a15=2) == EDTYPE
    for k, v in ((3, 0), (3, 16385), (4, 63), (6, 63), (8, 63), (10, 63), (23, 63), (25, 63), (2, -1)):
        assert call(**{f"a{k}": v}) == EINVAL, k
    for k in (7, 9, 11, 12, 13, 14):                                  # s, b and the statistics
        assert call(**{f"a{k}": None}) == EINVAL, k
    assert call(a0=None) == EINVAL                                    # dgamma without dh
    assert call(a0=None, a5=None, a26=None, a27=None) == EINVAL
    assert call(a16=0) == EINVAL and call(a15=1) == EINVAL            # post without post, betas of an RMS norm
    assert call(a32=ws - 1) == EWORKSPACE and call(a31=None) == EWORKSPACE


@needs_lib
def test_workspace_queries_over_the_range(lib):
    """Every size the entry points take has a workspace size, no tokens and the largest extents among them."""
    sizes = [1, 2, 15, 16, 63, 64, 65, 303, 1000, 4096, 4097, 11008, 1 << 16]
    for n in [0, *sizes, (1 << 27) - 1]:
        for di in sizes:
            for do in (1, 64, 303, 4096, 1 << 20):
                lib.lrc_int8_linear_workspace(n, di, do)
                lib.lrc_int8_gated_linear_workspace(n, di, do)
                for dt in (0, 1):
                    lib.lrc_gated_linear_workspace(dt, n, di, do)
                    lib.lrc_gated_linear_backward_workspace(dt, n, di, do)
    for n in (0, 1, 5000, (1 << 31) - 1):
        for d in [*sizes[:-1], 16384]:
            assert lib.lrc_block_norm_backward_workspace(n, d) <= 1024 * 4 * 16384 * 4
    # scratch stays near the operands' size
    n, di, df = 8192, 4096, 11008
    assert lib.lrc_gated_linear_workspace(1, n, di, df) < 1 << 20
    assert lib.lrc_gated_linear_backward_workspace(1, n, di, df) < 2 * n * (2 * df + di) + (64 << 20)
    assert lib.lrc_int8_linear_workspace(n, di, df) < n * di + (1 << 20)


def test_definitions():
    """The quantiser holds a value to half a step; gradients against central differences of the forward definitions."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((20, 150)) * np.exp(2 * rng.standard_normal((20, 1)))).astype(np.float32)
    q, s = ref.quantize(x)
    assert (np.abs(q * s[:, None].astype(float) - x) <= 0.5001 * s[:, None]).all() and np.abs(q.astype(int)).max() == 127
    w = rng.standard_normal((9, 150)).astype(np.float32)
    p, t = ref.quantize(w)
    y, z = ref.int8_linear(q, s, p, t, 0.5, "relu", 1.0)
    held = (q * s[:, None].astype(float)) @ (p * t[:, None].astype(float)).T
    assert np.allclose(z, held + 0.5) and np.allclose(y, np.maximum(z, 0) + 1)
    h = 1e-6
    x, wg, wu, dh = (rng.standard_normal(v) for v in ((3, 5), (7, 5), (7, 5), (3, 7)))
    for name in ("silu", "gelu", "none"):
        _, g, u = ref.gated(x, wg, wu, name)
        got = ref.gated_backward(dh, x, wg, wu, name, g, u)
        assert np.allclose(got[1], dh * base.act(g, name))
        for k, args in enumerate((x, wg, wu)):
            lo, hi = [v.copy() for v in (x, wg, wu)], [v.copy() for v in (x, wg, wu)]
            lo[k][2, 3] -= h
            hi[k][2, 3] += h
            want = ((ref.gated(*hi, name)[0] - ref.gated(*lo, name)[0]) * dh).sum() / (2 * h)
            assert abs(got[2 + k][2, 3] - want) < 1e-7 * max(1, abs(want)) + 1e-6
    d = 9
    b, r, dh, ds = (rng.standard_normal((4, d)) for _ in range(4))
    vec = [rng.standard_normal(d) for _ in range(5)]
    for kind in ("rms", "layer"):
        def f(b, r, pg, pb, gate, ga, be):
            s, y, _ = ref.block_norm(b, r, kind, 1e-5, (pg, pb), gate, 0.7, ga, be)
            return (s * ds).sum() + (y * dh).sum()
        s, _, st = ref.block_norm(b, r, kind, 1e-5, (vec[0], vec[1]), vec[2], 0.7, vec[3], vec[4])
        t, db, dga, dbe, dpg, dpb, dgate = ref.block_norm_backward(dh, ds, s, b, st, kind, (vec[0], vec[1]), vec[2], 0.7,
                                                                   vec[3])
        args = [b, r, *vec]
        for k, got in enumerate((db, t, dpg, dpb, dgate, dga, dbe)):
            at = (1, 4) if k < 2 else (4,)
            lo, hi = [v.copy() for v in args], [v.copy() for v in args]
            lo[k][at] -= h
            hi[k][at] += h
            assert abs(got[at] - (f(*hi) - f(*lo)) / (2 * h)) < 1e-6 * max(1, abs(got[at])) + 1e-7, (kind, k)
