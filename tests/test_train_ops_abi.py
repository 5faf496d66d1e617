"""Layer norm, linear and checkpoint entry points without a GPU: bad arguments are refused on the host before any
HIP call, and the fp64 definitions the GPU tests compare with are pinned."""
import ctypes
import os

import numpy as np
import pytest

from oracle import train_oracle as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "curvature_aware_rank_amd", "liblrc.so")
needs_lib = pytest.mark.skipif(not os.path.exists(LIB), reason="liblrc.so not built")

EINVAL, EDTYPE, EWORKSPACE = 1, 2, 3
P = ctypes.c_void_p(0x1000)   # never dereferenced: validation returns first


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
def test_pack_validation(lib):
    # x, dt, n, d, ldx, codes, exps, info, stream
    call = caller(lib.lrc_pack_activations, [P, 1, 4, 64, 64, P, P, None, None])
    assert call(a1=2) == EDTYPE and call(a2=-1) == EINVAL and call(a2=1 << 31) == EINVAL
    assert call(a3=0) == EINVAL and call(a3=(1 << 24) + 1, a4=1 << 25) == EINVAL and call(a4=63) == EINVAL
    assert call(a0=None) == EINVAL and call(a5=None) == EINVAL and call(a6=None) == EINVAL
    assert call(a2=0, a0=None, a5=None, a6=None) == 0
    # codes, exps, n, d, x, dt, ldx, stream
    call = caller(lib.lrc_unpack_activations, [P, P, 4, 64, P, 1, 64, None])
    assert call(a5=7) == EDTYPE and call(a6=63) == EINVAL and call(a0=None) == EINVAL and call(a1=None) == EINVAL
    assert call(a4=None) == EINVAL and call(a2=-5) == EINVAL and call(a3=0) == EINVAL and call(a2=0) == 0


@needs_lib
def test_layer_norm_validation(lib):
    # x, dt, n, d, ldx, gamma, beta, eps, y, ldy, mean, rstd, codes, exps, info, stream
    call = caller(lib.lrc_layer_norm, [P, 1, 4, 64, 64, None, None, 1e-5, P, 64, P, P, None, None, None, None])
    assert call(a1=3) == EDTYPE and call(a4=63) == EINVAL and call(a9=63) == EINVAL and call(a3=0) == EINVAL
    assert call(a7=-1e-5) == EINVAL and call(a7=float("nan")) == EINVAL
    assert call(a12=P) == EINVAL and call(a13=P) == EINVAL           # half a checkpoint
    for k in (0, 8, 10, 11):
        assert call(**{f"a{k}": None}) == EINVAL
    assert call(a2=0, a0=None, a8=None) == 0 and call(a2=1 << 31) == EINVAL


@needs_lib
def test_layer_norm_backward_validation(lib):
    # dy, dt, n, d, lddy, x, ldx, codes, exps, mean, rstd, gamma, dx, lddx, dgamma, dbeta, ws, ws_bytes, stream
    ws = lib.lrc_layer_norm_backward_workspace(4, 64)
    assert ws > 0 and lib.lrc_layer_norm_backward_workspace(4, 0) == 0
    call = caller(lib.lrc_layer_norm_backward,
                  [P, 1, 4, 64, 64, P, 64, None, None, P, P, None, P, 64, P, P, P, ws, None])
    assert call(a1=9) == EDTYPE and call(a4=63) == EINVAL and call(a6=63) == EINVAL and call(a13=63) == EINVAL
    assert call(a0=None) == EINVAL and call(a9=None) == EINVAL and call(a10=None) == EINVAL
    assert call(a5=None) == EINVAL and call(a5=None, a7=P) == EINVAL and call(a5=None, a8=P) == EINVAL
    assert call(a17=ws - 1) == EWORKSPACE and call(a16=None) == EWORKSPACE


@needs_lib
def test_linear_validation(lib):
    # x, dt, n, di, do, ldx, W, ldw, bias, act, res, ldr, y, ldy, z, ldz, zcodes, zexps, info, ws, ws_bytes, stream
    call = caller(lib.lrc_linear, [P, 1, 4, 64, 32, 64, P, 64, None, 0, None, 0, P, 32, None, 0, None, None, None, P,
                                   1 << 40, None])
    assert call(a1=5) == EDTYPE and call(a9=4) == EDTYPE and call(a9=-1) == EDTYPE
    for k, v in ((3, 0), (4, 0), (5, 63), (7, 63), (13, 31), (2, -1), (2, 1 << 31)):
        assert call(**{f"a{k}": v}) == EINVAL
    assert call(a3=(1 << 24) + 1, a5=1 << 25, a7=1 << 25) == EINVAL
    assert call(a10=P, a11=31) == EINVAL and call(a14=P, a15=31) == EINVAL
    assert call(a16=P) == EINVAL and call(a17=P) == EINVAL and call(a14=P, a15=32, a16=P, a17=P) == EINVAL
    for k in (0, 6, 12):
        assert call(**{f"a{k}": None}) == EINVAL
    assert call(a2=0, a0=None, a12=None) == 0
    need = lib.lrc_linear_workspace(1, 300, 4096, 512)
    if need:
        assert call(a2=300, a3=4096, a5=4096, a7=4096, a4=512, a13=512, a20=need - 1) == EWORKSPACE


@needs_lib
def test_linear_backward_validation(lib):
    # 0 dy, dt, n, di, do, 5 lddy, W, ldw, 8 x, ldx, xcodes, xexps, 12 act, z, ldz, zcodes, zexps, 17 dz, lddz, 19 dx,
    # lddx, 21 dW, dw_dt, lddw, 24 db, ws, ws_bytes, stream
    ws = lib.lrc_linear_backward_workspace(1, 4, 64, 32)
    assert ws > 0
    call = caller(lib.lrc_linear_backward,
                  [P, 1, 4, 64, 32, 32, P, 64, P, 64, None, None, 2, P, 32, None, None, P, 32, P, 64, P, 1, 64, P, P,
                   1 << 40, None])
    assert call(a1=5) == EDTYPE and call(a12=7) == EDTYPE and call(a22=2) == EDTYPE
    assert call(a1=0, a22=1) == EDTYPE                      # a bf16 dW of fp32 streams
    for k, v in ((3, 0), (4, 0), (5, 31), (7, 63), (9, 63), (14, 31), (18, 31), (20, 63), (23, 63), (2, -1)):
        assert call(**{f"a{k}": v}) == EINVAL, k
    for k in (0, 6, 8, 13, 17):
        assert call(**{f"a{k}": None}) == EINVAL, k
    assert call(a8=None, a10=P) == EINVAL and call(a13=None, a15=P) == EINVAL
    assert call(a26=ws - 1) == EWORKSPACE and call(a25=None) == EWORKSPACE


def test_definitions():
    """Checkpoint: what is held is within half a step and the step is the smallest that holds the block.  Gradients:
    against central differences."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 150)) * np.exp(2 * rng.standard_normal((20, 1)))
    codes, exps = ref.pack(x)
    held = ref.unpack(codes, exps)
    step = np.repeat(2.0 ** exps.astype(float), 64, 1)[:, :150]
    assert (np.abs(held - x) <= step / 2).all() and np.abs(codes.astype(int)).max() <= 127
    for b in range(3):
        assert (np.abs(x[:, 64 * b:64 * b + 64]).max(1) > 63.5 * 2.0 ** exps[:, b].astype(float)).all()
    again = ref.pack(held)
    assert np.array_equal(ref.unpack(*again), held)
    h = 1e-6
    z = np.linspace(-4, 4, 40) + 0.03
    for name in ("relu", "gelu", "silu"):
        diff = (ref.act(z + h, name) - ref.act(z - h, name)) / (2 * h)
        assert np.allclose(diff, ref.act_slope(z, name), atol=1e-8)
    x, dy, w = rng.standard_normal((3, 9)), rng.standard_normal((3, 9)), rng.standard_normal((9, 9))
    gamma = rng.standard_normal(9)
    _, mean, rstd = ref.layer_norm(x, gamma, 0.0, 1e-5)
    dx, dgamma, dbeta = ref.layer_norm_backward(dy, x, mean, rstd, gamma)
    e = np.zeros_like(x)
    e[1, 4] = h
    f = lambda v: (ref.layer_norm(v, gamma, 0.0, 1e-5)[0] * dy).sum()   # noqa: E731
    assert abs((f(x + e) - f(x - e)) / (2 * h) - dx[1, 4]) < 1e-7
    assert np.allclose(dgamma, (dy * (x - mean[:, None]) * rstd[:, None]).sum(0)) and np.allclose(dbeta, dy.sum(0))
    _, z = ref.linear(x, w, 0.0, "gelu", 0.0)
    dz, dxl, dw, db = ref.linear_backward(dy, x, w, "gelu", z)
    f = lambda v, m: (ref.linear(v, m, 0.0, "gelu", 0.0)[0] * dy).sum()   # noqa: E731
    assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dxl[1, 4]) < 1e-6
    e9 = np.zeros_like(w)
    e9[2, 7] = h
    assert abs((f(x, w + e9) - f(x, w - e9)) / (2 * h) - dw[2, 7]) < 1e-6


@needs_lib
def test_workspace_queries_over_the_range(lib):
    """Every size the entry points take has a workspace size, no tokens and the largest extents among them."""
    sizes = [1, 2, 63, 64, 65, 300, 1000, 4096, 4097, 11008, 1 << 20, 1 << 24]
    for dt in (0, 1):
        for n in [0, *sizes, (1 << 31) - 1]:
            for d_in in sizes:
                for d_out in (1, 64, 303, 4096, 1 << 24):
                    for f in (lib.lrc_linear_workspace, lib.lrc_linear_backward_workspace):
                        f(dt, n, d_in, d_out)
        for n in (0, 1, 5000, (1 << 31) - 1):
            for d in sizes:
                lib.lrc_layer_norm_backward_workspace(n, d)
        # a layer's scratch stays near its operands' size
        n, d_in, d_out = 8192, 4096, 11008
        assert lib.lrc_linear_workspace(1, n, d_in, d_out) < 1 << 20
        assert lib.lrc_linear_backward_workspace(1, n, d_in, d_out) < 2 * (2 * n * (d_in + d_out)) + (64 << 20)
        assert lib.lrc_linear_workspace(dt, n, d_in, 0) == lib.lrc_linear_workspace(dt, -1, d_in, d_out) == 0
