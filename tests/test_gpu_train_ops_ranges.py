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


# ----------------------------------------------------------------------------- the ends of the range
F32_WAYS = [(100, 300, 520), (700, 516, 1300), (6912, 1080, 1984)]   # any operand, fp32 tiles, three bf16 pieces


def three_products(lrc, a, b, m, n, k):
    """A B^T of A (m, k) and B (n, k) as y of the forward, dx and dW of the backward pass (sizes as given in each)."""
    y = lrc.lrc_linear(a, b)[0]
    dx = lrc.lrc_linear_backward(a, torch.zeros(m, n, dtype=a.dtype, device=dev()), b.t().contiguous())[1]
    w = torch.zeros(m, n, dtype=a.dtype, device=dev())
    dw = lrc.lrc_linear_backward(a.t().contiguous(), b.t().contiguous(), w)[2]
    return {"y": y, "dx": dx, "dW": dw}


@pytest.mark.parametrize("m,k,n", F32_WAYS)
def test_finite_fp32_entries_whose_product_overflows(lrc, m, k, n):
    """Finite entries near the largest number: an overflow is the infinity that the product's sign says, whatever
    pieces an entry is split in, and every other row is as accurate as before."""
    a, b = normal(1, m, k), normal(2, n, k)
    for i in range(16):   # mantissas whose lower bf16 pieces have either sign
        a[5 + i, 7] = (-1) ** (i // 8) * 2.0 ** 126 * (1 + i % 8 * 2.0 ** -9 + 2.0 ** -18)
    b[:, 7] = 2.0 ** 12
    b[3, 7] = -2.0 ** 12
    want = a.double() @ b.double().T
    bound = (k + 8) * 2 * U * (a.double().abs() @ b.double().abs().T)
    over = want.float().isinf()
    assert over[5:21].all() and int(over.sum()) == 16 * n
    for name, got in three_products(lrc, a, b, m, n, k).items():
        assert torch.equal(got[over], want.float()[over]), name
        assert ((got.double() - want).abs() <= bound)[~over].all(), name


def test_finite_fp32_entries_whose_product_with_a_checkpoint_overflows(lrc):
    """As above with x in 8 bits, whose values are one exact piece."""
    n, d_in, d_out = 6912, 1080, 1984
    x, dy = normal(1, n, d_in), normal(2, n, d_out)
    x[7] = 2.0 ** 120 * torch.where(torch.arange(d_in, device=dev()) % 3 == 0, -1.0, 1.0)
    dy[7] = 2.0 ** -100
    for i in range(16):
        dy[7, 5 + i] = (-1) ** (i // 8) * 2.0 ** 18 * (1 + i % 8 * 2.0 ** -9 + 2.0 ** -18)
    codes, exps, _ = lrc.lrc_pack_activations(x)
    held = lrc.lrc_unpack_activations(codes, exps, torch.float32)
    assert torch.equal(held[7], x[7])
    dw = lrc.lrc_linear_backward(dy, (codes, exps), torch.zeros(d_out, d_in, device=dev()))[2]
    want = dy.double().T.contiguous() @ held.double()
    over = want.float().isinf()
    assert over[5:21].all() and int(over.sum()) == 16 * d_in
    assert torch.equal(dw[over], want.float()[over])
    bound = (n + 8) * 2 * U * (dy.double().abs().T.contiguous() @ held.double().abs())
    assert ((dw.double() - want).abs() <= bound)[~over].all()


def test_an_infinity_moves_only_the_product_it_is_in(lrc):
    """An infinity in x does not change dx, nor one in W dW, at sizes that split fp32 entries: each has the bits of
    the call that asks for it alone."""
    n, d_in, d_out = 6912, 1080, 1984
    x, dy, w = normal(1, n, d_in), normal(2, n, d_out), normal(3, d_out, d_in)
    clean = lrc.lrc_linear_backward(dy, x, w)
    for where in ("x", "w"):
        t = {"x": x.clone(), "w": w.clone()}
        t[where][5, 7] = float("inf")
        joint = lrc.lrc_linear_backward(dy, t["x"], t["w"])
        kept = 1 if where == "x" else 2
        assert torch.equal(joint[kept], clean[kept]), where
        alone = lrc.lrc_linear_backward(dy, t["x"], t["w"], **{"need_dw" if where == "x" else "need_dx": False})
        assert torch.equal(alone[kept], clean[kept]), where
        other = joint[3 - kept]      # dW has an infinite column, dx one
        assert not other[:, 7].isfinite().any() and other[:, :7].isfinite().all() and other[:, 8:].isfinite().all()


# ----------------------------------------------------------------------------- entries that meet only zeros
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("n,d_in,d_out", [(5, 17, 9), (300, 136, 264), (1000, 521, 303), (2500, 1032, 2056)])
@pytest.mark.parametrize("held", [False, True])
def test_weight_gradient_with_values_in_masked_tokens(lrc, act, n, d_in, d_out, held):
    """Tokens that count for nothing hold large values on one side and zeros on the other: the type's lowest value in
    x where dy is zero, 1e30 in dy where x is zero, and 1e30 in single entries that meet a zero channel of x.  dW is
    as accurate as without them: to 2^-11 of its terms' magnitudes, element by element."""
    x, dy, z = normal(1, n, d_in).bfloat16(), normal(2, n, d_out).bfloat16(), normal(3, n, d_out).bfloat16()
    dy[1], x[1] = 0, BF16_LOWEST
    x[3], dy[3] = 0, 1e30
    if n > 100:
        dy[70::64], x[70::64] = 0, -BF16_LOWEST
        x[101::64], dy[101::64] = 0, -1e30
        x[:-20, 5:9], dy[:-20, 3] = 0, 1e30     # channels of x that only the last tokens feed
    w = torch.zeros(d_out, d_in, dtype=torch.bfloat16, device=dev())
    xa, xn = x, f64(x)
    if held:
        xa = lrc.lrc_pack_activations(x)[:2]
        xn = ref.unpack(xa[0].cpu().numpy(), xa[1].cpu().numpy())
    _, _, dw, _ = lrc.lrc_linear_backward(dy, xa, w, act=act, z=z, dw_dtype=torch.float32)
    dz = f64(dy) * ref.act_slope(f64(z), act)
    terms, got = np.abs(dz).T @ np.abs(xn), f64(dw)
    beyond = terms > 1e60      # 1e30 meets the lowest value: 3e68, which no fp32 number is near
    assert not beyond[:3].any() and not beyond[4:].any() and not np.isfinite(got[beyond]).any()
    assert (np.abs(got - dz.T @ xn) <= 2.0 ** -11 * terms)[~beyond].all()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_weight_gradient_with_an_infinite_activation(lrc, act):
    """An infinity or NaN in x gives its channel of dW what arithmetic gives, whatever the sign of dz's lower bits, and
    leaves the other channels' bits as they are."""
    n, d_in, d_out = 700, 264, 392
    x, dy, z = normal(1, n, d_in).bfloat16(), normal(2, n, d_out).bfloat16(), normal(3, n, d_out).bfloat16()
    w = torch.zeros(d_out, d_in, dtype=torch.bfloat16, device=dev())
    clean = lrc.lrc_linear_backward(dy, x, w, act=act, z=z)[2]
    bad = x.clone()
    bad[6, 40], bad[9, 41], bad[12, 42] = float("inf"), float("-inf"), float("nan")
    dw = lrc.lrc_linear_backward(dy, bad, w, act=act, z=z)[2]
    dz = torch.from_numpy(f64(dy) * ref.act_slope(f64(z), act)).to(dev())
    want = dz.T.contiguous()[:, [6, 9, 12]].sign() * torch.tensor([math.inf, -math.inf, math.nan], device=dev())
    assert torch.equal(torch.nan_to_num(dw[:, 40:43].double(), 9e9, 8e8, 7e7), torch.nan_to_num(want, 9e9, 8e8, 7e7))
    keep = [c for c in range(d_in) if not 40 <= c < 43]
    assert torch.equal(dw[:, keep], clean[:, keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [2, 65, 512, 1000, 2048, 4096, 11008, 16384, 20000])
def test_layer_norm_of_tokens_of_the_lowest_value(lrc, dtype, d):
    """Tokens that a mask filled with the type's lowest (or largest) value: their mean is that value, not an infinity,
    y is beta, the checkpoint is that of the tokens, and in the backward pass a dy of zeros there leaves the gradients'
    sums as they are without those tokens."""
    n = 12
    x, dy = normal(1, n, d).to(dtype), normal(2, n, d).to(dtype)
    gamma, beta = 1 + 0.1 * normal(3, d), normal(4, d)
    low = float(torch.finfo(dtype).min)
    x[3], x[7] = low, -low
    dy[3], dy[7] = 0, 0
    y, mean, rstd, kept, info = lrc.lrc_layer_norm(x, gamma, beta, checkpoint=True)
    assert torch.equal(y[[3, 7]], beta.to(dtype).expand(2, d)) and int(info.cpu()) == 0
    # a sum of d terms over per-thread runs and a tree (at most d / 64 + 24 deep), and 1 / d to half a step
    off = (mean[[3, 7]].double() - torch.tensor([low, -low], device=dev(), dtype=torch.float64)).abs() / -low
    assert (off <= (d / 64 + 26) * U).all() and rstd.isfinite().all()
    dx, dgamma, dbeta = lrc.lrc_layer_norm_backward(dy, x, mean, rstd, gamma)
    assert not dx[[3, 7]].any()
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    rows = [t for t in range(n) if t not in (3, 7)]
    want, terms = (dy.double() * xh)[rows].sum(0), (dy.double() * xh).abs()[rows].sum(0)
    # the sum, and xh's two roundings around the centred value
    slack = ((x.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None] * dy.double().abs())[rows].sum(0)
    assert ((dgamma.double() - want).abs() <= (n + 8) * U * terms + 2 * U * slack).all()
    assert ((dbeta.double() - dy.double().sum(0)).abs() <= (n + 8) * U * dy.double().abs().sum(0)).all()


# ----------------------------------------------------------------------------- alignment
@pytest.mark.parametrize("n,d_in,d_out", [(4200, 4096, 64), (4200, 64, 4096), (16400, 2048, 40)])
def test_large_products_of_a_narrow_unaligned_weight(lrc, n, d_in, d_out):
    """W of at most 64 rows, or columns, that start on no 16 bytes (a slice of a larger factor): the bits of an
    aligned W."""
    x, dy = normal(1, n, d_in).bfloat16(), normal(2, n, d_out).bfloat16()
    w = normal(3, d_out, d_in).bfloat16()
    far = torch.zeros(d_out, d_in + 8, dtype=torch.bfloat16, device=dev())[:, 3:3 + d_in]
    far.copy_(w)
    assert far.data_ptr() % 16 and torch.equal(lrc.lrc_linear(x, far, save="z")[1], lrc.lrc_linear(x, w, save="z")[1])
    for a, b in zip(lrc.lrc_linear_backward(dy, x, far), lrc.lrc_linear_backward(dy, x, w)):
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------- borders
def test_pack_at_the_borders_of_the_exponent(lrc):
    """Blocks whose largest magnitude lies one step below, at and one step above 127 * 2^e, over the whole range of e
    (the highest ones, and those from 127 * 2^114 on, among them), with ties below them: bit-exact."""
    rows = []
    for e in [-126, -125, -1, 0, 1, 60, 113, 114, 115, 119, 120, 121]:
        top = np.float32(127.0) * np.float32(2.0) ** e
        for big in (np.nextafter(top, np.float32(0)), top, np.nextafter(top, np.float32(np.inf))):
            rows.append([big, -big, top * 0.5, top * np.float32(2.5 / 127), -top * np.float32(63.5 / 127), 0.0])
    x = torch.from_numpy(np.array(rows, np.float32))
    codes, exps, info = lrc.lrc_pack_activations(x.to(dev()))
    qc, qe = ref.pack(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), qc) and np.array_equal(exps.cpu().numpy(), qe)
    assert int(info.cpu()) == 0


def relative_tail(x, name):
    """Bound of act(x) in fp32 relative to itself.  The exponential's argument goes through two roundings and a rounded
    constant, 3 u of itself for GELU (x^2 / 2) and 2 u for SiLU (x), which is the relative error of the exponential;
    the fit's error (5e-7) and ten more roundings, of two steps each where an instruction is good to one step."""
    return (1.5 * x * x if name == "gelu" else 2 * np.abs(x)) * U + 5e-7 + 20 * U


@pytest.mark.parametrize("name,low", [("gelu", -12.0), ("silu", -80.0)])
def test_activations_of_negative_tails(lrc, name, low):
    """act(z) of z down to where it is 1e-32: accurate relative to itself, not to z."""
    x = torch.linspace(low, 0, 20001, dtype=torch.float32)[:, None]
    y = lrc.lrc_linear(x.to(dev()), torch.ones(1, 1, device=dev()), act=name)[0]
    want = ref.act(f64(x), name)
    assert (np.abs(f64(y) - want) <= relative_tail(f64(x), name) * np.abs(want)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_operands_past_2_to_31_elements(lrc, dtype):
    """More than 2^31 elements in x and dx, on the pipelined tiles: small integers, exact in any order."""
    n, d_in, d_out = 524416, 4104, 72
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g, device=dev(), dtype=torch.int8).to(dtype)   # noqa: E731
    x, w, dy = ints(n, d_in), ints(d_out, d_in), ints(n, d_out)
    assert x.numel() > 1 << 31
    y = lrc.lrc_linear(x, w)[0]
    _, dx, dw, _ = lrc.lrc_linear_backward(dy, x, w, dw_dtype=torch.float32)
    total = torch.zeros(d_out, d_in, dtype=torch.float64, device=dev())
    for a in range(0, n, 65536):
        xs, ds = x[a:a + 65536].double(), dy[a:a + 65536].double()
        assert torch.equal(y[a:a + 65536], (xs @ w.double().T).to(dtype)), a
        assert torch.equal(dx[a:a + 65536], (ds @ w.double()).to(dtype)), a
        total += ds.T.contiguous() @ xs
    assert torch.equal(dw.double(), total)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d_in,d_out", [(24, 11008, 4096), (1000, 1024, 1024), (4096, 4096, 4104), (3900, 1100, 2500)])
def test_equal_inputs_give_equal_bits_on_every_tile(lrc, dtype, n, d_in, d_out):
    """Calls again and again on the same inputs, at sizes of one and several rounds of tiles and of split k."""
    x, dy, z = normal(1, n, d_in).to(dtype), normal(2, n, d_out).to(dtype), normal(3, n, d_out).to(dtype)
    w = normal(4, d_out, d_in, scale=1 / math.sqrt(d_in)).to(dtype)

    def call():
        y, (codes, exps), _ = lrc.lrc_linear(x, w, act="gelu", residual=dy, save="checkpoint")
        return (y, codes, exps, *lrc.lrc_linear_backward(dy, x, w, act="silu", z=z))

    first = call()
    for _ in range(6):
        for a, b in zip(call(), first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("n,d_in,d_out", [(37, 72, 104), (300, 264, 520), (300, 265, 521)])
def test_weight_gradient_beside_a_dz_of_any_pitch(lrc, act, n, d_in, d_out):
    """Through the C interface: dz rows of an odd pitch and start, dW with a gap behind its rows.  dW is as accurate as
    with rows of whole pieces, and what lies between the rows is left as it was."""
    x, dy, z = normal(1, n, d_in).bfloat16(), normal(2, n, d_out).bfloat16(), normal(3, n, d_out).bfloat16()
    w = normal(4, d_out, d_in).bfloat16()
    lddz, lddw = d_out + 3, d_in + 5
    dz = torch.full((n * lddz + 1,), 7.0, dtype=torch.bfloat16, device=dev())
    dw = torch.full((d_out, lddw), 7.0, device=dev())
    dx = torch.empty(n, d_in, dtype=torch.bfloat16, device=dev())
    size = lrc.lib.lrc_linear_backward_workspace(lrc.LRC_BF16, n, d_in, d_out)
    ws = torch.empty(size, dtype=torch.uint8, device=dev())
    assert lrc.lib.lrc_linear_backward(
        dy.data_ptr(), lrc.LRC_BF16, n, d_in, d_out, d_out, w.data_ptr(), d_in, x.data_ptr(), d_in, None, None,
        {"gelu": 2, "silu": 3}[act], z.data_ptr(), d_out, None, None, dz.data_ptr() + 2, lddz, dx.data_ptr(), d_in,
        dw.data_ptr(), lrc.LRC_F32, lddw, None, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream) == 0
    got = dz[1:].view(n, lddz)
    assert (got[:, d_out:] == 7).all() and (dz[0] == 7) and (dw[:, d_in:] == 7).all()
    want = lrc.lrc_linear_backward(dy, x, w, act=act, z=z, dw_dtype=torch.float32)
    assert torch.equal(got[:, :d_out], want[0])
    dzn = f64(dy) * ref.act_slope(f64(z), act)
    terms = np.abs(dzn).T @ np.abs(f64(x))
    for t in (dw[:, :d_in], want[2]):
        assert (np.abs(f64(t) - dzn.T @ f64(x)) <= 2.0 ** -11 * terms).all()
    # a product of the stream: dz to half a bf16 step, the sum in fp32, dx to half a step
    mags = np.abs(dzn) @ np.abs(f64(w))
    for t in (dx, want[1]):
        assert (np.abs(f64(t) - dzn @ f64(w)) <= 1.01 * (2.0 ** -8 * mags + 2.0 ** -8 * np.abs(dzn @ f64(w)))).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,h", [(96, 160), (512, 264), (4096, 96), (20000, 40)])
@pytest.mark.parametrize("held", [False, True])
def test_step_with_tokens_of_the_lowest_value(lrc, dtype, d, h, held):
    """norm -> linear (GELU) and back where a mask filled tokens of x with the lowest value: the norm sends them to beta
    as it does zeros, dy is zero there, and every output is that of a step whose masked tokens hold zeros."""
    n = 75
    x, dy = normal(1, n, d).to(dtype), normal(2, n, h, scale=0.01).to(dtype)
    w, b = normal(3, h, d, scale=1 / math.sqrt(d)).to(dtype), normal(4, h)
    gamma, beta = 1 + 0.1 * normal(5, d), normal(6, d)
    masked = torch.arange(n, device=dev()) % 9 == 4
    dy[masked] = 0
    got = []
    for fill in (torch.finfo(dtype).min, 0.0):
        x[masked] = fill
        a, mean, rstd, xk, _ = lrc.lrc_layer_norm(x, gamma, beta, checkpoint=True)
        y, zk, _ = lrc.lrc_linear(a, w, b, act="gelu", save="checkpoint" if held else "z")
        dz, da, dw, db = lrc.lrc_linear_backward(dy, lrc.lrc_pack_activations(a)[:2] if held else a, w, act="gelu", z=zk)
        dx, dgamma, dbeta = lrc.lrc_layer_norm_backward(da, xk if held else x, mean, rstd, gamma)
        got.append({"a": a, "y": y, "dz": dz, "da": da, "dw": dw, "db": db, "dgamma": dgamma, "dbeta": dbeta, "dx": dx})
    for k, t in got[0].items():
        assert torch.isfinite(t).all() and torch.equal(t, got[1][k]), k


def test_fp32_rows_beside_a_row_that_is_not_finite(lrc):
    """A token with a NaN at a size that splits fp32 entries: the other tokens as accurate as without it."""
    n, d_in, d_out = 6912, 1080, 1984
    x, w = normal(1, n, d_in), normal(2, d_out, d_in)
    x[5, 7] = float("nan")
    y = lrc.lrc_linear(x, w)[0]
    rows = [t for t in range(n) if t != 5]
    bound = (d_in + 8) * 2 * U * (x[rows].double().abs() @ w.double().abs().T)
    assert y[5].isnan().all() and ((y[rows].double() - x[rows].double() @ w.double().T).abs() <= bound).all()
