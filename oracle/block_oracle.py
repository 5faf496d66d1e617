"""Plain fp64 numpy definitions of the gated feed-forward block, the products in 8-bit integers and the norms
around a block.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the library's own path.  Written from
the formulas; it shares no code with the HIP kernels.
"""
import numpy as np

from oracle.train_oracle import act, act_slope


def quantize(x):
    """(codes int8, scale fp32) of rows: scale = fl32(max|x| / 127) over the finite entries, code = the nearest integer
    to fl32(x / scale), ties to even, held to +-127 (NaN: 0; a row whose scale is 0: zeros)."""
    x = np.asarray(x, np.float32)
    scale = np.where(np.isfinite(x), np.abs(x), np.float32(0)).max(1).astype(np.float32) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = np.clip(np.rint(x / scale[:, None]), -127, 127)
    q = np.where((scale[:, None] > 0) & ~np.isnan(x), q, 0)
    return q.astype(np.int8), scale


def int8_linear(xq, xs, wq, ws, bias, name, residual):
    """(y, z) of codes and scales; the integer sum is exact."""
    s = (xq.astype(np.int64) @ wq.astype(np.int64).T).astype(np.float64)
    z = s * ws.astype(np.float64) * xs.astype(np.float64)[:, None] + bias
    return act(z, name) + residual, z


def gated(x, wg, wu, name):
    g, u = x @ wg.T, x @ wu.T
    return act(g, name) * u, g, u


def gated_backward(dh, x, wg, wu, name, g, u):
    dg, du = dh * u * act_slope(g, name), dh * act(g, name)
    return dg, du, dg @ wg + du @ wu, dg.T @ x, du.T @ x


def _moments(x, kind, eps):
    mean = x.mean(1) if kind == "layer" else np.zeros(len(x))
    return mean, 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)


def block_norm(b, residual, kind, eps, post, gate, scale, gamma, beta):
    """post: None or (gamma, beta).  Returns s, h and (mean_b, rstd_b, mean_s, rstd_s)."""
    mean_b = rstd_b = None
    p = b
    if post is not None:
        mean_b, rstd_b = _moments(b, kind, eps)
        p = (b - mean_b[:, None]) * rstd_b[:, None] * post[0] + post[1]
    s = residual + scale * gate * p
    mean, rstd = _moments(s, kind, eps)
    return s, (s - mean[:, None]) * rstd[:, None] * gamma + beta, (mean_b, rstd_b, mean, rstd)


def _back(dy, xh, rstd, kind):
    v = dy - xh * (dy * xh).mean(1)[:, None]
    if kind == "layer":
        v = v - dy.mean(1)[:, None]
    return v * rstd[:, None]


def block_norm_backward(dh, ds, s, b, stats, kind, post, gate, scale, gamma):
    """(dresidual, db, dgamma, dbeta, dpost_gamma, dpost_beta, dgate)."""
    mean_b, rstd_b, mean, rstd = stats
    sh = (s - mean[:, None]) * rstd[:, None]
    t = ds + _back(dh * gamma, sh, rstd, kind)
    dp = scale * gate * t
    if post is None:
        return t, dp, (dh * sh).sum(0), dh.sum(0), None, None, (scale * t * b).sum(0)
    bh = (b - mean_b[:, None]) * rstd_b[:, None]
    p = bh * post[0] + post[1]
    return (t, _back(dp * post[0], bh, rstd_b, kind), (dh * sh).sum(0), dh.sum(0), (dp * bh).sum(0), dp.sum(0),
            (scale * t * p).sum(0))
