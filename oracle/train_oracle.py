"""Plain fp64 numpy definitions of the layer-norm, linear and 8-bit checkpoint operators.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the library's own path.  Written from
the formulas; it shares no code with the HIP kernels.
"""
import numpy as np
from scipy.special import erfc

BLOCK = 64


def pack(x):
    """(codes int8, exps int8) of rows: per 64 channels the smallest e with max|x| <= 127 * 2^e over the
    finite entries, held to [-126, 121]; q = rint(x / 2^e) held to +-127 (NaN: 0)."""
    x = np.asarray(x, np.float64)
    n, d = x.shape
    nb = -(-d // BLOCK)
    codes = np.zeros((n, d), np.int8)
    exps = np.full((n, nb), -126, np.int8)
    for b in range(nb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        m = np.where(np.isfinite(v), np.abs(v), 0).max(1)
        e = np.full(n, -126)
        while True:
            up = (m > 127 * 2.0 ** e) & (e < 121)
            if not up.any():
                break
            e = e + up
        exps[:, b] = e
        q = np.rint(np.where(np.isnan(v), 0, v) / 2.0 ** e[:, None])
        codes[:, b * BLOCK:(b + 1) * BLOCK] = np.clip(q, -127, 127)
    return codes, exps


def unpack(codes, exps):
    step = np.repeat(2.0 ** exps.astype(np.float64), BLOCK, 1)[:, :codes.shape[1]]
    return codes.astype(np.float64) * step


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0)
    if name == "gelu":
        return 0.5 * z * erfc(-z / np.sqrt(2))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * erfc(-z / np.sqrt(2)) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + z * s * (1 - s)
    return np.ones_like(z)


def layer_norm(x, gamma, beta, eps):
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / np.sqrt((c * c).mean(1) + eps)
    return c * rstd[:, None] * gamma + beta, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, gamma):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(1)[:, None] - xh * (g * xh).mean(1)[:, None])
    return dx, (dy * xh).sum(0), dy.sum(0)


def linear(x, w, bias, name, residual):
    z = x @ w.T + bias
    return act(z, name) + residual, z


def linear_backward(dy, x, w, name, z):
    dz = dy * act_slope(z, name) if name != "none" else dy
    return dz, dz @ w, dz.T @ x, dz.sum(0)
