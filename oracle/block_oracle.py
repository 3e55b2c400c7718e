"""fp64 CPU oracle of the MLP-block operators: 8-bit checkpoints, the
root-mean-square norm, linear layers with their epilogues, and the gradients.

TEST INFRASTRUCTURE ONLY; numpy in float64, one formula a function, nothing
shared with the CUDA path.
"""

from __future__ import annotations

import math

import numpy as np
from scipy.special import erfc

GROUP = 128


def ckpt_scales(t) -> np.ndarray:
    """Power-of-two scale of every 128-channel group of t [rows, C]: [rows, groups],
    NaN where the group holds a non-finite value."""
    t = np.asarray(t, np.float64)
    rows, C = t.shape
    out = np.empty((rows, -(-C // GROUP)))
    for g in range(out.shape[1]):
        with np.errstate(invalid="ignore"):
            top = np.abs(t[:, g * GROUP:(g + 1) * GROUP]).max(1)
        for i, a in enumerate(top):
            if not np.isfinite(a):
                out[i, g] = np.nan
                continue
            k = -120
            while k < 121 and a > 127 * 2.0 ** k:
                k += 1
            out[i, g] = 2.0 ** k
    return out


def ckpt_round(t) -> np.ndarray:
    """The values that the checkpoint of t stands for."""
    t = np.asarray(t, np.float64)
    s = np.repeat(ckpt_scales(t), GROUP, axis=1)[:, :t.shape[1]]
    with np.errstate(invalid="ignore"):
        return np.clip(np.rint(t / s), -127, 127) * s


def ckpt_encode(t):
    """Codes and scale bytes (q [rows, C to 16], s [groups, rows]) of t."""
    t = np.asarray(t, np.float64)
    rows, C = t.shape
    sc = ckpt_scales(t)
    s = np.repeat(sc, GROUP, axis=1)[:, :C]
    with np.errstate(invalid="ignore"):
        q = np.nan_to_num(np.clip(np.rint(t / s), -127, 127)).astype(np.int8)
    qp = np.zeros((rows, -(-C // 16) * 16), np.int8)
    qp[:, :C] = q
    code = np.where(np.isnan(sc), 255, np.round(np.log2(np.where(np.isnan(sc), 1, sc))) + 127)
    return qp, np.ascontiguousarray(code.T.astype(np.uint8))


def ckpt_decode(q, s, C) -> np.ndarray:
    """Values of codes q [rows, ld] with scale bytes s [groups, rows]."""
    s = np.asarray(s)
    sc = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127)).T
    return np.asarray(q, np.float64)[:, :C] * np.repeat(sc, GROUP, axis=1)[:, :C]


def act(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return np.where(z < 0, 0.0, z)
    if kind == "gelu":
        return 0.5 * z * erfc(-z / math.sqrt(2))
    if kind == "silu":
        return z / (1 + np.exp(-z))
    return z


def act_slope(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return np.where(z > 0, 1.0, np.where(z <= 0, 0.0, z))
    if kind == "gelu":
        return 0.5 * erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + z * s * (1 - s)
    return np.ones_like(z)


def rms_norm(x, gamma, residual=None, eps=1e-5):
    """(h, r, u, y)"""
    h = np.asarray(x, np.float64) + (0 if residual is None else residual)
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    u = h * r[:, None]
    return h, r, u, u * gamma


def rms_norm_backward(gy, u, r, gamma, residual=None):
    """(gx, ggamma) from the normalised rows u and the factor r."""
    d = gy * gamma
    c = (d * u).mean(1, keepdims=True)
    gx = np.asarray(r)[:, None] * (d - u * c)
    return gx + (0 if residual is None else residual), (gy * u).sum(0)


def linear_act(x, w, bias=None, kind="none", residual=None):
    """(z, y)"""
    z = x @ w.T + (0 if bias is None else bias)
    return z, act(z, kind) + (0 if residual is None else residual)


def linear_act_grad(gy, w, z=None, kind="none", residual=None):
    g = gy @ w
    if kind != "none":
        g = g * act_slope(z, kind)
    return g + (0 if residual is None else residual)


def grad_w(gy, v, col_scale=None):
    """(gw, gb)"""
    gw = gy.T @ v
    return gw if col_scale is None else gw * col_scale, gy.sum(0)
