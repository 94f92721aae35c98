"""Layer norm, linear layer and dropout of an OPT-style sub-block, with gradients (float64 numpy).

Layer norm over the rows:  n = (x - mean) / sqrt(var + eps),  y = n gamma + beta, var the
biased (1/h) variance.  Linear: y = act(x w^T + b) + residual.  Dropout: Philox4x32-10
(Salmon, Moraes, Dror, Shaw, SC'11), 16 random bits an element.
"""
import math

import numpy as np
from scipy.special import erf, expit


# ------------------------------------------------------------------ layer norm
def layernorm_fwd(x, gamma=None, beta=None, eps=1e-5):
    """-> (y, mean [rows], rstd [rows])."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layernorm_bwd(dy, x, mean, rstd, gamma=None):
    """-> (dx, dgamma, dbeta) for the given row statistics."""
    n = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - n * (g * n).mean(1, keepdims=True))
    return dx, (dy * n).sum(0), dy.sum(0)


# ------------------------------------------------------------------ linear
def act(z, kind):
    if kind == "relu":
        return np.maximum(z, 0.0)  # keeps a NaN
    if kind == "gelu":
        return 0.5 * z * (1.0 + erf(z / math.sqrt(2.0)))
    if kind == "silu":
        return z * expit(z)
    return z


def act_grad(z, kind):
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * (1.0 + erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "silu":
        s = expit(z)
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def linear_fwd(x, w, bias=None, kind="none", residual=None):
    """-> (y, z) with z = x w^T + bias."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + bias
    y = act(z, kind)
    return (y if residual is None else y + residual), z


def linear_bwd(dy, x, w, kind="none", pre=None):
    """-> (dx, dw, db, dz)."""
    dz = dy if kind == "none" else dy * act_grad(pre, kind)
    return dz @ w, dz.T @ x, dz.sum(0), dz


# ------------------------------------------------------------------ dropout
def philox4x32_10(counter, key):
    """Counter [..., 4] and key (2 words) of 32-bit words -> [..., 4] words."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter[..., i], np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & m, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def dropout_threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def dropout_mask(positions, cols, p, seed, offset):
    """Boolean keep mask [len(positions), cols]."""
    pos = np.asarray(positions, np.uint64)
    groups = (cols + 7) // 8
    ctr = np.zeros((len(pos), groups, 4), np.uint64)
    ctr[..., 0] = np.arange(groups, dtype=np.uint64)[None, :]
    ctr[..., 1] = pos[:, None]
    ctr[..., 2] = offset & 0xFFFFFFFF
    ctr[..., 3] = (offset >> 32) & 0xFFFFFFFF
    w = philox4x32_10(ctr, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(len(pos), groups * 8)
    return bits[:, :cols] >= dropout_threshold(p)


def dropout(x, positions, p, seed, offset, residual=None):
    t = dropout_threshold(p)
    keep = dropout_mask(positions, x.shape[1], p, seed, offset)
    y = np.where(keep, np.asarray(x, np.float64), 0.0) * (65536.0 / (65536 - t) if t < 65536 else 0.0)
    return y if residual is None else y + residual
