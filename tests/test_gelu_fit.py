"""Provenance of the polynomial behind GELU's normal tail (normal_tail in csrc/linear_tc.cuh).

P(Z > t) e^(t^2/2) = erfcx(t / sqrt 2) / 2 is a polynomial c1 r + ... + c9 r^9 in r = 1 / (1 + 0.34 t) whose
relative error is made equal-ripple (minimax) on t in [0, 14] by Lawson's iteratively reweighted least
squares (C. L. Lawson, 1961).  The test refits it, checks that the constants compiled into the
kernel reach the fit's error, and that the fp32 evaluation keeps the stated bound."""
import os
import re

import numpy as np
from scipy.special import erfc, erfcx

CUH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "token_sparse_long_b200", "csrc",
                   "linear_tc.cuh")
U = 2.0 ** -24
P = float(np.float32(0.34))


def ratio(t):
    return 0.5 * erfcx(t / np.sqrt(2.0))


def kernel_constants():
    """c1 .. c9 as written in normal_tail (the Horner chain starts from c9)."""
    src = open(CUH).read()
    body = src[src.index("__device__ __forceinline__ float normal_tail("):]
    body = body[:body.index("return")]
    vals = [float.fromhex(h[:-1]) for h in re.findall(r"-?0x[01]\.[0-9a-f]+p[-+]?\d+f", body)]
    assert len(vals) == 9 and "fmaf(0.34f, t, 1.f)" in body
    return np.array(vals[::-1])


def lawson_minimax_rel(deg=9, nodes=4000, iters=400):
    lo = 1.0 / (1.0 + P * 14.0)
    r = np.unique(np.concatenate([lo + (1 - lo) * (0.5 - 0.5 * np.cos(np.pi * (np.arange(nodes) + 0.5) / nodes)), [lo, 1.0]]))
    a = np.stack([r ** (k + 1) for k in range(deg)], 1) / ratio((1 / r - 1) / P)[:, None]
    w = np.full(len(r), 1.0 / len(r))
    best = np.inf
    for _ in range(iters):
        sw = np.sqrt(w)
        c, *_ = np.linalg.lstsq(a * sw[:, None], sw, rcond=None)
        e = np.abs(a @ c - 1.0)
        best = min(best, e.max())
        w = w * e
        w /= w.sum()
    return best


def test_kernel_polynomial_reaches_the_fit():
    t = np.linspace(0.0, 14.0, 200001)
    r = 1.0 / (1.0 + P * t)
    got = np.abs(sum(c * r ** (k + 1) for k, c in enumerate(kernel_constants())) / ratio(t) - 1.0).max()
    fit = lawson_minimax_rel()
    assert fit < 3.5e-8
    # nine constants rounded to fp32, each by half a step of itself
    slack = max(np.abs(sum(abs(c) * U * r ** (k + 1) for k, c in enumerate(kernel_constants())) / ratio(t)))
    assert got <= fit * 1.05 + slack


def test_fp32_evaluation_keeps_the_stated_bound():
    t = np.linspace(0.0, 13.0, 400001).astype(np.float32)
    T = t.astype(np.float64)
    f32 = lambda v: np.asarray(v, np.float64).astype(np.float32)
    r = f32(1.0 / f32(T * np.float32(0.34) + 1).astype(np.float64))
    c = kernel_constants()
    a = np.full_like(t, np.float32(c[8]))
    for k in range(7, -1, -1):  # fused multiply-adds: one rounding each
        a = f32(a.astype(np.float64) * r + c[k])
    e = f32(2.0 ** f32(f32(T * T).astype(np.float64) * np.float32(-0.72134752044448170)).astype(np.float64))
    q = f32(f32(a.astype(np.float64) * r).astype(np.float64) * e)
    rel = np.abs(q.astype(np.float64) / (0.5 * erfc(T / np.sqrt(2.0))) - 1.0)
    assert (rel <= 0.7 * (1.3 * (1 + T * T) + 12) * U).all(), float((rel / (1.3 * (1 + T * T) + 12) / U).max())
