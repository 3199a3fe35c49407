"""Plain float64 CPU oracle of what surrounds a sublayer on the kept tokens:
the norms before and after it, 8-bit activation checkpoints, the gated MLP
activation and the weight gradient from a checkpoint.

TEST INFRASTRUCTURE ONLY, like ``oracle.lemo_oracle``: nothing on the product
path imports it, and it shares no code with the CUDA library.  Inputs are
float64 arrays of bf16 values; outputs are float64, not rounded to bf16 (the
tests count that rounding in their tolerances).

Sources: the selective load and the in-place addition of "Jenga: Enhancing
LLM Long-Context Fine-tuning with Contextual Token Sparsity" (aipaper.cc
summary), section 4.2.3, around the usual RMS / layer norms; the SiLU-gated
activation of section 4.2.1, "Extend to MLP Block".
"""

from __future__ import annotations

import numpy as np

GROUP = 32


def statistics(v, norm: str, eps: float):
    """(mean, rstd) of every row; rms has mean 0, none has mean 0 and rstd 1."""
    K, d = v.shape
    mean, rstd = np.zeros(K), np.ones(K)
    for r in range(K):
        if norm == "layer":
            mean[r] = v[r].sum() / d
        if norm != "none":
            rstd[r] = 1.0 / np.sqrt(((v[r] - mean[r]) ** 2).sum() / d + eps)
    return mean, rstd


def norm_rows(v, norm: str, eps: float, weight=None, bias=None):
    """vhat weight + bias, with the statistics."""
    mean, rstd = statistics(v, norm, eps)
    n = (v - mean[:, None]) * rstd[:, None]
    if weight is not None:
        n = n * weight
    if bias is not None:
        n = n + bias
    return n, mean, rstd


def norm_backward(dn, v, mean, rstd, norm: str, weight=None):
    """Gradients (dv, dweight, dbias) of sum(dn * (vhat weight + bias)), with the
    given statistics' dependence on the row as the norm's formula has it."""
    K, d = v.shape
    vhat = (v - mean[:, None]) * rstd[:, None]
    g = dn if weight is None else dn * weight
    dv = np.empty_like(v)
    for r in range(K):
        if norm == "none":
            dv[r] = g[r]
            continue
        c = g[r] - vhat[r] * (np.dot(g[r], vhat[r]) / d)
        if norm == "layer":
            c = c - g[r].sum() / d
        dv[r] = rstd[r] * c
    return dv, (dn * vhat).sum(0), dn.sum(0)


def checkpoint_codes(v, fmt: str):
    """(values, scale bytes) of rows held in 8 bits: the value of every code
    times its group's scale, and the byte k + 127 per group of 32 columns."""
    K, d = v.shape
    most = 448.0 if fmt == "e4m3" else 127.0
    ng = -(-d // GROUP)
    out, codes = np.empty((K, d)), np.empty((K, ng), dtype=np.uint8)
    for r in range(K):
        for g in range(ng):
            x = v[r, g * GROUP:(g + 1) * GROUP]
            if not np.isfinite(x).all():
                codes[r, g] = 255
                out[r, g * GROUP:(g + 1) * GROUP] = np.nan
                continue
            k = -124
            peak = np.abs(x).max()
            while peak > most * 2.0 ** k:   # smallest k with peak / 2^k <= most
                k += 1
            codes[r, g] = k + 127
            q = round_to_grid(x / 2.0 ** k, fmt)
            over = np.abs(q) * 2.0 ** k >= 2.0 ** 128      # not a finite bf16: one code lower
            q[over] = np.copysign(240.0 if fmt == "e4m3" else 63.0, q[over])
            out[r, g * GROUP:(g + 1) * GROUP] = q * 2.0 ** k
    return out, codes


def round_to_grid(t, fmt: str):
    """Nearest representable value, ties to the even code."""
    if fmt == "int8":
        return np.rint(t)
    grid = e4m3_grid()
    hi = np.clip(np.searchsorted(grid, np.abs(t)), 1, len(grid) - 1)
    a, b = grid[hi - 1], grid[hi]
    up = np.abs(t) - a > b - np.abs(t)
    tie = np.abs(t) - a == b - np.abs(t)
    even_hi = hi % 2 == 0                       # a grid index is the code
    mag = np.where(up | (tie & even_hi), b, a)
    return np.copysign(mag, t)


def e4m3_grid():
    """The 127 non-negative values, index = code: 4 exponent bits of bias 7,
    3 mantissa bits, no infinities, code 127 (NaN) left out."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def gated(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def gated_backward(g, u, da):
    """(dgate, dup, a)."""
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return da * u * s * (1.0 + g * (1.0 - s)), da * g * s, g * s * u


def weight_grad(dy, xhat):
    return dy.T @ xhat
