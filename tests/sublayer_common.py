"""Shared helpers of the sublayer operator tests: seeded bf16 inputs, kept ids,
buffers with guard rows and padded strides, and the error bounds.

Bounds.  U32 = 2^-24 and U16 = 2^-8 are half a step of fp32 and bf16.  A row
sum of d fp32 terms taken in a tree of depth at most 64 (8 V values per thread
with V <= 4, five shuffles, 16 warps, a few operations per term) is off by at
most 64 U32 times the sum of magnitudes, whatever d is; ROW = 128 U32 covers a
row's statistics and the handful of roundings of one output value.  A sum over
K rows in any order is off by at most (K + 8) U32 times the sum of magnitudes.
"""

import numpy as np
import torch

from contextual_token_sparsity_b200 import lemo

U16, U32 = 2.0 ** -8, 2.0 ** -24
ROW = 128 * U32
FMT = {"e4m3": lemo.LEMO_CHECKPOINT_E4M3, "int8": lemo.LEMO_CHECKPOINT_INT8}
NORM = {"none": lemo.LEMO_NORM_NONE, "rms": lemo.LEMO_NORM_RMS, "layer": lemo.LEMO_NORM_LAYER}
EPS = 1e-5
GUARD = 3          # rows behind the buffers' documented ones
FILL = 7.0


def bf16(a):
    """float64 array of bf16 values -> device tensor."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16)


def draw(rng, *shape, scale=1.0, add=0.0):
    """Normal draws rounded to bf16, as float64."""
    t = torch.from_numpy((rng.normal(size=shape) * scale + add).astype(np.float32))
    return t.to(torch.bfloat16).double().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def strided(a, extra=0, rows=None, fill=FILL, dtype=torch.bfloat16):
    """(view, whole): a's values in a buffer of `rows` rows plus GUARD rows and
    `extra` more columns, everything else `fill`; the view has `rows` rows."""
    rows = a.shape[0] if rows is None else rows
    whole = torch.full((rows + GUARD, a.shape[1] + extra), fill, dtype=dtype, device="cuda")
    whole[: a.shape[0], : a.shape[1]] = torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)
    return whole[:rows, : a.shape[1]], whole


def kept(rng, L, K):
    return np.sort(rng.choice(L, K, replace=False)).astype(np.int32)


def dev_i32(a):
    a = np.atleast_1d(np.asarray(a, dtype=np.int32))
    return torch.from_numpy(a if a.size else np.zeros(1, np.int32)).cuda()


def make_ckpt(rows, d, fmt, extra=0):
    data = torch.full((rows + GUARD, -(-d // 16) * 16 + extra), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + GUARD, -(-d // 128) * 4 + (4 if extra else 0)), 0xCD,
                        dtype=torch.uint8, device="cuda")
    return lemo.make_checkpoint(data[:rows], scales[:rows], FMT[fmt], d), data, scales


def ckpt_values(c, K):
    """float64 values a checkpoint's first K rows stand for, and the scale bytes."""
    q = c.data[:K, : c.d].contiguous().cpu()
    e = c.scales[:K, : -(-c.d // 32)].cpu().numpy()
    t = q.view(torch.float8_e4m3fn if c.struct.format == FMT["e4m3"] else torch.int8).double().numpy()
    s = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))
    return t * np.repeat(s, 32, axis=1)[:, : c.d], e


def ok():
    st = lemo.lemo_get_error()
    assert st == lemo.LEMO_OK, lemo.STATUS.get(st, st)


def within(got, want, bound, what=""):
    """|got - want| <= bound element-wise; NaN only where NaN is wanted."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), what
    err = np.abs(got - want)[fin]
    lim = (np.broadcast_to(bound, want.shape) + 1e-37)[fin]
    bad = err > lim
    assert not bad.any(), (what, int(bad.sum()), float((err / lim).max()))


def norm_slop(v, mean, rstd, weight, bias):
    """fp32 error of vhat weight + bias, element-wise."""
    w = 1.0 if weight is None else np.abs(weight)
    b = 0.0 if bias is None else np.abs(bias)
    big = np.abs(v) + np.abs(v).mean(1, keepdims=True)
    return ROW * (big * rstd[:, None] * w + b)


def back_slop(g, vhat, rstd, norm):
    """fp32 error of rstd (g - vhat mean(g vhat) - mean(g)), element-wise."""
    if norm == "none":
        return ROW * np.abs(g)
    m1 = np.abs(g * vhat).mean(1, keepdims=True)
    m2 = np.abs(g).mean(1, keepdims=True) if norm == "layer" else 0.0
    return ROW * rstd[:, None] * (np.abs(g) + (np.abs(vhat) + 1) * m1 + m2)
