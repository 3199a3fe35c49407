"""Pins of the sublayer oracle: torch autograd and central differences for the
norms and the gated activation, hand-worked codes and torch's own 8-bit float
for the checkpoints."""

import numpy as np
import pytest
import torch

from oracle import sublayer_oracle as so


def _rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_norm_and_gradient_against_autograd(norm):
    rng = _rng(1)
    v, w, b, dn = rng.normal(size=(5, 24)), rng.normal(size=24), rng.normal(size=24), rng.normal(size=(5, 24))
    eps = 1e-5
    tv = torch.tensor(v, requires_grad=True)
    tw, tb = torch.tensor(w, requires_grad=True), torch.tensor(b, requires_grad=True)
    if norm == "layer":
        n = torch.nn.functional.layer_norm(tv, (24,), tw, tb, eps)
    else:
        n = torch.nn.functional.rms_norm(tv, (24,), tw, eps) + tb
    n.backward(torch.tensor(dn))
    got, mean, rstd = so.norm_rows(v, norm, eps, w, b)
    assert np.allclose(got, n.detach().numpy(), rtol=0, atol=1e-13)
    dv, dw, db = so.norm_backward(dn, v, mean, rstd, norm, w)
    assert np.allclose(dv, tv.grad.numpy(), rtol=0, atol=1e-12)
    assert np.allclose(dw, tw.grad.numpy(), rtol=0, atol=1e-12)
    assert np.allclose(db, tb.grad.numpy(), rtol=0, atol=1e-12)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_norm_gradient_against_differences(norm):
    rng = _rng(2)
    v, w, dn, eps, h = rng.normal(size=(2, 16)), rng.normal(size=16), rng.normal(size=(2, 16)), 1e-3, 1e-6
    _, mean, rstd = so.norm_rows(v, norm, eps, w)
    dv, _, _ = so.norm_backward(dn, v, mean, rstd, norm, w)
    for r in range(2):
        for c in range(16):
            p, m = v.copy(), v.copy()
            p[r, c] += h
            m[r, c] -= h
            diff = (dn * (so.norm_rows(p, norm, eps, w)[0] - so.norm_rows(m, norm, eps, w)[0])).sum() / (2 * h)
            # the third derivative of a norm of unit-size rows is O(10): h^2 10 plus cancellation 1e-16 / h
            assert abs(diff - dv[r, c]) < 1e-8


def test_gated_gradient_against_differences_and_torch():
    rng = _rng(3)
    g, u, da, h = 3 * rng.normal(size=200), rng.normal(size=200), rng.normal(size=200), 1e-6
    dg, du, a = so.gated_backward(g, u, da)
    assert np.allclose(a, so.gated(g, u), rtol=0, atol=1e-14)
    assert np.allclose(a, (torch.nn.functional.silu(torch.tensor(g)) * torch.tensor(u)).numpy(), atol=1e-14)
    assert np.allclose(dg, da * (so.gated(g + h, u) - so.gated(g - h, u)) / (2 * h), atol=1e-8)
    assert np.allclose(du, da * (so.gated(g, u + h) - so.gated(g, u - h)) / (2 * h), atol=1e-8)
    assert so.gated(np.array([-1000.0]), np.array([1.0]))[0] == 0.0


def test_e4m3_grid_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, so.e4m3_grid())
    t = _rng(4).uniform(-448, 448, 20000)
    t[:5000] *= 2.0 ** _rng(5).integers(-18, 0, 5000)
    mid = (so.e4m3_grid()[1:] + so.e4m3_grid()[:-1]) / 2      # every tie
    t = np.concatenate([t, mid, -mid]).astype(np.float32)
    want = torch.tensor(t).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(so.round_to_grid(t.astype(np.float64), "e4m3"), want)


def test_checkpoint_codes_by_hand():
    v = np.zeros((1, 96))
    v[0, 0], v[0, 1] = 448.0, 1.0            # scale 1: exact codes
    v[0, 32], v[0, 33] = 450.0, 3.0          # one step over: scale 2, 225 -> 224, 1.5
    val, codes = so.checkpoint_codes(v, "e4m3")
    assert codes.tolist() == [[127, 128, 3]]
    assert val[0, 0] == 448 and val[0, 1] == 1 and val[0, 32] == 448 and val[0, 33] == 3
    v[0, 0], v[0, 1], v[0, 32], v[0, 33] = 127.0, -0.5, 127.5, 2.0
    val, codes = so.checkpoint_codes(v, "int8")
    assert codes.tolist() == [[127, 128, 3]]
    assert val[0, 0] == 127 and val[0, 1] == 0 and val[0, 32] == 128 and val[0, 33] == 2
    v[0, 70] = np.inf
    val, codes = so.checkpoint_codes(v, "int8")
    assert codes[0, 2] == 255 and np.isnan(val[0, 64:]).all() and codes[0, 0] == 127


@pytest.mark.parametrize("fmt,half", [("e4m3", 2.0 ** -4), ("int8", None)])
def test_checkpoint_error_is_half_a_step(fmt, half):
    v = _rng(6).normal(size=(20, 100))
    val, codes = so.checkpoint_codes(v, fmt)
    scale = np.repeat(2.0 ** (codes.astype(np.float64) - 127), 32, axis=1)[:, :100]
    if fmt == "int8":
        assert (np.abs(val - v) <= scale / 2).all()
    else:
        assert (np.abs(val - v) <= np.maximum(half * np.abs(v), scale * 2.0 ** -10)).all()
