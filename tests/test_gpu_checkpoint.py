"""GPU parity of the 8-bit checkpoints, the gated MLP activation with its
backward pass from checkpoints, and the weight gradient from a checkpoint."""

import numpy as np
import pytest
import torch

from contextual_token_sparsity_b200 import lemo
from oracle import sublayer_oracle as so
from sublayer_common import (FILL, FMT, U16, U32, bf16, ckpt_values, dev_i32, draw, f64, kept,
                             make_ckpt, ok, strided, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    lemo.lemo_set_test_hooks(-1, 0)


def check_save_restore(v, idx, fmt, extra=0, pad_to=16):
    L, d = v.shape
    K = L if idx is None else len(idx)
    rows = -(-max(K, 1) // pad_to) * pad_to + 2
    xd, _ = strided(v, extra)
    ck, data, scales = make_ckpt(rows, d, fmt, 16 if extra else 0)
    K_d = dev_i32(K)
    lemo.lemo_checkpoint_save(xd, None if idx is None else dev_i32(idx), K_d, ck)
    ok()
    src = v if idx is None else v[idx]
    want, codes = so.checkpoint_codes(src, fmt)
    got, e = ckpt_values(ck, K)
    assert np.array_equal(e, codes)
    assert np.array_equal(got, want, equal_nan=True)
    assert (data[K:] == 0xAB).all() and (scales[K:] == 0xCD).all()
    assert (data[:, d:] == 0xAB).all() and (scales[:, -(-d // 32):] == 0xCD).all()
    y, y_all = strided(np.zeros((0, d)), extra, rows)
    lemo.lemo_checkpoint_restore(ck, K_d, pad_to, y)
    ok()
    K_pad = -(-K // pad_to) * pad_to
    back = f64(y_all)
    assert np.array_equal(back[:K, :d], want, equal_nan=True)     # exact in bf16
    assert (back[K:K_pad, :d] == 0).all()
    assert (back[K_pad:] == FILL).all() and (back[:, d:] == FILL).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [8, 24, 32, 40, 248, 256, 264, 1000, 4096, 11008])
def test_save_restore_widths(d, fmt):
    rng = np.random.default_rng([d, len(fmt)])
    check_save_restore(draw(rng, 29, d), kept(rng, 29, 13), fmt, extra=8 * (d % 3))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("K", [0, 1, 2, 700])
def test_save_restore_rows(K, fmt):
    rng = np.random.default_rng([K, 5])
    check_save_restore(draw(rng, 701, 136), kept(rng, 701, K), fmt, pad_to=128)


@pytest.mark.parametrize("L,K,d", [(10501, 10007, 40), (2400, 2300, 4104)])
def test_save_restore_more_than_the_grid_holds(L, K, d):
    """More rows, and more pieces of rows, than all warps take in one pass."""
    rng = np.random.default_rng([L, d])
    check_save_restore(draw(rng, L, d), kept(rng, L, K), "e4m3", extra=8, pad_to=128)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_magnitude_ties_and_nonfinite(fmt):
    """All bf16 exponents, both sides of the scale's switch, ties of the code
    grid, zero groups, signed zeros, infinities and NaN."""
    rows = []
    for e in range(-133, 128):
        m = np.array([1.0, 1.75, 1.7578125, 1.984375, 1.9921875, 1.0078125, 1.5, 0.0])
        r = np.zeros(32)
        with np.errstate(over="ignore"):
            r[:8] = m * 2.0 ** e
            r[8:16] = -m * 2.0 ** max(e - 6, -133)
            r[16:24] = m * 2.0 ** max(e - 14, -133)
        rows.append(r)
    v = torch.from_numpy(np.array(rows).astype(np.float32)).to(torch.bfloat16).double().numpy()
    ties = np.zeros((5, 32))
    ties[0, :32] = np.concatenate([[127.0], np.arange(31) + 0.5])
    ties[1, :32] = np.concatenate([[448.0], 17.0 + 2 * np.arange(31)])
    ties[2, 3], ties[3, 4] = np.inf, np.nan
    ties[4, 5] = -0.0
    check_save_restore(np.concatenate([v, ties]), None, fmt)


def test_save_takes_repeated_ids():
    rng = np.random.default_rng(2)
    check_save_restore(draw(rng, 6, 64), np.array([5, 0, 0, 5, 3]), "int8")


def check_gated(K, d, fmt_g, fmt_u, extra=0, pad_to=16, seed=0, scale=1.0):
    rng = np.random.default_rng([seed, K, d])
    g, u, da = (draw(rng, max(K, 1), d, scale=s)[:K] for s in (scale, 1.0, 0.5))
    rows = -(-max(K, 1) // pad_to) * pad_to + 2
    gd, ud, dad = (strided(t, extra, rows, fill=float("nan"))[0] for t in (g, u, da))
    cg, cu = make_ckpt(rows, d, fmt_g)[0], make_ckpt(rows, d, fmt_u)[0]
    K_d = dev_i32(K)
    a, a_all = strided(np.zeros((0, d)), extra, rows)
    lemo.lemo_gated_mlp(gd, ud, K_d, pad_to, a, cg, cu)
    ok()
    K_pad = -(-K // pad_to) * pad_to

    def out(whole, want, size, what):
        # e^-g: two units of the exponential's argument and result, |g| U32 each, and a quotient
        got = f64(whole)
        within(got[:K, :d], want, U16 * np.abs(want) + 1.01 * 16 * U32 * size, what)
        assert (got[K:K_pad, :d] == 0).all(), what
        assert (got[K_pad:] == FILL).all() and (got[:, d:] == FILL).all(), what

    want = so.gated(g, u)
    out(a_all, want, np.abs(want) * (1 + np.abs(g)), "a")
    qg, eg = so.checkpoint_codes(g, fmt_g)
    qu, eu = so.checkpoint_codes(u, fmt_u)
    for c, q, e in ((cg, qg, eg), (cu, qu, eu)):
        val, code = ckpt_values(c, K)
        assert np.array_equal(code, e) and np.array_equal(val, q)
    dg, dg_all = strided(np.zeros((0, d)), extra, rows)
    du, du_all = strided(np.zeros((0, d)), extra, rows)
    a2, a2_all = strided(np.zeros((0, d)), extra, rows)
    lemo.lemo_gated_mlp_backward(cg, cu, dad, K_d, pad_to, dg, du, a=a2)
    ok()
    rg, ru, ra = so.gated_backward(qg, qu, da)
    s = 1 / (1 + np.exp(-qg))
    grow = 1 + np.abs(qg)
    out(dg_all, rg, np.abs(da * qu) * (s + np.abs(qg) * s * (1 - s) * 2) * grow, "dgate")
    out(du_all, ru, np.abs(ru) * grow, "dup")
    out(a2_all, ra, np.abs(ra) * grow, "a again")
    lemo.lemo_gated_mlp(gd, ud, K_d, pad_to, a)                     # without checkpoints
    lemo.lemo_gated_mlp_backward(cg, cu, dad, K_d, pad_to, dg, du)  # without the activation
    ok()
    out(a_all, want, np.abs(want) * (1 + np.abs(g)), "a")
    out(dg_all, rg, np.abs(da * qu) * (s + np.abs(qg) * s * (1 - s) * 2) * grow, "dgate")


@pytest.mark.parametrize("d", [8, 40, 256, 264, 1000, 11008])
def test_gated_widths(d):
    check_gated(11, d, "e4m3", "int8", extra=8 * (d % 3))


@pytest.mark.parametrize("K", [0, 1, 128, 500])
def test_gated_rows(K):
    check_gated(K, 520, "int8", "e4m3", pad_to=128)


def test_gated_more_than_the_grid_holds():
    check_gated(1500, 2056, "int8", "e4m3", extra=8, pad_to=128)


def test_gated_saturated():
    check_gated(9, 256, "e4m3", "e4m3", scale=60.0)


def check_wgrad(K, n, d, fmt, extra=0, seed=0, rows=None):
    rng = np.random.default_rng([seed, K, n, d])
    v, dy = draw(rng, max(K, 1), d)[:K], draw(rng, max(K, 1), n, scale=0.5)[:K]
    rows = max(K, 1) + 5 if rows is None else rows
    ck, _, _ = make_ckpt(rows, d, fmt, 16 if extra else 0)
    xd, _ = strided(v, 0, rows)
    K_d = dev_i32(K)
    lemo.lemo_checkpoint_save(xd, None, K_d, ck)
    # rows past K hold NaN in both operands
    ck.data[K:] = 0x7F
    ck.scales[K:] = 255
    dyd, _ = strided(dy, extra, rows, fill=float("nan"))
    dw0 = rng.normal(size=(n, d)).astype(np.float32)
    dw, dw_all = strided(dw0, extra, dtype=torch.float32)
    lemo.lemo_checkpoint_weight_grad(ck, dyd, K_d, dw)
    ok()
    q, _ = so.checkpoint_codes(v, fmt)
    want = dw0 + so.weight_grad(dy, q)
    # products are exact; the fp32 sum of K terms in any order, each step off by at most one unit
    bound = 2 * (K + 8) * U32 * (np.abs(dy).T @ np.abs(q)) + 2 * U32 * (np.abs(dw0) + np.abs(want))
    got = f64(dw_all)
    within(got[:n, :d], want, bound, "dw")
    assert (got[n:] == FILL).all() and (got[:, d:] == FILL).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n,d", [(8, 8), (64, 72), (128, 128), (136, 264), (256, 256), (264, 520), (512, 40)])
def test_weight_grad_sizes(n, d, fmt):
    check_wgrad(100, n, d, fmt, extra=8 * (n % 3))


@pytest.mark.parametrize("K", [0, 1, 15, 16, 17, 63, 64, 65, 255, 1025, 3000])
def test_weight_grad_rows(K):
    check_wgrad(K, 264, 272, ["e4m3", "int8"][K % 2])


@pytest.mark.parametrize("K", [0, 1, 64, 100, 700, 2047, 2048, 5000, 8192])
def test_weight_grad_rows_split_over_a_cluster(K):
    """Few tiles and room for many rows: the rows of a tile are split over two or four CTA
    pairs, whatever the device's row count turns out to be."""
    check_wgrad(K, 512, 264, ["int8", "e4m3"][K % 2], rows=8192)
    check_wgrad(min(K, 1500), 136, 72, "e4m3", rows=1500)


def test_weight_grad_split_is_deterministic():
    rng = np.random.default_rng(6)
    K, n, d = 8192, 512, 512
    ck, _, _ = make_ckpt(K, d, "e4m3")
    lemo.lemo_checkpoint_save(bf16(draw(rng, K, d)), None, dev_i32(K), ck)
    dy = bf16(draw(rng, K, n))
    runs = [torch.zeros(n, d, device="cuda") for _ in range(4)]
    for dw in runs:
        lemo.lemo_checkpoint_weight_grad(ck, dy, dev_i32(K), dw)
    ok()
    assert all(torch.equal(runs[0], dw) for dw in runs[1:])


def test_weight_grad_many_tiles():
    check_wgrad(200, 2056, 2600, "e4m3")


def test_weight_grad_extreme_scales():
    """Scales over the whole range of the byte, and a NaN group only spoils its columns."""
    rng = np.random.default_rng(3)
    K, n, d = 40, 64, 128
    for fmt in ("e4m3", "int8"):
        ck, _, _ = make_ckpt(K, d, fmt)
        v = draw(rng, K, d)
        v[:, 32:64] *= 2.0 ** 90
        v[:, 64:96] *= 2.0 ** -100
        lemo.lemo_checkpoint_save(bf16(v), None, dev_i32(K), ck)
        ck.scales[7, 3] = 255
        dw = torch.zeros(n, d, device="cuda")
        dy = draw(rng, K, n)
        lemo.lemo_checkpoint_weight_grad(ck, bf16(dy), dev_i32(K), dw)
        ok()
        q, _ = so.checkpoint_codes(v, fmt)
        want = so.weight_grad(dy, q)
        want[:, 96:] = np.nan
        bound = 2 * (K + 8) * U32 * (np.abs(dy).T @ np.abs(q))
        within(f64(dw), want, bound)


def test_weight_grad_accumulates_and_is_deterministic():
    rng = np.random.default_rng(4)
    K, n, d = 1500, 520, 776
    ck, _, _ = make_ckpt(K, d, "int8")
    v, g = draw(rng, K, d), draw(rng, K, n)
    lemo.lemo_checkpoint_save(bf16(v), None, dev_i32(K), ck)
    dy = bf16(g)
    one, two = torch.zeros(n, d, device="cuda"), torch.zeros(n, d, device="cuda")
    for dw in (one, two, one, two):
        lemo.lemo_checkpoint_weight_grad(ck, dy, dev_i32(K), dw)
    ok()
    assert torch.equal(one, two)
    q, _ = so.checkpoint_codes(v, "int8")
    # two sums of K terms (check_wgrad's bound each) and their additions, which the K + 8 covers
    within(f64(one), 2 * so.weight_grad(g, q), 2 * 2 * (K + 8) * U32 * (np.abs(g).T @ np.abs(q)))


def test_too_many_rows_are_reported():
    d = 64
    x = torch.ones(10, d, dtype=torch.bfloat16, device="cuda")
    ck, data, _ = make_ckpt(4, d, "e4m3")
    lemo.lemo_checkpoint_save(x, None, dev_i32(9), ck)
    assert lemo.lemo_get_error() == lemo.LEMO_ERR_CAPACITY
    assert (data[4:] == 0xAB).all()
    lemo.lemo_checkpoint_save(x, dev_i32([0, 10, -1]), dev_i32(3), ck)
    assert lemo.lemo_get_error() == lemo.LEMO_ERR_INVALID_ARG
    y = torch.zeros(4, d, dtype=torch.bfloat16, device="cuda")
    lemo.lemo_checkpoint_restore(ck, dev_i32(9), 1, y)
    assert lemo.lemo_get_error() == lemo.LEMO_ERR_CAPACITY
    dw = torch.zeros(8, d, device="cuda")
    lemo.lemo_checkpoint_weight_grad(ck, x[:4, :8], dev_i32(9), dw)
    assert lemo.lemo_get_error() == lemo.LEMO_ERR_CAPACITY
