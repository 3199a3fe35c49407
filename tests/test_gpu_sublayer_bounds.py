"""Gradients and long sums of the sublayer operators at bounds that a wrong one exceeds: gradients
against central differences of the formulas in 64 bits, and sums over many rows against the
roundings that the kernels really make.  Each test also shows that its bound refuses what it is
there to refuse."""

import numpy as np
import pytest
import torch

from contextual_token_sparsity_b200 import lemo
from oracle import sublayer_oracle as so
from sublayer_common import (EPS, NORM, U16, U32, back_slop, bf16, dev_i32, draw, f64, make_ckpt, ok, within)

pytestmark = pytest.mark.gpu
H = 2.0 ** -12      # half a step of the differences: h^2 times a third derivative, and 2^-53 / h of rounding


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    lemo.lemo_set_test_hooks(-1, 0)


def differences(f, v, axis=None):
    """Central differences of the sum f(v) by every element of v (rows do not touch one another:
    with axis=1, f gives one value per row and a column of all rows moves at once)."""
    out = np.empty_like(v)
    where = range(v.shape[1]) if axis == 1 else np.ndindex(v.shape)
    for i in where:
        i = (slice(None), i) if axis == 1 else i
        p, m = v.copy(), v.copy()
        p[i] += H
        m[i] -= H
        out[i] = (f(p) - f(m)) / (2 * H)
    return out


def close(got, want, bound, what):
    """Within the bound, which neither a zero nor a negated gradient would be."""
    within(got, want, bound, what)
    big = np.abs(want) > bound
    assert big.mean() > 0.8, (what, float(big.mean()))      # |0 - want| and |-want - want| exceed it there


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_gather_gradients_against_differences(norm):
    rng = np.random.default_rng([1, len(norm)])
    K, d = 7, 72
    x, w, b, c = draw(rng, K, d, add=0.3), draw(rng, d, scale=0.3, add=1.0), draw(rng, d, scale=0.3), draw(rng, K, d)
    K_d = dev_i32(K)
    y, stats = torch.zeros(K, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(K, 2, device="cuda")
    lemo.lemo_norm_gather(NORM[norm], bf16(x), bf16(w), bf16(b), EPS, None, K_d, 1, y, stats=stats)
    dx = torch.zeros(K, d, dtype=torch.bfloat16, device="cuda")
    dw, db = torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
    ws = torch.empty(lemo.lemo_norm_workspace_size(d), dtype=torch.uint8, device="cuda")
    lemo.lemo_norm_gather_backward(NORM[norm], bf16(c), bf16(w), stats, None, K_d, dx, ws, x=bf16(x), dweight=dw,
                                   dbias=db)
    ok()
    vhat, _, rstd = so.norm_rows(x, norm, EPS)
    # differences: third derivatives of a row's norm are below 100 rstd^3 |c w| sums, times h^2 / 6
    cut = H * H * 100 * np.abs(c * w).sum(1).max()
    rows = differences(lambda t: (c * so.norm_rows(t, norm, EPS, w, b)[0]).sum(1), x, axis=1)
    close(f64(dx), rows, U16 * np.abs(rows) + 1.01 * back_slop(c * w, vhat, rstd, norm) + cut, "dx")
    by_w = differences(lambda t: (c * so.norm_rows(x, norm, EPS, t, b)[0]).sum(), w)
    by_b = differences(lambda t: (c * so.norm_rows(x, norm, EPS, w, t)[0]).sum(), b)
    # linear in w and b: only the rounding of the loss, 2^-53 / h of it, and fp32 statistics and sums
    size = np.abs(c * vhat).sum(0)
    close(f64(dw), by_w, 1e-9 + 1.01 * 128 * U32 * (size + np.abs(c).sum(0)), "dw")
    close(f64(db), by_b, 1e-9 + 16 * U32 * np.abs(c).sum(0), "db")


@pytest.mark.parametrize("norm,gate", [("none", "channel"), ("rms", "channel"), ("layer", "token"), ("layer", "channel"),
                                       ("rms", "token")])
def test_scatter_gradients_against_differences(norm, gate):
    rng = np.random.default_rng([2, len(norm), len(gate)])
    K, d, s = 7, 72, 0.75
    y, w, b, c = draw(rng, K, d, add=0.3), draw(rng, d, scale=0.3, add=1.0), draw(rng, d, scale=0.3), draw(rng, K, d)
    g = draw(rng, *((d,) if gate == "channel" else (K, d)), scale=0.3, add=0.6)
    if norm == "none":
        w = b = None
    K_d, on = dev_i32(K), norm != "none"
    stats = torch.zeros(K, 2, device="cuda") if on else None
    dev = [None if t is None else bf16(t) for t in (w, b)]
    lemo.lemo_norm_scatter(NORM[norm], torch.zeros(K, d, dtype=torch.bfloat16, device="cuda"), bf16(y), *dev, EPS,
                           bf16(g), s, None, K_d, stats=stats)
    dy = torch.zeros(K, d, dtype=torch.bfloat16, device="cuda")
    dw, db = (torch.zeros(d, device="cuda") if on else None for _ in range(2))
    dg = torch.zeros(d, device="cuda") if gate == "channel" else torch.zeros(K, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lemo.lemo_norm_workspace_size(d), dtype=torch.uint8, device="cuda")
    lemo.lemo_norm_scatter_backward(NORM[norm], bf16(c), *dev, stats, bf16(g), s, None, K_d, 1, dy, ws, y=bf16(y),
                                    dweight=dw, dbias=db, dgate=dg)
    ok()

    def n(t, w=w, b=b):
        return so.norm_rows(t, norm, EPS, w, b)[0]

    vhat, _, rstd = so.norm_rows(y, norm, EPS)
    ww = np.ones(d) if w is None else w
    cut = H * H * 100 * np.abs(s * c * g * ww).sum(1).max()
    rows = differences(lambda t: (s * c * g * n(t)).sum(1), y, axis=1)
    close(f64(dy), rows, U16 * np.abs(rows) + 1.01 * back_slop(s * c * g * ww, vhat, rstd, norm) + cut, "dy")
    size = np.abs(s * c) * (np.abs(vhat * ww) + (0 if b is None else np.abs(b)) + np.abs(ww))
    if gate == "channel":
        by_g = differences(lambda t: (s * c * t * n(y)).sum(), g)
        close(f64(dg), by_g, 1e-9 + 1.01 * 128 * U32 * size.sum(0), "dgate")
    else:
        by_g = differences(lambda t: (s * c * t * n(y)).sum(1), g, axis=1)
        close(f64(dg), by_g, U16 * np.abs(by_g) + 1e-9 + 1.01 * 128 * U32 * size, "dgate")
    if on:
        by_w = differences(lambda t: (s * c * g * n(y, w=t)).sum(), w)
        by_b = differences(lambda t: (s * c * g * n(y, b=t)).sum(), b)
        close(f64(dw), by_w, 1e-9 + 1.01 * 128 * U32 * (np.abs(s * c * g) * (np.abs(vhat) + 1)).sum(0), "dw")
        close(f64(db), by_b, 1e-9 + 16 * U32 * np.abs(s * c * g).sum(0), "db")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_gated_gradients_against_differences(fmt):
    """Of the checkpointed values, which the backward pass takes for g and u."""
    rng = np.random.default_rng([3, len(fmt)])
    K, d = 9, 72
    g, u = (so.checkpoint_codes(draw(rng, K, d, scale=2.0), fmt)[0] for _ in range(2))
    da, K_d = draw(rng, K, d), dev_i32(K)
    cg, cu = make_ckpt(K, d, fmt)[0], make_ckpt(K, d, fmt)[0]
    a, dg, du = (torch.zeros(K, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    lemo.lemo_gated_mlp(bf16(g), bf16(u), K_d, 1, a, cg, cu)
    lemo.lemo_gated_mlp_backward(cg, cu, bf16(da), K_d, 1, dg, du)
    ok()
    # element-wise, so all elements move at once; |SiLU'''| < 1
    by_g = (da * (so.gated(g + H, u) - so.gated(g - H, u))) / (2 * H)
    by_u = (da * (so.gated(g, u + H) - so.gated(g, u - H))) / (2 * H)
    cut = H * H * np.abs(da * u) + 1e-9
    slop = 1.01 * 32 * U32 * (1 + np.abs(g))
    close(f64(dg), by_g, U16 * np.abs(by_g) + cut + slop * np.abs(da * u) * (1 + np.abs(g)), "dgate")
    close(f64(du), by_u, U16 * np.abs(by_u) + 1e-9 + slop * np.abs(by_u), "dup")


# An accumulator takes 2048 rows, 16 at a step, each step's result cut to 24 bits: at most
# 128 x 2^-23 = 1.5e-5 of the sum of magnitudes.  Then one rounding to nearest per accumulator added
# to dW.  (One accumulator of all 8192 rows was measured to lose 3.5e-5 with one sign.)
def wgrad_bound(K):
    return 128 * 2.0 ** -23 + (-(-K // 2048) + 1) * U32


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("K,n,d", [(8192, 64, 96),       # rows split over a cluster's pairs
                                   (32768, 64, 96), (32768, 2056, 2440)])  # a pair walks over all rows
def test_weight_grad_of_many_rows(K, n, d, one_sign, fmt):
    gen = torch.Generator("cuda").manual_seed(K + n + one_sign)
    x, dy = (torch.randn(K, m, generator=gen, device="cuda").to(torch.bfloat16) for m in (d, n))
    if one_sign:
        x, dy = x.abs(), dy.abs()
    ck, _, _ = make_ckpt(K, d, fmt)
    K_d = dev_i32(K)
    lemo.lemo_checkpoint_save(x, None, K_d, ck)
    q = torch.empty_like(x)
    lemo.lemo_checkpoint_restore(ck, K_d, 1, q)
    dw = torch.zeros(n, d, device="cuda")
    lemo.lemo_checkpoint_weight_grad(ck, dy, K_d, dw)
    ok()
    want = dy.double().t() @ q.double()
    size = dy.double().abs().t() @ q.double().abs()
    bound = wgrad_bound(K) * size
    err = (dw.double() - want).abs()
    assert bool((err <= bound).all()), float((err / size).max())
    # it refuses sums held in 16 bits
    assert bool(((want.bfloat16().double() - want).abs() > bound).any())


@pytest.mark.parametrize("d,K", [(64, 4801), (520, 6000), (4096, 3001), (8192, 1500)])
def test_column_sums_of_many_rows(d, K):
    """dw, db and dgate at the depth of the sums: a thread's share of a CTA's rows, the groups of a
    CTA (16 at most), the CTAs in slices, and a few roundings per term."""
    rng = np.random.default_rng([d, K])
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    depth = -(-K // sms) + 16 + 8 + 32 + 8
    x, dy = draw(rng, K, d, add=0.3), draw(rng, K, d)
    w, b, gate = (draw(rng, d, scale=0.2, add=1.0) for _ in range(3))
    K_d, ws = dev_i32(K), torch.empty(lemo.lemo_norm_workspace_size(d), dtype=torch.uint8, device="cuda")
    stats, out = torch.zeros(K, 2, device="cuda"), torch.empty(K, d, dtype=torch.bfloat16, device="cuda")
    norm, s = NORM["layer"], 0.75
    lemo.lemo_norm_gather(norm, bf16(x), bf16(w), bf16(b), EPS, None, K_d, 1, out, stats=stats)
    dw, db, dw2, db2, dg = (torch.zeros(d, device="cuda") for _ in range(5))
    lemo.lemo_norm_gather_backward(norm, bf16(dy), bf16(w), stats, None, K_d, torch.zeros_like(out), ws, x=bf16(x),
                                   dweight=dw, dbias=db)
    lemo.lemo_norm_scatter_backward(norm, bf16(dy), bf16(w), bf16(b), stats, bf16(gate), s, None, K_d, 1, out, ws,
                                    y=bf16(x), dweight=dw2, dbias=db2, dgate=dg)
    ok()
    st = f64(stats)
    vhat = (x - st[:, :1]) * st[:, 1:]
    # vhat: the difference and the product, each half a step of what goes in
    vsize = (np.abs(x) + np.abs(st[:, :1])) * st[:, 1:]
    u = depth * U32
    sums = {"dw": (dw, dy * vhat, np.abs(dy) * vsize), "db": (db, dy, np.abs(dy)),
            "dw2": (dw2, s * dy * gate * vhat, np.abs(s * dy * gate) * vsize),
            "db2": (db2, s * dy * gate, np.abs(s * dy * gate)),
            "dgate": (dg, s * dy * (vhat * w + b), np.abs(s * dy) * (vsize * np.abs(w) + np.abs(b)))}
    for what, (got, terms, size) in sums.items():
        want, bound = terms.sum(0), u * size.sum(0)
        within(f64(got), want, bound, what)
        # it refuses partial sums held in 16 bits
        rough = torch.from_numpy(want).bfloat16().double().numpy()
        assert (np.abs(rough - want) > bound).any(), what
