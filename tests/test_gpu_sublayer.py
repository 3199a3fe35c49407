"""A run of the sublayer operators together, as a training step of a gated MLP
on the kept tokens uses them: scores -> selection -> pre-norm gather -> gate,
up and down projections (plain matrix products) -> post-norm scatter, then the
backward pass from 8-bit checkpoints.  Every step is compared with the float64
oracle on that step's own inputs, and the weight gradients with those of the
unquantised activations by an inequality of norms."""

import numpy as np
import pytest
import torch

from contextual_token_sparsity_b200 import lemo, synth
from contextual_token_sparsity_b200.pipeline import Layer, to_device_bf16
from oracle import sublayer_oracle as so
from sublayer_common import (EPS, U16, U32, back_slop, bf16, ckpt_values, draw, f64, norm_slop, ok,
                             within)

pytestmark = pytest.mark.gpu
RMS, LAYERNORM = lemo.LEMO_NORM_RMS, lemo.LEMO_NORM_LAYER


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    lemo.lemo_set_test_hooks(-1, 0)


def _mm(a, b):
    """bf16 product a b^T of padded rows (the caller's GEMM)."""
    return a @ b.t()


@pytest.mark.parametrize("fmt", [lemo.LEMO_CHECKPOINT_E4M3, lemo.LEMO_CHECKPOINT_INT8])
def test_training_step_of_a_gated_mlp_sublayer(fmt):
    lengths, H, dh, b, d, dff = [300, 1, 517], 4, 64, 64, 256, 640
    name = "e4m3" if fmt == lemo.LEMO_CHECKPOINT_E4M3 else "int8"
    rng = np.random.default_rng([fmt, 9])
    L = sum(lengths)
    layer = Layer(lengths, H, dh, b, d)
    q, k, _, _ = synth.qk_direct(lengths, H, dh, [0.1, 0.0, 0.1], seed=3)
    layer.score(to_device_bf16(q), to_device_bf16(k))
    theta = float(layer.block_scores.median())
    layer.select(theta)
    ok()
    K = int(layer.kept_total.item())
    idx = layer.kept_idx[:K].cpu().numpy()
    assert 0 < K < L
    rows = layer.y_rows

    x0, w1, w2 = draw(rng, L, d), draw(rng, d, scale=0.1, add=1.0), draw(rng, d, scale=0.1, add=1.0)
    b1, gate = draw(rng, d, scale=0.1), draw(rng, d, scale=0.1, add=0.5)
    wg, wu, wd = (draw(rng, n, m, scale=m ** -0.5) for n, m in ((dff, d), (dff, d), (d, dff)))
    x = bf16(x0)
    W = [bf16(t) for t in (wg, wu, wd)]
    scale = 0.7

    # forward
    cx, cy, cg, cu, ca, co = (layer.checkpoint(fmt, n) for n in (d, d, dff, dff, dff, d))
    y = layer.gather_norm(LAYERNORM, x, bf16(w1), bf16(b1), EPS, checkpoint=cx)
    lemo.lemo_checkpoint_save(y, None, layer.kept_total, cy)
    g, u = _mm(y, W[0]), _mm(y, W[1])
    a = torch.empty(rows, dff, dtype=torch.bfloat16, device="cuda")
    lemo.lemo_gated_mlp(g, u, layer.kept_total, layer.pad_to, a, cg, cu)
    lemo.lemo_checkpoint_save(a, None, layer.kept_total, ca)
    o = _mm(a, W[2])
    layer.scatter_norm(RMS, x, o, bf16(w2), None, EPS, gate=bf16(gate), scale=scale, checkpoint=co)
    ok()
    v = x0[idx]
    n1, mean, rstd = so.norm_rows(v, "layer", EPS, w1, b1)
    within(f64(y)[:K], n1, U16 * np.abs(n1) + 1.01 * norm_slop(v, mean, rstd, w1, b1), "y")
    yv, gv, uv, av, ov = (f64(t)[:K] for t in (y, g, u, a, o))
    want = so.gated(gv, uv)
    within(av, want, U16 * np.abs(want) + 17 * U32 * np.abs(want) * (1 + np.abs(gv)), "a")
    n2, _, rstd2 = so.norm_rows(ov, "rms", EPS, w2, None)
    want = x0.copy()
    want[idx] += scale * gate * n2
    slop = np.zeros_like(want)
    slop[idx] = 1.01 * np.abs(scale * gate) * norm_slop(ov, 0 * rstd2, rstd2, w2, None) + 4 * U32 * np.abs(x0[idx])
    bound = U16 * np.abs(want) + slop
    bound[np.setdiff1d(np.arange(L), idx)] = 0
    within(f64(x), want, bound, "x")
    for c, t in ((cx, v), (cy, yv), (cg, gv), (cu, uv), (ca, av), (co, ov)):
        val, codes = so.checkpoint_codes(t, name)
        got, e = ckpt_values(c, K)
        assert np.array_equal(e, codes) and np.array_equal(got, val)

    # backward
    dx0 = draw(rng, L, d, scale=0.1)
    dx = bf16(dx0)
    grads = [torch.zeros(s, device="cuda") for s in (d, d, d, d)]
    dw1, db1, dw2, dgate = grads
    dWg, dWu, dWd = (torch.zeros(t.shape, device="cuda") for t in W)
    do = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    layer.scatter_norm_backward(RMS, dx, do, bf16(w2), None, gate=bf16(gate), scale=scale,
                                checkpoint=co, dweight=dw2, dgate=dgate)
    lemo.lemo_checkpoint_weight_grad(ca, do, layer.kept_total, dWd)
    da = _mm(do, W[2].t())
    dg, du = torch.empty_like(a), torch.empty_like(a)
    lemo.lemo_gated_mlp_backward(cg, cu, da, layer.kept_total, layer.pad_to, dg, du)
    lemo.lemo_checkpoint_weight_grad(cy, dg, layer.kept_total, dWg)
    lemo.lemo_checkpoint_weight_grad(cy, du, layer.kept_total, dWu)
    dy = _mm(dg, W[0].t()) + _mm(du, W[1].t())
    layer.gather_norm_backward(LAYERNORM, dy, dx, bf16(w1), checkpoint=cx, dweight=dw1, dbias=db1)
    ok()

    qx, qy, qg, qu, qa, qo = (ckpt_values(c, K)[0] for c in (cx, cy, cg, cu, ca, co))
    st2, st1 = f64(layer.post_stats)[:K], f64(layer.pre_stats)[:K]
    dz = scale * dx0[idx]
    dn = dz * gate
    vhat = (qo - st2[:, :1]) * st2[:, 1:]
    want, rw2, _ = so.norm_backward(dn, qo, st2[:, 0], st2[:, 1], "rms", w2)
    within(f64(do)[:K], want, U16 * np.abs(want) + 1.01 * back_slop(dn * w2, vhat, st2[:, 1], "rms"), "do")
    assert (f64(do)[K: -(-K // layer.pad_to) * layer.pad_to] == 0).all()
    within(f64(dw2), rw2, (K + 8) * U32 * np.abs(dn * vhat).sum(0), "dw2")
    within(f64(dgate), (dz * vhat * w2).sum(0), (K + 8) * U32 * np.abs(dz * vhat * w2).sum(0), "dgate")
    dov, dav, dgv, duv, dyv = (f64(t)[:K] for t in (do, da, dg, du, dy))
    rg, ru, _ = so.gated_backward(qg, qu, dav)
    s = 1 / (1 + np.exp(-qg))
    size = np.abs(dav * qu) * (s + 2 * np.abs(qg) * s * (1 - s)) * (1 + np.abs(qg))
    within(dgv, rg, U16 * np.abs(rg) + 17 * U32 * size, "dg")
    within(duv, ru, U16 * np.abs(ru) + 17 * U32 * np.abs(ru) * (1 + np.abs(qg)), "du")
    for got, gr, act, exact in ((dWd, dov, qa, av), (dWg, dgv, qy, yv), (dWu, duv, qy, yv)):
        within(f64(got), so.weight_grad(gr, act), 2 * (K + 8) * U32 * (np.abs(gr).T @ np.abs(act)), "dW")
        # against the activations themselves: |dy^T (q - a)|_F <= |dy|_2 |q - a|_F
        off = np.linalg.norm(f64(got) - so.weight_grad(gr, exact))
        assert off <= np.linalg.norm(gr, 2) * np.linalg.norm(act - exact) * 1.001 + 1e-4 * np.linalg.norm(got.cpu())
    vhat = (qx - st1[:, :1]) * st1[:, 1:]
    dv, rw1, rb1 = so.norm_backward(dyv, qx, st1[:, 0], st1[:, 1], "layer", w1)
    want = dx0.copy()
    want[idx] += dv
    slop = np.zeros_like(want)
    slop[idx] = 1.01 * back_slop(dyv * w1, vhat, st1[:, 1], "layer") + 4 * U32 * np.abs(dx0[idx])
    bound = U16 * np.abs(want) + slop
    bound[np.setdiff1d(np.arange(L), idx)] = 0
    within(f64(dx), want, bound, "dx")
    within(f64(dw1), rw1, (K + 8) * U32 * np.abs(dyv * vhat).sum(0), "dw1")
    within(f64(db1), rb1, (K + 8) * U32 * np.abs(dyv).sum(0), "db1")


def test_nothing_kept():
    """A threshold above every score: no row moves, gradients of weights stay, tails are empty."""
    layer = Layer([200], 1, 64, 64, 128)
    layer.block_scores.zero_()
    layer.select(1.0)
    x = bf16(draw(np.random.default_rng(0), 200, 128))
    before = x.clone()
    layer.y.fill_(3.0)
    c = layer.checkpoint(lemo.LEMO_CHECKPOINT_INT8)
    layer.gather_norm(RMS, x, checkpoint=c)
    layer.scatter_norm(LAYERNORM, x, layer.y)
    dw = torch.ones(128, device="cuda")
    dy = torch.full_like(layer.y, 5.0)
    layer.scatter_norm_backward(LAYERNORM, x, dy, y_out=layer.y, dweight=dw)
    layer.gather_norm_backward(RMS, layer.y, x, checkpoint=c, dweight=dw)
    dW = torch.ones(64, 128, device="cuda")
    lemo.lemo_checkpoint_weight_grad(c, layer.y[:, :64], layer.kept_total, dW)
    ok()
    assert int(layer.kept_total.item()) == 0
    assert torch.equal(x, before) and (layer.y == 3).all() and (dy == 5).all()
    assert (dw == 1).all() and (dW == 1).all()


def test_two_streams_with_their_own_buffers():
    """Two calls that may overlap: separate streams, outputs and workspaces."""
    rng = np.random.default_rng(1)
    d, L = 1024, 2000
    K_d = torch.tensor([L], dtype=torch.int32, device="cuda")
    x, w = bf16(draw(rng, L, d)), bf16(draw(rng, d, add=1.0))
    dy = [bf16(draw(rng, L, d)) for _ in range(2)]
    y = torch.empty(L, d, dtype=torch.bfloat16, device="cuda")
    stats = torch.empty(L, 2, device="cuda")
    lemo.lemo_norm_gather(RMS, x, w, None, EPS, None, K_d, 1, y, stats=stats)
    out = []
    for parallel in (False, True):
        dx = [torch.zeros(L, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        dw = [torch.zeros(d, device="cuda") for _ in range(2)]
        ws = [torch.empty(lemo.lemo_norm_workspace_size(d), dtype=torch.uint8, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for i in range(2):
            st = streams[i] if parallel else None
            lemo.lemo_norm_gather_backward(RMS, dy[i], w, stats, None, K_d, dx[i], ws[i], x=x,
                                           dweight=dw[i], stream=st)
        torch.cuda.synchronize()
        out.append((dx, dw))
    ok()
    for i in range(2):
        assert torch.equal(out[0][0][i], out[1][0][i]) and torch.equal(out[0][1][i], out[1][1][i])


def test_weight_grad_in_two_graphs():
    """Captured calls read the device's row count at replay; the kernel has no workspace to share."""
    rng = np.random.default_rng(2)
    rows, n, d = 2300, 520, 264
    v, g = draw(rng, rows, d), draw(rng, rows, n)
    K_d = torch.tensor([rows], dtype=torch.int32, device="cuda")
    c = lemo.make_checkpoint(torch.zeros(rows, 272, dtype=torch.uint8, device="cuda"),
                             torch.zeros(rows, 12, dtype=torch.uint8, device="cuda"), 0, d)
    lemo.lemo_checkpoint_save(bf16(v), None, K_d, c)
    dy, dw = bf16(g), [torch.zeros(n, d, device="cuda") for _ in range(2)]
    lemo.lemo_checkpoint_weight_grad(c, dy, K_d, dw[0])
    ok()
    side = torch.cuda.Stream()
    graphs = []
    for i in range(2):
        side.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.stream(side), torch.cuda.graph(graphs[i], stream=side):
            lemo.lemo_checkpoint_weight_grad(c, dy, K_d, dw[i])
    torch.cuda.current_stream().wait_stream(side)
    q, _ = so.checkpoint_codes(v, "e4m3")
    for K in (rows, 77, 0, 1500):
        K_d.fill_(K)
        for t in dw:
            t.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        want = so.weight_grad(g[:K], q[:K])
        for t in dw:
            within(f64(t), want, 2 * (K + 8) * U32 * (np.abs(g[:K]).T @ np.abs(q[:K])))
    ok()


def test_offsets_past_32_bits():
    """Row strides that put the last rows more than 2^31 elements (2^32 bytes) behind the first."""
    rng = np.random.default_rng(3)
    d, ld, rows = 64, 1 << 17, 33000            # 33000 x 131072 = 4.3e9 elements
    idx = np.array([0, 5, 16385, 32766, 32999], dtype=np.int32)
    K = len(idx)
    K_d, idx_d = torch.tensor([K], dtype=torch.int32, device="cuda"), torch.from_numpy(idx).cuda()
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").as_strided((rows, d), (ld, 1))
    v = draw(rng, K, d)
    big[idx_d.long()] = bf16(v)
    y = torch.zeros(K, d, dtype=torch.bfloat16, device="cuda")
    stats = torch.zeros(K, 2, device="cuda")
    lemo.lemo_norm_gather(RMS, big, None, None, EPS, idx_d, K_d, 1, y, stats=stats, d=d)
    n, mean, rstd = so.norm_rows(v, "rms", EPS)
    within(f64(y), n, U16 * np.abs(n) + 1.01 * norm_slop(v, mean, rstd, None, None), "y")
    lemo.lemo_norm_scatter(lemo.LEMO_NORM_NONE, big, y, None, None, EPS, None, 1.0, idx_d, K_d, d=d)
    got, yv = f64(big[idx_d.long()]), f64(y)
    within(got, v + yv, U16 * np.abs(v + yv), "x")
    # a checkpoint whose rows are as far apart, its kept rows the last ones
    del big
    whole = torch.empty(rows * ld, dtype=torch.uint8, device="cuda").as_strided((rows, d), (ld, 1))
    c = lemo.make_checkpoint(whole, torch.zeros(rows, 4, dtype=torch.uint8, device="cuda"), 1, d)
    x = bf16(draw(rng, rows, d))
    R_d = torch.tensor([rows], dtype=torch.int32, device="cuda")
    lemo.lemo_checkpoint_save(x, None, R_d, c)
    back = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    lemo.lemo_checkpoint_restore(c, R_d, 1, back)
    ok()
    want, _ = so.checkpoint_codes(f64(x[-40:]), "int8")
    assert np.array_equal(f64(back[-40:]), want)
    dy = bf16(draw(rng, rows, 8))
    dw = torch.zeros(8, d, device="cuda")
    lemo.lemo_checkpoint_weight_grad(c, dy, R_d, dw)
    ok()
    a, b = f64(dy), f64(back)
    within(f64(dw), a.T @ b, 2 * (rows + 8) * U32 * (np.abs(a).T @ np.abs(b)), "dw")


@pytest.mark.parametrize("d", [64, 1000, 4096, 8192])
def test_a_wait_that_runs_out_is_reported(d):
    """With a limit of a nanosecond some waits of the norm kernels' rings run out: their warps
    go on without rows, the calls end, and the next ones are right."""
    rng = np.random.default_rng(d)
    K = 700
    K_d = torch.tensor([K], dtype=torch.int32, device="cuda")
    x, dy = bf16(draw(rng, K, d)), bf16(draw(rng, K, d))
    c = lemo.make_checkpoint(torch.zeros(K, -(-d // 16) * 16, dtype=torch.uint8, device="cuda"),
                             torch.zeros(K, -(-d // 128) * 4, dtype=torch.uint8, device="cuda"), 1, d)
    ws = torch.empty(lemo.lemo_norm_workspace_size(d), dtype=torch.uint8, device="cuda")

    def calls():
        y, dx = torch.zeros_like(x), torch.zeros_like(x)
        stats, dw = torch.zeros(K, 2, device="cuda"), torch.zeros(d, device="cuda")
        lemo.lemo_norm_gather(LAYERNORM, x, None, None, EPS, None, K_d, 1, y, stats=stats, checkpoint=c)
        lemo.lemo_norm_gather_backward(LAYERNORM, dy, None, stats, None, K_d, dx, ws, x=x, dweight=dw)
        return y, stats, dx, dw

    want = calls()
    ok()
    try:
        lemo.lemo_set_test_hooks(-1, 1)
        calls()
        assert lemo.lemo_get_error() in (lemo.LEMO_OK, lemo.LEMO_ERR_TIMEOUT)
    finally:
        lemo.lemo_set_test_hooks(-1, 0)
    got = calls()
    ok()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
