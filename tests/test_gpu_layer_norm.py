"""pipeline.Layer with norms on a GPU: sublayers that share one Layer."""

import ctypes

import numpy as np
import pytest
import torch

from contextual_token_sparsity_b200 import lemo
from contextual_token_sparsity_b200.pipeline import Layer
from sublayer_common import EPS, bf16, draw, ok

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


def _layer(lengths, d):
    layer = Layer(lengths, 1, 64, 64, d)
    layer.block_scores.copy_(torch.arange(layer.total_blocks, device="cuda") % 3)
    layer.select(0.5)
    ok()
    assert 0 < int(layer.kept_total.item()) < layer.total_L
    return layer


@pytest.mark.parametrize("saved", [False, True])
def test_two_sublayers_on_one_layer(saved):
    """Both forward passes before the first backward pass: every gradient is the one that a
    Layer per sublayer gives, bit for bit."""
    rng = np.random.default_rng([6, saved])
    lengths, d = [300, 129], 264
    L = sum(lengths)
    one, apart = _layer(lengths, d), [_layer(lengths, d) for _ in range(2)]
    rows = one.y_rows
    x0 = [bf16(draw(rng, L, d, scale=s)) for s in (1.0, 5.0)]      # statistics that differ
    o = [bf16(draw(rng, rows, d, scale=s, add=0.5)) for s in (0.2, 3.0)]
    w = [bf16(draw(rng, d, add=1.0)) for _ in range(4)]
    dy = [bf16(draw(rng, rows, d)) for _ in range(2)]
    dx0 = bf16(draw(rng, L, d))
    fmt = lemo.LEMO_CHECKPOINT_E4M3

    def run(layers, stats):
        grads, cks = [], []
        x = [t.clone() for t in x0]
        for i, layer in enumerate(layers):
            cks.append([layer.checkpoint(fmt) if saved else None for _ in range(2)])
            layer.gather_norm(RMS, x[i], w[i], None, EPS, checkpoint=cks[i][0], stats=stats[i][0])
            layer.scatter_norm(LAYERNORM, x[i], o[i], w[2 + i], None, EPS, checkpoint=cks[i][1],
                               stats=stats[i][1])
        for i in (1, 0):
            layer, dx = layers[i], dx0.clone()
            do, dw = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, d, device="cuda")
            layer.scatter_norm_backward(LAYERNORM, dx, do, w[2 + i], y_out=None if saved else o[i],
                                        checkpoint=cks[i][1], dweight=dw[0], dbias=dw[1], stats=stats[i][1])
            layer.gather_norm_backward(RMS, dy[i], dx, w[i], x=None if saved else x0[i],
                                       checkpoint=cks[i][0], dweight=dw[2], stats=stats[i][0])
            grads += [dx, do, dw]
        ok()
        return grads

    want = run(apart, [(None, None)] * 2)
    got = run([one, one], [[one.norm_stats() for _ in range(2)] for _ in range(2)])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # with the other call's statistics they are not (what the shared buffer used to give)
    wrong = run([one, one], [[s, t] for s, t in [(one.norm_stats(), one.norm_stats())]] * 2)
    assert not any(torch.equal(a, b) for a, b in zip(want[3:], wrong[3:]))


def test_backward_calls_on_two_streams(monkeypatch):
    """Calls of one Layer on two streams, and in two graphs, run on workspaces of their own and
    give what they give one after the other."""
    rng = np.random.default_rng(7)
    lengths, d = [1500, 700], 1024
    L = sum(lengths)
    layer = _layer(lengths, d)
    x, w = bf16(draw(rng, L, d)), bf16(draw(rng, d, add=1.0))
    dy = [bf16(draw(rng, layer.y_rows, d)) for _ in range(2)]
    layer.gather_norm(RMS, x, w)
    used, call = [], lemo.lemo_norm_gather_backward

    def spy(*a, **kw):
        used.append(a[7].data_ptr())
        call(*a, **kw)

    monkeypatch.setattr(lemo, "lemo_norm_gather_backward", spy)
    dx = [torch.zeros(L, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dw = [torch.zeros(d, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def run(where):
        for t in dx + dw:
            t.zero_()
        torch.cuda.synchronize()
        used.clear()
        where()
        torch.cuda.synchronize()
        ok()
        return [t.clone() for t in dx + dw]

    def back(i, stream=None):
        layer.gather_norm_backward(RMS, dy[i], dx[i], w, x=x, dweight=dw[i], stream=stream)

    want = run(lambda: [back(i) for i in range(2)])
    for handles in (streams, [s.cuda_stream for s in streams]):
        got = run(lambda: [back(i, handles[i]) for i in range(2)])
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert used[0] != used[1]
    assert all(torch.equal(a, b) for a, b in zip(want, run(lambda: [back(i, 0) for i in range(2)])))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    used.clear()
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            back(i)
    assert used[0] != used[1]

    def replay():
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()

    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, run(replay)))


def test_no_room_for_any_row():
    """Buffers of no rows: nothing is touched, and a kept total above zero is reported by every call
    of the shared rule."""
    lib = lemo.load()
    d = 64
    full, none = torch.ones(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    mem = torch.full((4, d), 3.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.ones(d, d, device="cuda")
    u8 = torch.zeros(4, d, dtype=torch.uint8, device="cuda")
    c = lemo.lemo_checkpoint(0, d, u8.data_ptr(), d, u8.data_ptr(), 4, 0)
    ck, m = ctypes.addressof(c), mem.data_ptr()
    for total, status in ((full, lemo.LEMO_ERR_CAPACITY), (none, lemo.LEMO_OK)):
        K = total.data_ptr()
        calls = [lambda: lib.lemo_checkpoint_weight_grad(ck, m, d, 0, d, K, dw.data_ptr(), d, None),
                 lambda: lib.lemo_checkpoint_restore(ck, K, 1, m, d, 0, None),
                 lambda: lib.lemo_checkpoint_save(m, d, 4, None, K, ck, None),
                 lambda: lib.lemo_gated_mlp(m, d, m, d, d, K, 1, m, d, 0, None, None, None),
                 lambda: lib.lemo_norm_gather(RMS, m, d, 4, d, None, None, EPS, None, K, 1, m, d, 0, None, None,
                                              None)]
        for call in calls:
            assert call() == lemo.LEMO_OK and lemo.lemo_get_error() == status
    assert (mem == 3).all() and (dw == 1).all() and (u8 == 0).all()
