"""The bounded waits of the sublayer kernels: with one arrival withheld they run out, the call
ends and reports it, what other clusters wrote is right, and so is the next call."""

import numpy as np
import pytest
import torch

from contextual_token_sparsity_b200 import lemo
from sublayer_common import bf16, dev_i32, draw, make_ckpt, ok

pytestmark = pytest.mark.gpu
LIMIT_NS = 50_000_000


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    lemo.lemo_set_test_hooks(-1, 0)
    lemo.lemo_set_sublayer_test_hook(False)


def withheld(call):
    """The call's outputs with one arrival withheld, after the status was checked."""
    try:
        lemo.lemo_set_test_hooks(-1, LIMIT_NS)
        lemo.lemo_set_sublayer_test_hook(True)
        out = call()
        assert lemo.lemo_get_error() == lemo.LEMO_ERR_TIMEOUT
    finally:
        lemo.lemo_set_sublayer_test_hook(False)
        lemo.lemo_set_test_hooks(-1, 0)
    return out


# K = 100: the loads are all under way before a wait runs out; 8192 rows are split over the pairs
# of a cluster (512 x 264) or go over several tiles of a pair (4104 x 5128)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("K,rows,n,d", [(100, 100, 264, 520), (8192, 8192, 512, 264),
                                        (300, 8192, 136, 72), (700, 700, 4104, 5128)])
def test_weight_grad(K, rows, n, d, fmt):
    rng = np.random.default_rng([K, n, d])
    ck, _, _ = make_ckpt(rows, d, fmt)
    lemo.lemo_checkpoint_save(bf16(draw(rng, rows, d)), None, dev_i32(K), ck)
    dy, K_d = bf16(draw(rng, rows, n)), dev_i32(K)

    def call():
        dw = torch.zeros(n, d, device="cuda")
        lemo.lemo_checkpoint_weight_grad(ck, dy, K_d, dw)
        return dw

    want = call()
    ok()
    got = withheld(call)
    missing = got != want
    assert missing.any() and (got[missing] == 0).all()     # the first cluster added nothing
    assert missing[0, 0]
    again = call()
    ok()
    assert torch.equal(want, again)


# enough rows that every CTA uses its first slot again: at most 8 slots of 32 (d <= 256), 16
# (512 and below), 8 (1024), 4, 2 or 1 rows on each of up to 296 CTAs
@pytest.mark.parametrize("d,K", [(64, 80000), (512, 40000), (1000, 20000), (2048, 11000), (4096, 6000),
                                 (5120, 5000), (8192, 5000), (16384, 2600)])
def test_norms(d, K):
    """The first CTA goes on without rows: its later rows are left as they were, everything else is
    the same."""
    rng = np.random.default_rng(d)
    norm = lemo.LEMO_NORM_LAYER
    g = torch.Generator("cuda").manual_seed(d)
    x, dy = (torch.randn(K, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w, K_d = bf16(draw(rng, d, add=1.0)), dev_i32(K)
    ck, data, scales = make_ckpt(K, d, "int8")
    stats = torch.zeros(K, 2, device="cuda")
    ws = torch.empty(lemo.lemo_norm_workspace_size(d), dtype=torch.uint8, device="cuda")

    def gather():
        y, st = torch.zeros_like(x), torch.zeros_like(stats)
        lemo.lemo_norm_gather(norm, x, w, None, 1e-5, None, K_d, 1, y, stats=st)
        return y, st

    def scatter():
        z = torch.zeros_like(x)
        lemo.lemo_norm_scatter(norm, z, x, w, None, 1e-5, None, 1.0, None, K_d)
        return (z,)

    def gather_backward(saved=False):
        dx, dw = torch.zeros_like(x), torch.zeros(d, device="cuda")
        lemo.lemo_norm_gather_backward(norm, dy, w, stats, None, K_d, dx, ws, x=None if saved else x,
                                       checkpoint=ck if saved else None, dweight=dw)
        return dx, dw

    def scatter_backward():
        dv, dg = torch.zeros_like(x), torch.zeros(d, device="cuda")
        lemo.lemo_norm_scatter_backward(norm, dy, w, None, stats, w, 0.5, None, K_d, 1, dv, ws, y=x, dgate=dg)
        return dv, dg

    lemo.lemo_norm_gather(norm, x, w, None, 1e-5, None, K_d, 1, torch.empty_like(x), stats=stats, checkpoint=ck)
    for call in (gather, scatter, gather_backward, lambda: gather_backward(True), scatter_backward):
        want = call()
        ok()
        got = withheld(call)
        missing = (got[0] != want[0]).any(1)
        assert missing.any() and (got[0][missing] == 0).all()
        # the first CTA's share at most: one CTA of an SM each, at least 100 of them
        assert int(missing.sum()) <= K // 100
        again = call()
        ok()
        assert all(torch.equal(a, b) for a, b in zip(want, again))
