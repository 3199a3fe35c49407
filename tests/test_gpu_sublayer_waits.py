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
