"""What the binding of the sublayer operators refuses, on CPU tensors that stand for device
tensors (the check of the device is told so): the library is not reached."""

import os
import shutil

import pytest
import torch

from contextual_token_sparsity_b200 import build as lemo_build
from contextual_token_sparsity_b200 import lemo

BAD = lemo.LEMO_ERR_INVALID_ARG


@pytest.fixture(autouse=True)
def on_cpu(monkeypatch):
    if shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc"):
        lemo_build.build()
    if not os.path.exists(lemo.LIB_PATH):
        pytest.skip("liblemo.so not built and nvcc unavailable")
    monkeypatch.setattr(lemo, "_device", lambda: -1)


def refused(fn, *a, **kw):
    with pytest.raises(lemo.LemoError) as e:
        fn(*a, **kw)
    assert e.value.status == BAD
    return str(e.value)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


@pytest.mark.parametrize("d", [8, 24, 40, 136])
def test_a_checkpoints_last_row_reaches_its_last_16_bytes(d):
    """Codes are read 16 bytes at a time; d is 8 past a multiple of 16 here."""
    ld = d + 8
    scales = u8(5, 8)
    # rows that are not followed by the bytes up to the next multiple of 16
    assert "16" in refused(lemo.make_checkpoint, u8(1, d), scales[:1], 0, d)
    flat = u8(5 * ld)
    for rows in (1, 2, 5):
        short = flat[: rows * ld - 8].clone().as_strided((rows, d), (ld, 1))
        refused(lemo.make_checkpoint, short, scales[:rows], 0, d)
        for good in (flat[: rows * ld].clone().as_strided((rows, d), (ld, 1)), u8(rows, ld)[:, :d],
                     u8(rows, ld), flat.as_strided((rows, d), (ld, 1), (5 - rows) * ld)):
            c = lemo.make_checkpoint(good, scales[:rows], 0, d)
            assert c.struct.ld_data == ld and c.rows == rows and c.d == d
    assert lemo.make_checkpoint(u8(1, 2 * ld)[:, :d], scales[:1], 0, d).struct.ld_data % 16 == 0
    assert lemo.make_checkpoint(u8(0, ld), scales[:0], 1, d).rows == 0


def test_missing_and_misshaped_arguments_raise_the_bindings_error():
    """None, another rank, an address or a number in place of a tensor, and anything that is no
    Checkpoint: LemoError(LEMO_ERR_INVALID_ARG) that names the argument."""
    x, K = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    ws, v = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(64)
    st = torch.zeros(4, 2)
    c = lemo.make_checkpoint(u8(4, 64), u8(4, 4), 0, 64)
    calls = {
        "lemo_norm_gather": dict(norm=1, x=x, weight=None, bias=None, eps=0.1, kept_idx=None, kept_total=K,
                                 pad_to=1, y=x, stats=st, checkpoint=c),
        "lemo_norm_gather_backward": dict(norm=1, dy=x, weight=None, stats=st, kept_idx=None, kept_total=K,
                                          dx=x, ws=ws, x=None, checkpoint=c, dweight=v, dbias=v),
        "lemo_norm_scatter": dict(norm=1, x=x, y=x, weight=None, bias=None, eps=0.1, gate=x, scale=1.0,
                                  kept_idx=None, kept_total=K, stats=st, checkpoint=c),
        "lemo_norm_scatter_backward": dict(norm=1, dx=x, weight=None, bias=None, stats=st, gate=x, scale=1.0,
                                           kept_idx=None, kept_total=K, pad_to=1, dy=x, ws=ws, y=None,
                                           checkpoint=c, dweight=v, dbias=v, dgate=x),
        "lemo_checkpoint_save": dict(x=x, kept_idx=None, kept_total=K, checkpoint=c),
        "lemo_checkpoint_restore": dict(checkpoint=c, kept_total=K, pad_to=1, y=x),
        "lemo_gated_mlp": dict(gate=x, up=x, kept_total=K, pad_to=1, a=x, gate_checkpoint=c, up_checkpoint=c),
        "lemo_gated_mlp_backward": dict(gate_checkpoint=c, up_checkpoint=c, da=x, kept_total=K, pad_to=1,
                                        dgate=x, dup=x, a=x),
        "lemo_checkpoint_weight_grad": dict(checkpoint=c, dy=x, kept_total=K, dw=torch.zeros(64, 64)),
    }
    optional = {"weight", "bias", "kept_idx", "stats", "gate", "dweight", "dbias", "dgate", "a", "x", "y",
                "checkpoint", "gate_checkpoint", "up_checkpoint"}
    needed = {"lemo_norm_gather": {"x", "y"}, "lemo_norm_gather_backward": {"dy", "dx", "ws", "kept_total"},
              "lemo_norm_scatter": {"x", "y"}, "lemo_norm_scatter_backward": {"dx", "dy", "ws"},
              "lemo_checkpoint_save": {"x", "checkpoint"}, "lemo_checkpoint_restore": {"y", "checkpoint"},
              "lemo_gated_mlp": {"gate", "up", "a"},
              "lemo_gated_mlp_backward": {"gate_checkpoint", "up_checkpoint", "da", "dgate", "dup"},
              "lemo_checkpoint_weight_grad": {"checkpoint", "dy", "dw"}}
    scalars = {"norm", "eps", "pad_to", "scale"}
    for name, good in calls.items():
        for arg in good:
            if arg in scalars:
                continue
            wrong = [0x10000, 1.5, "rows", torch.zeros(2, 2, 2, dtype=torch.bfloat16), torch.zeros(())]
            if arg == "ws":         # any contiguous tensor of enough bytes
                wrong = wrong[:3]
            if arg not in optional or arg in needed[name]:
                wrong.append(None)
            for bad in wrong:
                text = refused(getattr(lemo, name), **{**good, arg: bad})
                assert text.startswith(name + ":") and f" {arg} " in text, (name, arg, bad, text)
    for bad in (None, 0x10000, "rows", torch.zeros(4, dtype=torch.uint8), torch.zeros(4, 64)):
        assert " data " in refused(lemo.make_checkpoint, bad, u8(4, 4), 0, 64)
        assert " scales " in refused(lemo.make_checkpoint, u8(4, 64), bad, 0, 64)
