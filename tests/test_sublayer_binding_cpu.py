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
