"""CPU checks of the sublayer operators' refusals: every bad argument comes
back from the host before anything is enqueued (no GPU is needed: the calls
below must not reach CUDA), and the binding refuses tensors that do not fit."""

import ctypes
import os
import shutil

import pytest
import torch

from contextual_token_sparsity_b200 import build as lemo_build
from contextual_token_sparsity_b200 import lemo

BAD, NO = lemo.LEMO_ERR_INVALID_ARG, lemo.LEMO_ERR_UNSUPPORTED
BUF = 0x10000  # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc"):
        lemo_build.build()
    if not os.path.exists(lemo.LIB_PATH):
        pytest.skip("liblemo.so not built and nvcc unavailable")
    return lemo.load()


def _ckpt(**kw):
    a = dict(format=0, d=64, data=BUF, ld_data=64, scales=BUF, ld_scales=4, rows=8)
    a.update(kw)
    return lemo.lemo_checkpoint(a["format"], a["d"], a["data"], a["ld_data"], a["scales"],
                                a["ld_scales"], a["rows"])


def _caller(fn, names, good):
    def call(**kw):
        a = dict(good)
        a.update(kw)
        keep = [v for v in a.values() if isinstance(v, ctypes.Structure)]
        args = [ctypes.addressof(a[n]) if isinstance(a[n], ctypes.Structure) else a[n] for n in names]
        st = fn(*args)
        del keep
        return st
    return call


BAD_CKPT = [dict(format=2), dict(format=-1), dict(d=72), dict(data=None), dict(data=BUF + 8),
            dict(ld_data=48), dict(ld_data=72), dict(scales=None), dict(scales=BUF + 2),
            dict(ld_scales=0), dict(ld_scales=6), dict(rows=3)]
BIG = 1 << 30


def test_norm_gather(lib):
    names = "norm x ld_x x_rows d w b eps idx total pad y ld_y rows stats ck st".split()
    good = dict(norm=1, x=BUF, ld_x=64, x_rows=8, d=64, w=BUF, b=None, eps=1e-5, idx=BUF, total=BUF,
                pad=1, y=BUF, ld_y=64, rows=8, stats=None, ck=None, st=None)
    call = _caller(lib.lemo_norm_gather, names, good)
    for kw in [dict(norm=0), dict(norm=3), dict(x=None), dict(y=None), dict(x=BUF + 2), dict(y=BUF + 8),
               dict(ld_x=56), dict(ld_y=68), dict(d=0), dict(rows=-1), dict(rows=1 << 40),
               dict(x_rows=-1), dict(w=BUF + 2), dict(b=BUF + 4), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(idx=BUF + 2), dict(total=None),
               dict(total=BUF + 1), dict(pad=0), dict(stats=BUF + 4)]:
        assert call(**kw) == BAD, kw
    assert call(d=60) == NO
    assert call(d=16392, ld_x=16392, ld_y=16392) == NO
    for kw in BAD_CKPT:
        assert call(ck=_ckpt(**kw)) == BAD, kw


def test_norm_workspace_size(lib):
    assert lemo.lemo_norm_workspace_size(4096) == 296 * 2 * 4096 * 4
    assert lemo.lemo_norm_workspace_size(8) == -(-296 * 2 * 8 * 4 // 256) * 256
    for d in (0, -8, 12, 16392):
        assert lemo.lemo_norm_workspace_size(d) == 0


def test_norm_gather_backward(lib):
    names = ("norm dy ld_dy rows d w stats idx total x ld_x x_rows ck dx ld_dx dx_rows dw db ws "
             "ws_bytes st").split()
    good = dict(norm=2, dy=BUF, ld_dy=64, rows=8, d=64, w=None, stats=BUF, idx=BUF, total=BUF, x=BUF,
                ld_x=64, x_rows=8, ck=None, dx=BUF, ld_dx=64, dx_rows=8, dw=BUF, db=BUF, ws=BUF,
                ws_bytes=BIG, st=None)
    call = _caller(lib.lemo_norm_gather_backward, names, good)
    for kw in [dict(norm=0), dict(norm=7), dict(dy=None), dict(dx=None), dict(stats=None),
               dict(stats=BUF + 4), dict(x=None), dict(x=BUF, ck=_ckpt()), dict(ld_dy=60),
               dict(ld_dx=8), dict(ld_x=32), dict(x_rows=-2), dict(dx_rows=-1), dict(dw=BUF + 2),
               dict(db=BUF + 1), dict(ws=None), dict(ws=BUF + 16), dict(ws_bytes=1024), dict(d=0),
               dict(total=None), dict(w=BUF + 2)]:
        assert call(**kw) == BAD, kw
    assert call(d=12) == NO and call(d=16392) == NO
    for kw in BAD_CKPT:
        assert call(x=None, ck=_ckpt(**kw)) == BAD, kw


def test_norm_scatter(lib):
    names = "norm x ld_x x_rows d y ld_y rows w b eps gate ld_gate scale idx total stats ck st".split()
    good = dict(norm=1, x=BUF, ld_x=64, x_rows=8, d=64, y=BUF, ld_y=64, rows=8, w=None, b=None,
                eps=1e-5, gate=BUF, ld_gate=0, scale=1.0, idx=BUF, total=BUF, stats=None, ck=None,
                st=None)
    call = _caller(lib.lemo_norm_scatter, names, good)
    for kw in [dict(norm=-1), dict(norm=3), dict(norm=0, w=BUF), dict(norm=0, b=BUF),
               dict(norm=0, stats=BUF), dict(x=None), dict(y=None), dict(ld_x=32), dict(ld_y=9),
               dict(gate=BUF + 2), dict(ld_gate=32), dict(ld_gate=66), dict(ld_gate=-64),
               dict(gate=None, ld_gate=64), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(eps=-1e-9), dict(total=None), dict(stats=BUF + 4), dict(x_rows=-1)]:
        assert call(**kw) == BAD, kw
    assert call(d=20) == NO and call(d=16392, ld_x=16392, ld_y=16392) == NO
    for kw in BAD_CKPT:
        assert call(ck=_ckpt(**kw)) == BAD, kw


def test_norm_scatter_backward(lib):
    names = ("norm dx ld_dx dx_rows d w b stats gate ld_gate scale idx total y ld_y ck pad dy ld_dy "
             "rows dw db dgate dgr ld_dgr ws ws_bytes st").split()
    good = dict(norm=2, dx=BUF, ld_dx=64, dx_rows=8, d=64, w=None, b=None, stats=BUF, gate=BUF,
                ld_gate=0, scale=1.0, idx=BUF, total=BUF, y=BUF, ld_y=64, ck=None, pad=1, dy=BUF,
                ld_dy=64, rows=8, dw=BUF, db=BUF, dgate=BUF, dgr=None, ld_dgr=0, ws=BUF,
                ws_bytes=BIG, st=None)
    call = _caller(lib.lemo_norm_scatter_backward, names, good)
    for kw in [dict(norm=-1), dict(norm=3), dict(norm=0), dict(stats=None), dict(stats=BUF + 4),
               dict(dx=None), dict(dy=None), dict(ld_dx=8), dict(ld_dy=65), dict(y=None),
               dict(ck=_ckpt()), dict(ld_y=8), dict(gate=None), dict(ld_gate=64),
               dict(gate=BUF + 2), dict(dgr=BUF, ld_dgr=64), dict(dgate=None, dgr=BUF, ld_dgr=64),
               dict(ld_gate=64, dgate=None, dgr=BUF, ld_dgr=32), dict(scale=float("nan")),
               dict(pad=0), dict(ws=None), dict(ws=BUF + 8), dict(ws_bytes=8), dict(dgate=BUF + 2),
               dict(total=None), dict(idx=BUF + 1), dict(dx_rows=-1)]:
        assert call(**kw) == BAD, kw
    assert call(d=12) == NO and call(d=16392) == NO
    for kw in BAD_CKPT:
        assert call(y=None, ck=_ckpt(**kw)) == BAD, kw


def test_checkpoint_save_and_restore(lib):
    names = "x ld_x x_rows idx total ck st".split()
    good = dict(x=BUF, ld_x=64, x_rows=8, idx=None, total=BUF, ck=_ckpt(), st=None)
    call = _caller(lib.lemo_checkpoint_save, names, good)
    for kw in [dict(x=None), dict(x=BUF + 8), dict(ld_x=32), dict(x_rows=-1), dict(total=None),
               dict(ck=None), dict(idx=BUF + 2), dict(ck=_ckpt(rows=-1)), dict(ck=_ckpt(d=0))]:
        assert call(**kw) == BAD, kw
    assert call(ck=_ckpt(d=12)) == NO
    for kw in BAD_CKPT[:2] + BAD_CKPT[3:-1]:
        assert call(ck=_ckpt(**kw)) == BAD, kw
    names = "ck total pad y ld_y rows st".split()
    call = _caller(lib.lemo_checkpoint_restore, names,
                   dict(ck=_ckpt(), total=BUF, pad=1, y=BUF, ld_y=64, rows=8, st=None))
    for kw in [dict(ck=None), dict(total=None), dict(pad=0), dict(y=None), dict(y=BUF + 2),
               dict(ld_y=32), dict(rows=9), dict(rows=-1)]:
        assert call(**kw) == BAD, kw


def test_gated_mlp(lib):
    names = "g ld_g u ld_u d total pad a ld_a rows cg cu st".split()
    call = _caller(lib.lemo_gated_mlp, names,
                   dict(g=BUF, ld_g=64, u=BUF, ld_u=64, d=64, total=BUF, pad=1, a=BUF, ld_a=64,
                        rows=8, cg=None, cu=None, st=None))
    for kw in [dict(g=None), dict(u=None), dict(a=None), dict(ld_g=8), dict(ld_u=60), dict(ld_a=1),
               dict(total=None), dict(pad=-1), dict(rows=-1), dict(d=-8)]:
        assert call(**kw) == BAD, kw
    assert call(d=12) == NO
    for kw in BAD_CKPT:
        assert call(cg=_ckpt(**kw)) == BAD and call(cu=_ckpt(**kw)) == BAD, kw
    names = "cg cu da ld_da total pad dg ld_dg du ld_du a ld_a rows st".split()
    call = _caller(lib.lemo_gated_mlp_backward, names,
                   dict(cg=_ckpt(), cu=_ckpt(), da=BUF, ld_da=64, total=BUF, pad=1, dg=BUF, ld_dg=64,
                        du=BUF, ld_du=64, a=None, ld_a=0, rows=8, st=None))
    for kw in [dict(cg=None), dict(cu=None), dict(da=None), dict(dg=None), dict(du=None),
               dict(ld_da=8), dict(ld_dg=60), dict(ld_du=0), dict(a=BUF, ld_a=8), dict(pad=0),
               dict(total=None), dict(rows=9), dict(cu=_ckpt(d=72, ld_data=80))]:
        assert call(**kw) == BAD, kw


def test_weight_grad(lib):
    names = "ck dy ld_dy rows n total dw ld_dw st".split()
    call = _caller(lib.lemo_checkpoint_weight_grad, names,
                   dict(ck=_ckpt(), dy=BUF, ld_dy=64, rows=8, n=64, total=BUF, dw=BUF, ld_dw=64,
                        st=None))
    for kw in [dict(ck=None), dict(dy=None), dict(dy=BUF + 2), dict(ld_dy=32), dict(rows=9),
               dict(rows=-1), dict(n=0), dict(total=None), dict(dw=None), dict(dw=BUF + 4),
               dict(ld_dw=32), dict(ld_dw=66)]:
        assert call(**kw) == BAD, kw
    assert call(n=12) == NO
    for kw in BAD_CKPT[:2] + BAD_CKPT[3:]:
        assert call(ck=_ckpt(**kw)) == BAD, kw


def test_binding_refuses_tensors_that_do_not_fit(lib):
    """Tensors off the current CUDA device (here: on the CPU), of another type or
    too small never reach the library."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    K = torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(16, dtype=torch.uint8)
    u8 = torch.zeros(4, 64, dtype=torch.uint8)

    def refused(fn, *a, **kw):
        with pytest.raises(lemo.LemoError) as e:
            fn(*a, **kw)
        assert e.value.status == BAD

    refused(lemo.lemo_norm_gather, 1, x, None, None, 1e-5, None, K, 1, x)
    refused(lemo.lemo_norm_gather_backward, 1, x, None, None, None, K, x, ws, x=x)
    refused(lemo.lemo_norm_scatter, 1, x, x, None, None, 1e-5, None, 1.0, None, K)
    refused(lemo.lemo_norm_scatter_backward, 1, x, None, None, None, None, 1.0, None, K, 1, x, ws, y=x)
    refused(lemo.make_checkpoint, u8, u8[:, :4], 0, 64)
    refused(lemo.lemo_gated_mlp, x, x, K, 1, x)
    refused(lemo.lemo_norm_gather, 1, x.float(), None, None, 1e-5, None, K, 1, x)
