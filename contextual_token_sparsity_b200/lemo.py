"""ctypes binding of liblemo.so (C ABI in include/lemo.h), same entry-point names.

Argument marshalling only: tensors become device pointers, the stream is the
current torch stream unless one is given, and a non-OK status raises
``LemoError``.  Every step of the path runs in the library's CUDA kernels;
there is no CPU fallback - if the library is missing, every call raises.
"""

from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "liblemo.so")

STATUS = {0: "LEMO_OK", 1: "LEMO_ERR_INVALID_ARG", 2: "LEMO_ERR_UNSUPPORTED", 3: "LEMO_ERR_CUDA",
          4: "LEMO_ERR_CAPACITY", 5: "LEMO_ERR_TIMEOUT"}
LEMO_OK = 0
LEMO_ERR_INVALID_ARG = 1
LEMO_ERR_UNSUPPORTED = 2
LEMO_ERR_CUDA = 3
LEMO_ERR_CAPACITY = 4
LEMO_ERR_TIMEOUT = 5


class LemoError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(self.status, self.status)}")


class lemo_shape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p),
        ("total_L", ctypes.c_int32),
        ("max_seqlen", ctypes.c_int32),
        ("H", ctypes.c_int32),
        ("dh", ctypes.c_int32),
        ("block", ctypes.c_int32),
    ]


class lemo_checkpoint(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("data", ctypes.c_void_p),
        ("ld_data", ctypes.c_int64),
        ("scales", ctypes.c_void_p),
        ("ld_scales", ctypes.c_int64),
        ("rows", ctypes.c_int64),
    ]


LEMO_NORM_NONE = 0
LEMO_NORM_RMS = 1
LEMO_NORM_LAYER = 2
LEMO_CHECKPOINT_E4M3 = 0
LEMO_CHECKPOINT_INT8 = 1

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SIGS = {
    "lemo_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "lemo_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(lemo_shape)]),
    "lemo_block_max_elems": (_I64, [_I32, _P, _I32]),
    "lemo_score_blocks": (ctypes.c_int, [ctypes.POINTER(lemo_shape), _P, _P, ctypes.c_float, _P,
                                         _P, _P, ctypes.c_size_t, _P]),
    "lemo_score_blocks_shard": (ctypes.c_int, [ctypes.POINTER(lemo_shape), _P, _P, ctypes.c_float,
                                               _I32, _I32, _P, _P, _P, ctypes.c_size_t, _P]),
    "lemo_select": (ctypes.c_int, [ctypes.POINTER(lemo_shape), _P, ctypes.c_float, _P, _P, _P,
                                   _P, _P, ctypes.c_size_t, _P]),
    "lemo_select_static_ws": (ctypes.c_int, [ctypes.POINTER(lemo_shape), _P, ctypes.c_float, _P,
                                             _P, _P, _P, _P]),
    "lemo_gather_pad": (ctypes.c_int, [_P, _I64, _I64, _I32, _P, _P, _I32, _P, _I64, _I64, _P]),
    "lemo_scatter_residual": (ctypes.c_int, [_P, _I64, _I64, _I32, _P, _I64, _P, _P, _P]),
    "lemo_recompute_input": (ctypes.c_int, [_P, _I64, _I64, _I32, _P, _I64, _P, _P, _P]),
    "lemo_mlp_block_scores": (ctypes.c_int, [ctypes.POINTER(lemo_shape), _I32, _P, _P, _P, _I64,
                                             _P, _P, _P, ctypes.c_size_t, _P]),
    "lemo_predict_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(lemo_shape), _I32, _I32]),
    "lemo_predict_scores": (ctypes.c_int, [ctypes.POINTER(lemo_shape), _I32, _P, _I64, _P, _P, _P,
                                           _P, _I32, _P, _P, ctypes.c_size_t, _P]),
    "lemo_attention_workspace_size": (ctypes.c_size_t, [_I32]),
    "lemo_attention_kept": (ctypes.c_int, [ctypes.POINTER(lemo_shape), _P, _P, _P, _I64, _P, _P,
                                           _P, ctypes.c_float, _P, _I64, _P, _I64, _P,
                                           ctypes.c_size_t, _P]),
    "lemo_segment_loss_workspace_size": (ctypes.c_size_t, [_I64, _I32, _I32]),
    "lemo_segment_loss": (ctypes.c_int, [_P, _I64, _I64, _I32, _P, _I64, _I32, _P, _I32, _I32, _P,
                                         _P, _P, _I64, _P, _I64, _P, ctypes.c_size_t, _P]),
    "lemo_norm_gather": (ctypes.c_int, [_I32, _P, _I64, _I64, _I32, _P, _P, ctypes.c_float, _P, _P,
                                        _I32, _P, _I64, _I64, _P, _P, _P]),
    "lemo_norm_workspace_size": (ctypes.c_size_t, [_I32]),
    "lemo_norm_gather_backward": (ctypes.c_int, [_I32, _P, _I64, _I64, _I32, _P, _P, _P, _P, _P,
                                                 _I64, _I64, _P, _P, _I64, _I64, _P, _P, _P,
                                                 ctypes.c_size_t, _P]),
    "lemo_norm_scatter": (ctypes.c_int, [_I32, _P, _I64, _I64, _I32, _P, _I64, _I64, _P, _P,
                                         ctypes.c_float, _P, _I64, ctypes.c_float, _P, _P, _P, _P,
                                         _P]),
    "lemo_norm_scatter_backward": (ctypes.c_int, [_I32, _P, _I64, _I64, _I32, _P, _P, _P, _P, _I64,
                                                  ctypes.c_float, _P, _P, _P, _I64, _P, _I32, _P,
                                                  _I64, _I64, _P, _P, _P, _P, _I64, _P,
                                                  ctypes.c_size_t, _P]),
    "lemo_checkpoint_save": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P, _P]),
    "lemo_checkpoint_restore": (ctypes.c_int, [_P, _P, _I32, _P, _I64, _I64, _P]),
    "lemo_gated_mlp": (ctypes.c_int, [_P, _I64, _P, _I64, _I32, _P, _I32, _P, _I64, _I64, _P, _P,
                                      _P]),
    "lemo_gated_mlp_backward": (ctypes.c_int, [_P, _P, _P, _I64, _P, _I32, _P, _I64, _P, _I64, _P,
                                               _I64, _I64, _P]),
    "lemo_checkpoint_weight_grad": (ctypes.c_int, [_P, _P, _I64, _I64, _I32, _P, _P, _I64, _P]),
    "lemo_get_error": (ctypes.c_int, [_P]),
    "lemo_set_test_hooks": (None, [_I32, _I64]),
    "lemo_set_predict_test_hook": (None, [_I32]),
    "lemo_set_sublayer_test_hook": (None, [_I32]),
}

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblemo.so (once) and declare its signatures.  Raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"liblemo.so not found at {path}; build it with "
                               "`python -m contextual_token_sparsity_b200.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, device=None):
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # no Stream object per call
        if raw is not None:
            return raw(torch.cuda.current_device() if device is None else device)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, where: str):
    if st != LEMO_OK:
        raise LemoError(st, where)


def make_shape(cu_seqlens, total_L: int, max_seqlen: int, H: int = 1, dh: int = 64,
               block: int = 64) -> lemo_shape:
    """lemo_shape for a packed batch; ``cu_seqlens`` is a device int32 tensor."""
    return lemo_shape(int(cu_seqlens.numel()) - 1, _ptr(cu_seqlens), int(total_L),
                      int(max_seqlen), int(H), int(dh), int(block))


def lemo_workspace_size(shape: lemo_shape) -> int:
    return int(load().lemo_workspace_size(ctypes.byref(shape)))


def lemo_block_max_elems(lengths, block: int) -> int:
    arr = (ctypes.c_int32 * len(lengths))(*[int(v) for v in lengths])
    return int(load().lemo_block_max_elems(len(lengths), ctypes.cast(arr, ctypes.c_void_p), block))


def lemo_score_blocks(shape, q, k, scale, block_max, block_scores, ws, stream=None):
    _check(load().lemo_score_blocks(ctypes.byref(shape), _ptr(q), _ptr(k), float(scale),
                                    _ptr(block_max), _ptr(block_scores), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "lemo_score_blocks")


def lemo_score_blocks_shard(shape, q, k, scale, shard, nshards, block_max, block_scores, ws,
                            stream=None):
    _check(load().lemo_score_blocks_shard(ctypes.byref(shape), _ptr(q), _ptr(k), float(scale),
                                          int(shard), int(nshards), _ptr(block_max),
                                          _ptr(block_scores), _ptr(ws),
                                          ws.numel() * ws.element_size(), _stream(stream)),
           "lemo_score_blocks_shard")


def lemo_select(shape, block_scores, threshold, block_mask, kept_idx, cu_kept, kept_total, ws,
                stream=None):
    _check(load().lemo_select(ctypes.byref(shape), _ptr(block_scores), float(threshold),
                              _ptr(block_mask), _ptr(kept_idx), _ptr(cu_kept), _ptr(kept_total),
                              _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "lemo_select")


def lemo_select_static_ws(shape, block_scores, threshold, block_mask, kept_idx, cu_kept,
                          kept_total, stream=None):
    """lemo_select with the library's own device scratch (no workspace argument)."""
    _check(load().lemo_select_static_ws(ctypes.byref(shape), _ptr(block_scores), float(threshold),
                                        _ptr(block_mask), _ptr(kept_idx), _ptr(cu_kept),
                                        _ptr(kept_total), _stream(stream)),
           "lemo_select_static_ws")


def lemo_gather_pad(x, kept_idx, kept_total, pad_to, y, stream=None, d=None):
    """x [rows, ld_x] and y [capacity, ld_y] bf16/int16 2-D tensors (row-major)."""
    d = x.shape[1] if d is None else d
    _check(load().lemo_gather_pad(_ptr(x), x.stride(0), x.shape[0], int(d), _ptr(kept_idx),
                                  _ptr(kept_total), int(pad_to), _ptr(y), y.stride(0),
                                  y.shape[0], _stream(stream)),
           "lemo_gather_pad")


def lemo_scatter_residual(x, y, kept_idx, kept_total, stream=None, d=None):
    d = x.shape[1] if d is None else d
    _check(load().lemo_scatter_residual(_ptr(x), x.stride(0), x.shape[0], int(d), _ptr(y),
                                        y.stride(0), _ptr(kept_idx), _ptr(kept_total),
                                        _stream(stream)),
           "lemo_scatter_residual")


def lemo_recompute_input(x, y, kept_idx, kept_total, stream=None, d=None):
    """x [rows, ld_x] (in place), y [>= K, ld_y] bf16 2-D tensors."""
    d = x.shape[1] if d is None else d
    _check(load().lemo_recompute_input(_ptr(x), x.stride(0), x.shape[0], int(d), _ptr(y),
                                       y.stride(0), _ptr(kept_idx), _ptr(kept_total),
                                       _stream(stream)),
           "lemo_recompute_input")


def lemo_mlp_block_scores(shape, block_scores, ws, act=None, gate=None, up=None,
                          token_scores=None, stream=None):
    """act, or gate and up: bf16 [total_L, ld] tensors (d_ff = their width)."""
    ref = act if act is not None else gate
    _check(load().lemo_mlp_block_scores(ctypes.byref(shape), int(ref.shape[1]), _ptr(act),
                                        _ptr(gate), _ptr(up), ref.stride(0), _ptr(token_scores),
                                        _ptr(block_scores), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)),
           "lemo_mlp_block_scores")


def lemo_predict_workspace_size(shape: lemo_shape, d: int, rank: int) -> int:
    return int(load().lemo_predict_workspace_size(ctypes.byref(shape), int(d), int(rank)))


def lemo_predict_scores(shape, x, w1q, w2q, w1k, w2k, block_scores, ws, stream=None, d=None):
    """x [rows, ld_x] bf16; w1 [d, rank], w2 [rank, H*dh] bf16 row-major tensors."""
    d = x.shape[1] if d is None else d
    _check(load().lemo_predict_scores(ctypes.byref(shape), int(d), _ptr(x), x.stride(0),
                                      _ptr(w1q), _ptr(w2q), _ptr(w1k), _ptr(w2k),
                                      int(w1q.shape[1]), _ptr(block_scores), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)),
           "lemo_predict_scores")


def lemo_attention_workspace_size(batch: int) -> int:
    return int(load().lemo_attention_workspace_size(int(batch)))


def lemo_attention_kept(shape, q, k, v, kept_idx, cu_kept, kept_total, ws, x=None, o=None,
                        scale=None, stream=None):
    """q, k, v bf16 [total_L, ld] 2-D tensors (same stride); exactly one of x
    (residual, updated in place) or o (compact output) bf16 2-D tensors."""
    import math
    if scale is None:
        scale = 1.0 / math.sqrt(shape.dh)
    _check(load().lemo_attention_kept(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), q.stride(0), _ptr(kept_idx),
        _ptr(cu_kept), _ptr(kept_total), float(scale), _ptr(x),
        x.stride(0) if x is not None else 0, _ptr(o), o.stride(0) if o is not None else 0,
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
        "lemo_attention_kept")


def lemo_segment_loss_workspace_size(T: int, V: int, seg_rows: int) -> int:
    return int(load().lemo_segment_loss_workspace_size(int(T), int(V), int(seg_rows)))


def lemo_segment_loss(h, w, targets, seg_rows, loss, ws, token_loss=None, dh=None, dw=None,
                      ignore_index=-100, stream=None):
    """h [T, ld_h] and w [V, ld_w] bf16 2-D tensors, targets int32 [T]; dh
    bf16 [T, ld_dh] and dw fp32 [V, ld_dw] optional (dw is accumulated)."""
    _check(load().lemo_segment_loss(
        _ptr(h), h.stride(0), h.shape[0], int(h.shape[1]), _ptr(w), w.stride(0), int(w.shape[0]),
        _ptr(targets), int(ignore_index), int(seg_rows), _ptr(loss), _ptr(token_loss), _ptr(dh),
        dh.stride(0) if dh is not None else 0, _ptr(dw), dw.stride(0) if dw is not None else 0,
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
        "lemo_segment_loss")


# ---------------------------------------------------------------------------
# Norms around a sublayer and 8-bit checkpoints.  These calls take tensors
# (not addresses) and check, before anything is enqueued, that each one is on
# the current CUDA device and has the type, row layout and sizes the call
# needs; a tensor that does not fit raises LemoError(LEMO_ERR_INVALID_ARG).
# ---------------------------------------------------------------------------
_torch = _Tensor = _BF16 = _FP32 = _INT32 = _UINT8 = None  # torch and its types, set with the first _Fit

_NO_SHAPE = (AttributeError, ValueError, IndexError, TypeError)  # of unpacking the shape of something else


class _Fit:
    """Tensor checks of one call: its methods return the data pointer."""

    __slots__ = ("where", "dev")

    def __init__(self, where: str):
        if _BF16 is None:
            _bind_torch()
        self.where = where
        self.dev = _device()

    def bad(self, name, why):
        err = LemoError(LEMO_ERR_INVALID_ARG, self.where)
        err.args = (f"{self.where}: {name} {why}",)
        raise err

    def mat(self, t, name, dtype, cols, rows=0, unit=8):
        """(pointer, row stride) of a 2-D tensor with contiguous rows; a single
        row's own stride says nothing, so its width rounded up to `unit` stands in."""
        try:
            shape = t.shape
            if len(shape) == 2 and t.dtype is dtype and t.get_device() == self.dev:
                n, width = shape
                ld, step = t.stride()
                if n >= rows and width >= cols and (step == 1 or width == 1):
                    return t.data_ptr(), ld if n > 1 else -(-width // unit) * unit
        except AttributeError:  # not a tensor
            pass
        self.explain(t, name, dtype, (rows, cols))

    def vec(self, t, name, dtype, n):
        if t is None:
            return None
        try:
            if (t.dtype is dtype and t.dim() == 1 and t.numel() >= n and t.is_contiguous()
                    and t.get_device() == self.dev):
                return t.data_ptr()
        except AttributeError:  # not a tensor
            pass
        self.explain(t, name, dtype, (n,))

    def shapeless(self, **tensors):
        """Explains which of the tensors that `mat` is going to check has no rows and columns."""
        for name, t in tensors.items():
            if not isinstance(t, _Tensor) or t.dim() != 2:
                self.explain(t, name, _BF16, (0, 0))

    def explain(self, t, name, dtype, need):
        if t is None:
            self.bad(name, "is missing")
        if not isinstance(t, _Tensor):
            self.bad(name, "is not a tensor")
        if t.dtype is not dtype or t.dim() != len(need):
            self.bad(name, f"is not a {len(need)}-D {dtype} tensor")
        if t.get_device() != self.dev:
            self.bad(name, "is not on the current CUDA device")
        if any(have < want for have, want in zip(t.shape, need)):
            self.bad(name, f"has shape {tuple(t.shape)}, at least {need} is needed")
        self.bad(name, "does not have contiguous rows")

    def total(self, kept_total):
        if kept_total is None:
            self.bad("kept_total", "is missing")
        return self.vec(kept_total, "kept_total", _INT32, 1)

    def width(self, c, name):
        """d of a checkpoint that has to be there."""
        if not isinstance(c, Checkpoint):
            self.bad(name, "is missing" if c is None else "is not a Checkpoint")
        return c.d

    def ckpt(self, c, name, d, rows):
        if c is None:
            return None
        if not isinstance(c, Checkpoint):
            self.bad(name, "is not a Checkpoint")
        if c.device != self.dev:
            self.bad(name, "is not on the current CUDA device")
        if c.d != d or c.rows < rows:
            self.bad(name, f"holds {(c.rows, c.d)}, at least {(rows, d)} is needed")
        return c.ref


def _bind_torch():
    global _torch, _Tensor, _BF16, _FP32, _INT32, _UINT8
    import torch
    _torch, _Tensor = torch, torch.Tensor
    _BF16, _FP32, _INT32, _UINT8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _device() -> int:
    """Current CUDA device, or -2 where CUDA is not in use (no tensor is on it)."""
    cuda = _torch.cuda
    return cuda.current_device() if cuda.is_initialized() else -2


class Checkpoint:
    """Rows in 8 bits: ``data`` uint8 [rows, >= d] (row stride a multiple of 16
    bytes), ``scales`` uint8 [rows, >= ceil(d / 32)] (a multiple of 4).  Codes
    are read 16 bytes at a time, so the memory behind the last row's codes has
    to reach the next multiple of 16."""

    def __init__(self, data, scales, format: int, d: int):
        fit = _Fit("make_checkpoint")
        dp, ld_data = fit.mat(data, "data", _UINT8, d, 0, 16)
        sp, ld_scales = fit.mat(scales, "scales", _UINT8, -(-d // 32), data.shape[0], 4)
        self.data, self.scales, self.d, self.rows = data, scales, int(d), data.shape[0]
        end = data.storage_offset() + (self.rows - 1) * ld_data + -(-self.d // 16) * 16
        if self.rows and end > data.untyped_storage().nbytes():
            fit.bad("data", "ends before the last row's codes reach a multiple of 16 bytes")
        self.device = data.get_device()
        self.struct = lemo_checkpoint(int(format), int(d), dp, ld_data, sp, ld_scales, self.rows)
        self.ref = ctypes.addressof(self.struct)


def make_checkpoint(data, scales, format: int, d: int) -> Checkpoint:
    """Checkpoint handle over two uint8 tensors (kept alive by the handle)."""
    return Checkpoint(data, scales, format, d)


def _stats(fit, stats, rows):
    if stats is None:
        return None
    p, ld = fit.mat(stats, "stats", _FP32, 2, rows, 2)
    if ld != 2:
        fit.bad("stats", "is not a contiguous [rows, 2] tensor")
    return p


def _workspace(fit, ws, needed):
    if ws is None:
        if needed:
            fit.bad("ws", "is missing")
        return None, 0
    if not isinstance(ws, _Tensor) or ws.get_device() != fit.dev or not ws.is_contiguous():
        fit.bad("ws", "is not a contiguous tensor on the current CUDA device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _gate(fit, gate, d, rows):
    if gate is None:
        return None, 0
    if isinstance(gate, _Tensor) and gate.dim() == 1:
        return fit.vec(gate, "gate", _BF16, d), 0
    return fit.mat(gate, "gate", _BF16, d, rows)


def lemo_norm_gather(norm, x, weight, bias, eps, kept_idx, kept_total, pad_to, y, stats=None,
                     checkpoint=None, stream=None, d=None):
    """x bf16 [x_rows, >= d], y bf16 [rows, >= d], weight / bias bf16 [d] or
    None, stats fp32 [rows, 2] contiguous, kept_idx int32 (at least K) or None."""
    fit = _Fit("lemo_norm_gather")
    try:
        (x_rows, width), rows = x.shape, y.shape[0]
    except _NO_SHAPE:
        fit.shapeless(x=x, y=y)
    d = width if d is None else int(d)
    xp, ld_x = fit.mat(x, "x", _BF16, d)
    yp, ld_y = fit.mat(y, "y", _BF16, d)
    _check(load().lemo_norm_gather(
        norm, xp, ld_x, x_rows, d, fit.vec(weight, "weight", _BF16, d),
        fit.vec(bias, "bias", _BF16, d), eps, fit.vec(kept_idx, "kept_idx", _INT32, 1),
        fit.total(kept_total), pad_to, yp, ld_y, rows, _stats(fit, stats, rows),
        fit.ckpt(checkpoint, "checkpoint", d, rows), _stream(stream, fit.dev)),
        "lemo_norm_gather")


def lemo_norm_workspace_size(d: int) -> int:
    return int(load().lemo_norm_workspace_size(int(d)))


def lemo_norm_gather_backward(norm, dy, weight, stats, kept_idx, kept_total, dx, ws, x=None,
                              checkpoint=None, dweight=None, dbias=None, stream=None, d=None):
    """dy bf16 [rows, >= d], dx bf16 [tokens, >= d] (updated in place); exactly
    one of x (the forward call's input) and checkpoint; dweight / dbias fp32
    [d] optional (accumulated); ws may be None without them."""
    fit = _Fit("lemo_norm_gather_backward")
    try:
        rows, width = dy.shape
    except _NO_SHAPE:
        fit.shapeless(dy=dy)
    d = width if d is None else int(d)
    dyp, ld_dy = fit.mat(dy, "dy", _BF16, d)
    dxp, ld_dx = fit.mat(dx, "dx", _BF16, d)
    xp, ld_x = (None, 0) if x is None else fit.mat(x, "x", _BF16, d)
    wsp, ws_bytes = _workspace(fit, ws, dweight is not None or dbias is not None)
    _check(load().lemo_norm_gather_backward(
        norm, dyp, ld_dy, rows, d, fit.vec(weight, "weight", _BF16, d), _stats(fit, stats, rows),
        fit.vec(kept_idx, "kept_idx", _INT32, 1), fit.total(kept_total), xp, ld_x,
        0 if x is None else x.shape[0], fit.ckpt(checkpoint, "checkpoint", d, rows), dxp, ld_dx,
        dx.shape[0], fit.vec(dweight, "dweight", _FP32, d), fit.vec(dbias, "dbias", _FP32, d), wsp,
        ws_bytes, _stream(stream, fit.dev)),
        "lemo_norm_gather_backward")


def lemo_norm_scatter(norm, x, y, weight, bias, eps, gate, scale, kept_idx, kept_total,
                      stats=None, checkpoint=None, stream=None, d=None):
    """x bf16 [tokens, >= d] (updated in place), y bf16 [rows, >= d]; gate None,
    bf16 [d] (all tokens) or bf16 [rows, >= d] (per kept row)."""
    fit = _Fit("lemo_norm_scatter")
    try:
        (x_rows, width), rows = x.shape, y.shape[0]
    except _NO_SHAPE:
        fit.shapeless(x=x, y=y)
    d = width if d is None else int(d)
    xp, ld_x = fit.mat(x, "x", _BF16, d)
    yp, ld_y = fit.mat(y, "y", _BF16, d)
    gp, ld_gate = _gate(fit, gate, d, rows)
    _check(load().lemo_norm_scatter(
        norm, xp, ld_x, x_rows, d, yp, ld_y, rows, fit.vec(weight, "weight", _BF16, d),
        fit.vec(bias, "bias", _BF16, d), eps, gp, ld_gate, scale,
        fit.vec(kept_idx, "kept_idx", _INT32, 1), fit.total(kept_total), _stats(fit, stats, rows),
        fit.ckpt(checkpoint, "checkpoint", d, rows), _stream(stream, fit.dev)),
        "lemo_norm_scatter")


def lemo_norm_scatter_backward(norm, dx, weight, bias, stats, gate, scale, kept_idx, kept_total,
                               pad_to, dy, ws, y=None, checkpoint=None, dweight=None, dbias=None,
                               dgate=None, stream=None, d=None):
    """dx bf16 [tokens, >= d] (read), dy bf16 [rows, >= d] (written); exactly one
    of y and checkpoint; dgate fp32 [d] (accumulated) for a gate of one row,
    bf16 [rows, >= d] (written) for a gate row per kept row."""
    fit = _Fit("lemo_norm_scatter_backward")
    try:
        (dx_rows, width), rows = dx.shape, dy.shape[0]
    except _NO_SHAPE:
        fit.shapeless(dx=dx, dy=dy)
    d = width if d is None else int(d)
    dxp, ld_dx = fit.mat(dx, "dx", _BF16, d)
    dyp, ld_dy = fit.mat(dy, "dy", _BF16, d)
    yp, ld_y = (None, 0) if y is None else fit.mat(y, "y", _BF16, d, rows)
    gp, ld_gate = _gate(fit, gate, d, rows)
    dg, dgr, ld_dgr = None, None, 0
    if isinstance(dgate, _Tensor) and dgate.dim() == 2:
        dgr, ld_dgr = fit.mat(dgate, "dgate", _BF16, d, rows)
    else:
        dg = fit.vec(dgate, "dgate", _FP32, d)
    wsp, ws_bytes = _workspace(fit, ws, dweight is not None or dbias is not None or dg is not None)
    _check(load().lemo_norm_scatter_backward(
        norm, dxp, ld_dx, dx_rows, d, fit.vec(weight, "weight", _BF16, d),
        fit.vec(bias, "bias", _BF16, d), _stats(fit, stats, rows), gp, ld_gate, scale,
        fit.vec(kept_idx, "kept_idx", _INT32, 1), fit.total(kept_total), yp, ld_y,
        fit.ckpt(checkpoint, "checkpoint", d, rows), pad_to, dyp, ld_dy, rows,
        fit.vec(dweight, "dweight", _FP32, d), fit.vec(dbias, "dbias", _FP32, d), dg, dgr, ld_dgr,
        wsp, ws_bytes, _stream(stream, fit.dev)),
        "lemo_norm_scatter_backward")


def lemo_checkpoint_save(x, kept_idx, kept_total, checkpoint, stream=None):
    """x bf16 [tokens, >= checkpoint.d]; kept_idx int32 or None (row r is token r)."""
    fit = _Fit("lemo_checkpoint_save")
    d = fit.width(checkpoint, "checkpoint")
    xp, ld_x = fit.mat(x, "x", _BF16, d)
    _check(load().lemo_checkpoint_save(
        xp, ld_x, x.shape[0], fit.vec(kept_idx, "kept_idx", _INT32, 1), fit.total(kept_total),
        fit.ckpt(checkpoint, "checkpoint", d, 0), _stream(stream, fit.dev)),
        "lemo_checkpoint_save")


def lemo_checkpoint_restore(checkpoint, kept_total, pad_to, y, stream=None):
    """y bf16 [rows, >= checkpoint.d], rows <= checkpoint.rows."""
    fit = _Fit("lemo_checkpoint_restore")
    d = fit.width(checkpoint, "checkpoint")
    try:
        rows = y.shape[0]
    except _NO_SHAPE:
        fit.shapeless(y=y)
    yp, ld_y = fit.mat(y, "y", _BF16, d)
    _check(load().lemo_checkpoint_restore(
        fit.ckpt(checkpoint, "checkpoint", d, rows), fit.total(kept_total), pad_to, yp, ld_y, rows,
        _stream(stream, fit.dev)),
        "lemo_checkpoint_restore")


def lemo_gated_mlp(gate, up, kept_total, pad_to, a, gate_checkpoint=None, up_checkpoint=None,
                   stream=None, d=None):
    """gate, up, a bf16 [rows, >= d]; a = SiLU(gate) up."""
    fit = _Fit("lemo_gated_mlp")
    try:
        rows, width = a.shape
    except _NO_SHAPE:
        fit.shapeless(a=a)
    d = width if d is None else int(d)
    gp, ld_g = fit.mat(gate, "gate", _BF16, d, rows)
    up_, ld_u = fit.mat(up, "up", _BF16, d, rows)
    ap, ld_a = fit.mat(a, "a", _BF16, d)
    _check(load().lemo_gated_mlp(
        gp, ld_g, up_, ld_u, d, fit.total(kept_total), pad_to, ap, ld_a, rows,
        fit.ckpt(gate_checkpoint, "gate_checkpoint", d, rows),
        fit.ckpt(up_checkpoint, "up_checkpoint", d, rows), _stream(stream, fit.dev)),
        "lemo_gated_mlp")


def lemo_gated_mlp_backward(gate_checkpoint, up_checkpoint, da, kept_total, pad_to, dgate, dup,
                            a=None, stream=None):
    """da, dgate, dup and the optional recomputed activation a: bf16 [rows, >= d]."""
    fit = _Fit("lemo_gated_mlp_backward")
    d = fit.width(gate_checkpoint, "gate_checkpoint")
    fit.width(up_checkpoint, "up_checkpoint")
    try:
        rows = dgate.shape[0]
    except _NO_SHAPE:
        fit.shapeless(dgate=dgate)
    dap, ld_da = fit.mat(da, "da", _BF16, d, rows)
    dgp, ld_dg = fit.mat(dgate, "dgate", _BF16, d)
    dup_, ld_du = fit.mat(dup, "dup", _BF16, d, rows)
    ap, ld_a = (None, 0) if a is None else fit.mat(a, "a", _BF16, d, rows)
    _check(load().lemo_gated_mlp_backward(
        fit.ckpt(gate_checkpoint, "gate_checkpoint", d, rows),
        fit.ckpt(up_checkpoint, "up_checkpoint", d, rows), dap, ld_da, fit.total(kept_total),
        pad_to, dgp, ld_dg, dup_, ld_du, ap, ld_a, rows, _stream(stream, fit.dev)),
        "lemo_gated_mlp_backward")


def lemo_checkpoint_weight_grad(checkpoint, dy, kept_total, dw, stream=None, n=None):
    """dw fp32 [n, >= d] += dy^T xhat; dy bf16 [rows, >= n], n = dy's width."""
    fit = _Fit("lemo_checkpoint_weight_grad")
    d = fit.width(checkpoint, "checkpoint")
    try:
        rows, width = dy.shape
    except _NO_SHAPE:
        fit.shapeless(dy=dy)
    n = width if n is None else int(n)
    dyp, ld_dy = fit.mat(dy, "dy", _BF16, n)
    dwp, ld_dw = fit.mat(dw, "dw", _FP32, d, n, 4)
    _check(load().lemo_checkpoint_weight_grad(
        fit.ckpt(checkpoint, "checkpoint", d, rows), dyp, ld_dy, rows, n, fit.total(kept_total),
        dwp, ld_dw, _stream(stream, fit.dev)),
        "lemo_checkpoint_weight_grad")


def lemo_get_error(stream=None) -> int:
    """Synchronise the stream; return (and clear) the device error status."""
    return int(load().lemo_get_error(_stream(stream)))


def lemo_set_test_hooks(select_skip_publish_tile: int = -1, spin_limit_ns: int = 0):
    load().lemo_set_test_hooks(int(select_skip_publish_tile), int(spin_limit_ns))


def lemo_set_predict_test_hook(skip_cta: int = -1):
    load().lemo_set_predict_test_hook(int(skip_cta))


def lemo_set_sublayer_test_hook(withhold: bool = False):
    load().lemo_set_sublayer_test_hook(int(withhold))
