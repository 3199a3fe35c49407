"""One layer of the path on a packed batch: device buffers and the four calls.

``Layer`` allocates (with torch, on the device) every buffer the C ABI
needs for a fixed batch layout and exposes the steps in order:

    layer.score(q, k)          block scores               (lemo_score_blocks)
    layer.select(theta)        mask + kept ids            (lemo_select)
    layer.gather(x)            y = x[kept] + zero tail     (lemo_gather_pad)
    layer.scatter(x, y_out)    x[kept] += y_out, in place  (lemo_scatter_residual)

A sublayer with norms takes, in place of the last two, the forms that fuse
them with the movement, and their backward passes:

    layer.gather_norm(...)     y = norm(x[kept]) w + b     (lemo_norm_gather)
    layer.scatter_norm(...)    x[kept] += s gate norm(y)   (lemo_norm_scatter)
    layer.checkpoint(...)      8-bit rows for one kept-row buffer (make_checkpoint)
    layer.norm_stats()         row statistics of one forward call, for its backward call

No step copies anything to the host; K stays on the device.
"""

from __future__ import annotations

import numpy as np

from . import lemo


def _round_up(v: int, m: int) -> int:
    return (v + m - 1) // m * m


class Layer:
    def __init__(self, lengths, H: int, dh: int, block: int, d: int, pad_to: int = 128,
                 device="cuda", keep_block_max: bool = False):
        import torch
        self.torch = torch
        self.lengths = [int(v) for v in lengths]
        self.H, self.dh, self.block, self.d, self.pad_to = H, dh, block, d, pad_to
        self.total_L = int(sum(self.lengths))
        cu = np.zeros(len(self.lengths) + 1, dtype=np.int32)
        cu[1:] = np.cumsum(self.lengths)
        self.cu_host = cu
        self.cu = torch.from_numpy(cu).to(device)
        self.shape = lemo.make_shape(self.cu, self.total_L, max(self.lengths), H, dh, block)
        ws = lemo.lemo_workspace_size(self.shape)
        if ws == 0:
            raise ValueError("invalid shape")
        self.ws = torch.empty(ws, dtype=torch.uint8, device=device)
        self.nblocks = [-(-L // block) for L in self.lengths]
        self.total_blocks = int(sum(self.nblocks))
        self.block_scores = torch.empty(max(self.total_blocks, 1), dtype=torch.float32,
                                        device=device)
        self.block_max = (torch.full((max(lemo.lemo_block_max_elems(self.lengths, block), 1),),
                                     float("nan"), dtype=torch.float32, device=device)
                          if keep_block_max else None)
        self.mask = torch.empty(max(self.total_blocks, 1), dtype=torch.uint8, device=device)
        self.kept_idx = torch.empty(max(self.total_L, 1), dtype=torch.int32, device=device)
        self.cu_kept = torch.empty(len(self.lengths) + 1, dtype=torch.int32, device=device)
        self.kept_total = torch.empty(1, dtype=torch.int32, device=device)
        self.y_rows = max(_round_up(self.total_L, pad_to), pad_to)
        self.y = torch.empty((self.y_rows, d), dtype=torch.bfloat16, device=device)
        self.pre_stats, self.post_stats = self.norm_stats(), self.norm_stats()
        # forward calls that wrote these since a backward call read them, and whether one has
        self._forwards = {"pre_stats": 0, "post_stats": 0}
        self._read = {"pre_stats": False, "post_stats": False}

    # -- the four steps ------------------------------------------------------
    def score(self, q, k, scale: float = 1.0, stream=None):
        lemo.lemo_score_blocks(self.shape, q, k, scale, self.block_max, self.block_scores,
                               self.ws, stream)
        return self.block_scores

    def select(self, theta: float, stream=None):
        lemo.lemo_select(self.shape, self.block_scores, theta, self.mask, self.kept_idx,
                         self.cu_kept, self.kept_total, self.ws, stream)

    def gather(self, x, stream=None):
        lemo.lemo_gather_pad(x, self.kept_idx, self.kept_total, self.pad_to, self.y, stream)
        return self.y

    def scatter(self, x, y_out, stream=None):
        lemo.lemo_scatter_residual(x, y_out, self.kept_idx, self.kept_total, stream)

    def step(self, q, k, theta: float, x, y_out, scale: float = 1.0, stream=None):
        """score -> select -> gather -> scatter on one stream."""
        self.score(q, k, scale, stream)
        self.select(theta, stream)
        self.gather(x, stream)
        self.scatter(x, y_out, stream)

    # -- norms around the sublayer, 8-bit checkpoints ---------------------------
    # A forward call leaves the statistics (mean, rstd) of its rows in `stats`, and the backward
    # call that follows it takes the same buffer.  Without `stats` both use the Layer's own
    # (pre_stats for gather_norm, post_stats for scatter_norm), which hold one forward call:
    # after a second one a backward call without `stats` is refused, since it could belong to
    # either.  Two sublayers on one selection, micro-batches and forward calls that no backward
    # call follows take a buffer each.  Every row has the Layer's d values (of wider tensors the
    # first d columns).
    def norm_stats(self):
        """An empty buffer for the statistics of one gather_norm or scatter_norm call."""
        t = self.torch
        return t.empty((self.y_rows, 2), dtype=t.float32, device=self.y.device)

    def _norm_ws(self, sums: bool, stream):
        """Workspace of one backward call, from the allocator's memory of the stream that the call
        runs on (of the graph, where it is captured): calls that overlap do not share it."""
        if not sums:
            return None
        t = self.torch
        if isinstance(stream, int):
            stream = (t.cuda.default_stream(self.y.device) if stream < 2 else
                      t.cuda.ExternalStream(stream, self.y.device))
        with t.cuda.stream(stream):
            return t.empty(lemo.lemo_norm_workspace_size(self.d), dtype=t.uint8, device=self.y.device)

    def _own_stats(self, which: str, where: str):
        """The Layer's own statistics, for a backward call."""
        n = self._forwards[which]
        if n != 1:
            err = lemo.LemoError(lemo.LEMO_ERR_INVALID_ARG, where)
            err.args = (f"{where}: {n} forward calls wrote the layer's own statistics; pass the same "
                        "stats to a forward call and its backward call",)
            raise err
        return getattr(self, which)

    def _wrote(self, which: str, own: bool):
        """After a forward call: once read, the own statistics end with the next one."""
        if self._read[which]:
            self._forwards[which], self._read[which] = 0, False
        self._forwards[which] += own

    def checkpoint(self, format: int, width: int | None = None):
        """An empty checkpoint for a kept-row buffer of `width` columns (d by default)."""
        t, dev, d = self.torch, self.y.device, self.d if width is None else width
        return lemo.make_checkpoint(
            t.empty((self.y_rows, _round_up(d, 16)), dtype=t.uint8, device=dev),
            t.empty((self.y_rows, _round_up(-(-d // 32), 4)), dtype=t.uint8, device=dev), format, d)

    def gather_norm(self, norm, x, weight=None, bias=None, eps: float = 1e-5, checkpoint=None,
                    stream=None, stats=None):
        lemo.lemo_norm_gather(norm, x, weight, bias, eps, self.kept_idx, self.kept_total,
                              self.pad_to, self.y, stats=self.pre_stats if stats is None else stats,
                              checkpoint=checkpoint, stream=stream, d=self.d)
        self._wrote("pre_stats", stats is None)
        return self.y

    def gather_norm_backward(self, norm, dy, dx, weight=None, x=None, checkpoint=None, dweight=None,
                             dbias=None, stream=None, stats=None):
        """dx[kept] += d loss / d x[kept], in place, from the gradient dy of gather_norm's rows."""
        own = stats is None
        if own:
            stats = self._own_stats("pre_stats", "gather_norm_backward")
        ws = self._norm_ws(dweight is not None or dbias is not None, stream)
        lemo.lemo_norm_gather_backward(norm, dy, weight, stats, self.kept_idx, self.kept_total, dx,
                                       ws, x=x, checkpoint=checkpoint, dweight=dweight, dbias=dbias,
                                       stream=stream, d=self.d)
        if own:
            self._read["pre_stats"] = True

    def scatter_norm(self, norm, x, y_out, weight=None, bias=None, eps: float = 1e-5, gate=None,
                     scale: float = 1.0, checkpoint=None, stream=None, stats=None):
        own = stats is None and norm != lemo.LEMO_NORM_NONE
        lemo.lemo_norm_scatter(norm, x, y_out, weight, bias, eps, gate, scale, self.kept_idx,
                               self.kept_total, stats=self.post_stats if own else stats,
                               checkpoint=checkpoint, stream=stream, d=self.d)
        if norm != lemo.LEMO_NORM_NONE:
            self._wrote("post_stats", own)

    def scatter_norm_backward(self, norm, dx, dy_out, weight=None, bias=None, gate=None,
                              scale: float = 1.0, y_out=None, checkpoint=None, dweight=None,
                              dbias=None, dgate=None, stream=None, stats=None):
        """dy_out = the gradient of scatter_norm's y_out, zero-padded; dx is only read."""
        own = stats is None and norm != lemo.LEMO_NORM_NONE
        if own:
            stats = self._own_stats("post_stats", "scatter_norm_backward")
        ws = self._norm_ws(any(g is not None for g in (dweight, dbias, dgate)), stream)
        lemo.lemo_norm_scatter_backward(norm, dx, weight, bias, stats, gate, scale, self.kept_idx,
                                        self.kept_total, self.pad_to, dy_out, ws, y=y_out,
                                        checkpoint=checkpoint, dweight=dweight, dbias=dbias,
                                        dgate=dgate, stream=stream, d=self.d)
        if own:
            self._read["post_stats"] = True

    # -- helpers for checking results ----------------------------------------
    def block_max_list(self):
        """Per-sequence [N_b, N_b] numpy views of block_max (host copy)."""
        bm = self.block_max.cpu().numpy()
        out, off = [], 0
        for nb in self.nblocks:
            out.append(bm[off:off + nb * nb].reshape(nb, nb))
            off += nb * nb
        return out


def to_device_bf16(bits: np.ndarray, device="cuda"):
    """bf16 bit patterns (uint16 numpy) -> torch bfloat16 device tensor."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device).view(
        torch.bfloat16)


def to_host_bits(t) -> np.ndarray:
    """torch bfloat16 tensor -> bf16 bit patterns (uint16 numpy)."""
    import torch
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
