"""The norm methods of pipeline.Layer without a GPU: what each one hands to the
library (recorded by stand-ins of the binding's functions), and what it refuses."""

import os
import shutil

import pytest
import torch

from contextual_token_sparsity_b200 import build as lemo_build
from contextual_token_sparsity_b200 import lemo
from contextual_token_sparsity_b200.pipeline import Layer

NONE, RMS, LAYERNORM = lemo.LEMO_NORM_NONE, lemo.LEMO_NORM_RMS, lemo.LEMO_NORM_LAYER
D = 64


@pytest.fixture
def layer():
    if shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc"):
        lemo_build.build()
    if not os.path.exists(lemo.LIB_PATH):
        pytest.skip("liblemo.so not built and nvcc unavailable")
    return Layer([40, 9], 1, 64, 64, D, device="cpu")


class Calls:
    """Stand-ins of the four norm calls that keep what they were given."""

    def __init__(self, monkeypatch):
        self.seen = []
        for name, stats_at in (("lemo_norm_gather", None), ("lemo_norm_gather_backward", 3),
                               ("lemo_norm_scatter", None), ("lemo_norm_scatter_backward", 4)):
            monkeypatch.setattr(lemo, name, self.record(name, stats_at))

    def record(self, name, stats_at):
        def call(*a, **kw):
            self.seen.append((name, a[stats_at] if stats_at else kw.get("stats"), a, kw))
        return call

    def stats(self):
        return [s for _, s, _, _ in self.seen]


@pytest.fixture
def calls(monkeypatch):
    return Calls(monkeypatch)


def _rows(layer):
    return torch.zeros(layer.y_rows, D, dtype=torch.bfloat16)


def test_a_backward_call_takes_the_statistics_of_its_forward_call(layer, calls):
    x, y = torch.zeros(49, D, dtype=torch.bfloat16), _rows(layer)
    pre, post = ([layer.norm_stats() for _ in range(2)] for _ in range(2))
    for i in range(2):
        layer.gather_norm(RMS, x, stats=pre[i])
        layer.scatter_norm(LAYERNORM, x, y, stats=post[i])
    for i in (1, 0):
        layer.scatter_norm_backward(LAYERNORM, x, y, y_out=y, stats=post[i])
        layer.gather_norm_backward(RMS, y, x, x=x, stats=pre[i])
    want = [pre[0], post[0], pre[1], post[1], post[1], pre[1], post[0], pre[0]]
    assert all(a is b for a, b in zip(calls.stats(), want)) and len(calls.seen) == 8
    assert all(t.shape == (layer.y_rows, 2) and t.dtype == torch.float32 for t in pre + post)
    assert len({t.data_ptr() for t in pre + post}) == 4


def test_overwritten_statistics_are_refused(layer, calls):
    """Two forward calls into the Layer's own statistics: no backward call can tell which it
    follows, so it has to be told."""
    x, y = torch.zeros(49, D, dtype=torch.bfloat16), _rows(layer)

    def refused(fn, *a, **kw):
        n = len(calls.seen)
        with pytest.raises(lemo.LemoError) as e:
            fn(*a, **kw)
        assert e.value.status == lemo.LEMO_ERR_INVALID_ARG and len(calls.seen) == n

    refused(layer.gather_norm_backward, RMS, y, x, x=x)          # no forward call at all
    refused(layer.scatter_norm_backward, RMS, x, y, y_out=y)
    for _ in range(2):                                           # one forward call each: fine, again and again
        layer.gather_norm(RMS, x)
        layer.scatter_norm(RMS, x, y)
        for _ in range(2):
            layer.scatter_norm_backward(RMS, x, y, y_out=y)
            layer.gather_norm_backward(RMS, y, x, x=x)
    layer.gather_norm(RMS, x, stats=layer.norm_stats())          # not in the own ones, which were read
    refused(layer.gather_norm_backward, RMS, y, x, x=x)
    layer.gather_norm(RMS, x)
    layer.gather_norm(RMS, x, stats=layer.norm_stats())          # not read yet: they stay
    layer.gather_norm_backward(RMS, y, x, x=x)
    layer.gather_norm(RMS, x)
    layer.gather_norm(RMS, x)
    refused(layer.gather_norm_backward, RMS, y, x, x=x)
    refused(layer.gather_norm_backward, RMS, y, x, x=x)
    layer.scatter_norm(RMS, x, y)
    layer.scatter_norm_backward(RMS, x, y, y_out=y)              # the other norm's are its own
    layer.gather_norm(RMS, x, stats=layer.norm_stats())
    refused(layer.gather_norm_backward, RMS, y, x, x=x)
    layer.gather_norm_backward(RMS, y, x, x=x, stats=layer.norm_stats())
    layer.scatter_norm(RMS, x, y)
    layer.scatter_norm(NONE, x, y)                               # no norm: no statistics
    layer.scatter_norm_backward(NONE, x, y, y_out=y)
    layer.scatter_norm_backward(RMS, x, y, y_out=y)
    assert calls.stats()[-2] is None and calls.stats()[-3] is None


def test_the_layers_own_statistics(layer, calls):
    x, y = torch.zeros(49, D, dtype=torch.bfloat16), _rows(layer)
    layer.gather_norm(RMS, x)
    layer.scatter_norm(RMS, x, y)
    layer.scatter_norm_backward(RMS, x, y, y_out=y)
    layer.gather_norm_backward(RMS, y, x, x=x)
    own = [layer.pre_stats, layer.post_stats, layer.post_stats, layer.pre_stats]
    assert all(a is b for a, b in zip(calls.stats(), own))
    assert layer.pre_stats.data_ptr() != layer.post_stats.data_ptr()


def test_a_refused_forward_call_writes_nothing(layer, calls, monkeypatch):
    x, y = torch.zeros(49, D, dtype=torch.bfloat16), _rows(layer)
    layer.gather_norm(RMS, x)
    layer.scatter_norm(RMS, x, y)
    for name in ("lemo_norm_gather", "lemo_norm_scatter"):
        def fail(*a, name=name, **kw):
            raise lemo.LemoError(lemo.LEMO_ERR_INVALID_ARG, name)
        with monkeypatch.context() as m:
            m.setattr(lemo, name, fail)
            for _ in range(2):
                with pytest.raises(lemo.LemoError):
                    layer.gather_norm(RMS, x) if name.endswith("gather") else layer.scatter_norm(RMS, x, y)
    layer.scatter_norm_backward(RMS, x, y, y_out=y)
    layer.gather_norm_backward(RMS, y, x, x=x)


def test_backward_calls_do_not_share_a_workspace(layer, calls):
    """Each call has its own (calls on two streams may overlap); without column sums there is none."""
    x, y, dw = torch.zeros(49, D, dtype=torch.bfloat16), _rows(layer), torch.zeros(D)
    layer.gather_norm(RMS, x)
    layer.scatter_norm(RMS, x, y)
    for _ in range(2):
        layer.scatter_norm_backward(RMS, x, y, y_out=y, dgate=dw)
        layer.gather_norm_backward(RMS, y, x, x=x, dbias=dw)
    ws = [a[7 if name.endswith("gather_backward") else 11] for name, _, a, _ in calls.seen[2:]]
    assert len({t.data_ptr() for t in ws}) == 4
    assert all(t.numel() == lemo.lemo_norm_workspace_size(D) for t in ws)
    layer.scatter_norm_backward(RMS, x, y, y_out=y)
    layer.gather_norm_backward(RMS, y, x, x=x)
    assert calls.seen[-1][2][7] is None and calls.seen[-2][2][11] is None


def test_rows_of_another_width_are_refused(layer, monkeypatch):
    """Every row has the Layer's width: narrower ones would leave the rest of y as it was; of wider
    ones the first d columns are taken."""
    monkeypatch.setattr(lemo, "_device", lambda: -1)      # CPU tensors pass the device check
    x, y = torch.zeros(49, D, dtype=torch.bfloat16), _rows(layer)
    for name, args in (("gather_norm", (RMS, x[:, :32])), ("scatter_norm", (RMS, x[:, :32], y)),
                       ("scatter_norm", (RMS, x, y[:, :32])),
                       ("scatter_norm_backward", (NONE, x[:, :32], y)),
                       ("gather_norm_backward", (RMS, y[:, :32], x)),
                       ("gather_norm_backward", (RMS, y, x[:, :32]))):
        kw = {} if name in ("gather_norm", "scatter_norm") else {"stats": layer.norm_stats()}
        if name == "gather_norm_backward":
            kw["x"] = x
        if name == "scatter_norm_backward":
            kw["y_out"] = y
        with pytest.raises(lemo.LemoError) as e:
            getattr(layer, name)(*args, **kw)
        assert e.value.status == lemo.LEMO_ERR_INVALID_ARG and "has shape" in str(e.value), name
    seen = Calls(monkeypatch).seen
    wide = torch.zeros(49, 2 * D, dtype=torch.bfloat16)
    layer.gather_norm(RMS, wide)
    layer.scatter_norm(RMS, wide, y)
    layer.scatter_norm_backward(RMS, wide, y, y_out=y)
    layer.gather_norm_backward(RMS, y, wide, x=wide)
    assert [kw.get("d") for _, _, _, kw in seen] == [D] * 4
