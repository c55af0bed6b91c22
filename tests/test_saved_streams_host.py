"""What a training step's forward call saves may be dropped as soon as the backward call returns: each tensor is marked for every
stream that a call was given, so that its memory is not handed out while that stream still reads it.  Without a GPU: the library
and the streams are stood in for, the tensors write down what they are marked for."""
from __future__ import annotations

import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from prefix_scan_gb300 import _lib, delta, recurrence  # noqa: E402

CURRENT, SIDE, THIRD = (SimpleNamespace(cuda_stream=i, name=n) for i, n in ((11, "current"), (12, "side"), (13, "third")))


class Tensor(torch.Tensor):
    def record_stream(self, stream):
        self.marks = getattr(self, "marks", []) + [stream.name]


@pytest.fixture
def streams(monkeypatch):
    here = [CURRENT]

    @contextlib.contextmanager
    def inside(s):
        here.append(s)
        yield
        here.pop()

    for module in (delta, recurrence):
        monkeypatch.setattr(module, "enter", lambda device, stream: ((stream or CURRENT).cuda_stream, inside(stream or CURRENT)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here[-1])
    done = lambda *a: _lib.PS_OK  # noqa: E731
    size = lambda *a: 512  # noqa: E731
    lib = SimpleNamespace(ps_linrec_forward=done, ps_linrec_backward=done, ps_linrec_workspace_size=size, ps_delta_forward=done,
                          ps_delta_backward=done, ps_delta_workspace_size=size)
    monkeypatch.setattr(_lib, "load", lambda: lib)
    monkeypatch.setattr(recurrence, "_check_inputs", lambda *a: None)
    monkeypatch.setattr(delta, "_check_inputs", lambda *a: None)


def tensor(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Tensor)


def marks(t):
    return set(getattr(t, "marks", []))


def recurrence_step(forward, backward):
    x, g, cu, h0 = tensor(6, 4), tensor(6, 4), torch.tensor([0, 6], dtype=torch.int32).as_subclass(Tensor), tensor(1, 4)
    ws, dh, dht = tensor(512, dtype=torch.uint8), tensor(6, 4), tensor(1, 4)
    *_, saved = recurrence.linear_recurrence_forward(x, g, cu_seqlens=cu, initial_state=h0, workspace=ws, stream=forward)
    after = [marks(t) for t in (x, g, cu, h0, ws)]
    recurrence.linear_recurrence_backward(saved, dh, d_final_state=dht, stream=backward)
    return after, [marks(t) for t in (x, g, cu, h0, ws)], [marks(t) for t in (dh, dht)]


def delta_step(forward, backward):
    q, k, v = (tensor(6, 2, 4) for _ in range(3))
    g, beta, cu, h0 = tensor(6, 2), tensor(6, 2), torch.tensor([0, 6], dtype=torch.int32).as_subclass(Tensor), tensor(1, 2, 4, 4)
    ws, do, dht = tensor(512, dtype=torch.uint8), tensor(6, 2, 4), tensor(1, 2, 4, 4)
    *_, saved = delta.delta_rule_forward(q, k, v, g, beta, cu_seqlens=cu, initial_state=h0, workspace=ws, stream=forward)
    after = [marks(t) for t in (q, k, cu, ws)]
    delta.delta_rule_backward(saved, do, d_final_state=dht, stream=backward)
    return after, [marks(t) for t in (q, k, cu, ws)], [marks(t) for t in (do, dht)]


@pytest.mark.parametrize("step", [recurrence_step, delta_step])
@pytest.mark.parametrize("forward,backward", [(None, None), (None, SIDE), (SIDE, None), (SIDE, SIDE), (SIDE, THIRD), (CURRENT, CURRENT)])
def test_saved_tensors_are_marked_for_the_streams_that_read_them(streams, step, forward, backward):
    after_forward, held, gradients = step(forward, backward)
    for m in after_forward:
        assert forward is None or forward.name in m
    for m in held:
        assert all(s is None or s.name in m for s in (forward, backward))
        # the other way round: a backward call on the current stream after a forward call on another
        assert (forward or CURRENT) is (backward or CURRENT) or (backward or CURRENT).name in m
        assert forward is not None or backward is not None or not m   # one stream for all: nothing to mark
    for m in gradients:
        assert backward is None or backward.name in m
