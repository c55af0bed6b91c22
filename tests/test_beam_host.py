"""Beam search's choice and the reordering of pages without a GPU: sizes and refusals before anything is enqueued."""
from __future__ import annotations

import struct

import pytest

from prefix_scan_gb300 import _lib
from prefix_scan_gb300 import build as nvbuild

torch = pytest.importorskip("torch")

FAKE = 1 << 40   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    if not nvbuild.is_fresh():
        try:
            nvbuild.build()
        except RuntimeError as e:  # pragma: no cover - toolchain missing
            pytest.skip(f"cannot build the CUDA library here: {e}")
    return _lib.load()


@pytest.fixture
def no_device():
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses are only passed on hosts without a GPU")


def shape(batch=2, beams=4, width=4, vocab=1000, item=4000, beam=1000, code=_lib.PS_REAL_F32, eos=-1):
    return _lib.BEAM_SHAPE.pack(batch, beams, width, vocab, item, beam, code, eos)


def test_workspace_size(lib):
    f = lib.ps_beam_workspace_size
    assert f(shape(batch=0)) == 0 and f(None) == 0
    for bad in (dict(batch=-1), dict(beams=0), dict(beams=257), dict(width=0), dict(width=65), dict(vocab=0), dict(vocab=1 << 31),
                dict(code=5), dict(eos=-2), dict(batch=1 << 30)):
        assert f(shape(**bad)) == 0, bad
    for vocab in (1, 4096, 100000):
        for width in (1, 64):
            n = f(shape(vocab=vocab, width=width))
            assert n % 256 == 0 and n >= 8 * (12 + 8 * width)   # of each row a sum, a maximum and `width` candidates


def test_select_refusals(lib, no_device):
    s = shape()
    need = lib.ps_beam_workspace_size(s)
    X, SC, EN, A, B, C, D, WS = (FAKE + (i << 32) for i in range(8))
    base = [s, X, SC, EN, A, B, C, D, WS, need, None]

    def f(**change):
        names = ("shape", "logits", "scores", "ended", "o1", "o2", "o3", "o4", "ws", "bytes", "stream")
        return lib.ps_beam_select(*[change.get(n, v) for n, v in zip(names, base)])

    assert f(shape=shape(batch=0), logits=None) == _lib.PS_OK
    for bad in (dict(shape=None), dict(logits=None), dict(scores=None), dict(o1=None), dict(o2=None), dict(o3=None), dict(ws=None),
                dict(logits=X + 2), dict(scores=SC + 1), dict(o2=B + 2), dict(ws=WS + 64), dict(shape=shape(width=65))):
        assert f(**bad) == _lib.PS_ERR_INVALID_ARG, bad
    assert f(bytes=need - 1) == _lib.PS_ERR_WORKSPACE_TOO_SMALL
    for bad in (dict(o1=X + 400), dict(o2=A + 16), dict(o4=EN), dict(o1=SC), dict(o3=WS + 128), dict(scores=WS + 256)):
        assert f(**bad) == _lib.PS_ERR_OVERLAP, bad


def test_reorder_refusals(lib, no_device):
    pool = lambda *x: struct.pack("@" + "Pq" * (len(x) // 2), *x)  # noqa: E731
    A, B, C, D, E, WS = (FAKE + (i << 32) for i in range(6))
    need = lib.ps_pages_workspace_size(8, 100)
    f = lambda *a: lib.ps_pages_reorder(*a, None)  # noqa: E731
    base = [A, B, 8, pool(E, 64), 1, 100, C, D, WS, need]
    bad = lambda i, v: f(*(base[:i] + [v] + base[i + 1:]))  # noqa: E731
    assert bad(0, None) == bad(1, None) == bad(6, None) == bad(8, None) == _lib.PS_ERR_INVALID_ARG
    assert bad(0, A + 1) == bad(6, C + 2) == bad(8, WS + 16) == bad(2, -1) == bad(4, 129) == _lib.PS_ERR_INVALID_ARG
    assert bad(9, need - 1) == _lib.PS_ERR_WORKSPACE_TOO_SMALL
    assert bad(6, A) == bad(6, B + 16) == bad(0, E + 64) == bad(7, C) == bad(6, WS + 64) == _lib.PS_ERR_OVERLAP


def test_python_layer_refuses_what_it_cannot_run():
    from prefix_scan_gb300 import api
    x, s = torch.zeros(2, 3, 5), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="CUDA"):
        api.beam_select(x, s)
    with pytest.raises(ValueError, match="requires gradients"):
        api.beam_select(x.clone().requires_grad_(), s)
    with pytest.raises(TypeError, match="float64"):
        api.beam_workspace_size(x.double())
    with pytest.raises(ValueError, match="CUDA"):
        api.pages_reorder(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2))
