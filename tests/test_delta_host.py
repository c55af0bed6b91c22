"""The gated delta rule and the page operations without a GPU: sizes, refusals before anything is enqueued, the rule that
cuts long sequences, and the 64-bit reference's gradients against its own differences."""
from __future__ import annotations

import pytest

from prefix_scan_gb300 import _lib
from prefix_scan_gb300 import build as nvbuild

torch = pytest.importorskip("torch")

import delta_reference as ref  # noqa: E402

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


def shape(seqs=2, tokens=100, cu=0, hk=2, hv=4, k=64, v=64, code=_lib.PS_REAL_BF16, beta=_lib.PS_REAL_F32, scale=1.0):
    return _lib.DELTA_SHAPE.pack(seqs, tokens, cu, hk, hv, k, v, code, beta, scale)


def inputs(hk=2, hv=4, size=64, tokens=100, **data):
    where = {name: FAKE + (i << 32) for i, name in enumerate("qkvgb")}
    where.update(data)
    rows = ((hk * size, size), (hk * size, size), (hv * size, size), (hv, 1), (hv, 1))
    return _lib.DELTA_INPUTS.pack(*[x for name, (tok, head) in zip("qkvgb", rows) for x in (where[name], tokens * tok, tok, head)])


WS, OUT, H0, HT = FAKE + (6 << 32), FAKE + (7 << 32), FAKE + (8 << 32), FAKE + (9 << 32)


def test_workspace_size(lib):
    f = lib.ps_delta_workspace_size
    assert f(shape(seqs=0), 0) == 0 and f(shape(tokens=0), 1) == 0
    for bad in (dict(hv=3), dict(hk=0), dict(k=129), dict(k=0), dict(v=1025), dict(code=7), dict(beta=_lib.PS_REAL_F16),
                dict(seqs=-1), dict(tokens=-1), dict(tokens=1 << 32)):
        assert f(shape(**bad), 0) == 0, bad
    one = f(shape(seqs=1, tokens=64), 0)
    assert one % 256 == 0 and one >= 4 * 4 * 8192     # T and P of four value heads, in pairs
    assert f(shape(seqs=1, tokens=65), 0) == 2 * one  # a chunk of one token takes a chunk's room
    assert f(shape(seqs=1, tokens=64), 1) > 2 * one
    # packed sequences: any way to cut 100 tokens into 3 fits
    assert f(shape(seqs=3, tokens=100, cu=FAKE), 0) == f(shape(seqs=1, tokens=64 * 4), 0)


def test_forward_refusals(lib, no_device):
    s, x = shape(), inputs()
    need = lib.ps_delta_workspace_size(s, 0)
    f = lib.ps_delta_forward
    assert f(shape(seqs=0), x, None, None, None, 0, None, 0, None) == _lib.PS_OK
    assert f(None, x, None, None, OUT, 0, WS, need, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, None, None, None, OUT, 0, WS, need, None) == _lib.PS_ERR_INVALID_ARG
    for bad in (dict(q=0), dict(k=FAKE + 1), dict(g=FAKE + 2), dict(b=0)):
        assert f(s, inputs(**bad), None, None, OUT, 0, WS, need, None) == _lib.PS_ERR_INVALID_ARG, bad
    assert f(s, x, None, None, None, 0, WS, need, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, None, None, OUT + 1, 0, WS, need, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, H0 + 2, None, OUT, 0, WS, need, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, None, None, OUT, 0, WS + 16, need, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, None, None, OUT, 0, None, need, None) == _lib.PS_ERR_INVALID_ARG
    assert f(shape(cu=FAKE + 2), x, None, None, OUT, 0, WS, need, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, None, None, OUT, 0, WS, need - 1, None) == _lib.PS_ERR_WORKSPACE_TOO_SMALL
    assert f(s, x, None, None, OUT, 1, WS, need, None) == _lib.PS_ERR_WORKSPACE_TOO_SMALL   # training keeps more
    v = FAKE + (2 << 32)
    assert f(s, x, None, None, v + 4096, 0, WS, need, None) == _lib.PS_ERR_OVERLAP          # output in v
    assert f(s, x, None, OUT + 256, OUT, 0, WS, need, None) == _lib.PS_ERR_OVERLAP          # state in the output
    assert f(s, x, H0, H0 + 256, OUT, 0, WS, need, None) == _lib.PS_ERR_OVERLAP             # states meet, not the same
    assert f(s, x, None, None, WS + 512, 0, WS, need, None) == _lib.PS_ERR_OVERLAP


def test_backward_refusals(lib, no_device):
    s = shape(beta=_lib.PS_REAL_BF16)
    need = lib.ps_delta_workspace_size(s, 1)
    t = lambda p, h, d: _lib.DELTA_TENSOR.pack(p, 100 * h * d, h * d, d)  # noqa: E731
    q, k, do = t(FAKE, 2, 64), t(FAKE + (1 << 32), 2, 64), t(FAKE + (2 << 32), 4, 64)
    o = [OUT + (i << 28) for i in range(6)]   # dq, dk, dv, dg, dbeta, dh0
    f = lambda *a: lib.ps_delta_backward(s, *a, None)  # noqa: E731
    assert f(q, k, do, None, *o, WS, need - 1) == _lib.PS_ERR_WORKSPACE_TOO_SMALL
    assert f(q, k, None, None, *o, WS, need) == _lib.PS_ERR_INVALID_ARG
    for i in range(5):
        assert f(q, k, do, None, *(p if j != i else None for j, p in enumerate(o)), WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(q, k, do, None, o[0], o[0] + 64, *o[2:], WS, need) == _lib.PS_ERR_OVERLAP
    assert f(q, k, do, None, FAKE, *o[1:], WS, need) == _lib.PS_ERR_OVERLAP        # dq in q
    assert f(q, k, do, o[5] + 64, *o, WS, need) == _lib.PS_ERR_OVERLAP             # states' gradients meet


def test_step_refusals(lib, no_device):
    s, x = shape(tokens=1), inputs(tokens=1)
    f = lib.ps_delta_step
    assert f(shape(tokens=0), x, H0, 2, None, None, OUT, None) == _lib.PS_OK
    assert f(shape(cu=FAKE), x, H0, 2, None, None, OUT, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, H0, -1, None, None, OUT, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, None, 2, None, None, OUT, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, H0, 2, HT + 1, None, OUT, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, H0, 2, None, None, None, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, H0, 2, None, None, H0 + 64, None) == _lib.PS_ERR_OVERLAP
    assert f(s, x, H0, 2, H0 + 64, None, OUT, None) == _lib.PS_ERR_OVERLAP


def test_pages_refusals(lib, no_device):
    import struct
    pool = lambda *x: struct.pack("@" + "Pq" * (len(x) // 2), *x)  # noqa: E731
    A, B, C, D, E = (FAKE + (i << 32) for i in range(5))
    need = lib.ps_pages_workspace_size(4, 100)
    assert need % 256 == 0 and need >= 4 * (4 + 300) and lib.ps_pages_workspace_size(-1, 5) == 0
    copy = lib.ps_pages_copy
    assert copy(pool(A, 64), 1, 100, B, C, 0, None) == _lib.PS_OK
    assert copy(pool(A, 0), 1, 100, B, C, 3, None) == _lib.PS_ERR_INVALID_ARG
    assert copy(pool(A, 64), 129, 100, B, C, 3, None) == _lib.PS_ERR_INVALID_ARG
    assert copy(pool(A, 64), 1, 100, None, C, 3, None) == _lib.PS_ERR_INVALID_ARG
    assert copy(pool(A, 64), 1, 100, B + 2, C, 3, None) == _lib.PS_ERR_INVALID_ARG
    assert copy(pool(A, 64, A + 640, 64), 2, 100, B, C, 3, None) == _lib.PS_ERR_OVERLAP
    assert copy(pool(A, 64), 1, 100, A + 640, C, 3, None) == _lib.PS_ERR_OVERLAP
    fork = lambda *a: lib.ps_pages_fork(*a, None)  # noqa: E731
    base = [A, B, 4, 8, C, 4, 16, D, pool(E, 64), 1, 100, A + (1 << 20), B + (1 << 20), None, WS, need]
    bad = lambda i, v: fork(*(base[:i] + [v] + base[i + 1:]))  # noqa: E731
    assert bad(6, 0) == bad(4, None) == bad(7, None) == bad(2, -1) == bad(0, None) == _lib.PS_ERR_INVALID_ARG
    assert bad(14, WS + 64) == bad(14, None) == _lib.PS_ERR_INVALID_ARG
    assert bad(15, need - 1) == _lib.PS_ERR_WORKSPACE_TOO_SMALL
    assert bad(11, A + 64) == bad(12, D) == bad(13, E + 64) == bad(7, WS + 64) == _lib.PS_ERR_OVERLAP
    grow = lambda *a: lib.ps_pages_grow(*a, None)  # noqa: E731
    assert grow(A, B, C, 4, 8, 0, D, 100, None, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert grow(A, B, None, 4, 8, 16, D, 100, None, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert grow(A, B, C, 4, 8, 16, A + 8, 100, None, WS, need) == _lib.PS_ERR_OVERLAP
    assert lib.ps_pages_free(A, 4, 8, None, A + 8, 100, None) == _lib.PS_ERR_OVERLAP
    assert lib.ps_pages_free(None, 4, 8, None, D, 100, None) == _lib.PS_ERR_INVALID_ARG
    assert lib.ps_pages_free(None, 0, 8, None, None, 0, None) == _lib.PS_OK
    assert lib.ps_pages_free(A, 1 << 20, 1 << 20, None, D, 100, None) == _lib.PS_ERR_INVALID_ARG
    assert lib.ps_pages_compact(A, 4, 8, D, pool(E, 64), 1, 100, None, WS, 100, None) == _lib.PS_ERR_WORKSPACE_TOO_SMALL
    assert lib.ps_pages_compact(A, 4, 8, D, pool(E, 64), 1, 100, E, WS, need, None) == _lib.PS_ERR_OVERLAP


def test_python_layer_refuses_cpu_tensors():
    from prefix_scan_gb300 import api
    x = [torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2), torch.zeros(1, 4, 2)]
    for call in (api.delta_rule, api.delta_rule_forward, lambda *a: api.delta_rule_step(*a, torch.zeros(1, 2, 8, 8))):
        with pytest.raises(ValueError, match="CUDA"):
            call(*x)
    table = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.pages_free(table, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        api.pages_copy(torch.zeros(4, 4), table[0], table[0])


def test_reference_gradients_against_differences():
    # the tests' reference itself, in 64 bits: central differences of third-order error, relative 1e-7
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    T, hk, hv, k, v = 9, 1, 2, 4, 3
    x = [r(T, hk, k), r(T, hk, k), r(T, hv, v), -r(T, hv).abs(), torch.sigmoid(r(T, hv)), r(hv, k, v)]
    do, dht = r(T, hv, v), r(hv, k, v)
    d = ref.sequence(*x[:5], 0.5, x[5], do, dht)

    def value(y):
        out = ref.sequence(*y[:5], 0.5, y[5])
        return float((out["o"] * do).sum() + (out["state"] * dht).sum())

    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dh0")):
        step = 1e-4 * r(*x[i].shape)
        a, b = ([t + s * step if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        slope = (value(a) - value(b)) / 2
        want = float((d[name] * step).sum())
        assert abs(slope - want) <= 1e-6 * float(d[name].norm() * step.norm()), name
