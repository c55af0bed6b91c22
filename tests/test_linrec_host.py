"""The gated linear recurrence without a GPU: sizes, refusals before anything is enqueued, the 64-bit reference's gradients
against its own differences, and that its tolerances find planted mistakes."""
from __future__ import annotations

import pytest

from prefix_scan_gb300 import _lib
from prefix_scan_gb300 import build as nvbuild

torch = pytest.importorskip("torch")

import linrec_reference as ref  # noqa: E402

FAKE = 1 << 40   # never dereferenced: every call below fails validation first
BF16, F16, F32 = _lib.PS_REAL_BF16, _lib.PS_REAL_F16, _lib.PS_REAL_F32


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


def shape(seqs=2, tokens=300, cu=0, channels=64, code=BF16, gate=F32, tied=0):
    return _lib.LINREC_SHAPE.pack(seqs, tokens, cu, channels, code, gate, tied)


def tensor(p, tokens=300, channels=64):
    return _lib.LINREC_TENSOR.pack(p, tokens * channels, channels)


X, G, DH, H0, HT, OUT, OUT2, WS = (FAKE + (i << 32) for i in range(8))


def test_workspace_size(lib):
    f = lib.ps_linrec_workspace_size
    assert f(shape(seqs=0), 0) == 0 and f(shape(tokens=0), 0) % 256 == 0
    for bad in (dict(channels=0), dict(code=7), dict(gate=F16), dict(seqs=-1), dict(tokens=-1), dict(tokens=1 << 32), dict(cu=FAKE + 2),
                dict(seqs=1 << 20, tokens=1 << 11), dict(tokens=(1 << 31) - 512, seqs=1), dict(channels=1 << 31),
                dict(channels=1 << 30, tokens=1 << 15), dict(seqs=1 << 30, tokens=1, channels=1 << 10)):
        assert f(shape(**bad), 0) == 0, bad
    for d in (1, 63, 64, 65, 4096):
        for tokens in (1, 128, 129, 4096):
            infer, train = f(shape(seqs=1, tokens=tokens, channels=d), 0), f(shape(seqs=1, tokens=tokens, channels=d), 1)
            tiles = -(-tokens // 512)
            assert infer % 256 == 0 and train % 256 == 0
            assert infer >= 4 * d + (tiles * d * 12 + 256 if tiles > 1 else 0)   # a copy of the states; maps and states of tiles
            assert train >= infer + tiles * d * 4                                # the states before the tiles
    assert f(None, 0) == 0


def test_forward_refusals(lib, no_device):
    s, x, g = shape(), tensor(X), tensor(G)
    need = lib.ps_linrec_workspace_size(s, 0)
    f = lambda *a: lib.ps_linrec_forward(*a, None)  # noqa: E731
    assert f(shape(seqs=0), None, None, None, None, None, 0, None, 0) == _lib.PS_OK
    assert f(None, x, g, None, None, OUT, 0, WS, need) == _lib.PS_ERR_INVALID_ARG
    for bx, bg in ((None, g), (x, None), (tensor(0), g), (x, tensor(0)), (tensor(X + 1), g), (x, tensor(G + 2))):
        assert f(s, bx, bg, None, None, OUT, 0, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, H0 + 2, None, OUT, 0, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, None, HT + 1, OUT, 0, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, None, None, None, 0, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, None, None, OUT + 1, 0, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, None, None, OUT, 0, None, need) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, None, None, OUT, 0, WS + 16, need) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, None, None, OUT, 0, WS, need - 1) == _lib.PS_ERR_WORKSPACE_TOO_SMALL
    assert f(s, x, g, None, None, OUT, 1, WS, need) == _lib.PS_ERR_WORKSPACE_TOO_SMALL   # training keeps more
    assert f(s, x, g, None, None, X + 512, 0, WS, need) == _lib.PS_ERR_OVERLAP           # output in x
    assert f(s, x, g, None, None, X, 0, WS, need) == _lib.PS_ERR_OVERLAP                 # in place of x
    assert f(s, x, g, None, OUT + 256, OUT, 0, WS, need) == _lib.PS_ERR_OVERLAP          # state in the output
    assert f(s, x, g, H0, H0 + 256, OUT, 0, WS, need) == _lib.PS_ERR_OVERLAP             # states meet, not the same
    assert f(s, x, g, H0, H0, OUT, 1, WS, lib.ps_linrec_workspace_size(s, 1)) == _lib.PS_ERR_OVERLAP   # the backward pass reads h0
    assert f(s, x, g, None, None, WS + 512, 0, WS, need) == _lib.PS_ERR_OVERLAP
    assert f(s, x, g, WS + 256, None, OUT, 0, WS, need) == _lib.PS_ERR_OVERLAP


def test_backward_refusals(lib, no_device):
    s, x, g, dh = shape(), tensor(X), tensor(G), tensor(DH)
    need = lib.ps_linrec_workspace_size(s, 1)
    f = lambda *a: lib.ps_linrec_backward(s, *a, None)  # noqa: E731
    assert f(x, g, None, dh, None, OUT, OUT2, None, WS, need - 1) == _lib.PS_ERR_WORKSPACE_TOO_SMALL
    for bad in ((None, g, dh), (x, None, dh), (x, g, None), (tensor(X + 1), g, dh)):
        assert f(*bad[:2], None, bad[2], None, OUT, OUT2, None, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(x, g, None, dh, None, None, OUT2, None, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(x, g, None, dh, None, OUT, None, None, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(x, g, None, dh, None, OUT, OUT2 + 2, None, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(x, g, H0 + 1, dh, None, OUT, OUT2, None, WS, need) == _lib.PS_ERR_INVALID_ARG
    assert f(x, g, None, dh, None, OUT, OUT2, None, WS + 8, need) == _lib.PS_ERR_INVALID_ARG
    assert f(x, g, None, dh, None, OUT, OUT + 64, None, WS, need) == _lib.PS_ERR_OVERLAP
    assert f(x, g, None, dh, None, X, OUT2, None, WS, need) == _lib.PS_ERR_OVERLAP
    assert f(x, g, H0, dh, None, OUT, OUT2, H0, WS, need) == _lib.PS_ERR_OVERLAP         # dh0 in place of h0
    assert f(x, g, H0, dh, HT, OUT, OUT2, HT + 64, WS, need) == _lib.PS_ERR_OVERLAP      # states' gradients meet


def test_step_refusals(lib, no_device):
    s, x, g = shape(tokens=1), tensor(X, 1), tensor(G, 1)
    f = lambda *a: lib.ps_linrec_step(*a, None)  # noqa: E731
    assert f(shape(tokens=0), x, g, H0, 2, None, None, OUT) == _lib.PS_OK
    assert f(shape(cu=FAKE), x, g, H0, 2, None, None, OUT) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, H0, -1, None, None, OUT) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, None, 2, None, None, OUT) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, H0, 2, HT + 1, None, OUT) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, H0, 2, None, HT + 2, OUT) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, H0, 2, None, None, None) == _lib.PS_ERR_INVALID_ARG
    assert f(s, x, g, H0, 2, None, None, H0 + 64) == _lib.PS_ERR_OVERLAP
    assert f(s, x, g, H0, 2, H0 + 64, None, OUT) == _lib.PS_ERR_OVERLAP
    assert f(s, x, g, H0, 2, None, None, X) == _lib.PS_ERR_OVERLAP


def test_python_layer_refuses_what_it_cannot_run():
    from prefix_scan_gb300 import api
    x = torch.zeros(2, 4, 8)
    calls = [api.linear_recurrence, api.linear_recurrence_forward, lambda *a: api.linear_recurrence_step(*a, torch.zeros(2, 8))]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call(x, x)
    for which in range(2):
        y = [x, x.clone()]
        y[which] = y[which].clone().requires_grad_()
        for call in (calls[0], calls[2]):
            with pytest.raises(ValueError, match="requires gradients"):
                call(*y)
        with pytest.raises(ValueError, match="CUDA"):   # which has a backward pass of its own
            calls[1](*y)
    with pytest.raises(TypeError, match="float64"):
        api.linear_recurrence_workspace_size(x.double())
    with pytest.raises(ValueError, match="packed"):
        api.linear_recurrence_workspace_size(x[0])


@pytest.mark.parametrize("tied", [False, True])
def test_reference_gradients_against_differences(tied):
    # central differences in 64 bits: the third-order term of a step of 1e-4 is below 1e-7 of the slope
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x = [r(9, 3), -r(9, 3).abs(), r(3)]
    dh, dht = r(9, 3), r(3)
    d = ref.sequence(*x, tied, dh, dht)

    def value(y):
        out = ref.sequence(*y, tied)
        return float((out["h"][0] * dh).sum() + (out["state"][0] * dht).sum())

    for i, name in enumerate(("dx", "dg", "dh0")):
        step = 1e-4 * r(*x[i].shape)
        a, b = ([t + s * step if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        slope, want = (value(a) - value(b)) / 2, float((d[name][0] * step).sum())
        assert abs(slope - want) <= 1e-6 * float(d[name][0].norm() * step.norm()), name


def test_tolerances_find_planted_mistakes():
    gen = torch.Generator().manual_seed(5)
    x, g = torch.randn(600, 8, generator=gen), -0.05 * torch.rand(600, 8, generator=gen)
    want = ref.sequence(x, g, dh=x)
    h, dg = want["h"][0].float(), want["dg"][0].float()
    ref.check(h, want["h"])
    ref.check(dg, want["dg"])
    off = []
    lost = h.clone()                                    # the state is lost at a tile's start
    lost[128:] = ref.sequence(x[128:], g[128:])["h"][0].float()
    off.append((lost, "h"))
    off.append((h.roll(1, 0), "h"))                     # a token too late
    off.append((ref.sequence(x, g.bfloat16())["h"][0].float(), "h"))   # decays of 16 bits
    off.append((ref.sequence(x, g, dh=x.bfloat16())["dg"][0].float(), "dg"))
    off.append((dg + 1e-4 * dg.abs().mean(), "dg"))
    for got, name in off:
        with pytest.raises(AssertionError):
            ref.check(got, want[name])
