"""Tied weights 1 - exp(g) of the gated linear recurrence in 32 bits, where nothing else hides them: sequences of one token from
states of 0, so that h = (1 - exp(g)) x and dx = (1 - exp(g)) dh.

Tolerance, relative, u = 2^-24.  Above g = -7/16 (-5/32 for inputs of 16 bits, whose states are of 32) the weight is a polynomial
times g: within 2^-22.7 (the polynomial 2^-24.3, its last two roundings u each, those before them less than u in all), the
product with x u.  Below, it is 1 - a from the hardware's 2^x: 2^-22 a / (1 - a) of 2^x itself, |g| a / (1 - a) <= 1 times 1.5 u of
its argument (a product by a rounded constant), half a step of 1 - a, u / (1 - a), and u of the product."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402

DEV, U = "cuda", 2.0 ** -24


def gates(n, d):
    gen = torch.Generator().manual_seed(1)
    g = -torch.exp(-12 * torch.rand(n, d, generator=gen)) * 2        # from -2 up, over five orders of magnitude
    g[:, ::4] = -0.5 * torch.rand(n, (d + 3) // 4, generator=gen)    # and dense around where the two ways meet
    g[:, 1::4] = -0.0625 * (1 + 0.1 * torch.rand(n, (d + 2) // 4, generator=gen))
    return g


def check(got, g, x, name, near=-7 / 16):
    w = -torch.expm1(g.double())
    a = g.double().exp()
    tol = torch.where(g > near, torch.full_like(w, 2.0 ** -22.7), (2.0 ** -22 + U) * a / w + 1.5 * U + U / w) + U
    off = (got.cpu().double() / (w * x.double()) - 1).abs()
    worst = (off / tol).argmax()
    assert (off <= tol).all(), (name, float(g.flatten()[worst]), float(off.flatten()[worst]), float(tol.flatten()[worst]))


def data(n, d):
    gen = torch.Generator().manual_seed(2)
    return tuple(torch.randn(n, d, generator=gen) + 3 for _ in range(2))   # away from 0


@pytest.mark.parametrize("n,d", [(3000, 64), (700, 33)])
def test_whole_sequences_and_gradients(n, d):
    g, (x, dh) = gates(n, d), data(n, d)
    for cu in (None, torch.arange(n + 1, dtype=torch.int32, device=DEV)):
        view = (lambda t: t[:, None]) if cu is None else lambda t: t
        h, _, saved = api.linear_recurrence_forward(view(x.to(DEV)), view(g.to(DEV)), tied=True, cu_seqlens=cu)
        dx, _, _ = api.linear_recurrence_backward(saved, view(dh.to(DEV)))
        check(h.view(n, d), g, x, "h")
        check(dx.view(n, d), g, dh, "dx")


@pytest.mark.parametrize("n,d", [(3000, 64), (40, 2052)])
def test_steps(n, d):
    g, (x, _) = gates(n, d), data(n, d)
    state = torch.zeros(n, d, device=DEV)
    h = api.linear_recurrence_step(x.to(DEV)[:, None], g.to(DEV)[:, None], state, tied=True)
    check(h.view(n, d), g, x, "h")
    check(state, g, x, "state")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_states_of_16_bit_inputs(dtype):
    n, d = 2000, 64
    g, x = gates(n, d), data(n, d)[0].to(dtype)
    _, state = api.linear_recurrence(x.to(DEV)[:, None], g.to(DEV)[:, None], tied=True, output_final_state=True)
    check(state, g, x, "state", -5 / 32)
    state = torch.zeros(n, d, device=DEV)
    api.linear_recurrence_step(x.to(DEV)[:, None], g.to(DEV)[:, None], state, tied=True)
    check(state, g, x, "state of a step", -5 / 32)
    g = g.to(dtype)
    _, state = api.linear_recurrence(x.to(DEV)[:, None], g.to(DEV)[:, None], tied=True, output_final_state=True)
    check(state, g.float(), x, "state of gates of 16 bits", -5 / 32)
