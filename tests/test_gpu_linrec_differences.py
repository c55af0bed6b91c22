"""Gradients of the gated linear recurrence against central differences of its own outputs along themselves, for the training
calls as they are used.

L(x) = <d_h, h> + <d_ht, h_T>.  The direction is the gradient plus noise of half its norm, 1 % of the input's norm long.  L is
linear in x and the initial state, and along g its third-order term is below 0.05 % of the slope (log decays change by 1 % of their
size, memories of up to 100 tokens with them: (0.01)^2 / 6 x a factor of some tens).  f32 outputs leave less than that.  A gradient
that is zero, halved, turned round or another's is off by half or more."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402

DEV = "cuda"
TOLERANCE = 0.005


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("lens", [[150], [40, 0, 200, 1], [700]])
@pytest.mark.parametrize("which", ["dx", "dg", "dh0"])
def test_against_differences(which, lens, tied):
    gen = torch.Generator(device=DEV).manual_seed(7)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    n, d = sum(lens), 40
    cu = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    base = {"dx": rnd(n, d), "dg": -0.3 * rnd(n, d).abs() - 0.01, "dh0": rnd(len(lens), d)}
    dh, dht = rnd(n, d), rnd(len(lens), d)
    h, _, saved = api.linear_recurrence_forward(base["dx"], base["dg"], tied=tied, cu_seqlens=cu, initial_state=base["dh0"],
                                                output_final_state=True)
    got = dict(zip(("dx", "dg", "dh0"), api.linear_recurrence_backward(saved, dh, d_final_state=dht)))[which].double()

    def value(changed):
        y = {**base, which: changed}
        h, last = api.linear_recurrence(y["dx"], y["dg"], tied=tied, cu_seqlens=cu, initial_state=y["dh0"], output_final_state=True)
        return float((h.double() * dh).sum() + (last.double() * dht).sum())

    step = got + 0.5 * got.norm() / got.numel() ** 0.5 * rnd(*got.shape)
    step *= 0.01 * base[which].norm() / step.norm()
    plus, minus = (base[which] + step).float(), (base[which] - step).float()
    slope = (value(plus) - value(minus)) / 2
    want = float((got * (plus.double() - minus.double())).sum()) / 2
    assert abs(slope - want) <= TOLERANCE * abs(want)
