"""The training half of the beam-search example: the gradients that it steps against, compared with differences of its own loss.

L = |h - target|^2 / 2.  The direction is the gradient plus noise of half its norm, 0.1 % of the input's norm long.  L is
quadratic in x, so central differences have no error there.  Along g the slope's third-order term is (0.001)^2 / 6 of it times
a factor of some hundreds (memories of up to a thousand tokens change by as much as their decays do, cubed): below 1e-4.  The N
outputs, of 32 bits and off independently by 2^-21 of themselves or so, leave N^0.5 2^-21 of L, and the slope is 0.001 N times a few
tenths: below 1e-4 of it for N of some thousands and more.  A gradient that is zero, halved, turned round or another's
is off by half or more."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import searching  # noqa: E402

DEV = "cuda"
TOLERANCE = 0.005


@pytest.mark.parametrize("which", ["x", "g"])
@pytest.mark.parametrize("lens", [[70, 5], [300, 7, 1, 129]])
def test_gradients_against_differences_of_the_loss(lens, which):
    gen = torch.Generator(device=DEV).manual_seed(9)
    model = searching.Model(300, 96, 4)
    prompt = torch.randint(1, 300, (sum(lens),), device=DEV, generator=gen)
    cu = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    at = {"x": model.x[prompt], "g": model.g[prompt]}
    target = torch.randn(at["x"].shape, device=DEV, generator=gen)
    _, dx, dg = searching.gradients(at["x"], at["g"], cu, target)
    got = {"x": dx, "g": dg}[which].double()

    def loss(value):
        h, _, _ = searching.gradients(**{**at, which: value}, cu=cu, target=target)
        return float((h.double() - target).square().sum() / 2)

    step = got + 0.5 * got.norm() / got.numel() ** 0.5 * torch.randn(got.shape, device=DEV, generator=gen)
    step *= 0.001 * at[which].norm() / step.norm()
    plus, minus = (at[which] + step).float(), (at[which] - step).float()
    slope = (loss(plus) - loss(minus)) / 2
    want = float((got * (plus.double() - minus.double())).sum()) / 2
    assert abs(slope - want) <= TOLERANCE * abs(want)
