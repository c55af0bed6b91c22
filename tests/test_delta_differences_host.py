"""That the check of gradients against differences can fail: mistakes planted in the 64-bit reference's gradients, on the CPU."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import delta_reference as ref  # noqa: E402
from delta_differences import NAMES, agrees  # noqa: E402

MISTAKES = {"zero": lambda t, r: 0 * t, "half": lambda t, r: t / 2, "turned round": lambda t, r: -t, "a tenth too large": lambda t, r: 1.1 * t,
            "another direction": lambda t, r: t.norm() * r / r.norm()}


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("which", range(6))
def test_planted_mistakes_are_found(which, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    lens, n, k, v = [150, 61], 211, 64, 48
    g = -torch.rand(n, 2, generator=gen, dtype=torch.float64) * torch.logspace(-3, 0, 2, dtype=torch.float64)
    x = [unit(rnd(n, 1, k)), unit(rnd(n, 1, k)), rnd(n, 2, v), g, torch.sigmoid(rnd(n, 2)), 0.3 * rnd(2, 2, k, v)]
    do, dht = rnd(n, 2, v), 0.3 * rnd(2, 2, k, v)
    right = ref.packed(*x[:5], k ** -0.5, lens, x[5], do, dht)[NAMES[which]]

    def value(changed):
        y = [changed if i == which else t for i, t in enumerate(x)]
        out = ref.packed(*y[:5], k ** -0.5, lens, y[5])
        return ((out["o"] * do).sum() + (out["state"] * dht).sum()).item()

    ok, slope, want = agrees(value, x[which], right, NAMES[which], gen)
    assert ok, (slope, want)
    for name, wrong in MISTAKES.items():
        ok, slope, want = agrees(value, x[which], wrong(right, rnd(*right.shape)), NAMES[which], gen)
        assert not ok, (name, slope, want)
