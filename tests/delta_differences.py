"""Differences of the gated delta rule's outputs along a gradient, for the tests.

L(x) = <d_o, o> + <d_ht, h_T>.  The direction d is the gradient that is to be checked plus noise of half its norm, scaled to
|d| = SIZE of the input's norm.  So <gradient, d> is 0.89 |gradient| |d|, and a gradient that is zero, halved, turned round or of
another direction is off by half of that or more.

Tolerance: 1 % of <gradient, d>.  In 64 bits (L(x + d) - L(x - d)) / 2 is off by at most 0.05 % for k, 0.26 % for g, at 150
tokens and log decays down to -1, and by less than that for the others (nothing at all for q, v and h0, in which L is linear).
Values of L off by 6 x 2^-17 of each of its terms, independently, add 0.01 % of the slope, and 0.08 % for g with its smaller d;
three times as much is 0.24 %."""
from __future__ import annotations

import torch

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")
SIZE = {"dg": 0.002}
TOLERANCE = 0.01


def agrees(value, base, got, name, generator):
    """Whether ``value``'s central difference at ``base`` along ``got`` (and noise) is what ``got`` says.  ``value`` takes the
    changed input."""
    d = got.double() + 0.5 * got.double().norm() / base.numel() ** 0.5 * torch.randn(
        base.shape, dtype=torch.float64, device=base.device, generator=generator)
    if d.norm() == 0:
        d = torch.randn(base.shape, dtype=torch.float64, device=base.device, generator=generator)
    d *= SIZE.get(name, 0.02) * base.double().norm() / d.norm()
    plus, minus = ((base.double() + s * d).to(base.dtype) for s in (1, -1))
    slope = (value(plus) - value(minus)) / 2
    want = (got.double() * (plus.double() - minus.double())).sum().item() / 2   # as rounded
    return abs(slope - want) <= TOLERANCE * abs(slope), slope, want
