"""Calls through which no gradients pass refuse inputs that require them (before anything touches a GPU)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from prefix_scan_gb300 import api  # noqa: E402


@pytest.mark.parametrize("which", range(6))
def test_inputs_that_require_gradients_are_refused(which):
    x = [torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2), torch.zeros(1, 4, 2),
         torch.zeros(1, 2, 8, 8)]
    x[which].requires_grad_()
    calls = [lambda: api.delta_rule(*x[:5], initial_state=x[5]), lambda: api.delta_rule_step(*x)]
    for call in calls:
        with pytest.raises(ValueError, match="requires gradients"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="CUDA"):   # which has a backward pass of its own
        api.delta_rule_forward(*x[:5], initial_state=x[5])
