"""Single-step calls with very many tokens, of which few count: zeros for the rest, 2^31 and more (token, column) places of a
block of 32 columns."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import delta_reference as ref  # noqa: E402
from prefix_scan_gb300 import api  # noqa: E402
from test_gpu_delta import BF16, DEV, STEP, near  # noqa: E402


def test_outputs_that_do_not_count():
    t, n = (1 << 26) + 5, 3
    one = lambda x, dtype, *size: torch.full((), x, dtype=dtype, device=DEV).expand(1, t, 1, *size)  # noqa: E731
    x = [one(0.5, BF16, 1), one(0.75, BF16, 1), one(1.25, BF16, 1), one(-0.125, torch.float32), one(0.5, BF16)]
    state = torch.full((1, 1, 1, 1), 2.0, device=DEV)
    out = torch.full((1, t, 1, 1), float("nan"), dtype=BF16, device=DEV)
    want = ref.sequence(*(y[0, :n] for y in x), 1.0, state[0].clone())
    api.delta_rule_step(*x, state, lengths=torch.tensor([n], dtype=torch.int32, device=DEV), scale=1.0, out=out)
    near(out[0, :n], want["o"], STEP)
    near(state[0], want["state"], STEP)
    assert (out[0, n:] == 0).all()
