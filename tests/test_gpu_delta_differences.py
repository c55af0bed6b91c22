"""Gradients of the gated delta rule on the GPU against differences along themselves (delta_differences.py has the tolerance and
its derivation; test_delta_differences_host.py shows that the check finds planted mistakes)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from delta_differences import NAMES, agrees  # noqa: E402
from prefix_scan_gb300 import api  # noqa: E402
from test_gpu_delta import DEV, F32, cu_of, inputs, states  # noqa: E402


@pytest.mark.parametrize("hk,hv,k,v", [(1, 2, 64, 48), (2, 2, 128, 130)])
@pytest.mark.parametrize("which", range(6))
def test_gradients_against_differences_along_them(which, hk, hv, k, v):
    lens = [150, 61]
    x = [*inputs(sum(lens), hk, hv, k, v, F32, 91), states(2, hv, k, v, 92)]
    dht, do = states(2, hv, k, v, 93), torch.randn(sum(lens), hv, v, device=DEV, generator=torch.Generator(device=DEV).manual_seed(95))
    _, _, saved = api.delta_rule_forward(*x[:5], cu_seqlens=cu_of(lens), initial_state=x[5])
    got = api.delta_rule_backward(saved, do, d_final_state=dht)[which]

    def value(changed):
        y = [changed if i == which else t for i, t in enumerate(x)]
        o, last = api.delta_rule(*y[:5], cu_seqlens=cu_of(lens), initial_state=y[5], output_final_state=True)
        return ((o.double() * do.double()).sum() + (last.double() * dht.double()).sum()).item()

    ok, slope, want = agrees(value, x[which], got, NAMES[which], torch.Generator(device=DEV).manual_seed(94))
    assert ok, (slope, want)
