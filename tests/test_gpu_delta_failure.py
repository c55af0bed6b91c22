"""A chain of the gated delta rule whose bounded waits ran out: nothing that was computed from it looks like a result.

A correct launch never runs out of a wait, so the test sets the word by which such a chain tells the kernels after it (256
bytes before the end of the training workspace) and no wait is made to run out."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402
from test_gpu_delta import BF16, DEV, F16, F32, inputs, states  # noqa: E402


@pytest.mark.parametrize("dtype,beta_dtype", [(BF16, BF16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("hk,hv,k,v,cu", [(2, 4, 64, 48, [3, 70, 70, 203]), (1, 2, 37, 200, [0, 1900]), (2, 4, 128, 128, list(range(0, 2501, 50)))])
def test_gradients_after_a_failed_chain(dtype, beta_dtype, hk, hv, k, v, cu):
    tokens, n = cu[-1] + 5, len(cu) - 1
    x = inputs(tokens, hk, hv, k, v, dtype, 5, beta_dtype=beta_dtype)
    offsets = torch.tensor(cu, dtype=torch.int32, device=DEV)
    h0, dht, do = states(n, hv, k, v, 6), states(n, hv, k, v, 7), torch.randn(x[2].shape, device=DEV).to(dtype)
    # whatever the workspace held before
    ws = torch.full((api.delta_rule_workspace_size(x[0], x[2], offsets, train=True),), 255, dtype=torch.uint8, device=DEV)
    forward = lambda: api.delta_rule_forward(*x, cu_seqlens=offsets, initial_state=h0, workspace=ws)[2]  # noqa: E731
    saved = forward()
    want = api.delta_rule_backward(saved, do, d_final_state=dht)
    assert all(torch.isfinite(t).all() for t in want)
    ws[-256:-252].view(torch.int32).fill_(1)
    for _ in range(2):
        got = api.delta_rule_backward(saved, do, d_final_state=dht)
        for t in got[:5]:
            assert torch.isnan(t[cu[0]:cu[-1]]).all()
            assert (t[:cu[0]] == 0).all() and (t[cu[-1]:] == 0).all()
        assert torch.isnan(got[5]).all()
    for a, b in zip(api.delta_rule_backward(forward(), do, d_final_state=dht), want):   # the next forward call starts anew
        assert torch.equal(a, b)
