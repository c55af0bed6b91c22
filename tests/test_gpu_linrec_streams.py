"""Training of the gated linear recurrence on a stream that both calls are given, with tensors of the current stream that are
dropped, and whose memory is written over, as soon as the calls return."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402
from test_gpu_linrec import BF16, DEV, check_packed, cu_of, make, states  # noqa: E402


def test_both_calls_on_a_stream_that_is_not_the_tensors():
    lens = [900, 300]
    host = make(sum(lens), 128, BF16, BF16, 33)
    h0, dht = states(2, 128, 34)
    x, g, dh = (t.to(DEV) for t in host)
    cu, start, end = cu_of(lens), h0.to(DEV), dht.to(DEV)
    workspace = torch.empty(api.linear_recurrence_workspace_size(x, cu, train=True), dtype=torch.uint8, device=DEV)
    side, big = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            big @ big
    h, state, saved = api.linear_recurrence_forward(x, g, cu_seqlens=cu, initial_state=start, output_final_state=True,
                                                    workspace=workspace, stream=side)
    dx, dg, dh0 = api.linear_recurrence_backward(saved, dh, d_final_state=end, stream=side)
    sizes = [t.numel() * t.element_size() for t in (workspace, x, g, cu, dh, start, end)]
    del saved, workspace, x, g, cu, dh, start, end
    new = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes]   # on the current stream, at once
    torch.cuda.synchronize()
    del new
    check_packed({"h": h, "state": state, "dx": dx, "dg": dg, "dh0": dh0}, *host[:2], lens, host[2], h0, dht, False)


def test_two_calls_at_once():
    # their tiles share the SMs, each call's wait for one another only
    sides = [torch.cuda.Stream() for _ in range(2)]
    data = [[t.to(DEV).view(4, 2048, 700) for t in make(4 * 2048, 700, BF16, BF16, 50 + i)] for i in range(2)]

    def run(x, g, dh, stream=None):
        h, state, saved = api.linear_recurrence_forward(x, g, output_final_state=True, stream=stream)
        return (h, state, *api.linear_recurrence_backward(saved, dh, stream=stream)[:2])

    want = [run(*d) for d in data]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [run(*d, stream=s) for d, s in zip(data, sides)]
        torch.cuda.synchronize()
        for one, w in zip(got, want):
            assert all(torch.equal(a, b) and a.isfinite().all() for a, b in zip(one, w))
