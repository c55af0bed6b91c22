"""Arguments that the torch wrappers of the gated delta rule and the page operations judge by themselves, without a GPU."""
from __future__ import annotations

from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from prefix_scan_gb300 import _streams, api  # noqa: E402


def test_a_stream_of_another_device_is_refused():
    # the kernels would be launched there, on memory of the tensors' device
    elsewhere = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=1)
    with pytest.raises(ValueError, match="cuda:1"):
        _streams.enter(torch.device("cuda", 0), elsewhere)


def test_workspace_size_of_an_unknown_type():
    x = torch.zeros(1, 4, 2, 8, dtype=torch.float64)
    with pytest.raises(TypeError, match="float64"):
        api.delta_rule_workspace_size(x, x)
