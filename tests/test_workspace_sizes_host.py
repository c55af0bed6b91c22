"""The workspace sizes that the torch wrappers tell: for what a call would refuse they refuse too, instead of telling 0 bytes."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from prefix_scan_gb300 import api  # noqa: E402


def test_log_decays_of_a_type_that_does_not_go_with_the_inputs():
    for dtype, gate in ((torch.bfloat16, torch.float16), (torch.float32, torch.bfloat16), (torch.float16, torch.float64)):
        x = torch.zeros(2, 300, 64, dtype=dtype)
        for train in (False, True):
            with pytest.raises(TypeError, match=str(gate).split(".")[1]):
                api.linear_recurrence_workspace_size(x, gate_dtype=gate, train=train)
            assert api.linear_recurrence_workspace_size(x, gate_dtype=dtype, train=train) > 0
            assert api.linear_recurrence_workspace_size(x, train=train) > 0


def test_beams_and_widths_that_the_choice_does_not_take():
    logits = torch.zeros(2, 65, 10)
    for width in (None, 0, 65):
        with pytest.raises(ValueError, match="64 candidates"):
            api.beam_workspace_size(logits, width=width)
    with pytest.raises(ValueError, match="256 beams"):
        api.beam_workspace_size(torch.zeros(2, 257, 10), width=4)
    assert api.beam_workspace_size(logits, width=64) > 0
    assert api.beam_workspace_size(torch.zeros(0, 4, 10)) == 0   # nothing to do
