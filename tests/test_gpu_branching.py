"""The serving and training example: sequences branch in a pool of states, survive compaction and agree with their whole
token streams; a step against the gradient lowers the loss.

The branches' states pass the chunked kernel once and f32 steps after it, the whole streams the chunked kernel alone: each is
off by at most 6 x 2^-17 (test_gpu_delta.py)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import branching  # noqa: E402


@pytest.mark.parametrize("lens,heads", [([1], 1), ([700, 234, 1, 164], 8), ([64, 63, 65], 3)])
def test_serving(lens, heads):
    assert branching.serve(lens, heads) <= 12 * 2.0 ** -17


def test_training():
    before, after = branching.train([700, 234, 1, 164], 4)
    assert after < before
