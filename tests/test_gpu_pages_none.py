"""Page operations over no pools at all, as the C ABI has them: only tables and counts change."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402
from test_gpu_pages import ints  # noqa: E402


def test_no_pools():
    api.pages_copy([], ints([0, 1]), ints([2, 3]))
    table, ref = ints([[4, 0], [2, -1]]), ints([1, 0, 1, 0, 1])
    new, lengths, missing = api.pages_fork(table, ints([6, 3]), ints([1, 0]), ref, [], page_tokens=4)
    assert new.tolist() == [[1, -1], [4, 3]] and lengths.tolist() == [3, 6] and missing.item() == 0
    assert ref.tolist() == [1, 1, 1, 1, 2]
    api.pages_free(table, ref)
    assert api.pages_compact(new, ref, []).item() == 3
    assert new.tolist() == [[1, -1], [2, 0]] and ref.tolist() == [1, 1, 1, 0, 0]
