"""The look-back of the gated linear recurrence under load: long chains of tiles whose states become known in ever another order.
What one warp decides there it has to decide for all of its lanes; every call ends, and every result is the first one's, bit for
bit."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402

DEV = "cuda"


@pytest.mark.parametrize("seqs,tokens,d", [(1, 40000, 32), (1, 9000, 700), (3, 5120, 96)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_chains_beside_other_work(dtype, seqs, tokens, d):
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(seqs, tokens, d, device=DEV, generator=gen).to(dtype)
    g = (-0.02 * torch.rand(seqs, tokens, d, device=DEV, generator=gen)).to(dtype)   # states of hundreds of tokens: all tiles matter

    def run():
        h, state, saved = api.linear_recurrence_forward(x, g, tied=True, output_final_state=True)
        return (h, state, *api.linear_recurrence_backward(saved, x)[:2])

    want = run()
    assert all(t.isfinite().all() for t in want)
    other, a = torch.cuda.Stream(), torch.randn(1024, 1024, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(200):
            a @ a
            a * 2
    for _ in range(25):
        for got, w in zip(run(), want):
            assert torch.equal(got, w)
    torch.cuda.synchronize()
