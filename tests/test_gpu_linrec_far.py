"""The gated linear recurrence on tensors of more than 2^31 numbers: outputs and every gradient of the last rows, which lie more than
2^32 bytes behind the first ones, against the recurrence in 64 bits (rows differ, so that a row from elsewhere is found)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import linrec_reference as ref  # noqa: E402
from prefix_scan_gb300 import api  # noqa: E402

DEV, BF16 = "cuda", torch.bfloat16


@pytest.mark.parametrize("packed", [False, True])
def test_rows_behind_2_to_the_32_bytes(packed):
    tokens, d = (1 << 15) + 300, 1 << 16
    if torch.cuda.mem_get_info()[0] < 50 << 30:
        pytest.skip("not enough free memory")
    gen = torch.Generator(device=DEV).manual_seed(3)
    wide = lambda t: t.to(BF16).repeat(1, d // 512)  # noqa: E731
    x, dh = (wide(torch.randn(tokens, 512, device=DEV, generator=gen)) for _ in range(2))
    g = wide(-0.5 * torch.rand(tokens, 512, device=DEV, generator=gen))
    cu = torch.tensor([0, 5, tokens], dtype=torch.int32, device=DEV) if packed else None
    view = (lambda t: t) if packed else lambda t: t[None]
    h, state, saved = api.linear_recurrence_forward(view(x), view(g), cu_seqlens=cu, output_final_state=True)
    dx, dg, _ = api.linear_recurrence_backward(saved, view(dh))
    rows, columns = slice(tokens - 1200, tokens), slice(d - 40, d)
    want = ref.sequence(x[rows, columns].cpu(), g[rows, columns].cpu(), dh=dh[rows, columns].cpu())
    # a state of 900 tokens before is forgotten: e^(-0.25 * 900) of it is left
    for name, t in (("h", h), ("dx", dx), ("dg", dg)):
        ref.check(t.view(tokens, d)[-300:, columns], tuple(y[-300:] for y in want[name]), name)
    ref.check(state[-1, columns], want["state"], "state")
    # and the first rows are still the first rows'
    want = ref.sequence(x[:5, :40].cpu(), g[:5, :40].cpu())
    ref.check(h.view(tokens, d)[:5, :40], want["h"], "the first rows' h")
