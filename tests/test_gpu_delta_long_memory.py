"""States that the chunked kernels carry over very many chunks.

With gates of 0 nothing is written and a state only decays: h_T = exp(sum of g) h_0.  Each of n chunks multiplies it by a factor that
is rounded to f32 and rounds the product, errors of at most 2^-25 each and of random sign, rms 2^-25.8: 4 standard deviations of 2 n of them."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402
from test_gpu_delta import BF16, DEV, inputs, off, states  # noqa: E402


def test_decays_of_many_chunks():
    # 160 heads: the sequence is not cut
    T, hv = 16384, 160
    q, k, v, g, beta = inputs(T, 1, hv, 8, 8, BF16, 3, seqs=1)
    g = -torch.rand(1, T, hv, device=DEV, generator=torch.Generator(device=DEV).manual_seed(4)) * torch.logspace(-6, -3.5, hv, device=DEV)
    h0 = states(1, hv, 8, 8, 5)
    _, last = api.delta_rule(q, k, v, g, torch.zeros_like(beta), initial_state=h0, output_final_state=True)
    want = h0.double() * g.double().sum(1).exp()[..., None, None]
    assert off(last, want) <= 4 * (2 * T / 64) ** 0.5 * 2.0 ** -25.8
