"""Whole prompts by the single-step kernel, which works in f32 throughout: what a caller uses who needs more than the 16 bits that
the chunked kernels' operands keep.

Tolerance 2^-20: each token's sums have up to 128 terms of f32, random roundings of 2^-25 each: 2^-21.5 of the terms, independent from
token to token, so the states and outputs, sums over tokens, are off by that much too; 300 roundings of the state add 2^-21."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import delta_reference as ref  # noqa: E402
from prefix_scan_gb300 import api  # noqa: E402
from test_gpu_delta import DEV, F32, STEP, inputs, near, states  # noqa: E402


@pytest.mark.parametrize("hk,hv,k,v", [(1, 3, 80, 56), (2, 2, 128, 128)])
def test_prompts_by_steps(hk, hv, k, v):
    lens = [300, 1, 0, 129]
    x = inputs(300, hk, hv, k, v, F32, 7, seqs=len(lens), decay=0.05)
    state = states(len(lens), hv, k, v, 8)
    was = state.clone()
    o = api.delta_rule_step(*x, state, lengths=torch.tensor(lens, dtype=torch.int32, device=DEV))
    for i, n in enumerate(lens):
        assert (o[i, n:] == 0).all()
        if n:
            want = ref.sequence(*(t[i, :n] for t in x), k ** -0.5, was[i])
            near(o[i, :n], want["o"], STEP)
            near(state[i], want["state"], STEP)
        else:
            assert torch.equal(state[i], was[i])
