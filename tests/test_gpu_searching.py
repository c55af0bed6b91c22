"""The beam-search example: hypotheses found step by step, on states that are reordered in place, have the scores of their whole
token streams; the search finds what a search over all sequences finds where the beam is wide enough for it; gradients of the
training half against differences.

Tolerance of a score: each token's log softmax comes from logits of 96 products of 32 bits.  Products may be taken in tf32 nowhere
(torch's default), so a logit is off by 96 x 2^-24 of the sum of its terms' magnitudes, some 3 x 0.8 x 96^0.5 = 24: 1.4e-4 at
worst, on both sides, and states differ by their own roundings, less than that; 40 tokens of it: 40 x 2 x 1.4e-4."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api, searching  # noqa: E402

A_TOKEN = 2 * 1.4e-4


@pytest.mark.parametrize("lens,beams,steps", [([300, 7, 1, 129], 4, 40), ([1], 1, 3), ([64, 5], 8, 12), ([20] * 30, 3, 5)])
def test_hypotheses_have_their_whole_streams_scores(lens, beams, steps):
    scores, off = searching.search(lens, beams, steps)
    assert off <= steps * A_TOKEN
    assert (scores[:, :-1] >= scores[:, 1:]).all()


def test_a_wide_beam_finds_the_best_sequence_of_all():
    # 6 tokens, 3 steps: 36 beams hold every prefix of two tokens, so the best of all 216 (or ended sooner) is found
    scores, _ = searching.search([9], 36, 3, vocab=6, channels=32, seed=5)
    model = searching.Model(6, 32, 5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    prompt = torch.randint(1, 6, (9,), device="cuda", generator=gen)
    best = -float("inf")
    every = [[a] for a in range(6)]
    for _ in range(2):
        every = [s + [a] for s in every for a in range(6) if s[-1] != 0] + [s for s in every if s[-1] == 0]
    for said in every:
        stream = torch.cat([prompt, torch.tensor(said, device="cuda")])
        h, _ = api.linear_recurrence(model.x[stream][None], model.g[stream][None], tied=True)
        at = torch.log_softmax(model.logits(h[0, 8:-1]).double(), -1)
        best = max(best, float(at.gather(1, torch.tensor(said, device="cuda")[:, None]).sum()))
    assert abs(float(scores[0, 0]) - best) <= 3 * A_TOKEN


def test_training_runs():
    before, after = searching.train([300, 7, 1, 129])
    assert before > 0 and after == after
