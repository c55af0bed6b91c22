"""A small example: beam search on a gated-linear-recurrence layer, and one training step of it.

    python -m prefix_scan_gb300.searching [--beams 4] [--tokens 40]

A model of one layer: a token's embedding gives input and log decays, the layer's state gives logits.  Searching: prompts of
different lengths run in one packed batch and their states go into pages of a pool, a page a beam; then, token after token,
beam_select chooses the best continuations of all of an item's beams, pages_reorder gives each beam the state of the beam that
it continues, and linear_recurrence_step takes the chosen tokens in.  Every hypothesis' score is compared with that of its whole
token stream, run at once.  Training: the layer forward and backward over the packed prompts, with a step against the gradient.
Synthetic weights and prompts; needs a GPU.
"""
from __future__ import annotations

import argparse

import torch

from . import api


class Model:
    """Weights of one layer: tokens to inputs and log decays, states to logits."""

    def __init__(self, vocab: int, channels: int, seed: int):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.x = rnd(vocab, channels)
        self.g = -torch.nn.functional.softplus(rnd(vocab, channels) - 2)
        self.out = 3 * rnd(channels, vocab) / channels ** 0.5

    def logits(self, h: torch.Tensor) -> torch.Tensor:
        return h @ self.out


def search(lens: list, beams: int, steps: int, vocab: int = 300, channels: int = 96, seed: int = 0) -> tuple[torch.Tensor, float]:
    """Runs the searching half; returns the hypotheses' scores [items, beams], best first, and how far they are from those of
    their whole token streams at most."""
    model = Model(vocab, channels, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    n, eos = len(lens), 0
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    prompt = torch.randint(1, vocab, (sum(lens),), device="cuda", generator=gen)
    h, states = api.linear_recurrence(model.x[prompt], model.g[prompt], tied=True, cu_seqlens=cu, output_final_state=True)

    # the first choice has one beam an item; its state is what every beam starts from
    slots = torch.arange(n * beams, dtype=torch.int32, device="cuda")
    pool = torch.empty(n * beams, channels, device="cuda")
    pool[::beams] = states
    scores = torch.full((n, beams), float("-inf"), device="cuda")
    scores[:, 0] = 0
    ended = torch.zeros(n, beams, dtype=torch.uint8, device="cuda")
    logits = model.logits(states)[:, None].expand(n, beams, vocab)
    history = torch.empty(n * beams, 0, dtype=torch.int64, device="cuda")
    for _ in range(steps):
        choice = api.beam_select(logits, scores, ended=ended, eos_token=eos)
        scores, ended = choice.scores, choice.ended
        slots, _ = api.pages_reorder(slots, choice.parents, pool)
        tokens = choice.tokens.flatten().long()
        history = torch.cat([history[choice.parents.flatten().long()], tokens[:, None]], 1)
        out = api.linear_recurrence_step(model.x[tokens][:, None], model.g[tokens][:, None], pool, tied=True, slots=slots)
        logits = model.logits(out[:, 0]).view(n, beams, vocab)

    # the same hypotheses from their whole token streams
    off = 0.0
    for i in range(n):
        for b in range(beams):
            said = history[i * beams + b]
            end = (said == eos).nonzero()[:, 0]
            said = said[:int(end[0]) + 1] if len(end) else said
            stream = torch.cat([prompt[int(cu[i]):int(cu[i + 1])], said])
            h, _ = api.linear_recurrence(model.x[stream][None], model.g[stream][None], tied=True)
            at = torch.log_softmax(model.logits(h[0, lens[i] - 1:-1]).double(), -1)
            off = max(off, abs(float(at.gather(1, said[:, None]).sum()) - float(scores[i, b])))
    return scores, off


def gradients(x: torch.Tensor, g: torch.Tensor, cu: torch.Tensor, target: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The layer's outputs h over packed prompts, and the gradients of the loss |h - target|^2 / 2 of its inputs and log decays."""
    h, _, saved = api.linear_recurrence_forward(x, g, tied=True, cu_seqlens=cu)
    dx, dg, _ = api.linear_recurrence_backward(saved, h - target)
    return h, dx, dg


def train(lens: list, vocab: int = 300, channels: int = 96, seed: int = 2) -> tuple[float, float]:
    """The loss |h - target|^2 / 2 before and after a short step of the inputs and log decays against its gradient."""
    model = Model(vocab, channels, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    prompt = torch.randint(1, vocab, (sum(lens),), device="cuda", generator=gen)
    x, g = model.x[prompt], model.g[prompt]
    target = torch.randn(x.shape, device="cuda", generator=gen)
    losses = []
    for _ in range(2):
        h, dx, dg = gradients(x, g, cu, target)
        losses.append(float((h - target).square().sum() / 2))
        x, g = x - 0.05 * dx, (g - 0.01 * dg).clamp(max=0)
    return losses[0], losses[1]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=40, help="tokens to search for")
    a = ap.parse_args()
    scores, off = search([300, 7, 1, 129], a.beams, a.tokens)
    print(f"searching: best scores {[round(float(s), 2) for s in scores[:, 0]]}, off their whole streams' by {off:.1e} at most")
    before, after = train([300, 7, 1, 129])
    print(f"training: loss {before:.1f} -> {after:.1f}")


if __name__ == "__main__":
    main()
