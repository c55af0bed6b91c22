"""A small example: one gated-delta-rule layer serving branching sequences, and one training step of it.

    python -m prefix_scan_gb300.branching [--heads 8] [--tokens 700]

Serving: prompts of different lengths run in one packed batch, their states go into pages of a pool; each sequence branches
into candidates (pages_fork copies the state's page, which every token changes), the candidates take tokens of their own,
the best one of each stays and the others are freed, and the pool is compacted.  What the surviving sequences computed is
compared with running their whole token streams at once.  Training: the same layer forward and backward over the packed
prompts, with a step against the gradient that has to lower the loss.  Synthetic inputs; needs a GPU.
"""
from __future__ import annotations

import argparse

import torch

from . import api

ONE_PAGE = 1 << 30   # tokens "per page": a state's page is never full, so a branch always copies it


def layer_inputs(lead: tuple, heads: int, gen: torch.Generator):
    """q, k (unit norm), v in bf16, log decays and gates of ``lead`` tokens."""
    rnd = lambda *s: torch.randn(*lead, *s, device="cuda", generator=gen)  # noqa: E731
    q, k = (torch.nn.functional.normalize(rnd(heads, 64), dim=-1).bfloat16() for _ in range(2))
    return q, k, rnd(heads, 64).bfloat16(), -torch.nn.functional.softplus(rnd(heads)), torch.sigmoid(rnd(heads)).bfloat16()


def serve(lens: list, heads: int, branches: int = 4, draft: int = 5, seed: int = 0) -> float:
    """Runs the serving half; returns how far the surviving branches' states are from their whole token streams' at once."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = len(lens)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    prompt = layer_inputs((sum(lens),), heads, gen)
    _, states = api.delta_rule(*prompt, cu_seqlens=cu, output_final_state=True)

    pages = n * (branches + 2)
    pool = torch.zeros(pages, heads, 64, 64, device="cuda")
    refcount = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    api.pages_grow(table, torch.zeros_like(lengths), lengths, refcount, page_tokens=ONE_PAGE)
    pool[table[:, 0].long()] = states

    # every sequence branches, its branches read `draft` tokens of their own
    parents = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(branches)
    rows, row_lengths, missing = api.pages_fork(table, lengths, parents, refcount, pool, page_tokens=ONE_PAGE)
    tokens = layer_inputs((n * branches, draft), heads, gen)
    out = api.delta_rule_step(*tokens, pool, slots=rows[:, 0].contiguous())

    # the branch with the largest last output of each sequence stays; the rest, and the trunk, go
    best = out[:, -1].float().flatten(1).norm(dim=1).view(n, branches).argmax(1) + torch.arange(n, device="cuda") * branches
    drop = torch.ones(n * branches, dtype=torch.uint8, device="cuda")
    drop[best] = 0
    api.pages_free(rows, refcount, flags=drop)
    api.pages_free(table, refcount)
    used = api.pages_compact(rows, refcount, pool)

    kept = pool[rows[best, 0].long()]
    whole = [torch.cat([t for i in range(n) for t in (p[int(cu[i]):int(cu[i + 1])], d[best[i]])]) for p, d in zip(prompt, tokens)]
    ends = torch.tensor([0] + [x + draft for x in lens], device="cuda").cumsum(0).to(torch.int32)
    _, want = api.delta_rule(*whole, cu_seqlens=ends, output_final_state=True)
    assert int(missing) == 0 and int(used) == n and int(row_lengths.sum()) == branches * sum(lens)
    return float((kept - want).norm() / want.norm())


def train(lens: list, heads: int, seed: int = 1) -> tuple[float, float]:
    """The loss |o - target|^2 / 2 before and after a short step of the values against its gradient."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    q, k, v, g, beta = layer_inputs((sum(lens),), heads, gen)
    target = torch.randn(v.shape, device="cuda", generator=gen)
    losses = []
    for _ in range(2):
        o, _, saved = api.delta_rule_forward(q, k, v, g, beta, cu_seqlens=cu)
        d = o.float() - target
        losses.append(float(d.square().sum() / 2))
        dv = api.delta_rule_backward(saved, d.bfloat16())[2]
        v = (v.float() - 0.5 * dv.float()).bfloat16()
    return losses[0], losses[1]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=700, help="tokens of the longest prompt")
    a = ap.parse_args()
    lens = [a.tokens, a.tokens // 3 + 1, 1, a.tokens // 7 + 64]
    print(f"serving: branches' states are {serve(lens, a.heads):.1e} from their whole sequences'")
    before, after = train(lens, a.heads)
    print(f"training: loss {before:.1f} -> {after:.1f}")


if __name__ == "__main__":
    main()
