"""PyTorch-facing wrapper of beam search's choice (``include/prefix_scan_beam.h``)."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from ._streams import enter
from .delta import REAL_CODES, _workspace


class BeamChoice(NamedTuple):
    scores: torch.Tensor
    parents: torch.Tensor
    tokens: torch.Tensor
    ended: torch.Tensor | None


def _check_sizes(fn, beams, width):
    if beams > _lib.PS_BEAM_MAX_BEAMS or not 1 <= width <= _lib.PS_BEAM_MAX_WIDTH:
        raise ValueError(f"{fn}: up to {_lib.PS_BEAM_MAX_BEAMS} beams and {_lib.PS_BEAM_MAX_WIDTH} candidates are supported")


def _check(fn, logits, scores, width, ended, eos_token):
    device = logits.device
    if not logits.is_cuda:
        raise ValueError(f"{fn}: logits must be a CUDA tensor (there is no CPU path)")
    if logits.dtype not in REAL_CODES:
        raise TypeError(f"{fn} supports logits of float32, bfloat16 or float16, not {logits.dtype}")
    if logits.dim() != 3 or logits.shape[-1] < 1 or logits.shape[1] < 1:
        raise ValueError(f"{fn}: logits are [batch, beams, vocabulary]")
    if logits.shape[-1] > 1 and logits.numel() > 0 and logits.stride(-1) != 1:
        raise ValueError(f"{fn}: logits must be contiguous in their last dimension")
    _check_sizes(fn, logits.shape[1], width)
    for name, t, dtype in (("scores", scores, torch.float32), ("ended", ended, torch.uint8)):
        if t is not None and (t.dtype != dtype or t.shape != logits.shape[:2] or t.device != device or not t.is_contiguous()):
            raise ValueError(f"{fn}: {name} must be a contiguous {dtype} CUDA tensor [batch, beams]")
    if ended is not None and eos_token < 0:
        raise ValueError(f"{fn}: beams can have ended only with an eos_token")


_plans: dict = {}   # packed shapes and workspace sizes by what they follow from: kept from call to call (never data)


def _goes_with(plan, t, dtype, device) -> bool:
    return t.dtype == dtype and t.shape == plan[2] and t.device == device and t.is_contiguous()


def beam_select(logits: torch.Tensor, scores: torch.Tensor, *, width: int | None = None, ended: torch.Tensor | None = None,
                eos_token: int = -1, workspace: torch.Tensor | None = None, stream=None) -> BeamChoice:
    """The best continuations of an item's beams: ``(scores, parents, tokens, ended)``, each [batch, width], best first.

    ``logits``: [batch, beams, vocabulary], float32, bfloat16 or float16, of any strides with a contiguous last dimension;
    ``scores`` (float32, [batch, beams]): the beams' scores, -infinity for a beam that takes no part.  A continuation's total
    is score + log_softmax(logits)[token]; equal totals go to the lower beam, then to the larger logit, then to the lower token.
    A beam's own continuations are compared exactly, those of different beams in 64 bits from row sums of 32 bits (off by 2^-19 at
    most, as a rule by 2^-22: closer totals may change places).  ``width`` (the number of beams if not given, at most 64): how many to choose.  ``parents`` (int32) are
    rows item * beams + beam, as :func:`pages_fork` and :func:`pages_reorder` take them.  With ``ended`` (uint8, [batch, beams])
    a beam at its end offers itself once, with its score as it is and ``eos_token``, and the ``ended`` returned says which of
    the chosen are at theirs (None without).  Where candidates run out: score -infinity, parent and token -1.
    """
    fn = "beam_select"
    if (logits.requires_grad or scores.requires_grad) and torch.is_grad_enabled():
        raise ValueError(f"{fn}: an input requires gradients, which do not pass through this call; call it under torch.no_grad()")
    device = logits.device
    key = (logits.shape, logits.stride(), logits.dtype, device, width, eos_token)
    plan = _plans.get(key)
    if plan is None or not _goes_with(plan, scores, torch.float32, device) \
            or ended is not None and (eos_token < 0 or not _goes_with(plan, ended, torch.uint8, device)):
        w = logits.shape[1] if width is None and logits.dim() == 3 else width
        _check(fn, logits, scores, w if w is not None else 1, ended, eos_token)
        st = logits.stride()
        shape = _lib.BEAM_SHAPE.pack(logits.shape[0], logits.shape[1], w, logits.shape[2], st[0], st[1], REAL_CODES[logits.dtype], eos_token)
        if len(_plans) >= 4096:
            _plans.clear()
        plan = _plans[key] = (shape, _lib.load().ps_beam_workspace_size(shape), logits.shape[:2], (logits.shape[0], w))
    shape, need, _, picks = plan
    s, ctx = enter(device, stream)
    with ctx:
        out_scores = torch.empty(picks, dtype=torch.float32, device=device)
        parents = torch.empty(picks, dtype=torch.int32, device=device)
        tokens = torch.empty(picks, dtype=torch.int32, device=device)
        out_ended = torch.empty(picks, dtype=torch.uint8, device=device) if ended is not None else None
        workspace = _workspace(fn, workspace, need, device)
        st = _lib.load().ps_beam_select(shape, logits.data_ptr(), scores.data_ptr(), ended.data_ptr() if ended is not None else None,
                                        out_scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
                                        out_ended.data_ptr() if ended is not None else None, workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), s)
    _lib.check("ps_beam_select", st)
    return BeamChoice(out_scores, parents, tokens, out_ended)


def beam_workspace_size(logits: torch.Tensor, *, width: int | None = None) -> int:
    """Bytes of workspace :func:`beam_select` needs for such logits."""
    if logits.dtype not in REAL_CODES:
        raise TypeError(f"beam_workspace_size supports float32, bfloat16 and float16, not {logits.dtype}")
    if logits.dim() != 3:
        raise ValueError("beam_workspace_size: logits are [batch, beams, vocabulary]")
    w = logits.shape[1] if width is None else width
    _check_sizes("beam_workspace_size", logits.shape[1], w)
    return int(_lib.load().ps_beam_workspace_size(_lib.BEAM_SHAPE.pack(
        logits.shape[0], logits.shape[1], w, logits.shape[2], logits.stride(0), logits.stride(1), REAL_CODES[logits.dtype], -1)))
