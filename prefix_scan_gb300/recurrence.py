"""PyTorch-facing wrappers of the gated linear recurrence (``include/prefix_scan_recurrence.h``).

The recurrence, for each channel of each sequence::

    h_t = exp(g_t) h_{t-1} + w_t x_t        w = 1, or 1 - exp(g_t) where input and decay are tied

Tensors are passed as raw device pointers with their strides and the current
(or given) CUDA stream; every step runs in ``libprefixscan.so``.
"""
from __future__ import annotations

from dataclasses import dataclass, field

import torch

from . import _lib
from ._streams import enter, read_here
from .delta import REAL_CODES, _check_state, _workspace


@dataclass(frozen=True)
class _Plan:
    """What follows from the inputs' shapes, strides, types and device: kept from call to call (never their data)."""
    seqs: int          # sequences without cu_seqlens
    tokens: int
    channels: int
    codes: tuple       # of x's type, of g's type, tied
    strides: tuple     # (seq, tok) of x, then of g
    sizes: dict = field(default_factory=dict)   # bytes of workspace by (sequences, train)


_plans: dict = {}


def _check_inputs(fn, x, g, cu_seqlens):
    dims = 3 if cu_seqlens is None else 2
    lead = "[sequences, tokens" if cu_seqlens is None else "for packed sequences [tokens"
    for name, t in (("x", x), ("g", g)):
        if not t.is_cuda or t.device != x.device:
            raise ValueError(f"{fn}: {name} must be a CUDA tensor on x's device (there is no CPU path)")
        if t.dim() != dims or t.shape != x.shape:
            raise ValueError(f"{fn}: x and g are {lead}, channels], of one shape")
        if t.shape[-1] > 1 and t.numel() > 0 and t.stride(-1) != 1:
            raise ValueError(f"{fn}: {name} must be contiguous in its last dimension")
    if x.dtype not in REAL_CODES or g.dtype not in (torch.float32, x.dtype):
        raise TypeError(f"{fn} supports x of float32, bfloat16 or float16, and g of that type or float32, not {x.dtype}, {g.dtype}")
    if x.shape[-1] < 1:
        raise ValueError(f"{fn}: at least one channel is needed")
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 \
                or cu_seqlens.device != x.device or not cu_seqlens.is_contiguous():
            raise ValueError(f"{fn}: cu_seqlens must be a contiguous 1-D int32 CUDA tensor of one offset more than sequences")


def _strides(t: torch.Tensor, packed: bool) -> tuple:
    st = t.stride()
    return (0, st[0]) if packed else (st[0], st[1])


def _plan(fn, x, g, cu_seqlens, tied) -> _Plan:
    packed = cu_seqlens is not None
    key = (packed, x.shape, g.shape, x.stride(), g.stride(), x.dtype, g.dtype, x.device, g.device, bool(tied))
    plan = _plans.get(key)
    if plan is None or (packed and (cu_seqlens.dtype != torch.int32 or cu_seqlens.device != x.device
                                    or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous())):
        _check_inputs(fn, x, g, cu_seqlens)
        plan = _Plan(0 if packed else x.shape[0], x.shape[0] if packed else x.shape[1], x.shape[-1],
                     (REAL_CODES[x.dtype], REAL_CODES[g.dtype], int(bool(tied))), (_strides(x, packed), _strides(g, packed)))
        if len(_plans) >= 4096:
            _plans.clear()
        _plans[key] = plan
    return plan


def _shape(plan: _Plan, cu_seqlens) -> bytes:
    """ps_linrec_shape"""
    seqs, cu = (plan.seqs, 0) if cu_seqlens is None else (cu_seqlens.numel() - 1, cu_seqlens.data_ptr())
    return _lib.LINREC_SHAPE.pack(seqs, plan.tokens, cu, plan.channels, *plan.codes)


def _need(lib, plan: _Plan, shape: bytes, seqs: int, train: int) -> int:
    need = plan.sizes.get((seqs, train))
    if need is None:
        need = plan.sizes[(seqs, train)] = lib.ps_linrec_workspace_size(shape, train)
    return need


def _check_no_graph(fn, tensors):
    """Outputs have no autograd graph: where torch would record one, gradients would be lost without a word."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{fn}: an input requires gradients, which do not pass through this call; use linear_recurrence_forward "
                         "and linear_recurrence_backward, or call it under torch.no_grad()")


def linear_recurrence_workspace_size(x: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *, train: bool = False,
                                     gate_dtype: torch.dtype = torch.float32) -> int:
    """Bytes of workspace :func:`linear_recurrence` needs for such inputs, log decays of ``gate_dtype`` (``train``: the buffer
    that :func:`linear_recurrence_forward` leaves for the backward pass)."""
    if x.dtype not in REAL_CODES:
        raise TypeError(f"linear_recurrence_workspace_size supports float32, bfloat16 and float16, not {x.dtype}")
    if gate_dtype not in (torch.float32, x.dtype):
        raise TypeError(f"linear_recurrence_workspace_size supports log decays of x's type or float32, not {gate_dtype} with {x.dtype}")
    packed = cu_seqlens is not None
    if x.dim() != (2 if packed else 3):
        raise ValueError("linear_recurrence_workspace_size: x is [sequences, tokens, channels], or [tokens, channels] packed")
    code = REAL_CODES[x.dtype]
    shape = _lib.LINREC_SHAPE.pack(cu_seqlens.numel() - 1 if packed else x.shape[0], x.shape[0] if packed else x.shape[1],
                                   cu_seqlens.data_ptr() if packed else 0, x.shape[-1], code,
                                   REAL_CODES[gate_dtype], 0)
    return int(_lib.load().ps_linrec_workspace_size(shape, int(train)))


@dataclass
class LinearRecurrenceSaved:
    """What :func:`linear_recurrence_forward` keeps for :func:`linear_recurrence_backward`."""
    x: torch.Tensor
    g: torch.Tensor
    cu_seqlens: torch.Tensor | None
    initial_state: torch.Tensor | None
    plan: object
    shape: bytes
    states: tuple
    workspace: torch.Tensor
    stream: int   # handle of the stream that the forward call ran on


def _forward(fn, x, g, tied, cu_seqlens, initial_state, output_final_state, out, final_state, workspace, stream, train):
    plan = _plan(fn, x, g, cu_seqlens, tied)
    device = x.device
    seqs = plan.seqs if cu_seqlens is None else cu_seqlens.numel() - 1
    states = (seqs, plan.channels)
    if initial_state is not None:
        _check_state(fn, "initial_state", initial_state, states, device)
    if final_state is not None:
        _check_state(fn, "final_state", final_state, states, device)
    if out is not None and (out.dtype != x.dtype or out.shape != x.shape or out.device != device or not out.is_contiguous()):
        raise ValueError(f"{fn}: `out` must be contiguous and match x's shape, type and device")
    shape = _shape(plan, cu_seqlens)
    lib = _lib.load()
    s, ctx = enter(device, stream)
    with ctx:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=device)
        if final_state is None and output_final_state:
            final_state = torch.empty(states, dtype=torch.float32, device=device)
        workspace = _workspace(fn, workspace, _need(lib, plan, shape, seqs, train), device)
        st = lib.ps_linrec_forward(shape, _lib.LINREC_TENSOR.pack(x.data_ptr(), *plan.strides[0]),
                                   _lib.LINREC_TENSOR.pack(g.data_ptr(), *plan.strides[1]),
                                   initial_state.data_ptr() if initial_state is not None else None,
                                   final_state.data_ptr() if final_state is not None else None, out.data_ptr(), train,
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
        if train and stream is not None:   # what is saved may be dropped while the stream given still reads it
            read_here(device, x, g, cu_seqlens, initial_state, workspace)
    _lib.check("ps_linrec_forward", st)
    return out, final_state, plan, shape, states, workspace, s


def linear_recurrence(x: torch.Tensor, g: torch.Tensor, *, tied: bool = False, cu_seqlens: torch.Tensor | None = None,
                      initial_state: torch.Tensor | None = None, output_final_state: bool = False,
                      out: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """The gated linear recurrence over whole sequences: ``(h, final_state)``.

    ``x`` (inputs) and ``g`` (log decays, of x's type or float32): [sequences, tokens, channels].  With ``cu_seqlens``
    (int32, on the device, one offset more than sequences, never falling) the first two dimensions are one that packs all
    sequences' tokens.  Any strides go, as long as the last dimension is contiguous.  ``tied``: the input is weighted by
    1 - exp(g) instead of 1.  ``initial_state``: [sequences, channels] float32 (0 if not given); the states at the end are
    written to ``final_state`` (which may be ``initial_state``), or returned in a new tensor with ``output_final_state``.
    States and sums are float32 throughout, and results repeat bit for bit.  Asynchronous on ``stream`` (default: the
    current stream).  With ``cu_seqlens``, outputs of tokens that no sequence holds are not written.  No gradients pass
    through (inputs that require them are refused where torch records them): see :func:`linear_recurrence_forward`.
    """
    _check_no_graph("linear_recurrence", (x, g, initial_state))
    return _forward("linear_recurrence", x, g, tied, cu_seqlens, initial_state, output_final_state, out, final_state, workspace,
                    stream, 0)[:2]


def linear_recurrence_forward(x: torch.Tensor, g: torch.Tensor, *, tied: bool = False, cu_seqlens: torch.Tensor | None = None,
                              initial_state: torch.Tensor | None = None, output_final_state: bool = False,
                              out: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, stream=None
                              ) -> tuple[torch.Tensor, torch.Tensor | None, LinearRecurrenceSaved]:
    """:func:`linear_recurrence` for training: ``(h, final_state, saved)``.

    The outputs have no autograd graph: ``saved`` goes to :func:`linear_recurrence_backward`, whose results a
    ``torch.autograd.Function`` can hand on.  It holds x, g and the initial state (which must not change until then, so
    ``final_state`` must be another tensor) and a workspace of ``linear_recurrence_workspace_size(x, cu_seqlens, train=True)``
    bytes.
    """
    out, final_state, plan, shape, states, workspace, s = _forward(
        "linear_recurrence_forward", x, g, tied, cu_seqlens, initial_state, output_final_state, out, final_state, workspace,
        stream, 1)
    return out, final_state, LinearRecurrenceSaved(x, g, cu_seqlens, initial_state, plan, shape, states, workspace, s)


def linear_recurrence_backward(saved: LinearRecurrenceSaved, d_h: torch.Tensor, *, d_final_state: torch.Tensor | None = None,
                               stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor | None]:
    """Gradients ``(dx, dg, d_initial_state)`` of one :func:`linear_recurrence_forward` call.

    ``d_h``: the gradient of ``h``, of its shape and type (any strides with a contiguous last dimension);
    ``d_final_state``: that of the final states (0 if not given).  ``d_initial_state`` is None where the forward call had
    no initial state.  Bitwise reproducible.  Gradients of tokens that no sequence holds are 0; those of broadcast inputs
    (stride 0) come for every place, to be summed by the caller.
    """
    fn = "linear_recurrence_backward"
    x, g, cu = saved.x, saved.g, saved.cu_seqlens
    packed = cu is not None
    if d_h.shape != x.shape or d_h.dtype != x.dtype or d_h.device != x.device:
        raise ValueError(f"{fn}: d_h must match h's shape, type and device")
    if d_final_state is not None:
        _check_state(fn, "d_final_state", d_final_state, saved.states, x.device)
    lib = _lib.load()
    s, ctx = enter(x.device, stream)
    with ctx:
        if d_h.numel() and d_h.shape[-1] > 1 and d_h.stride(-1) != 1:
            d_h = d_h.contiguous()   # on the call's stream
        new = torch.zeros if packed and saved.states[0] == 0 else torch.empty   # with no sequence nothing is enqueued
        dx = new(x.shape, dtype=x.dtype, device=x.device)
        dg = new(x.shape, dtype=g.dtype, device=x.device)
        h0 = saved.initial_state
        dh0 = torch.empty(saved.states, dtype=torch.float32, device=x.device) if h0 is not None else None
        strides = saved.plan.strides
        st = lib.ps_linrec_backward(saved.shape, _lib.LINREC_TENSOR.pack(x.data_ptr(), *strides[0]),
                                    _lib.LINREC_TENSOR.pack(g.data_ptr(), *strides[1]), h0.data_ptr() if h0 is not None else None,
                                    _lib.LINREC_TENSOR.pack(d_h.data_ptr(), *_strides(d_h, packed)),
                                    d_final_state.data_ptr() if d_final_state is not None else None, dx.data_ptr(), dg.data_ptr(),
                                    dh0.data_ptr() if dh0 is not None else None, saved.workspace.data_ptr(),
                                    saved.workspace.numel() * saved.workspace.element_size(), s)
        if stream is not None or s != saved.stream:   # `saved` may be dropped while this stream still reads what it holds
            read_here(x.device, saved.workspace, x, g, cu, h0, d_h, d_final_state)
    _lib.check("ps_linrec_backward", st)
    return dx, dg, dh0


def linear_recurrence_step(x: torch.Tensor, g: torch.Tensor, state: torch.Tensor, *, tied: bool = False,
                           slots: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The next token (or few) of many sequences: the outputs, with ``state`` advanced in place.

    ``x`` and ``g`` as for :func:`linear_recurrence` without ``cu_seqlens``.  ``state``: a pool of pages, [pages, channels]
    float32.  ``slots`` (int32, one per sequence, all different): the page of each sequence's state, -1 for one that takes no
    part; page i for sequence i if not given.  ``lengths`` (int32, one per sequence): how many of the tokens count.  Outputs
    of tokens that do not count are 0.  Inputs that require gradients are refused where torch records them: there is no
    backward pass of single steps.
    """
    fn = "linear_recurrence_step"
    _check_no_graph(fn, (x, g, state))
    plan = _plan(fn, x, g, None, tied)
    device = x.device
    if state.dim() != 2 or state.shape[1] != plan.channels:
        raise ValueError(f"{fn}: state must be [pages, channels]")
    _check_state(fn, "state", state, state.shape, device)
    for name, t in (("slots", slots), ("lengths", lengths)):
        if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or t.numel() != plan.seqs or t.device != device
                              or not t.is_contiguous()):
            raise ValueError(f"{fn}: {name} must be a contiguous int32 CUDA tensor with one entry per sequence")
    if slots is None and state.shape[0] < plan.seqs:
        raise ValueError(f"{fn}: fewer pages than sequences")
    if out is not None and (out.dtype != x.dtype or out.shape != x.shape or out.device != device or not out.is_contiguous()):
        raise ValueError(f"{fn}: `out` must be contiguous and match x's shape, type and device")
    s, ctx = enter(device, stream)
    with ctx:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=device)
        st = _lib.load().ps_linrec_step(_shape(plan, None), _lib.LINREC_TENSOR.pack(x.data_ptr(), *plan.strides[0]),
                                        _lib.LINREC_TENSOR.pack(g.data_ptr(), *plan.strides[1]), state.data_ptr(), state.shape[0],
                                        slots.data_ptr() if slots is not None else None,
                                        lengths.data_ptr() if lengths is not None else None, out.data_ptr(), s)
    _lib.check("ps_linrec_step", st)
    return out
