"""PyTorch-facing wrappers of the gated delta rule (``include/prefix_scan_delta.h``).

The recurrence, for each value head of each sequence, of a K x V state S::

    S <- exp(g) S;   u = beta (v - k^T S);   S <- S + k u^T;   o = scale q^T S

Tensors are passed as raw device pointers with their strides and the current
(or given) CUDA stream; every step runs in ``libprefixscan.so``.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _lib
from ._streams import enter, read_here

REAL_CODES = {torch.float32: _lib.PS_REAL_F32, torch.bfloat16: _lib.PS_REAL_BF16, torch.float16: _lib.PS_REAL_F16}


def _check_inputs(fn, q, k, v, g, beta, cu_seqlens):
    dims = 4 if cu_seqlens is None else 3
    lead = "[sequences, tokens" if cu_seqlens is None else "for packed sequences [tokens"
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        if not t.is_cuda or t.device != q.device:
            raise ValueError(f"{fn}: {name} must be a CUDA tensor on q's device (there is no CPU path)")
        if t.dim() != dims - (name in ("g", "beta")):
            raise ValueError(f"{fn}: q, k, v are {lead}, heads, size], g and beta the same without size")
        if name in "qkv" and t.shape[-1] > 1 and t.numel() > 0 and t.stride(-1) != 1:
            raise ValueError(f"{fn}: {name} must be contiguous in its last dimension")
    if q.dtype not in REAL_CODES or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError(f"{fn} supports q, k and v of one type, float32, bfloat16 or float16, not {q.dtype}, {k.dtype}, {v.dtype}")
    if g.dtype != torch.float32 or beta.dtype not in (torch.float32, q.dtype):
        raise TypeError(f"{fn}: g is float32, and beta float32 or q's type")
    if k.shape != q.shape or v.shape[:-2] != q.shape[:-2] or g.shape != v.shape[:-1] or beta.shape != v.shape[:-1]:
        raise ValueError(f"{fn}: shapes of q, k, v, g and beta do not go together")
    hk, hv = q.shape[-2], v.shape[-2]
    if hk < 1 or hv < 1 or hv % hk:
        raise ValueError(f"{fn}: the value heads ({hv}) must be a multiple of the key heads ({hk})")
    if not 1 <= q.shape[-1] <= 128 or not 1 <= v.shape[-1] <= 1024:
        raise ValueError(f"{fn}: key sizes up to 128 and value sizes up to 1024 are supported")
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 \
                or cu_seqlens.device != q.device or not cu_seqlens.is_contiguous():
            raise ValueError(f"{fn}: cu_seqlens must be a contiguous 1-D int32 CUDA tensor of one offset more than sequences")


@dataclass(frozen=True)
class _Plan:
    """What follows from the inputs' shapes, strides, types and device: kept from call to call (never their data)."""
    dims: tuple       # tokens, key heads, value heads, K, V and the codes of both types
    seqs: int         # sequences without cu_seqlens
    states: tuple     # shape of the states, without the number of sequences
    strides: tuple    # (seq, tok, head) of q, k, v, g, beta
    scale: float


_plans: dict = {}


def _strides(t: torch.Tensor, packed: bool, inner: bool) -> tuple:
    """The strides of a [sequences,] tokens, heads[, size] tensor."""
    st = t.stride()
    head = -2 if inner else -1
    return (0 if packed else st[0], st[head - 1], st[head])


def _plan(fn, q, k, v, g, beta, cu_seqlens) -> _Plan:
    packed = cu_seqlens is not None
    key = (packed, q.shape, v.shape, q.stride(), k.stride(), v.stride(), g.stride(), beta.stride(), k.shape, g.shape, beta.shape,
           q.dtype, k.dtype, v.dtype, g.dtype, beta.dtype, q.device, k.device, v.device, g.device, beta.device)
    plan = _plans.get(key)
    if plan is None or (packed and (cu_seqlens.dtype != torch.int32 or cu_seqlens.device != q.device
                                    or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous())):
        _check_inputs(fn, q, k, v, g, beta, cu_seqlens)
        hk, hv, ks, vs = q.shape[-2], v.shape[-2], q.shape[-1], v.shape[-1]
        plan = _Plan((q.shape[0] if packed else q.shape[1], hk, hv, ks, vs, REAL_CODES[q.dtype], REAL_CODES[beta.dtype]),
                     q.shape[0], (hv, ks, vs),
                     tuple(_strides(t, packed, inner) for t, inner in ((q, True), (k, True), (v, True), (g, False), (beta, False))),
                     ks ** -0.5)
        if len(_plans) >= 4096:
            _plans.clear()
        _plans[key] = plan
    return plan


def _shape(plan: _Plan, cu_seqlens, scale) -> bytes:
    """ps_delta_shape"""
    tokens, hk, hv, ks, vs, code, beta_code = plan.dims
    seqs, cu = (plan.seqs, 0) if cu_seqlens is None else (cu_seqlens.numel() - 1, cu_seqlens.data_ptr())
    return _lib.DELTA_SHAPE.pack(seqs, tokens, cu, hk, hv, ks, vs, code, beta_code, plan.scale if scale is None else scale)


def _inputs(plan: _Plan, q, k, v, g, beta) -> bytes:
    """The array of five ps_delta_tensor"""
    sq, sk, sv, sg, sb = plan.strides
    return _lib.DELTA_INPUTS.pack(q.data_ptr(), *sq, k.data_ptr(), *sk, v.data_ptr(), *sv, g.data_ptr(), *sg, beta.data_ptr(), *sb)


def _check_no_graph(fn, tensors):
    """Outputs have no autograd graph: where torch would record one, gradients would be lost without a word."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{fn}: an input requires gradients, which do not pass through this call; use delta_rule_forward and "
                         "delta_rule_backward, or call it under torch.no_grad()")


def _check_state(fn, name, t, shape, device):
    if t.dtype != torch.float32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous float32 CUDA tensor of shape {list(shape)}")


def _workspace(fn, workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < need or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace needs {need} contiguous bytes on {device}")
    return workspace


def delta_rule_workspace_size(q: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
                              train: bool = False) -> int:
    """Bytes of workspace :func:`delta_rule` needs for such inputs (``train``: the buffer that
    :func:`delta_rule_forward` leaves for the backward pass)."""
    if q.dtype not in REAL_CODES:
        raise TypeError(f"delta_rule_workspace_size supports float32, bfloat16 and float16, not {q.dtype}")
    packed = cu_seqlens is not None
    shape = _lib.DELTA_SHAPE.pack(cu_seqlens.numel() - 1 if packed else q.shape[0], q.shape[0] if packed else q.shape[1],
                                  cu_seqlens.data_ptr() if packed else 0, q.shape[-2], v.shape[-2], q.shape[-1], v.shape[-1],
                                  REAL_CODES[q.dtype], _lib.PS_REAL_F32, 1.0)
    return int(_lib.load().ps_delta_workspace_size(shape, int(train)))


@dataclass
class DeltaRuleSaved:
    """What :func:`delta_rule_forward` keeps for :func:`delta_rule_backward`."""
    q: torch.Tensor
    k: torch.Tensor
    v_shape: torch.Size
    beta_dtype: torch.dtype
    cu_seqlens: torch.Tensor | None
    plan: object
    shape: bytes
    states: tuple
    has_initial_state: bool
    workspace: torch.Tensor
    stream: int   # handle of the stream that the forward call ran on


def _forward(fn, q, k, v, g, beta, scale, cu_seqlens, initial_state, output_final_state, out, final_state, workspace,
             stream, train):
    plan = _plan(fn, q, k, v, g, beta, cu_seqlens)
    device = q.device
    states = (plan.seqs if cu_seqlens is None else cu_seqlens.numel() - 1, *plan.states)
    if initial_state is not None:
        _check_state(fn, "initial_state", initial_state, states, device)
    if final_state is not None:
        _check_state(fn, "final_state", final_state, states, device)
    if out is not None and (out.dtype != q.dtype or out.shape != v.shape or out.device != device or not out.is_contiguous()):
        raise ValueError(f"{fn}: `out` must be contiguous and match v's shape, type and device")
    shape, inputs = _shape(plan, cu_seqlens, scale), _inputs(plan, q, k, v, g, beta)
    lib = _lib.load()
    s, ctx = enter(device, stream)
    with ctx:
        if out is None:
            out = torch.empty(v.shape, dtype=q.dtype, device=device)
        if final_state is None and output_final_state:
            final_state = torch.empty(states, dtype=torch.float32, device=device)
        need = lib.ps_delta_workspace_size(shape, train)
        workspace = _workspace(fn, workspace, need, device)
        st = lib.ps_delta_forward(shape, inputs, initial_state.data_ptr() if initial_state is not None else None,
                                  final_state.data_ptr() if final_state is not None else None, out.data_ptr(), train,
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
        if train and stream is not None:   # what is saved may be dropped while the stream given still reads it
            read_here(device, q, k, cu_seqlens, workspace)
    _lib.check("ps_delta_forward", st)
    return out, final_state, plan, shape, states, workspace, s


def delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, *,
               scale: float | None = None, cu_seqlens: torch.Tensor | None = None,
               initial_state: torch.Tensor | None = None, output_final_state: bool = False,
               out: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """The gated delta rule over whole sequences: ``(o, final_state)``.

    ``q``, ``k``: [sequences, tokens, key heads, K]; ``v``: [sequences, tokens, value heads, V]; ``g`` (log decays,
    float32) and ``beta`` (gates, float32 or q's type): [sequences, tokens, value heads].  With ``cu_seqlens``
    (int32, on the device, one offset more than sequences, never falling) the first two dimensions are one that packs
    all sequences' tokens.  Any strides go, as long as the last dimension is contiguous.  ``initial_state``:
    [sequences, value heads, K, V] float32 (0 if not given); the states at the end are written to
    ``final_state`` (which may be ``initial_state``), or returned in a new tensor with ``output_final_state``.
    ``scale`` is K ** -0.5 if not given.  Matrix products take operands of 16 significant bits, float32 q and k too, so
    float32 results are off by some 1e-6 to 5e-6; :func:`delta_rule_step`, which is float32 throughout, takes whole
    prompts as well, token after token.  Asynchronous on ``stream`` (default: the current stream).  With
    ``cu_seqlens``, outputs of tokens that no sequence holds are not written.  No gradients pass through
    (inputs that require them are refused where torch records them): see :func:`delta_rule_forward`.
    """
    _check_no_graph("delta_rule", (q, k, v, g, beta, initial_state))
    return _forward("delta_rule", q, k, v, g, beta, scale, cu_seqlens, initial_state, output_final_state, out, final_state,
                    workspace, stream, 0)[:2]


def delta_rule_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, *,
                       scale: float | None = None, cu_seqlens: torch.Tensor | None = None,
                       initial_state: torch.Tensor | None = None, output_final_state: bool = False,
                       out: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None
                       ) -> tuple[torch.Tensor, torch.Tensor | None, DeltaRuleSaved]:
    """:func:`delta_rule` for training: ``(o, final_state, saved)``.

    The outputs have no autograd graph: ``saved`` goes to :func:`delta_rule_backward`, whose results a
    ``torch.autograd.Function`` can hand on.  It holds q and k (which must not change until then) and a workspace of
    ``delta_rule_workspace_size(q, v, cu_seqlens, train=True)`` bytes.
    """
    out, final_state, plan, shape, states, workspace, s = _forward(
        "delta_rule_forward", q, k, v, g, beta, scale, cu_seqlens, initial_state, output_final_state, out, final_state, workspace,
        stream, 1)
    return out, final_state, DeltaRuleSaved(q, k, v.shape, beta.dtype, cu_seqlens, plan, shape, states, initial_state is not None,
                                            workspace, s)


def delta_rule_backward(saved: DeltaRuleSaved, d_o: torch.Tensor, *, d_final_state: torch.Tensor | None = None, stream=None
                        ) -> tuple[torch.Tensor, ...]:
    """Gradients ``(dq, dk, dv, dg, dbeta, d_initial_state)`` of one :func:`delta_rule_forward` call.

    ``d_o``: the gradient of ``o``, of its shape and type (any strides with a contiguous last dimension);
    ``d_final_state``: that of the final states (0 if not given).  dq and dk are summed over the value heads that share a
    key head; ``d_initial_state`` is None where the forward call had no initial state.  Bitwise reproducible.  Gradients
    of tokens that no sequence holds are 0.
    """
    fn = "delta_rule_backward"
    q, k, packed = saved.q, saved.k, saved.cu_seqlens is not None
    if d_o.shape != saved.v_shape or d_o.dtype != q.dtype or d_o.device != q.device:
        raise ValueError(f"{fn}: d_o must match o's shape, type and device")
    if d_final_state is not None:
        _check_state(fn, "d_final_state", d_final_state, saved.states, q.device)
    lib = _lib.load()
    s, ctx = enter(q.device, stream)
    with ctx:
        if d_o.numel() and d_o.shape[-1] > 1 and d_o.stride(-1) != 1:
            d_o = d_o.contiguous()   # on the call's stream
        new = torch.zeros if packed and saved.cu_seqlens.numel() == 1 else torch.empty   # with no sequence nothing is enqueued
        heads = saved.v_shape[:-1]
        dq, dk = (new(q.shape, dtype=q.dtype, device=q.device) for _ in range(2))
        dv = new(saved.v_shape, dtype=q.dtype, device=q.device)
        dg = new(heads, dtype=torch.float32, device=q.device)
        dbeta = new(heads, dtype=saved.beta_dtype, device=q.device)
        dh0 = torch.empty(saved.states, dtype=torch.float32, device=q.device) if saved.has_initial_state else None
        strides = (saved.plan.strides[0], saved.plan.strides[1], _strides(d_o, packed, True))
        ts = [_lib.DELTA_TENSOR.pack(t.data_ptr(), *st) for t, st in zip((q, k, d_o), strides)]
        ptr = lambda t: t.data_ptr() if t is not None and t.numel() else None  # noqa: E731
        st = lib.ps_delta_backward(saved.shape, *ts, ptr(d_final_state), ptr(dq),
                                   ptr(dk), ptr(dv), ptr(dg), ptr(dbeta), ptr(dh0), saved.workspace.data_ptr(),
                                   saved.workspace.numel() * saved.workspace.element_size(), s)
        if stream is not None or s != saved.stream:   # `saved` may be dropped while this stream still reads what it holds
            read_here(q.device, saved.workspace, q, k, saved.cu_seqlens, d_o, d_final_state)
    _lib.check("ps_delta_backward", st)
    return dq, dk, dv, dg, dbeta, dh0


def delta_rule_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                    state: torch.Tensor, *, slots: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                    scale: float | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The next token (or few) of many sequences: the outputs, with ``state`` advanced in place.

    ``q`` .. ``beta`` as for :func:`delta_rule` without ``cu_seqlens``.  ``state``: a pool of pages, [pages, value
    heads, K, V] float32.  ``slots`` (int32, one per sequence, all different): the page of each sequence's state, -1
    for one that takes no part; page i for sequence i if not given.  ``lengths`` (int32, one per sequence): how many
    of the tokens count.  Outputs of tokens that do not count are 0.  Inputs that require gradients are refused where
    torch records them: there is no backward pass of single steps.
    """
    fn = "delta_rule_step"
    _check_no_graph(fn, (q, k, v, g, beta, state))
    plan = _plan(fn, q, k, v, g, beta, None)
    device = q.device
    if state.dim() != 4 or state.shape[1:] != plan.states:
        raise ValueError(f"{fn}: state must be [pages, value heads, K, V]")
    _check_state(fn, "state", state, state.shape, device)
    for name, t in (("slots", slots), ("lengths", lengths)):
        if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or t.numel() != plan.seqs or t.device != device
                              or not t.is_contiguous()):
            raise ValueError(f"{fn}: {name} must be a contiguous int32 CUDA tensor with one entry per sequence")
    if slots is None and state.shape[0] < plan.seqs:
        raise ValueError(f"{fn}: fewer pages than sequences")
    if out is not None and (out.dtype != q.dtype or out.shape != v.shape or out.device != device or not out.is_contiguous()):
        raise ValueError(f"{fn}: `out` must be contiguous and match v's shape, type and device")
    s, ctx = enter(device, stream)
    with ctx:
        if out is None:
            out = torch.empty(v.shape, dtype=q.dtype, device=device)
        st = _lib.load().ps_delta_step(_shape(plan, None, scale), _inputs(plan, q, k, v, g, beta), state.data_ptr(), state.shape[0],
                                       slots.data_ptr() if slots is not None else None,
                                       lengths.data_ptr() if lengths is not None else None, out.data_ptr(), s)
    _lib.check("ps_delta_step", st)
    return out
