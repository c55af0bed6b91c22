"""PyTorch-facing wrappers of the page operations (``include/prefix_scan_pages.h``).

A cache is one pool or several (per layer, say; keys and values): tensors [pages, ...], contiguous, with the same number
of pages.  ``refcount`` (int32, [pages]) counts the table entries that hold each page, 0 for a free one; ``table`` (int32,
[rows, width]) names each row's pages in order, -1 where there is none; ``lengths`` (int32, [rows]) counts its tokens, of
which a page holds ``page_tokens``.  Pages are handed out lowest first in the order of rows.  All calls are asynchronous
on ``stream`` (default: the current stream) and never synchronise.
"""
from __future__ import annotations

import struct

import torch

from . import _lib
from ._streams import enter


def _check_ints(fn, device, **tensors):
    cuda = device.type == "cuda"
    for name, (t, dims) in tensors.items():
        if not cuda or t.dtype != torch.int32 or t.device != device or t.dim() != dims or not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be a contiguous {dims}-D int32 tensor on one CUDA device with the others")


def _pools(fn, pools, pages, device):
    if isinstance(pools, torch.Tensor):
        pools = [pools]
    if len(pools) > _lib.PS_PAGES_MAX_POOLS:
        raise ValueError(f"{fn}: at most {_lib.PS_PAGES_MAX_POOLS} pools in one call")
    out, like, dtype, size = [], None, None, 0
    for p in pools:
        shape = p.shape
        if shape != like or p.dtype is not dtype:   # pools are often of one shape and type
            if p.dim() < 1 or shape[0] != pages:
                raise ValueError(f"{fn}: pools must be contiguous CUDA tensors of {pages} pages on one device")
            like, dtype, size = shape, p.dtype, p.numel() // pages * p.element_size() if pages else 1
            if size == 0:
                raise ValueError(f"{fn}: pages must not be empty")
        if p.device != device or not p.is_contiguous():
            raise ValueError(f"{fn}: pools must be contiguous CUDA tensors of {pages} pages on one device")
        out += (p.data_ptr(), size)
    return struct.pack("@" + "Pq" * len(pools), *out), len(pools)   # ps_page_pool


def pages_workspace_size(rows: int, pages: int) -> int:
    """Bytes of workspace for tables of up to ``rows`` rows and pools of ``pages`` pages."""
    return int(_lib.load().ps_pages_workspace_size(rows, pages))


def _workspace(fn, lib, workspace, rows, pages, device):
    need = lib.ps_pages_workspace_size(rows, pages)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < need or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace needs {need} contiguous bytes on {device}")
    return workspace


def pages_copy(pools, src: torch.Tensor, dst: torch.Tensor, *, stream=None) -> None:
    """Copies page ``src[i]`` to page ``dst[i]`` of every pool, for all i.  Pairs with an index outside the pools are left
    out; no page may be written twice, or written and read."""
    fn = "pages_copy"
    _check_ints(fn, src.device, src=(src, 1), dst=(dst, 1))
    if src.numel() != dst.numel():
        raise ValueError(f"{fn}: src and dst differ in length")
    pools = [pools] if isinstance(pools, torch.Tensor) else pools
    pages = pools[0].shape[0] if len(pools) else 0
    arr, n = _pools(fn, pools, pages, src.device)
    s, ctx = enter(src.device, stream)
    with ctx:
        st = _lib.load().ps_pages_copy(arr, n, pages, src.data_ptr(), dst.data_ptr(), src.numel(), s)
    _lib.check("ps_pages_copy", st)


def pages_fork(table: torch.Tensor, lengths: torch.Tensor, parents: torch.Tensor, refcount: torch.Tensor, pools, *,
               page_tokens: int, out_table: torch.Tensor | None = None, out_lengths: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Branches of rows: ``(new_table, new_lengths, missing)``, row i a branch of row ``parents[i]``.

    Whole pages are shared (``refcount`` rises in place); a part-filled last page is copied, in every pool, to a free
    page.  ``missing`` (int32, one entry): how many last pages found no free page; their places are -1.  A recurrent
    state, which changes with every token, is a page that is never full: give it a ``page_tokens`` above any length.
    """
    fn = "pages_fork"
    device = table.device
    _check_ints(fn, device, table=(table, 2), lengths=(lengths, 1), parents=(parents, 1), refcount=(refcount, 1))
    rows, width = table.shape
    new_rows, pages = parents.numel(), refcount.numel()
    if lengths.numel() != rows:
        raise ValueError(f"{fn}: one length per row of the table is needed")
    if page_tokens < 1:
        raise ValueError(f"{fn}: page_tokens must be positive")
    arr, n = _pools(fn, pools, pages, device)
    lib = _lib.load()
    s, ctx = enter(device, stream)
    with ctx:
        if out_table is None:
            out_table = torch.empty((new_rows, width), dtype=torch.int32, device=device)
        if out_lengths is None:
            out_lengths = torch.empty(new_rows, dtype=torch.int32, device=device)
        _check_ints(fn, device, out_table=(out_table, 2), out_lengths=(out_lengths, 1))
        if tuple(out_table.shape) != (new_rows, width) or out_lengths.numel() != new_rows:
            raise ValueError(f"{fn}: out_table and out_lengths have one row per parent")
        missing = torch.empty(1, dtype=torch.int32, device=device)
        workspace = _workspace(fn, lib, workspace, new_rows, pages, device)
        st = lib.ps_pages_fork(table.data_ptr(), lengths.data_ptr(), rows, width, parents.data_ptr(), new_rows, page_tokens,
                               refcount.data_ptr(), arr, n, pages, out_table.data_ptr(), out_lengths.data_ptr(),
                               missing.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
    _lib.check("ps_pages_fork", st)
    return out_table, out_lengths, missing


def pages_reorder(slots: torch.Tensor, parents: torch.Tensor, pools, *, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Branches of rows in place, for states that fill a page each: ``(new_slots, missing)``, row i a branch of row ``parents[i]``.

    ``slots`` (int32, all different, -1 for none): each row's page, which no other row shares, so there are no counts.  The
    lowest row of a parent takes over its page; the others get, in order, the pages that no row continues, and the parent's
    page is copied there in every pool.  ``parents`` (int32, as many): as ``beam_select`` gives them, -1 for none; such rows
    get what pages are left, as they are.  ``missing`` (int32, one entry): how many branches found no page; their places are
    -1.  Any shapes go, as long as both are contiguous; the result has the shape of ``slots``, or is ``out``, another tensor.
    """
    fn = "pages_reorder"
    device = slots.device
    _check_ints(fn, device, slots=(slots, slots.dim()), parents=(parents, parents.dim()))
    rows = slots.numel()
    if parents.numel() != rows:
        raise ValueError(f"{fn}: one parent per row is needed")
    pools = [pools] if isinstance(pools, torch.Tensor) else pools
    pages = pools[0].shape[0] if len(pools) else 0
    arr, n = _pools(fn, pools, pages, device)
    lib = _lib.load()
    s, ctx = enter(device, stream)
    with ctx:
        if out is None:
            out = torch.empty(slots.shape, dtype=torch.int32, device=device)
        else:
            _check_ints(fn, device, out=(out, slots.dim()))
            if out.shape != slots.shape:
                raise ValueError(f"{fn}: out must have the shape of slots")
        missing = torch.empty(1, dtype=torch.int32, device=device)
        workspace = _workspace(fn, lib, workspace, rows, pages, device)
        st = lib.ps_pages_reorder(slots.data_ptr(), parents.data_ptr(), rows, arr, n, pages, out.data_ptr(), missing.data_ptr(),
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
    _lib.check("ps_pages_reorder", st)
    return out, missing


def pages_grow(table: torch.Tensor, lengths: torch.Tensor, new_lengths: torch.Tensor, refcount: torch.Tensor, *,
               page_tokens: int, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gives each row the pages it needs for ``new_lengths`` tokens instead of ``lengths`` (``table`` and ``refcount``
    change in place; nothing is taken away where a length falls).  Returns ``missing`` (int32, one entry): places that
    found no free page or lie past the table's width."""
    fn = "pages_grow"
    device = table.device
    _check_ints(fn, device, table=(table, 2), lengths=(lengths, 1), new_lengths=(new_lengths, 1), refcount=(refcount, 1))
    rows, width = table.shape
    if lengths.numel() != rows or new_lengths.numel() != rows:
        raise ValueError(f"{fn}: one length per row of the table is needed")
    if page_tokens < 1:
        raise ValueError(f"{fn}: page_tokens must be positive")
    lib = _lib.load()
    s, ctx = enter(device, stream)
    with ctx:
        missing = torch.empty(1, dtype=torch.int32, device=device)
        workspace = _workspace(fn, lib, workspace, rows, refcount.numel(), device)
        st = lib.ps_pages_grow(table.data_ptr(), lengths.data_ptr(), new_lengths.data_ptr(), rows, width, page_tokens,
                               refcount.data_ptr(), refcount.numel(), missing.data_ptr(), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), s)
    _lib.check("ps_pages_grow", st)
    return missing


def pages_free(table: torch.Tensor, refcount: torch.Tensor, *, flags: torch.Tensor | None = None, stream=None) -> None:
    """Lets go of all pages of the rows with ``flags`` (uint8, one per row) != 0, or of all rows: their counts fall, their
    places in ``table`` become -1 (both in place)."""
    fn = "pages_free"
    device = table.device
    _check_ints(fn, device, table=(table, 2), refcount=(refcount, 1))
    rows, width = table.shape
    if flags is not None and (flags.dtype != torch.uint8 or tuple(flags.shape) != (rows,) or flags.device != device
                              or not flags.is_contiguous()):
        raise ValueError(f"{fn}: flags must be a contiguous uint8 CUDA tensor with one entry per row")
    s, ctx = enter(device, stream)
    with ctx:
        st = _lib.load().ps_pages_free(table.data_ptr(), rows, width, flags.data_ptr() if flags is not None else None,
                                       refcount.data_ptr(), refcount.numel(), s)
    _lib.check("ps_pages_free", st)


def pages_compact(table: torch.Tensor, refcount: torch.Tensor, pools, *, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Moves pages so that the m pages in use are pages 0 .. m-1, in every pool; ``table`` and ``refcount`` follow in
    place.  Pages below m stay; the others fill the free places in order.  Returns m (int32, one entry, on the device)."""
    fn = "pages_compact"
    device = table.device
    _check_ints(fn, device, table=(table, 2), refcount=(refcount, 1))
    rows, width = table.shape
    pages = refcount.numel()
    arr, n = _pools(fn, pools, pages, device)
    lib = _lib.load()
    s, ctx = enter(device, stream)
    with ctx:
        used = torch.empty(1, dtype=torch.int32, device=device)
        workspace = _workspace(fn, lib, workspace, 0, pages, device)
        st = lib.ps_pages_compact(table.data_ptr(), rows, width, refcount.data_ptr(), arr, n, pages, used.data_ptr(),
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
    _lib.check("ps_pages_compact", st)
    return used
