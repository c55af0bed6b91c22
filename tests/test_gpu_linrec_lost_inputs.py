"""The gated linear recurrence where a tile's inputs do not come: the bounded waits run out, the call ends, and whatever rests on
the tile is NaN.

A correct launch never gets there.  So the kernels are built a second time, with a limit of 50 ms, so that one tile (its number
TILE, of the first 32 channels) is never copied and nothing completes the barrier that its warps wait at.  What they find in
shared memory instead is numbers that no index is made of."""
from __future__ import annotations

import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import _lib, api  # noqa: E402
from prefix_scan_gb300 import build as nvbuild  # noqa: E402

DEV = "cuda"
TILE = 3
LENS = [1400, 0, 1160, 1536]   # their starts and ends lie before, in and behind the tile, whatever its length
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def lossy():
    note = nvbuild.BUILD_DIR / "linrec_lost" / "note.cu"
    note.parent.mkdir(parents=True, exist_ok=True)
    note.write_text('#include "scan_internal.h"\nvoid ps::note_cuda_error(cudaError_t) {}\n')
    path = nvbuild.build_variant("linrec_lost", {"PS_TESTING_LOST_TILE": TILE, "PS_LINREC_WAIT_LIMIT_NS": 50_000_000},
                                 only=[note] + [p for p in nvbuild.sources() if p.name.startswith("linrec_")])
    lib = ctypes.CDLL(str(path))
    for name, (res, args) in _lib.SIGNATURES.items():
        if name.startswith("ps_linrec_"):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
    return lib


def nan_or(got, want):
    return (torch.isnan(got) | (got == want)).all()


@pytest.mark.parametrize("dtype,gtype,forward_tile,backward_tile", [(F32, F32, 256, 128), (BF16, F32, 256, 256), (F16, F16, 512, 256)])
def test_what_rests_on_a_tile_that_does_not_come_is_nan(lossy, monkeypatch, dtype, gtype, forward_tile, backward_tile):
    gen = torch.Generator(device=DEV).manual_seed(5)
    n, d = sum(LENS), 40
    x, dh = (torch.randn(n, d, device=DEV, generator=gen).to(dtype) for _ in range(2))
    g = (-0.01 * torch.rand(n, d, device=DEV, generator=gen)).to(gtype)
    h0, dht = (torch.randn(len(LENS), d, device=DEV, generator=gen) for _ in range(2))
    ends = torch.tensor(LENS).cumsum(0).tolist()
    starts = [0] + ends[:-1]
    cu = torch.tensor([0] + ends, dtype=torch.int32, device=DEV)

    def forward():
        return api.linear_recurrence_forward(x, g, tied=True, cu_seqlens=cu, initial_state=h0, output_final_state=True)

    h, state, saved = forward()
    dx, dg, dh0 = api.linear_recurrence_backward(saved, dh, d_final_state=dht)
    assert all(t.isfinite().all() for t in (h, state, dx, dg, dh0))
    with monkeypatch.context() as m:
        m.setattr(_lib, "load", lambda: lossy)
        lost_h, lost_state, lost_saved = forward()
        lost = api.linear_recurrence_backward(saved, dh, d_final_state=dht)
    torch.cuda.synchronize()

    first, last = TILE * forward_tile, (TILE + 1) * forward_tile   # the tile; then on to the end of the sequence that goes on behind it
    last = max([last] + [e for s, e in zip(starts, ends) if s < last < e])
    assert torch.isnan(lost_h[first:last, :32]).all()
    assert nan_or(lost_h, h) and nan_or(lost_state, state) and not torch.isnan(lost_h[:, :32]).all()
    for i, e in enumerate(ends):
        if LENS[i] and first < e <= last:
            assert torch.isnan(lost_state[i, :32]).all()
    assert torch.equal(lost_state[1], state[1])   # an empty sequence's

    first, last = TILE * backward_tile, (TILE + 1) * backward_tile   # and back to the start of the sequence that goes on before it
    first = min([first] + [s for s, e in zip(starts, ends) if s < first < e])
    for name, got, want in zip(("dx", "dg"), lost, (dx, dg)):
        assert torch.isnan(got[first:last, :32]).all(), name
        assert nan_or(got, want) and not torch.isnan(got[:, :32]).all(), name
    assert nan_or(lost[2], dh0) and torch.equal(lost[2][1], dh0[1])
    for i, s in enumerate(starts):
        if LENS[i] and first <= s < last:
            assert torch.isnan(lost[2][i, :32]).all()

    # a backward pass of what a lossy forward pass left is NaN where it needs its states, and the next calls are whole again
    assert nan_or(api.linear_recurrence_backward(lost_saved, dh, d_final_state=dht)[1], dg)
    again = forward()
    for got, want in zip((*again[:2], *api.linear_recurrence_backward(again[2], dh, d_final_state=dht)), (h, state, dx, dg, dh0)):
        assert torch.equal(got, want)
