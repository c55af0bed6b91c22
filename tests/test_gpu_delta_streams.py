"""The gated delta rule beside other work on the GPU: results do not depend on when its kernels' parts come to run.

Every comparison is bit for bit: the kernels have one order of sums, so any difference is a missing wait."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import _lib, api  # noqa: E402
from test_gpu_delta import BF16, CHUNKED, DEV, F16, F32, cu_of, inputs, off, states  # noqa: E402


class Busy:
    """Small kernels of memory traffic and matrix products on another stream while the block runs."""

    def __enter__(self):
        self.stream = torch.cuda.Stream()
        a, b = torch.randn(1024, 1024, device=DEV), torch.randn(1 << 22, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.stream(self.stream):
            for _ in range(150):
                a @ a
                b * 2
        return self.stream

    def __exit__(self, *_):
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("k,v,lens", [(128, 128, [700, 65, 0, 330]), (64, 64, [700, 65, 0, 330]), (128, 200, [1900]), (40, 24, [1900])])
def test_results_repeat_beside_other_work(dtype, k, v, lens):
    x = inputs(sum(lens), 2, 4, k, v, dtype, 3)
    h0, dht = states(len(lens), 4, k, v, 4), states(len(lens), 4, k, v, 5)
    do = torch.randn(x[2].shape, device=DEV).to(dtype)

    def run():
        o, last, saved = api.delta_rule_forward(*x, cu_seqlens=cu_of(lens), initial_state=h0, output_final_state=True)
        return (o, last, *api.delta_rule_backward(saved, do, d_final_state=dht))

    want = run()
    torch.cuda.synchronize()
    with Busy():
        for _ in range(10):
            for a, b in zip(run(), want):
                assert torch.equal(a, b)


# 2 to 8 chains of 14 to 72 chunks are cut into segments, and so are 22 of 160 (more segments than run at once)
CUT = [(BF16, 2, 128, 128, [1900]), (F32, 2, 64, 200, [1900]), (F16, 2, 80, 136, [2000, 900, 0, 1500]), (BF16, 8, 64, 40, [4608]),
       (BF16, 22, 128, 128, [10240])]


@pytest.mark.parametrize("dtype,hv,k,v,lens", CUT)
def test_state_in_place_of_cut_sequences(dtype, hv, k, v, lens):
    # the last segment writes the state at the end where the first one has read the state at the start
    x = inputs(sum(lens), 1, hv, k, v, dtype, 17, decay=0.05)
    h0, cu = states(len(lens), hv, k, v, 18), cu_of(lens)
    o, last = api.delta_rule(*x, cu_seqlens=cu, initial_state=h0, output_final_state=True)
    with Busy():
        for _ in range(8):
            h = h0.clone()
            again = api.delta_rule(*x, cu_seqlens=cu, initial_state=h, final_state=h)[0]
            assert torch.equal(again, o) and torch.equal(h, last)


def test_long_prompt_in_pieces():
    # pieces long enough to be cut, the state carried in place, against the whole prompt
    x = inputs(4096, 1, 2, 128, 128, BF16, 19, seqs=1, decay=0.02)
    _, want = api.delta_rule(*x, output_final_state=True)
    h = torch.zeros_like(want)
    for i in range(0, 4096, 2048):
        api.delta_rule(*(t[:, i:i + 2048] for t in x), initial_state=h, final_state=h)
    assert off(h, want.double()) <= 2 * CHUNKED


@pytest.mark.parametrize("dtype,hv,k,v,lens", CUT)
def test_state_gradient_in_place_of_cut_sequences(dtype, hv, k, v, lens):
    # the C ABI lets the gradient of the state at the start take the place of the one at the end
    x = inputs(sum(lens), 1, hv, k, v, dtype, 27, decay=0.05)
    h0, dht = states(len(lens), hv, k, v, 28), states(len(lens), hv, k, v, 29)
    do = torch.randn(x[2].shape, device=DEV).to(dtype)
    _, _, saved = api.delta_rule_forward(*x, cu_seqlens=cu_of(lens), initial_state=h0)
    want = api.delta_rule_backward(saved, do, d_final_state=dht)
    got = [torch.empty_like(t) for t in want[:5]]
    ts = [_lib.DELTA_TENSOR.pack(t.data_ptr(), 0, t.stride(0), t.stride(1)) for t in (*x[:2], do)]
    with Busy():
        for _ in range(8):
            d = dht.clone()
            st = _lib.load().ps_delta_backward(saved.shape, *ts, d.data_ptr(), *(t.data_ptr() for t in got), d.data_ptr(),
                                               saved.workspace.data_ptr(), saved.workspace.numel(), torch.cuda.current_stream().cuda_stream)
            assert st == _lib.PS_OK
            for a, b in zip((*got, d), want):
                assert torch.equal(a, b)


def test_backward_on_another_stream():
    # a gradient that has to be made contiguous first: the copy, too, belongs to the given stream.  Its old memory holds NaN,
    # and the current stream is held up, so that a copy made there would come late.
    x = inputs(600, 1, 2, 64, 64, BF16, 37, seqs=2)
    o, _, saved = api.delta_rule_forward(*x)
    grads = [torch.ones((), device=DEV, dtype=BF16).expand(o.shape),
             torch.randn(2, 600, 64, 2, device=DEV).to(BF16).transpose(2, 3)]
    s, big = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    for do in grads:
        want = api.delta_rule_backward(saved, do.contiguous())
        torch.cuda.synchronize()
        held = [torch.full(o.shape, float("nan"), device=DEV, dtype=BF16) for _ in range(4)]
        del held
        for _ in range(20):
            big @ big
        got = api.delta_rule_backward(saved, do, stream=s)
        for _ in range(4):   # what the current stream is given next
            torch.full(o.shape, float("nan"), device=DEV, dtype=BF16)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert a is b is None or torch.equal(a, b)


def test_saved_memory_outlives_a_backward_call_on_another_stream():
    # `saved`, its workspace and the inputs are dropped right after the call; the forward call's stream gets their memory next
    def inputs_and_saved():
        x = inputs(900, 2, 4, 64, 64, BF16, 47, seqs=2)
        return x, api.delta_rule_forward(*x)[2]

    do = torch.randn(2, 900, 4, 64, device=DEV).to(BF16)
    x, saved = inputs_and_saved()
    want = api.delta_rule_backward(saved, do)
    del x, saved
    big, s = torch.randn(4096, 4096, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (True, False):
        x, saved = inputs_and_saved()
        sizes = [t.numel() * t.element_size() for t in (saved.workspace, *x[:2])]
        gradient = do.clone()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(20):
                big @ big
            if not given:
                got = api.delta_rule_backward(saved, gradient)
        if given:
            got = api.delta_rule_backward(saved, gradient, stream=s)
        del x, saved, gradient
        new = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in (*sizes, do.numel() * 2)]
        torch.cuda.synchronize()
        del new
        for a, b in zip(got, want):
            assert a is b is None or torch.equal(a, b)
