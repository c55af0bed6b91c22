"""Gradients of the gated delta rule on the GPU: against the recurrence's own in 64 bits, and against differences.

Tolerances (2-norm of the difference over 2-norm of the result; see test_gpu_delta.py for the allowance of a 16-bit
result's own rounding): a pair of bf16 is off by 2^-17 (root-mean-square).  A gradient passes the forward chain's three
dependent products, the backward chain's three and two more in the last kernel, of two operands each: 16 x 2^-17.

Differences: L(x) = <d_o, o> + <d_ht, h_T> along a random unit direction of one input at a time, in f32,
(L(x + e) - L(x - e)) / 2.  The forward values are off by 6 x 2^-17 of the terms of L, whose independent errors add up to
about 6 x 2^-17 sqrt(|d_o|^2 |o|^2 / n) over n numbers, and the quotient's own error is of third order in e: with |e| = 1e-1
of an input's norm spread over all its numbers that is 1e-2 of the derivative at most.  2 % of |gradient| |e| is allowed.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import delta_reference as ref  # noqa: E402
from prefix_scan_gb300 import api  # noqa: E402
from test_gpu_delta import BF16, DEV, F16, F32, cu_of, inputs, off, states  # noqa: E402

GRAD = 16 * 2.0 ** -17
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


def near(x, y, bound, name=""):
    assert x.shape == y.shape
    if x.dtype in (BF16, F16):
        bound = off(y.to(x.dtype), y) + 2 * bound
    assert off(x, y) <= bound, (name, off(x, y), bound)


def gradients(x, lens=None, h0=None, dht=None, seed=7, scale=None):
    do = torch.randn(x[2].shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)).to(x[2].dtype)
    o, last, saved = api.delta_rule_forward(*x, cu_seqlens=None if lens is None else cu_of(lens), initial_state=h0,
                                            output_final_state=True, scale=scale)
    return do, o, last, saved, api.delta_rule_backward(saved, do, d_final_state=dht)


def check(x, lens, h0=None, dht=None, scale=None):
    do, o, last, _, got = gradients(x, lens, h0, dht, scale=scale)
    want = ref.packed(*x, x[0].shape[-1] ** -0.5 if scale is None else scale, lens, h0, do, dht)
    plain = api.delta_rule(*x, cu_seqlens=cu_of(lens), initial_state=h0, output_final_state=True, scale=scale)
    assert torch.equal(o, plain[0]) and torch.equal(last, plain[1])
    for name, t in zip(NAMES, got):
        if t is not None:
            near(t, want[name], GRAD, name)
    assert (got[5] is None) == (h0 is None)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("hk,hv,k,v", [(1, 1, 128, 128), (2, 6, 64, 128), (3, 3, 80, 56), (1, 2, 37, 19), (2, 2, 8, 200), (1, 3, 128, 64)])
def test_gradients(dtype, hk, hv, k, v):
    lens = [1, 64, 0, 63, 65, 130, 7, 200]
    n = len(lens)
    check(inputs(sum(lens), hk, hv, k, v, dtype, 11), lens, states(n, hv, k, v, 12), states(n, hv, k, v, 13))


@pytest.mark.parametrize("tokens", [1, 2, 16, 17, 63, 64, 65, 128, 700])
def test_lengths(tokens):
    check(inputs(tokens, 2, 4, 128, 128, BF16, tokens, beta_dtype=F32), [tokens], scale=0.5)


@pytest.mark.parametrize("dtype,k,v", [(BF16, 128, 128), (F32, 64, 64), (F16, 80, 136)])
@pytest.mark.parametrize("lens", [[1900], [2000, 900, 0, 1500]])
def test_sequences_cut_into_segments(dtype, k, v, lens):
    n = len(lens)
    x = inputs(sum(lens), 1, 2, k, v, dtype, 7, decay=0.05)
    check(x, lens, states(n, 2, k, v, 8), states(n, 2, k, v, 9))


def test_batch_layout_and_strided_gradient():
    x = inputs(100, 1, 2, 64, 64, BF16, 21, seqs=3)
    do, _, _, saved, got = gradients(x)
    flat = [t.reshape(300, *t.shape[2:]) for t in x]
    want = ref.packed(*flat, 64 ** -0.5, [100] * 3, None, do.reshape(300, 2, 64))
    for name, t in zip(NAMES[:5], got):
        near(t.reshape(300, *t.shape[2:]), want[name], GRAD, name)
    wide = torch.randn(3, 100, 2, 3, 64, device=DEV).to(BF16)
    wide[..., 1, :] = do
    for g2, g1 in zip(api.delta_rule_backward(saved, wide[..., 1, :]), got):
        assert g1 is None or torch.equal(g1, g2)
    # heads outermost, and a gradient of one number for all
    turned = do.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    for g2, g1 in zip(api.delta_rule_backward(saved, turned), got):
        assert g1 is None or torch.equal(g1, g2)
    one = torch.ones((), device=DEV, dtype=BF16).expand(do.shape)
    for g2, g1 in zip(api.delta_rule_backward(saved, one), api.delta_rule_backward(saved, one.contiguous())):
        assert g1 is None or torch.equal(g1, g2)


def test_forgetting():
    T = 140
    x = inputs(T, 1, 2, 64, 64, F32, 31)
    g = x[3]
    g[5], g[6], g[70, 0], g[128], g[139, 1], g[0, 0] = -torch.inf, -200.0, -100.0, -torch.inf, -torch.inf, -torch.inf
    h0, dht = states(1, 2, 64, 64, 32), states(1, 2, 64, 64, 33)
    do, _, _, _, got = gradients(x, [T], h0, dht)
    gr = torch.where(g <= -87, -torch.inf, g)   # what exp(-100) would leave is dropped
    want = ref.packed(*x[:3], gr, x[4], 64 ** -0.5, [T], h0, do, dht)
    for name, t in zip(NAMES, got):
        near(t, want[name].nan_to_num(), GRAD, name)
    assert (got[3][g <= -87] == 0).all()


def test_gates_of_zero_and_one():
    x = inputs(100, 1, 2, 64, 32, F32, 41)
    x[4][::3], x[4][1::3] = 0.0, 1.0
    check(x, [100], states(1, 2, 64, 32, 42), states(1, 2, 64, 32, 43))
    x[4].zero_()
    check(x, [100], states(1, 2, 64, 32, 42), states(1, 2, 64, 32, 43))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("k,v", [(37, 19), (64, 64), (128, 19)])
def test_value_gradients_do_not_depend_on_how_fast_they_are_stored(dtype, k, v):
    # many chunks behind rows that are stored number by number, again and again
    lens = [700, 640, 65, 0, 330]
    x = inputs(sum(lens), 2, 4, k, v, dtype, 14)
    do, _, _, saved, got = gradients(x, lens)
    want = ref.packed(*x, k ** -0.5, lens, None, do)
    for name, t in zip(NAMES, got):
        if t is not None:
            near(t, want[name], GRAD, name)
    for _ in range(30):
        for a, b in zip(api.delta_rule_backward(saved, do), got):
            assert a is None or torch.equal(a, b)


def test_reproducible_and_repeatable():
    x = inputs(500, 2, 6, 128, 128, BF16, 51)
    do, _, _, saved, got = gradients(x, [200, 300])
    for _ in range(3):
        for a, b in zip(api.delta_rule_backward(saved, do), got):
            assert a is None or torch.equal(a, b)


def test_tokens_of_no_sequence_have_no_gradient():
    x = inputs(100, 1, 1, 64, 64, BF16, 61)
    cu = torch.tensor([10, 50, 90], dtype=torch.int32, device=DEV)
    _, _, saved = api.delta_rule_forward(*x, cu_seqlens=cu)
    for t in api.delta_rule_backward(saved, torch.ones_like(x[2]))[:5]:
        assert (t[:10] == 0).all() and (t[90:] == 0).all() and torch.isfinite(t).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", [[0, 5], [7, 7], [130, 130, 200, 250], [3, 300], [300, 300], [90, 20, 40]])
def test_tokens_of_no_sequence_in_used_memory(dtype, cu):
    # new tensors come from memory that held NaN; offsets that fall count as empty sequences
    x = inputs(300, 2, 4, 24, 40, dtype, 51)
    o, _, saved = api.delta_rule_forward(*x, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    held = [torch.full_like(t, float("nan")) for t in (*x, *x)]
    del held
    grads = api.delta_rule_backward(saved, torch.ones_like(o))[:5]
    outside = torch.ones(300, dtype=torch.bool, device=DEV)
    for a, b in zip(cu, cu[1:]):
        outside[a:max(a, b)] = False
    for grad in grads:
        assert (grad[outside] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_gradients_stay_in_their_sequence(bad):
    lens = [70, 33, 90]
    x = inputs(sum(lens), 1, 2, 64, 64, BF16, 71)
    do, _, _, saved, want = gradients(x, lens)
    do[70:103] = bad
    for a, b in zip(api.delta_rule_backward(saved, do)[:5], want):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[103:], b[103:])


def test_no_tokens():
    x = inputs(0, 1, 2, 64, 64, BF16, 81, seqs=3)
    h0, dht = states(3, 2, 64, 64, 82), states(3, 2, 64, 64, 83)
    _, _, _, _, got = gradients(x, None, h0, dht)
    assert torch.equal(got[5], dht) and got[0].shape == x[0].shape


@pytest.mark.parametrize("which", range(6))
def test_against_differences(which):
    lens = [150, 61]
    n = sum(lens)
    x = list(inputs(n, 1, 2, 64, 48, F32, 91))
    h0, dht = states(2, 2, 64, 48, 92), states(2, 2, 64, 48, 93)
    do, _, _, _, got = gradients(x, lens, h0, dht)
    base = h0 if which == 5 else x[which]
    d = torch.randn(base.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(94)) * got[which].abs()
    d *= 0.1 * base.norm() / d.norm() / base[0].numel() ** 0.5

    def value(sign):
        y, h = list(x), h0
        if which == 5:
            h = h0 + sign * d
        else:
            y[which] = x[which] + sign * d
        o, last = api.delta_rule(*y, cu_seqlens=cu_of(lens), initial_state=h, output_final_state=True)
        return (o.double() * do.double()).sum().item() + (last.double() * dht.double()).sum().item()

    slope = (value(1) - value(-1)) / 2
    want = (got[which].double() * d.double()).sum().item()
    assert abs(slope - want) <= 0.02 * got[which].double().norm().item() * d.double().norm().item(), (slope, want)


def test_refusals():
    x = inputs(10, 2, 4, 64, 64, BF16, 101)
    _, _, saved = api.delta_rule_forward(*x, cu_seqlens=cu_of([10]))
    with pytest.raises(ValueError, match="d_o"):
        api.delta_rule_backward(saved, x[2].float())
    with pytest.raises(ValueError, match="d_o"):
        api.delta_rule_backward(saved, x[2][:9])
    with pytest.raises(ValueError, match="d_final_state"):
        api.delta_rule_backward(saved, x[2], d_final_state=torch.zeros(1, 4, 64, 63, device=DEV))
