"""The gated delta rule on the GPU against the recurrence in 64 bits, token by token.

Tolerances (2-norm of the difference over 2-norm of the result).  An output y of a 16-bit type is the rounding of a
32-bit value x' near the true x; as the rounding of x' is the number nearest to x', |y - x| <= |round(x) - x| + 2 |x' - x|,
so an output may be off by the true result's own rounding and twice what the 32-bit values may be off.  bf16 has 8
significant bits: a pair hi + lo is off by at most 2^-16 of the number, 2^-17 root-mean-square and less (uniform errors).
A chunk's results pass three dependent products of two operands each: 6 x 2^-17.  The single-step kernel works in f32
throughout: 2^-20 for sums of up to 128 terms.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import delta_reference as ref  # noqa: E402
from prefix_scan_gb300 import api  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CHUNKED, STEP = 6 * 2.0 ** -17, 2.0 ** -20


def inputs(tokens, hk, hv, k, v, dtype, seed, beta_dtype=None, decay=1.0, seqs=None):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    lead = (tokens,) if seqs is None else (seqs, tokens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, key = unit(rnd(*lead, hk, k)).to(dtype), unit(rnd(*lead, hk, k)).to(dtype)
    g = -decay * torch.rand(*lead, hv, device=DEV, generator=gen) * torch.logspace(-3, 0, hv, device=DEV)
    beta = torch.sigmoid(rnd(*lead, hv)).to(beta_dtype or dtype)
    return q, key, rnd(*lead, hv, v).to(dtype), g, beta


def states(n, hv, k, v, seed):
    return 0.3 * torch.randn(n, hv, k, v, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))


def cu_of(lens):
    return torch.tensor([0] + list(lens), device=DEV).cumsum(0).to(torch.int32)


def off(x, y):
    d = (x.double() - y).norm().item()
    n = y.norm().item()
    return d / n if n else d


def near(x, y, bound):
    assert x.shape == y.shape
    if x.dtype in (BF16, F16):
        bound = off(y.to(x.dtype), y) + 2 * bound
    assert off(x, y) <= bound, (off(x, y), bound)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("hk,hv,k,v", [(1, 1, 128, 128), (2, 6, 64, 128), (3, 3, 80, 56), (1, 2, 37, 19), (2, 2, 8, 200),
                                       (1, 1, 1, 1), (1, 3, 128, 64)])
def test_sequences(dtype, hk, hv, k, v):
    lens = [1, 64, 0, 63, 65, 130, 7, 200]
    x = inputs(sum(lens), hk, hv, k, v, dtype, 11)
    h0 = states(len(lens), hv, k, v, 12)
    o, last = api.delta_rule(*x, cu_seqlens=cu_of(lens), initial_state=h0, output_final_state=True)
    want = ref.packed(*x, k ** -0.5, lens, h0)
    near(o, want["o"], CHUNKED)
    near(last, want["state"], CHUNKED)
    assert torch.equal(last[2], h0[2])   # the empty sequence hands its state on


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000])
def test_lengths_batch(tokens):
    x = inputs(tokens, 2, 4, 128, 128, BF16, tokens, seqs=3, beta_dtype=F32)
    o, last = api.delta_rule(*x, scale=0.7, output_final_state=True)
    for i in range(3):
        want = ref.sequence(*(t[i] for t in x), 0.7)
        near(o[i], want["o"], CHUNKED)
        near(last[i], want["state"], CHUNKED)


def test_long_memory_and_long_sequence():
    x = inputs(5000, 1, 2, 128, 128, BF16, 5, decay=1e-3)
    o, last = api.delta_rule(*x, cu_seqlens=cu_of([5000]), output_final_state=True)
    want = ref.packed(*x, 128 ** -0.5, [5000])
    near(o, want["o"], CHUNKED)
    near(last, want["state"], CHUNKED)


@pytest.mark.parametrize("dtype,k,v", [(BF16, 128, 128), (F32, 64, 64), (F16, 80, 136), (BF16, 64, 40)])
@pytest.mark.parametrize("lens", [[1900], [2000, 900, 0, 1500], [3000, 1, 1, 3000]])
def test_sequences_cut_into_segments(dtype, k, v, lens):
    # few heads and many chunks: the states at the segments' starts come from a first pass and a join
    x = inputs(sum(lens), 1, 2, k, v, dtype, 7, decay=0.05)
    h0 = states(len(lens), 2, k, v, 8)
    o, last = api.delta_rule(*x, cu_seqlens=cu_of(lens), initial_state=h0, output_final_state=True)
    want = ref.packed(*x, k ** -0.5, lens, h0)
    near(o, want["o"], CHUNKED)
    near(last, want["state"], CHUNKED)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_alignment(dtype):
    T, hk, hv, k, v = 150, 2, 4, 64, 64
    q, key, val, g, beta = inputs(T, hk, hv, k, v, dtype, 21)
    want, wlast = api.delta_rule(q, key, val, g, beta, cu_seqlens=cu_of([T]), output_final_state=True)

    def check(q, key, val, g, beta):
        o, last = api.delta_rule(q, key, val, g, beta, cu_seqlens=cu_of([T]), output_final_state=True)
        assert torch.equal(o, want) and torch.equal(last, wlast)

    fused = torch.cat([t.reshape(T, -1) for t in (q, key, val)], 1)   # views of one projection
    a, b = hk * k, 2 * hk * k
    check(fused[:, :a].unflatten(1, (hk, k)), fused[:, a:b].unflatten(1, (hk, k)), fused[:, b:].unflatten(1, (hv, v)), g, beta)
    heads_first = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    check(*(heads_first(t) for t in (q, key, val, g, beta)))
    odd = [torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape).copy_(t) for t in (q, key, val)]
    check(*odd, g, beta)   # rows off the 16-byte boundary
    gb = torch.stack([g, beta.float()], -1)
    check(q, key, val, gb[..., 0], gb[..., 1].to(dtype))
    # backwards in memory, and one key head for all (stride 0)
    check(q.flip(0).contiguous().flip(0), key, val, g, beta)
    one = api.delta_rule(q[:, :1].expand(T, hv, k), key[:, :1].expand(T, hv, k), val, g, beta, cu_seqlens=cu_of([T]))[0]
    assert torch.equal(one, api.delta_rule(q[:, :1], key[:, :1], val, g, beta, cu_seqlens=cu_of([T]))[0])


def test_forgetting():
    # log decays at and below the smallest normal number's, and -inf, between ordinary ones
    T = 140
    q, k, v, g, beta = inputs(T, 1, 2, 64, 64, F32, 31)
    g[5], g[6], g[70, 0], g[128], g[139, 1] = -torch.inf, -200.0, -100.0, -torch.inf, -torch.inf
    h0 = states(1, 2, 64, 64, 32)
    o, last = api.delta_rule(q, k, v, g, beta, cu_seqlens=cu_of([T]), initial_state=h0, output_final_state=True)
    want = ref.packed(q, k, v, g, beta, 64 ** -0.5, [T], h0)
    near(o, want["o"], CHUNKED)
    near(last, want["state"], CHUNKED)
    # an infinite state is forgotten too
    h0[0, 0] = torch.inf
    g[0] = -torch.inf
    o, last = api.delta_rule(q, k, v, g, beta, cu_seqlens=cu_of([T]), initial_state=h0, output_final_state=True)
    assert torch.isfinite(o[:, 1]).all() and torch.isfinite(last[0, 1]).all()


def test_gates_of_zero_and_one():
    q, k, v, g, beta = inputs(100, 1, 2, 64, 32, F32, 41)
    beta[::3], beta[1::3] = 0.0, 1.0
    o, last = api.delta_rule(q, k, v, g, beta, cu_seqlens=cu_of([100]), output_final_state=True)
    want = ref.packed(q, k, v, g, beta, 64 ** -0.5, [100])
    near(o, want["o"], CHUNKED)
    near(last, want["state"], CHUNKED)
    beta.zero_()
    o, last = api.delta_rule(q, k, v, g, beta, cu_seqlens=cu_of([100]), output_final_state=True)
    assert o.abs().max() < 1e-15 and last.abs().max() < 1e-15


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_sequence(bad):
    lens = [70, 33, 90]
    x = inputs(sum(lens), 1, 2, 64, 64, BF16, 51)
    want, wlast = api.delta_rule(*x, cu_seqlens=cu_of(lens), output_final_state=True)
    for t in x:
        y = [u.clone() for u in x]
        y[[u.data_ptr() for u in x].index(t.data_ptr())][70:103] = bad
        o, last = api.delta_rule(*y, cu_seqlens=cu_of(lens), output_final_state=True)
        assert torch.equal(o[:70], want[:70]) and torch.equal(o[103:], want[103:])
        assert torch.equal(last[0], wlast[0]) and torch.equal(last[2], wlast[2])
        assert not torch.isfinite(o[70:103].float()).all()


def test_offsets_out_of_range_are_clamped():
    x = inputs(100, 1, 1, 64, 64, BF16, 61)
    cu = torch.tensor([-5, 40, 30, 4000, 1 << 30], dtype=torch.int32, device=DEV)   # [0,40) [40,40) [30,100) [100,100)
    o, last = api.delta_rule(*x, cu_seqlens=cu, output_final_state=True)
    torch.cuda.synchronize()
    assert torch.equal(o[:30], api.delta_rule(*(t[:40] for t in x), cu_seqlens=cu_of([40]))[0][:30])
    assert last[1].abs().max() == 0 and last[3].abs().max() == 0


def test_no_tokens_and_no_sequences():
    x = inputs(0, 1, 2, 64, 64, BF16, 71, seqs=3)
    h0 = states(3, 2, 64, 64, 72)
    o, last = api.delta_rule(*x, initial_state=h0, output_final_state=True)
    assert o.shape == (3, 0, 2, 64) and torch.equal(last, h0)
    o, last = api.delta_rule(*x, output_final_state=True)
    assert last.abs().max() == 0
    x = inputs(5, 1, 2, 64, 64, BF16, 73, seqs=0)
    o, last = api.delta_rule(*x, output_final_state=True)
    assert o.shape == (0, 5, 2, 64) and last.shape == (0, 2, 64, 64)


def test_state_in_place_and_in_pieces():
    # two calls over the halves of a sequence, the state carried in place, against one call
    x = inputs(256, 2, 2, 128, 128, F32, 81, seqs=2)
    want, wlast = api.delta_rule(*x, output_final_state=True)
    h = torch.zeros(2, 2, 128, 128, device=DEV)
    parts = [api.delta_rule(*(t[:, a:b] for t in x), initial_state=h, final_state=h)[0] for a, b in ((0, 128), (128, 256))]
    assert torch.equal(torch.cat(parts, 1), want) and torch.equal(h, wlast)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("n,t,hk,hv,k,v", [(1, 1, 16, 32, 128, 128), (3, 5, 2, 6, 64, 64), (70, 1, 4, 8, 128, 128),
                                           (5, 11, 1, 3, 40, 72), (2, 3, 1, 2, 33, 7), (300, 2, 1, 1, 16, 24), (2, 1, 2, 2, 1, 300)])
def test_step(dtype, n, t, hk, hv, k, v):
    x = inputs(t, hk, hv, k, v, dtype, 91, seqs=n)
    pool = states(n + 3, hv, k, v, 92)
    was = pool.clone()
    slots = torch.randperm(n + 3, device=DEV)[:n].to(torch.int32)
    o = api.delta_rule_step(*x, pool, slots=slots)
    for i in range(n):
        want = ref.sequence(*(y[i] for y in x), k ** -0.5, was[slots[i].long()])
        near(o[i], want["o"], STEP)
        near(pool[slots[i].long()], want["state"], STEP)
    rest = [p for p in range(n + 3) if p not in slots.tolist()]
    assert torch.equal(pool[rest], was[rest])


def test_step_lengths_and_absent_sequences():
    x = inputs(6, 2, 4, 64, 64, BF16, 101, seqs=5)
    pool = states(5, 4, 64, 64, 102)
    was = pool.clone()
    slots = torch.tensor([4, -1, 2, 99, 0], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([3, 6, 0, 6, 70], dtype=torch.int32, device=DEV)
    o = api.delta_rule_step(*x, pool, slots=slots, lengths=lengths)
    for i, (page, n) in enumerate(((4, 3), (None, 0), (2, 0), (None, 0), (0, 6))):
        assert o[i, n:].abs().max() == 0 if n < 6 else True
        if n:
            want = ref.sequence(*(y[i, :n] for y in x), 64 ** -0.5, was[page])
            near(o[i, :n], want["o"], STEP)
            near(pool[page], want["state"], STEP)
    assert torch.equal(pool[[1, 2, 3]], was[[1, 2, 3]])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("n,t,hk,hv,k,v", [(160, 1, 2, 4, 128, 128), (77, 3, 2, 8, 100, 68), (210, 4, 1, 3, 65, 124),
                                           (400, 2, 2, 4, 64, 64), (160, 4, 1, 4, 33, 36), (90, 1, 8, 8, 128, 60), (90, 2, 4, 8, 48, 128),
                                           (110, 1, 3, 6, 72, 200)])
def test_step_many_states(dtype, n, t, hk, hv, k, v):
    # enough heads for states to pass through shared memory; some sequences absent, some with fewer tokens
    x = inputs(t, hk, hv, k, v, dtype, 95, seqs=n)
    x[3][5:9] = -float("inf")
    pool = states(n + 3, hv, k, v, 96)
    slots = torch.randperm(n + 3, device=DEV)[:n].to(torch.int32)
    pool[slots[6].long()] = float("nan")
    slots[11], slots[12] = -1, n + 3
    lengths = torch.randint(0, t + 2, (n,), device=DEV).to(torch.int32)
    lengths[5:9] = t
    was = pool.clone()
    o = api.delta_rule_step(*x, pool, slots=slots, lengths=lengths)
    untouched = torch.ones(n + 3, dtype=torch.bool, device=DEV)
    for i in range(n):
        count = min(int(lengths[i]), t) if 0 <= slots[i] < n + 3 else 0
        assert (o[i, count:] == 0).all()
        if count:
            page = int(slots[i])
            untouched[page] = False
            before = torch.zeros_like(was[page]) if 5 <= i < 9 else was[page]
            want = ref.sequence(*(y[i, :count] for y in x), k ** -0.5, before)
            near(o[i, :count], want["o"], STEP)
            near(pool[page], want["state"], STEP)
    assert torch.equal(pool[untouched], was[untouched])


def test_many_sequences_of_different_lengths():
    # more chains than run at once, in another order than they come; and more sequences than are ordered
    for n, hv in ((100, 4), (300, 2)):
        lens = [(37 * i) % 131 for i in range(n)]
        x = inputs(sum(lens), 1, hv, 32, 40, F32, 131)
        h0 = states(n, hv, 32, 40, 132)
        o, last = api.delta_rule(*x, cu_seqlens=cu_of(lens), initial_state=h0, output_final_state=True)
        want = ref.packed(*x, 32 ** -0.5, lens, h0)
        near(o, want["o"], CHUNKED)
        near(last, want["state"], CHUNKED)


def test_steps_continue_a_prompt():
    # a prompt by chunks, its state handed to single steps, against the whole sequence
    x = inputs(80, 2, 4, 128, 128, F32, 111, seqs=2)
    want, wlast = api.delta_rule(*x, output_final_state=True)
    _, pool = api.delta_rule(*(t[:, :70] for t in x), output_final_state=True)
    outs = [api.delta_rule_step(*(t[:, i:i + 1] for t in x), pool) for i in range(70, 80)]
    near(torch.cat(outs, 1), want[:, 70:].double(), 2 * CHUNKED)
    near(pool, wlast.double(), 2 * CHUNKED)


def test_step_unaligned_pool():
    x = inputs(1, 1, 2, 64, 64, F32, 121, seqs=2)
    pool = states(2, 2, 64, 64, 122)
    other = torch.empty(pool.numel() + 1, device=DEV)[1:].view(pool.shape).copy_(pool)
    assert torch.equal(api.delta_rule_step(*x, pool), api.delta_rule_step(*x, other))
    assert torch.equal(pool, other)


def test_another_stream_and_graph():
    x = inputs(200, 1, 2, 64, 64, BF16, 131, seqs=2)
    want, wlast = api.delta_rule(*x, output_final_state=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, last = api.delta_rule(*x, output_final_state=True, stream=s)
    s.synchronize()
    assert torch.equal(o, want) and torch.equal(last, wlast)
    shape = api.delta_rule_workspace_size(x[0], x[2])
    ws, out, fin = torch.empty(shape, dtype=torch.uint8, device=DEV), torch.empty_like(want), torch.empty_like(wlast)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.delta_rule(*x, out=out, final_state=fin, workspace=ws)
    new = inputs(200, 1, 2, 64, 64, BF16, 132, seqs=2)
    for a, b in zip(x, new):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    want, wlast = api.delta_rule(*new, output_final_state=True)
    assert torch.equal(out, want) and torch.equal(fin, wlast)


def test_refusals():
    q, k, v, g, beta = inputs(10, 2, 4, 64, 64, BF16, 141)
    cu = cu_of([10])
    call = lambda *x, **kw: api.delta_rule(*x, **{"cu_seqlens": cu, **kw})  # noqa: E731
    with pytest.raises(TypeError):
        call(q.float(), k, v, g, beta)
    with pytest.raises(TypeError):
        call(q, k, v, g.to(BF16), beta)
    with pytest.raises(TypeError):
        call(q.double(), k.double(), v.double(), g, beta)
    with pytest.raises(ValueError, match="go together"):
        call(q, k[:9], v, g, beta)
    with pytest.raises(ValueError, match="multiple"):
        call(q, k, v[:, :3], g[:, :3], beta[:, :3])
    with pytest.raises(ValueError, match="cu_seqlens"):
        call(q, k, v, g, beta, cu_seqlens=cu.long())
    with pytest.raises(ValueError, match="sequences"):
        call(q[None], k[None], v[None], g[None], beta[None])
    with pytest.raises(ValueError, match="contiguous"):
        call(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, g, beta)
    with pytest.raises(ValueError, match="initial_state"):
        call(q, k, v, g, beta, initial_state=torch.zeros(2, 4, 64, 64, device=DEV))
    with pytest.raises(ValueError, match="workspace"):
        call(q, k, v, g, beta, workspace=torch.empty(100, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="up to 128"):
        call(*(torch.zeros(10, 2, 136, dtype=BF16, device=DEV) for _ in range(2)), v, g, beta)
    from prefix_scan_gb300 import PrefixScanError
    with pytest.raises(PrefixScanError, match="OVERLAP"):
        call(q, k, v, g, beta, out=v)
    x = inputs(1, 2, 4, 64, 64, BF16, 142, seqs=2)
    with pytest.raises(ValueError, match="fewer pages"):
        api.delta_rule_step(*x, torch.zeros(1, 4, 64, 64, device=DEV))
    with pytest.raises(ValueError, match="slots"):
        api.delta_rule_step(*x, torch.zeros(3, 4, 64, 64, device=DEV), slots=torch.zeros(3, dtype=torch.int32, device=DEV))
