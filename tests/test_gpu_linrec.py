"""The gated linear recurrence against the recurrence in 64 bits (linrec_reference.py states the tolerances)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import linrec_reference as ref  # noqa: E402
from prefix_scan_gb300 import api  # noqa: E402

DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]
INF, NAN = float("inf"), float("nan")


def make(tokens, d, dtype, gtype, seed, slow=6.0):
    """Inputs on the host; log decays from long memory to short, channel by channel."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, d, generator=gen)
    rate = torch.exp(-slow + slow * torch.rand(d, generator=gen))
    g = -rate * torch.nn.functional.softplus(torch.randn(tokens, d, generator=gen))
    return x.to(dtype), g.to(gtype), torch.randn(tokens, d, generator=gen).to(dtype)


def states(n, d, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(n, d, generator=gen), torch.randn(n, d, generator=gen)


def cu_of(lens, first=0):
    return torch.tensor([first] + lens).cumsum(0).to(torch.int32).to(DEV)


def run_packed(x, g, lens, dh, h0, dht, tied, first=0):
    """Forward and backward over packed sequences; everything by name."""
    dev = [None if t is None else t.to(DEV) for t in (x, g, dh, h0, dht)]
    out = torch.full(x.shape, 7.0, dtype=x.dtype, device=DEV)
    h, state, saved = api.linear_recurrence_forward(dev[0], dev[1], tied=tied, cu_seqlens=cu_of(lens, first), initial_state=dev[3],
                                                    output_final_state=True, out=out)
    assert h is out
    dx, dg, dh0 = api.linear_recurrence_backward(saved, dev[2], d_final_state=dev[4])
    return {"h": h, "state": state, "dx": dx, "dg": dg, "dh0": dh0}


def check_packed(got, x, g, lens, dh, h0, dht, tied, first=0):
    want, held = ref.packed(x, g, lens, first, h0, tied, dh, dht)
    for name, value in got.items():
        if value is None:
            continue
        if name in ("state", "dh0"):
            ref.check(value, want[name], name)
            continue
        value = value.cpu()
        ref.check(value[held], tuple(y[held] for y in want[name]), name)
        assert (value[~held] == (7 if name == "h" else 0)).all(), f"{name} of tokens that no sequence holds"


LENS = {"one token": [1], "a tile": [128], "a tile and one": [129], "many tiles": [1500],
        "ragged": [5, 0, 131, 1, 1, 16, 127, 300, 0, 0, 17, 400, 2], "short ones": [1, 2, 3, 1, 0, 1] * 40, "all empty but one": [0, 0, 3, 0]}


@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_packed(types, tied, lens):
    d = 70
    x, g, dh = make(sum(lens), d, *types, 1)
    h0, dht = states(len(lens), d, 2)
    check_packed(run_packed(x, g, lens, dh, h0, dht, tied), x, g, lens, dh, h0, dht, tied)


@pytest.mark.parametrize("d", [1, 2, 31, 64, 65, 130, 257])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F16, F32)], ids=str)
def test_channels(types, d):
    lens = [200, 3, 150]
    x, g, dh = make(sum(lens), d, *types, 3)
    h0, dht = states(len(lens), d, 4)
    check_packed(run_packed(x, g, lens, dh, h0, dht, True), x, g, lens, dh, h0, dht, True)


@pytest.mark.parametrize("types", TYPES, ids=str)
def test_no_states_given(types):
    lens = [90, 300]
    x, g, dh = make(sum(lens), 66, *types, 5)
    got = run_packed(x, g, lens, dh, None, None, False)
    assert got["dh0"] is None
    check_packed(got, x, g, lens, dh, None, None, False)


@pytest.mark.parametrize("first,lens,tokens", [(3, [200, 0, 41], 400), (130, [1, 2], 133), (0, [5], 700), (300, [0, 0], 301), (0, [128], 257)])
def test_tokens_that_no_sequence_holds(first, lens, tokens):
    # they hold NaN, which must not reach anything; outputs there stay, gradients are 0
    x, g, dh = make(tokens, 66, BF16, F32, 7)
    h0, dht = states(len(lens), 66, 8)
    last = first + sum(lens)
    for t in (x, g, dh):
        t[:first] = NAN
        t[last:] = NAN
    check_packed(run_packed(x, g, lens, dh, h0, dht, True, first), x, g, lens, dh, h0, dht, True, first)


@pytest.mark.parametrize("seqs,tokens", [(1, 1), (3, 1), (2, 128), (5, 37), (300, 2), (2, 700), (1, 12000), (4, 0)])
@pytest.mark.parametrize("d", [33, 96])
def test_equal_lengths(seqs, tokens, d):
    x, g, dh = make(seqs * tokens, d, F16, F16, 9)
    h0, dht = states(seqs, d, 10)
    h, state, saved = api.linear_recurrence_forward(x.view(seqs, tokens, d).to(DEV), g.view(seqs, tokens, d).to(DEV),
                                                    initial_state=h0.to(DEV), output_final_state=True)
    dx, dg, dh0 = api.linear_recurrence_backward(saved, dh.view(seqs, tokens, d).to(DEV), d_final_state=dht.to(DEV))
    got = {"h": h.flatten(0, 1), "state": state, "dx": dx.flatten(0, 1), "dg": dg.flatten(0, 1), "dh0": dh0}
    check_packed(got, x, g, [tokens] * seqs, dh, h0, dht, False)


def test_long_and_narrow():
    # more tiles than a look-back window holds, over a single block of channels
    x, g, dh = make(40000, 5, F32, F32, 11, slow=9.0)
    h0, dht = states(1, 5, 12)
    check_packed(run_packed(x, g, [40000], dh, h0, dht, True), x, g, [40000], dh, h0, dht, True)


def test_fixed_slow_decay_does_not_drift():
    # the same decay in every token: a factor's error to one side adds up over a memory of 20000 tokens
    tokens = 60000
    gen = torch.Generator().manual_seed(13)
    x = torch.randn(tokens, 8, generator=gen) + 1
    g = torch.full((tokens, 8), -5e-5) * torch.arange(1, 9)
    for tied in (False, True):
        h, state = api.linear_recurrence(x[None].to(DEV), g[None].to(DEV), tied=tied, output_final_state=True)
        want = ref.sequence(x, g, tied=tied)
        ref.check(h[0], want["h"], "h")
        # all inputs near 1: what is left of the errors is that of the factors, 2^-22.5, and of 60000 roundings
        assert float(((state[0].cpu().double() - want["state"][0]) / want["state"][0]).abs().max()) < 2.0 ** -22.5 + 6 * U_OF(20000)


def U_OF(memory):
    """The deviation of a sum of `memory` roundings of u each, relative to a state that they make up."""
    return memory ** 0.5 * ref.U


def strided(t, how):
    """`t` [sequences, tokens, d] with other strides, on the device."""
    t = t.to(DEV)
    n, m, d = t.shape
    if how == "projection":
        return torch.cat([torch.full_like(t, NAN), t, torch.full_like(t, NAN)], -1)[..., d:2 * d]
    if how == "odd":
        big = torch.full((n, m, 2 * d + 3), NAN, dtype=t.dtype, device=DEV)
        big[..., 1:d + 1] = t
        return big[..., 1:d + 1]
    if how == "tokens first":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    big = torch.full((n + 1, 2 * m, d), NAN, dtype=t.dtype, device=DEV)   # every other token
    big[:n, ::2] = t
    return big[:n, ::2]


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32)], ids=str)
@pytest.mark.parametrize("seqs,tokens,d", [(3, 1024, 40), (5, 512, 16), (2, 4096, 30), (7, 1536, 300)])
def test_equal_sequences_that_take_turns(types, seqs, tokens, d):
    # of whole tiles: those of one sequence are not next to one another in the order of work
    x, g, dh = make(seqs * tokens, d, *types, 35)
    h0, dht = states(seqs, d, 36)
    view = lambda t: t.view(seqs, tokens, d).to(DEV)  # noqa: E731
    for _ in range(3):
        h, state, saved = api.linear_recurrence_forward(view(x), view(g), tied=True, initial_state=h0.to(DEV), output_final_state=True)
        dx, dg, dh0 = api.linear_recurrence_backward(saved, view(dh), d_final_state=dht.to(DEV))
    got = {"h": h.flatten(0, 1), "state": state, "dx": dx.flatten(0, 1), "dg": dg.flatten(0, 1), "dh0": dh0}
    check_packed(got, x, g, [tokens] * seqs, dh, h0, dht, True)


def test_many_chains_under_way_at_once():
    # more tiles than run at once, of many chains, alone and one call after another: every result the same, and finite
    x, g, dh = (t.to(DEV).view(8, 2048, 1024) for t in make(8 * 2048, 1024, BF16, BF16, 37))
    want = None
    for i in range(30):
        h, state, saved = api.linear_recurrence_forward(x, g, output_final_state=True)
        got = (h, state, *api.linear_recurrence_backward(saved, dh)[:2])
        if i % 3 == 0:
            torch.cuda.synchronize()
        want = got if want is None else want
        for a, b in zip(got, want):
            assert torch.equal(a, b) and a.isfinite().all()


@pytest.mark.parametrize("how", ["projection", "odd", "tokens first", "every other"])
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_strides(types, how):
    n, m, d = 3, 170, 68
    x, g, dh = make(n * m, d, *types, 15)
    h0, dht = states(n, d, 16)
    view = lambda t: strided(t.view(n, m, d), how)  # noqa: E731
    h, state, saved = api.linear_recurrence_forward(view(x), view(g), tied=True, initial_state=h0.to(DEV), output_final_state=True)
    dx, dg, dh0 = api.linear_recurrence_backward(saved, view(dh), d_final_state=dht.to(DEV))
    got = {"h": h.flatten(0, 1), "state": state, "dx": dx.flatten(0, 1), "dg": dg.flatten(0, 1), "dh0": dh0}
    check_packed(got, x, g, [m] * n, dh, h0, dht, True)


def test_broadcast_decay():
    # one log decay a channel for all tokens, and a gradient of all ones: stride 0
    n, m, d = 2, 300, 64
    x, g, _ = make(n * m, d, F32, F32, 17)
    g = g[:1].expand(n * m, d)
    h, _, saved = api.linear_recurrence_forward(x.view(n, m, d).to(DEV), g[:1].to(DEV).view(1, 1, d).expand(n, m, d))
    dx, dg, _ = api.linear_recurrence_backward(saved, torch.ones(1, 1, 1, device=DEV).expand(n, m, d))
    check_packed({"h": h.flatten(0, 1), "dx": dx.flatten(0, 1), "dg": dg.flatten(0, 1)}, x, g, [m] * n, torch.ones(n * m, d), None, None,
                 False)


def test_extreme_decays():
    lens = [400]
    x, g, dh = make(400, 64, F32, F32, 19)
    g[7] = -INF
    g[130, ::2] = -INF
    g[200:210] = -200.0
    g[::3, 5] = 0.0
    g[:, 9] = 0.0
    g[:, 11] = -1e-7
    g[:, 13] = -30.0
    g[129, 15] = 0.4      # above 0 now and then
    x[:130] *= 1e6        # which a closed gate forgets
    h0, dht = states(1, 64, 20)
    check_packed(run_packed(x, g, lens, dh, h0, dht, True), x, g, lens, dh, h0, dht, True)
    check_packed(run_packed(x, g, lens, dh, h0, dht, False), x, g, lens, dh, h0, dht, False)


def test_not_finite_stays_in_its_sequence_and_channel():
    lens = [200, 3, 90, 400]
    x, g, dh = make(sum(lens), 66, BF16, BF16, 21)
    h0, dht = states(4, 66, 22)
    clean = run_packed(x, g, lens, dh, h0, dht, True)
    x[250, 3], g[210, 5], x[300, 40] = NAN, NAN, INF     # all in the third sequence: 203 ... 292; the fourth: 293 ...
    got = run_packed(x, g, lens, dh, h0, dht, True)
    dirty = torch.zeros(sum(lens), 66, dtype=torch.bool)
    dirty[203:293, 3] = dirty[203:293, 5] = dirty[293:, 40] = True
    for name in ("h", "dx", "dg"):
        assert torch.equal(got[name].cpu()[~dirty], clean[name].cpu()[~dirty])
    assert not got["h"][250:293, 3].isfinite().any() and got["h"][203:250, 3].isfinite().all()
    assert not got["h"][300:, 40].isfinite().any()
    for name in ("state", "dh0"):
        assert torch.equal(got[name][:2], clean[name][:2])


@pytest.mark.parametrize("types", [(BF16, F32), (F32, F32)], ids=str)
def test_state_in_place(types):
    # a prompt in pieces, the state carried in place, is the whole prompt
    d, lens = 64, [1000]
    x, g, _ = make(1000, d, *types, 23)
    h0, _ = states(1, d, 24)
    want, _ = ref.packed(x, g, lens, 0, h0, True)
    state, out = h0.to(DEV), []
    for i in (0, 300, 301, 700):
        j = {0: 300, 300: 301, 301: 700, 700: 1000}[i]
        h, last = api.linear_recurrence(x[None, i:j].to(DEV), g[None, i:j].to(DEV), tied=True, initial_state=state, final_state=state)
        assert last is state
        out.append(h[0])
    # each piece starts from a state rounded to 32 bits: nothing more than a token's rounding
    ref.check(torch.cat(out), want["h"], "h")
    ref.check(state, want["state"], "state")


def test_results_repeat_bit_for_bit():
    # beside other work, so that states become known in another order
    lens = [3000, 1, 0, 777, 5000]
    x, g, dh = (t.to(DEV) for t in make(sum(lens), 200, BF16, F32, 25))
    h0, dht = (t.to(DEV) for t in states(len(lens), 200, 26))
    cu = cu_of(lens)

    def run():
        h, state, saved = api.linear_recurrence_forward(x, g, cu_seqlens=cu, initial_state=h0, output_final_state=True)
        return (h, state, *api.linear_recurrence_backward(saved, dh, d_final_state=dht))

    want = run()
    other, a = torch.cuda.Stream(), torch.randn(1024, 1024, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(150):
            a @ a
    for _ in range(20):
        for got, w in zip(run(), want):
            assert torch.equal(got, w)
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 66, 33, 1, 1000])
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("t", [1, 4])
def test_step(types, d, t):
    n, pages = 9, 14
    x, g, _ = make(n * t, d, *types, 27)
    pool, _ = states(pages, d, 28)
    slots = torch.tensor([3, 0, -1, 13, 7, 99, 5, 6, 1], dtype=torch.int32)
    lengths = torch.tensor([t, 0, t, t, 1, t, 99, -3, max(t - 1, 0)], dtype=torch.int32)
    for tied in (False, True):
        state = pool.to(DEV)
        h = api.linear_recurrence_step(x.view(n, t, d).to(DEV), g.view(n, t, d).to(DEV), state, tied=tied, slots=slots.to(DEV),
                                       lengths=lengths.to(DEV)).cpu()
        left = torch.ones(pages, dtype=torch.bool)
        for i in range(n):
            p, m = int(slots[i]), max(0, min(t, int(lengths[i])))
            if not 0 <= p < pages:
                m = 0
            want = ref.sequence(x.view(n, t, d)[i, :m], g.view(n, t, d)[i, :m], pool[p] if m else None, tied)
            ref.check(h[i, :m], want["h"], f"h {i}")
            assert (h[i, m:] == 0).all()
            if m:
                ref.check(state[p], want["state"], f"state {i}")
                left[p] = False
        assert torch.equal(state.cpu()[left], pool[left])


@pytest.mark.parametrize("n,d", [(3000, 1), (1111, 12), (700, 104), (130, 255), (129, 256), (65, 257), (30, 704), (20, 1001), (9, 1024), (9, 1028),
                                 (5, 2052), (3, 5000)])
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_step_of_many_sequences_and_of_many_channels(types, n, d):
    t = 2
    x, g, _ = make(n * t, d, *types, n)
    pool, _ = states(n + 3, d, 30)
    slots = torch.randperm(n + 3, generator=torch.Generator().manual_seed(d))[:n].to(torch.int32)
    state = pool.to(DEV)
    h = api.linear_recurrence_step(x.view(n, t, d).to(DEV), g.view(n, t, d).to(DEV), state, tied=True, slots=slots.to(DEV)).cpu()
    # a sequence's channels are as other channels
    flat = lambda y: y.view(n, t, d).transpose(0, 1).reshape(t, n * d)  # noqa: E731
    want = ref.sequence(flat(x), flat(g), pool[slots.long()].reshape(n * d), True)
    ref.check(flat(h), want["h"])
    ref.check(state.cpu()[slots.long()].reshape(n * d), want["state"])
    rest = torch.ones(n + 3, dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(state.cpu()[rest], pool[rest])


def test_step_takes_whole_prompts():
    x, g, _ = make(2 * 500, 64, F32, F32, 29)
    state = torch.zeros(2, 64, device=DEV)
    h = api.linear_recurrence_step(x.view(2, 500, 64).to(DEV), g.view(2, 500, 64).to(DEV), state)
    for i in range(2):
        want = ref.sequence(x.view(2, 500, 64)[i], g.view(2, 500, 64)[i])
        ref.check(h[i], want["h"])
        ref.check(state[i], want["state"])


def _capture(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    return graph


def test_captured_and_replayed():
    lens, d = [700, 0, 65, 1300], 66
    cu = cu_of(lens)
    bufs = [t.to(DEV) for t in (*make(sum(lens), d, BF16, BF16, 31), *states(len(lens), d, 32))]
    pool = torch.zeros(5, d, device=DEV)
    box = {}

    def step():
        h, state, saved = api.linear_recurrence_forward(bufs[0], bufs[1], tied=True, cu_seqlens=cu, initial_state=bufs[3],
                                                        output_final_state=True)
        box["all"] = (h, state, *api.linear_recurrence_backward(saved, bufs[2], d_final_state=bufs[4]))
        pool[:4] = state
        box["step"] = api.linear_recurrence_step(bufs[0][:4, None], bufs[1][:4, None], pool)

    graph = _capture(step)
    for seed in range(3):
        new = (*make(sum(lens), d, BF16, BF16, 40 + seed), *states(len(lens), d, 50 + seed))
        for b, t in zip(bufs, new):
            b.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = dict(zip(("h", "state", "dx", "dg", "dh0"), box["all"]))
        x, g, dh, h0, dht = new
        got["h"] = got["h"].clone()
        check_packed(got, x, g, lens, dh, h0, dht, True)
        for i in range(4):
            ref.check(box["step"][i], ref.sequence(x[i:i + 1], g[i:i + 1], got["state"][i].cpu())["h"])


def test_on_another_stream_with_memory_given_up_after_the_call():
    lens = [900, 300]
    host = make(sum(lens), 128, BF16, BF16, 33)
    h0, dht = states(2, 128, 34)
    x, g, dh = (t.to(DEV) for t in host)
    cu, start, end = cu_of(lens), h0.to(DEV), dht.to(DEV)
    side, big = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    h, state, saved = api.linear_recurrence_forward(x, g, cu_seqlens=cu, initial_state=start, output_final_state=True)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            big @ big
    got = api.linear_recurrence_backward(saved, dh, d_final_state=end, stream=side)
    sizes = [t.numel() * t.element_size() for t in (saved.workspace, x, g, dh, start, end)]
    del saved, x, g, dh, start, end
    new = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda.synchronize()
    del new
    check_packed({"h": h, "state": state, "dx": got[0], "dg": got[1], "dh0": got[2]}, *host[:2], lens, host[2], h0, dht, False)


def test_offsets_beyond_32_bits():
    # 2^31 numbers and more a tensor: the last rows against the recurrence from the state before them
    tokens, d = (1 << 15) + 300, 1 << 16
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough free memory")
    x = torch.randn(tokens, 512, device=DEV).to(BF16).repeat(1, d // 512)
    g = (-0.5 * torch.rand(tokens, 512, device=DEV)).to(BF16).repeat(1, d // 512)
    h, state, saved = api.linear_recurrence_forward(x[None], g[None], output_final_state=True)
    dx, dg, _ = api.linear_recurrence_backward(saved, x[None])
    for name, t in (("h", h), ("dx", dx), ("dg", dg)):
        assert torch.equal(t[0, -500:, :512], t[0, -500:, -512:]), name   # equal channels, whose places differ by 2^32 bytes and more
    rows = slice(tokens - 1200, tokens)
    want = ref.sequence(x[rows, -40:].cpu(), g[rows, -40:].cpu(), dh=x[rows, -40:].cpu())
    # a state of 900 tokens before is forgotten: e^(-0.25 * 900) of it is left
    for name, t in (("h", h), ("dg", dg)):
        ref.check(t[0, -300:, -40:], tuple(y[-300:] for y in want[name]), name)
    ref.check(state[0, -40:], want["state"], "state")
