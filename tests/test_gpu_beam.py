"""Beam search's choice against a full sort of all continuations in 64 bits.

Tolerance of a total: its row's log of the sum of exponentials.  An exponential of the hardware's is off by 2^-22 of itself, its
argument y <= 0 by 2^-24 |y|, of which |y| e^y <= 0.37 remains (2^-25.4); up to 32 numbers are added in 32 bits, 32 x 2^-24 of the
sum at most, then in 64.  A score returned is rounded to 32 bits besides: 2^-24 of itself."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402

DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF, NAN = float("inf"), float("nan")
TOLERANCE = 2.0 ** -22 + 2.0 ** -25.4 + 32 * 2.0 ** -24


def reference(logits, scores, width, ended=None, eos=-1):
    """[(total, beam, token), ...] of each item, best first, in 64 bits, at most ``width``."""
    out = []
    for i in range(logits.shape[0]):
        every = []
        for b in range(logits.shape[1]):
            s = scores[i, b].double()
            if not s.isfinite():
                continue
            if ended is not None and ended[i, b]:
                every.append((float(s), b, eos, 0.0))
                continue
            x = logits[i, b].double() + 0.0
            if x.isnan().any() or (x == INF).any() or (x == -INF).all():
                continue
            total = s + torch.log_softmax(x, 0)
            best = torch.sort(x, descending=True, stable=True)[1][:width]
            every += [(float(total[t]), b, int(t), -float(x[t])) for t in best if x[t] > -INF]
        every.sort(key=lambda c: (-c[0], c[1], c[3], c[2]))
        out.append([c[:3] for c in every[:width]])
    return out


def check(choice, logits, scores, width, ended=None, eos=-1):
    logits, scores = logits.cpu(), scores.cpu()
    beams = logits.shape[1]
    want = reference(logits, scores, width, ended, eos)
    got = [t.cpu() for t in choice[:3]]
    assert all(t.shape == (logits.shape[0], width) for t in got)
    for i, w in enumerate(want):
        n = len(w)
        assert (got[0][i, n:] == -INF).all() and (got[1][i, n:] == -1).all() and (got[2][i, n:] == -1).all()
        if ended is not None:
            assert (choice.ended[i, n:] == 0).all()
        seen, last = set(), {}
        for r in range(n):
            total, beam, token = w[r]
            score, parent, mine = float(got[0][i, r]), int(got[1][i, r]) - i * beams, int(got[2][i, r])
            tol = TOLERANCE + abs(total) * 2.0 ** -24
            assert abs(score - total) <= tol, (i, r, score, total)
            assert 0 <= parent < beams and (parent, mine) not in seen
            seen.add((parent, mine))
            if ended is not None and ended[i, parent]:
                assert mine == eos and score == float(scores[i, parent]) and choice.ended[i, r] == 1
                continue
            if ended is not None:
                assert int(choice.ended[i, r]) == (mine == eos)
            # where no other beam's total is within the tolerance this is the one; a beam's own order is exact
            x = logits[i, parent].double() + 0.0
            own = float(scores[i, parent].double() + torch.log_softmax(x, 0)[mine])
            assert abs(own - total) <= 2 * tol
            key = (-float(x[mine]), mine)
            assert last.get(parent, (-INF, -1)) < key
            last[parent] = key
        for b, key in last.items():   # no better one of a beam was left out
            x = logits[i, b].double() + 0.0
            taken = {t for p, t in seen if p == b}
            better = [t for t in torch.nonzero(x >= -key[0])[:, 0].tolist() if (-float(x[t]), t) < key]
            assert set(better) <= taken


def make(batch, beams, vocab, dtype, seed, spread=2.5):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    logits = (spread * torch.randn(batch, beams, vocab, device=DEV, generator=gen)).to(dtype)
    return logits, -20 + 2 * torch.randn(batch, beams, device=DEV, generator=gen)


@pytest.mark.parametrize("vocab", [1, 2, 7, 63, 511, 512, 513, 2048, 4096, 4097, 16384, 16385, 50021])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_vocabularies(dtype, vocab):
    logits, scores = make(3, 4, vocab, dtype, vocab)
    check(api.beam_select(logits, scores), logits, scores, 4)


@pytest.mark.parametrize("batch,beams,width", [(1, 1, 1), (1, 1, 64), (5, 3, 6), (2, 32, 32), (1, 64, 64), (40, 2, 5), (2, 256, 16), (0, 4, 4)])
@pytest.mark.parametrize("vocab", [1000, 40001])
def test_beams_and_widths(batch, beams, width, vocab):
    logits, scores = make(batch, beams, vocab, BF16, beams)
    check(api.beam_select(logits, scores, width=width), logits, scores, width)


def test_many_rows_take_larger_parts():
    # more than 152 parts of 32 KiB: 32 (16-bit) and 16 (f32) numbers a thread
    for dtype, vocab in ((BF16, 70000), (F32, 35003), (F16, 33001)):
        logits, scores = make(10, 8, vocab, dtype, 5)
        check(api.beam_select(logits, scores), logits, scores, 8)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(dtype):
    logits, scores = make(3, 4, 3001, dtype, 7)
    wide = torch.full((3, 4, 3008), NAN, dtype=dtype, device=DEV)
    wide[..., :3001] = logits
    check(api.beam_select(wide[..., :3001], scores), logits, scores, 4)          # padded rows
    odd = torch.full((3, 4, 3005), NAN, dtype=dtype, device=DEV)
    odd[..., 1:3002] = logits
    check(api.beam_select(odd[..., 1:3002], scores), logits, scores, 4)          # off the boundaries
    first = logits.transpose(0, 1).contiguous().transpose(0, 1)
    check(api.beam_select(first, scores), logits, scores, 4)                     # beams first
    same = logits[:, :1].expand(3, 4, 3001)
    check(api.beam_select(same, scores), same, scores, 4)                        # one row for all beams


@pytest.mark.parametrize("pieces", [True, False])
def test_equal_numbers_go_to_the_lowest(pieces):
    # equal rows have equal sums, so equal totals go by beam and token
    vocab = 40000 if pieces else 39999
    logits = torch.zeros(2, 3, vocab, device=DEV)
    scores = torch.full((2, 3), -1.0, device=DEV)
    c = api.beam_select(logits, scores, width=64)
    assert (c.parents.cpu() == torch.tensor([[0], [3]])).all() and (c.tokens.cpu() == torch.arange(64)).all()
    logits[:, 1, 7777] = 1.0
    logits[:, 2, 7777] = 1.0
    c = api.beam_select(logits, scores, width=4)
    assert c.parents.cpu().tolist() == [[1, 2, 0, 0], [4, 5, 3, 3]] and c.tokens.cpu().tolist() == [[7777, 7777, 0, 1]] * 2
    logits[:, :, ::2] = -0.0
    c = api.beam_select(logits, scores, width=4)
    assert c.tokens.cpu().tolist() == [[7777, 7777, 0, 1]] * 2
    # many beams, each with a tie of all tokens: more candidates reach the threshold than there is room for
    c = api.beam_select(torch.zeros(1, 40, 9000, device=DEV), torch.zeros(1, 40, device=DEV), width=48)
    assert (c.parents == 0).all() and (c.tokens.cpu() == torch.arange(48)).all()


def test_few_distinct_values():
    gen = torch.Generator(device=DEV).manual_seed(3)
    logits = torch.randint(0, 3, (4, 5, 20011), device=DEV, generator=gen).to(BF16)
    scores = -torch.rand(4, 5, device=DEV, generator=gen)
    check(api.beam_select(logits, scores, width=12), logits, scores, 12)


def test_rising_and_falling():
    up = torch.linspace(-30, 30, 30011, device=DEV)
    logits = torch.stack([up, up.flip(0), up * 0.5])[None]
    scores = torch.tensor([[-1.0, -1.5, -2.0]], device=DEV)
    check(api.beam_select(logits, scores, width=20), logits, scores, 20)


def test_large_logits():
    # the sum's exponents are near 1e4: no accuracy is lost to their size beyond 32 bits of the difference
    gen = torch.Generator(device=DEV).manual_seed(13)
    logits = 1e4 + torch.randn(2, 3, 5000, device=DEV, generator=gen)
    scores = torch.zeros(2, 3, device=DEV)
    check(api.beam_select(logits, scores), logits, scores, 3)
    logits = torch.full((1, 2, 9), -3e38, device=DEV)
    logits[0, 0, 3], logits[0, 1, 5] = 3e38, 1.0
    c = api.beam_select(logits, torch.zeros(1, 2, device=DEV), width=2)
    assert c.parents.cpu().tolist() == [[0, 1]] and c.tokens.cpu().tolist() == [[3, 5]] and c.scores.cpu().tolist() == [[0.0, 0.0]]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [10, 18, 20, 22, 24, 31, 40, 64, 99, 101, 126])
def test_logits_of_any_size(exponent, sign):
    # numbers a few steps of their type around one size, and a few far below
    g = torch.Generator().manual_seed(exponent)
    for dtype, bits, vocab in ((F32, 23, 5000), (F32, 23, 333), (BF16, 7, 20000)):
        steps = torch.randint(-6, 7, (2, 3, vocab), generator=g)
        x = (sign * 2.0 ** exponent * (1 + steps.double() * 2.0 ** -bits)).to(dtype)
        x[:, :, ::7] = -(2.0 ** exponent)
        x[1, 1] = (-(2.0 ** exponent) * (1 + steps[1, 1].double() * 2.0 ** -bits)).to(dtype)
        s = torch.randn(2, 3, generator=g)
        check(api.beam_select(x.to(DEV), s.to(DEV), width=5), x, s, 5)


@pytest.mark.parametrize("width", [3, 17, 64])
@pytest.mark.parametrize("vocab", [700, 40000])
def test_scores_of_any_size(width, vocab):
    # one beam has them all; beams far apart; scores at the end of their type
    for row in ([0.0, -1e4, -1e4, -1e4], [-50.0, -50.5, -2e30, -3e38], [3.4e38, 3.4e38, 1e38, -3e38], [-3e38] * 4, [2e36, 0.0, -2e36, -INF]):
        logits, _ = make(2, 4, vocab, F32, width)
        logits[1] *= 1e36
        scores = torch.tensor([row] * 2, device=DEV)
        check(api.beam_select(logits, scores, width=width), logits, scores, width)


def test_totals_beyond_32_bits_are_chosen_last():
    logits = torch.tensor([[[0.0, -3e38, -INF]]], device=DEV)
    c = api.beam_select(logits, torch.tensor([[-3e38]], device=DEV), width=3)
    assert c.parents.cpu().tolist() == [[0, 0, -1]] and c.tokens.cpu().tolist() == [[0, 1, -1]]
    assert c.scores.cpu().tolist() == [[torch.tensor(-3e38).item(), -INF, -INF]]


def test_many_lists_with_equal_numbers():
    # 256 beams of 10 parts each, more equal totals than there is room for
    gen = torch.Generator(device=DEV).manual_seed(23)
    logits = torch.randint(0, 2, (1, 256, 80000), device=DEV, generator=gen).to(BF16)
    logits[0, 17, 79999] = 2
    scores = torch.zeros(1, 256, device=DEV)
    scores[0, ::3] = -INF
    # every row's sum is another, so beams differ; equal rows are equal
    logits[0, 40:60] = logits[0, 40]
    check(api.beam_select(logits, scores, width=64), logits, scores, 64)
    logits[:] = 1
    c = api.beam_select(logits, scores, width=64)
    assert c.parents.cpu().tolist() == [[1] * 64] and c.tokens.cpu().tolist() == [list(range(64))]


@pytest.mark.parametrize("dtype", [F32, F16])
def test_masks_and_what_offers_nothing(dtype):
    logits, scores = make(8, 4, 5000, dtype, 11)
    low = torch.finfo(dtype).min
    logits[0, 1] = -INF                      # a row with nothing
    logits[1] = -INF                         # an item with nothing
    logits[2, :, 3:] = -INF                  # fewer than the width
    logits[3, 0, 17], logits[3, 1, 4999], logits[3, 2, 0] = NAN, INF, -INF
    scores[4, 2], scores[4, 0] = -INF, NAN
    scores[5] = -INF
    scores[5, 3] = INF
    logits[6] = low                          # masked by the type's lowest value, all and all but two
    logits[7, :, 2:] = low
    check(api.beam_select(logits, scores, width=24), logits, scores, 24)
    check(api.beam_select(logits, scores, width=4), logits, scores, 4)
    first = scores.clone()                   # a search's first step: one beam takes part
    first[:, 1:] = -INF
    check(api.beam_select(logits, first, width=4), logits, first, 4)


@pytest.mark.parametrize("vocab", [300, 60001])
def test_ended_beams(vocab):
    logits, scores = make(6, 5, vocab, BF16, 17)
    ended = torch.zeros(6, 5, dtype=torch.uint8)
    ended[0, 2] = ended[1] = ended[2, 0] = ended[2, 4] = ended[3, 1] = 1
    logits[2, 0] = NAN                       # not read
    scores[3, 1] = -INF                      # ended and out
    scores[4] = 0.0
    logits[5, :, 9] = 40.0                   # the token that ends a beam wins
    check(api.beam_select(logits, scores, ended=ended.to(DEV), eos_token=9), logits, scores, 5, ended, 9)
    check(api.beam_select(logits, scores, ended=ended.to(DEV), eos_token=9, width=11), logits, scores, 11, ended, 9)


def test_captured_replayed_and_on_another_stream():
    logits, scores = make(3, 4, 9000, F32, 23)
    ended = torch.zeros(3, 4, dtype=torch.uint8, device=DEV)
    ws = torch.empty(api.beam_workspace_size(logits), dtype=torch.uint8, device=DEV)
    box = {}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    box["c"] = api.beam_select(logits, scores, ended=ended, eos_token=1, workspace=ws, stream=s)
    torch.cuda.synchronize()
    check(box["c"], logits, scores, 4, ended.cpu(), 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        box["c"] = api.beam_select(logits, scores, ended=ended, eos_token=1, workspace=ws)
    for seed in range(4):
        new = make(3, 4, 9000, F32, 30 + seed)
        logits.copy_(new[0])
        scores.copy_(new[1])
        ended.copy_((torch.rand(3, 4) < 0.3).to(torch.uint8))
        ws.fill_(255)   # whatever it holds
        graph.replay()
        torch.cuda.synchronize()
        check(box["c"], logits, scores, 4, ended.cpu(), 1)


def test_rows_beyond_32_bits():
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("not enough free memory")
    logits = torch.zeros(9, 256, 1 << 20, dtype=BF16, device=DEV)   # 2^31 numbers and more
    for i in range(9):
        logits[i, 255, (1 << 20) - 1 - i] = 9.0
        logits[i, 3, i] = 8.0
    scores = torch.zeros(9, 256, device=DEV)
    c = api.beam_select(logits, scores, width=2)
    assert c.parents.cpu().tolist() == [[i * 256 + 255, i * 256 + 3] for i in range(9)]
    assert c.tokens.cpu().tolist() == [[(1 << 20) - 1 - i, i] for i in range(9)]
