"""Measured cases of the gated linear recurrence, of beam search's choice and of the states that follow it.

The gated linear recurrence is, for each channel of a sequence,

    h_t = exp(g_t) h_{t-1} + w_t x_t        w = 1, or 1 - exp(g_t) where input and decay are tied

``prompt`` runs whole sequences, ``train`` runs them forward and backward, ``step`` advances the states of many sequences by
a token or a few, in place, in a pool of pages.  ``beam`` chooses, for each item of a batch, the best continuations of all of
its beams by score + log softmax(logits); ``reorder`` gives each beam the state of the beam that it continues, in place.

Each case's plain form is elementary torch operations in 32 bits (64 where candidates of different beams are compared);
``exact`` works in 64 bits.
"""
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one user's next token: latency counts
        dict(name="step: one sequence", kind="step", n=1, t=1, d=4096, dtype="bf16", gtype="bf16", tied=False, spare=3),
        # the next token of a full serving batch, a layer of 2048 channels: 268 MB of state move
        dict(name="step: full batch", kind="step", n=16384, t=1, d=2048, dtype="bf16", gtype="f32", tied=True, spare=40),
        # prompts of very different lengths in one packed batch, as a server takes them in, gates in 32 bits
        dict(name="prompt: ragged batch", kind="prompt", n=48, tokens=24571, spread=7, d=4096, dtype="bf16", gtype="f32",
             tied=False, fused=False),
        # one long document and few channels: a long way to go and little to do at a time
        dict(name="prompt: one long", kind="prompt", n=1, tokens=131072, spread=0, d=512, dtype="bf16", gtype="bf16",
             tied=True, fused=True),
        # an ordinary training batch
        dict(name="train: batch", kind="train", n=4, tokens=32768, spread=0, d=4096, dtype="bf16", gtype="bf16", tied=False,
             fused=True, h0=False),
        # a long training context in 32 bits
        dict(name="train: long f32", kind="train", n=1, tokens=65536, spread=0, d=512, dtype="f32", gtype="f32", tied=True,
             fused=False, h0=True),
        # packed documents of a small model, an odd number of channels, states carried in and gradients carried out
        dict(name="train: ragged f16", kind="train", n=9, tokens=3001, spread=5, d=1001, dtype="f16", gtype="f32", tied=False,
             fused=False, h0=True),
        # four beams of one sentence in 32 bits: latency
        dict(name="beam: one sentence", kind="beam", batch=1, beams=4, width=4, vocab=32000, pad=0, dtype="f32", ended=False),
        # a batch of beams over a large vocabulary, some of them at their end
        dict(name="beam: batch", kind="beam", batch=64, beams=8, width=8, vocab=128000, pad=0, dtype="bf16", ended=True),
        # wide beams over an odd vocabulary, as a view of a projection with padded rows, twice as many candidates
        dict(name="beam: wide, odd", kind="beam", batch=12, beams=16, width=32, vocab=50021, pad=27, dtype="f16", ended=False),
        # the states of one sentence's beams in a few layers: latency
        dict(name="reorder: one sentence", kind="reorder", batch=1, beams=4, pages=8, elems=4096, pools=4, dtype="f32"),
        # the states of a batch of beams in all layers
        dict(name="reorder: batch", kind="reorder", batch=64, beams=8, pages=520, elems=4096, pools=24, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["step", "prompt", "prompt", "train", "train", "beam", "beam", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    gtype = rng.choice([dtype, "f32"])
    d = _log(rng, 64, 8192)
    d = rng.choice([d, -(-d // 64) * 64, -(-d // 2) * 2])
    if kind == "step":
        t = rng.choice([1, 1, 1, 2, 3, 5])
        return dict(kind=kind, n=_log(rng, 1, max(2, (1 << 25) // d // t)), t=t, d=d, dtype=dtype, gtype=gtype,
                    tied=rng.random() < 0.5, spare=rng.randrange(1, 40))
    if kind in ("prompt", "train"):
        tokens = min(262144, _log(rng, 33, (1 << 26) // d))
        n = _log(rng, 1, max(2, min(200, tokens // 16)))
        c = dict(kind=kind, n=n, tokens=tokens, spread=rng.randrange(0, 1000), d=d, dtype=dtype, gtype=gtype,
                 tied=rng.random() < 0.5, fused=rng.random() < 0.5 and gtype == dtype)
        return dict(c, h0=rng.random() < 0.5) if kind == "train" else c
    if kind == "beam":
        vocab, beams = _log(rng, 500, 262144), rng.choice([1, 2, 3, 4, 5, 8, 10, 16, 32])
        vocab = rng.choice([vocab, -(-vocab // 64) * 64])
        return dict(kind=kind, batch=_log(rng, 1, max(2, min(512, (1 << 26) // vocab // beams))), beams=beams,
                    width=rng.choice([beams, beams, 2 * beams]), vocab=vocab, pad=rng.choice([0, 0, 64 - vocab % 64]),
                    dtype=dtype, ended=rng.random() < 0.5)
    beams, pools = rng.choice([2, 3, 4, 5, 8, 16]), rng.choice([1, 2, 5, 12, 24])
    elems = rng.choice([256, 1000, 2048, 4096, 16384])
    batch = _log(rng, 1, max(2, min(512, (1 << 27) // (beams * elems * pools))))
    return dict(kind=kind, batch=batch, beams=beams, pages=batch * beams + rng.randrange(0, 30), elems=elems, pools=pools,
                dtype=dtype)


# ---- sizes that follow from a case ------------------------------------------------------------------------------------

def _lengths(c):
    """The sequences' lengths: equal where spread is 0, else drawn over three orders of magnitude (an empty one among many)."""
    n, total = c["n"], c["tokens"]
    if c["spread"] == 0 or n == 1:
        return [total // n] * n
    r = random.Random(c["spread"])
    w = [10 ** (2.5 * r.random()) for _ in range(n)]
    lens = [int(total * x / sum(w)) for x in w]
    if n > 6:
        lens[r.randrange(n)] = 0
    lens[max(range(n), key=lens.__getitem__)] += total - sum(lens)
    return lens


def _parents(c):
    """Which row of the batch each row continues: one of its own item's, the better (lower) ones more often."""
    r = random.Random(c["batch"] * 131 + c["beams"])
    return [i * c["beams"] + int(c["beams"] * r.random() ** 1.5) for i in range(c["batch"]) for _ in range(c["beams"])]


def work(c):
    kind = c["kind"]
    if kind in ("step", "prompt", "train"):
        tokens = c["n"] * c["t"] if kind == "step" else sum(_lengths(c))
        x, g = tokens * c["d"] * BYTES[c["dtype"]], tokens * c["d"] * BYTES[c["gtype"]]
        state, flops = c["n"] * c["d"] * 4, tokens * c["d"] * (6 if c["tied"] else 3)
        if kind != "train":
            return {"bytes": 2 * x + g + 2 * state, "flops": flops}
        # x, g and the output's gradient in; the output and the gradients of x and g out
        return {"bytes": 4 * x + 2 * g + (3 * state if c["h0"] else 0), "flops": 3 * flops}
    if kind == "beam":
        rows = c["batch"] * c["beams"]
        return {"bytes": rows * c["vocab"] * BYTES[c["dtype"]] + rows * 5 + c["batch"] * c["width"] * 13,
                "flops": 4 * rows * c["vocab"]}
    copies = c["batch"] * c["beams"] - len(set(_parents(c)))
    return {"bytes": 2 * copies * c["elems"] * BYTES[c["dtype"]] * c["pools"] + 12 * c["batch"] * c["beams"], "flops": 0}


# ---- inputs -----------------------------------------------------------------------------------------------------------

def _inputs(c, shape, gen, fused):
    """Normal inputs, and log decays from long memory (a thousand tokens) to short, channel by channel."""
    x = torch.randn(*shape, c["d"], device=DEV, generator=gen)
    rate = torch.exp(-6.9 + 6.9 * torch.rand(c["d"], device=DEV, generator=gen))
    g = -rate * torch.nn.functional.softplus(torch.randn(*shape, c["d"], device=DEV, generator=gen))
    x, g = x.to(TYPES[c["dtype"]]), g.to(TYPES[c["gtype"]])
    if fused:  # views of one projection's output, as a layer has them
        both = torch.cat([x, g], -1)
        x, g = both[..., :c["d"]], both[..., c["d"]:]
    return {"x": x, "g": g}


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind = c["kind"]
    normal = lambda *shape: torch.randn(*shape, device=DEV, generator=gen)  # noqa: E731
    if kind == "step":
        s = _inputs(c, (c["n"], c["t"]), gen, False)
        pages = c["n"] + c["spare"]
        s["slots"] = torch.randperm(pages, device=DEV, generator=gen)[:c["n"]].to(torch.int32)
        return dict(s, case=c, state=normal(pages, c["d"]))
    if kind in ("prompt", "train"):
        lens, uniform = _lengths(c), c["spread"] == 0
        s = _inputs(c, (c["n"], lens[0]) if uniform else (sum(lens),), gen, c["fused"])
        s["cu"] = None if uniform else torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        s["h0"] = normal(c["n"], c["d"]) if kind == "prompt" or c["h0"] else None
        if kind == "train":
            s["dh"] = normal(*s["x"].shape).to(s["x"].dtype)
            s["dht"] = normal(c["n"], c["d"]) if c["h0"] else None
        return dict(s, case=c, longest=max(lens))
    if kind == "beam":
        logits = (2.5 * normal(c["batch"], c["beams"], c["vocab"] + c["pad"])).to(TYPES[c["dtype"]])[..., :c["vocab"]]
        scores = -20 + 2 * normal(c["batch"], c["beams"])
        ended = (torch.rand(c["batch"], c["beams"], device=DEV, generator=gen) < 0.2).to(torch.uint8) if c["ended"] else None
        return {"case": c, "logits": logits, "scores": scores, "ended": ended, "eos": 2}
    perm = torch.randperm(c["pages"], device=DEV, generator=gen)[:c["batch"] * c["beams"]].to(torch.int32)
    return {"case": c, "pools": [normal(c["pages"], c["elems"]).to(TYPES[c["dtype"]]) for _ in range(c["pools"])],
            "slots": perm, "parents": torch.tensor(_parents(c), dtype=torch.int32, device=DEV)}


# ---- the plain forms --------------------------------------------------------------------------------------------------

def _scan(g, b, longest):
    """b_t + e^{g_t} (b_{t-1} + e^{g_{t-1}} (...)) for every t, by doubling: the maps of 1, 2, 4, ... tokens composed, their
    decays as sums of logarithms, which lose less than products do."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], b[step:] + g[step:].exp() * b[:-step]])
        g = torch.cat([g[:step], g[step:] + g[:-step]])
        step *= 2
    return b


def _bounds(s):
    """The sequences that hold a token, and their first and last tokens, counted over all sequences."""
    c = s["case"]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(c["n"] + 1, device=DEV) * s["x"].shape[1]
    live = cu[1:] > cu[:-1]
    return live, cu[:-1][live], cu[1:][live] - 1


def _plain_forward(s):
    c = s["case"]
    x, g = (s[name].float().reshape(-1, c["d"]) for name in ("x", "g"))
    live, first, last = _bounds(s)
    a, w = g.exp(), -torch.expm1(g) if c["tied"] else torch.ones_like(g)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(c["n"], c["d"], device=DEV)
    b, kept = w * x, g.clone()
    b[first] += a[first] * h0[live]
    kept[first] = float("-inf")
    h, state = _scan(kept, b, s["longest"]), h0.clone()
    state[live] = h[last]
    return x, g, w, h0, h, state


def _plain_prompt(s):
    _, _, _, _, h, state = _plain_forward(s)
    return {"h": h.to(s["x"].dtype).view(s["x"].shape), "state": state}


def _plain_train(s):
    c = s["case"]
    x, g, w, h0, h, _ = _plain_forward(s)
    a = g.exp()
    live, first, last = _bounds(s)
    d = s["dh"].float().reshape(-1, c["d"]).clone()
    if s["dht"] is not None:
        d[last] += s["dht"][live]
    after = torch.cat([g[1:], g[:1]])
    after[last] = float("-inf")
    lam = _scan(after.flip(0), d.flip(0), s["longest"]).flip(0)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = h0[live]
    dg = lam * a * (before - x if c["tied"] else before)
    out = {"h": h.to(s["x"].dtype).view(s["x"].shape), "dx": (lam * w).to(s["x"].dtype).view(s["x"].shape),
           "dg": dg.to(s["g"].dtype).view(s["x"].shape)}
    if s["h0"] is not None:
        out["dh0"] = s["dht"].clone()
        out["dh0"][live] = (lam * a)[first]
    return out


def _plain_step(s):
    c, at = s["case"], s["slots"].long()
    x, g = s["x"].float(), s["g"].float()
    a, b = g.exp(), -torch.expm1(g) * x if c["tied"] else x
    h = torch.cat([s["state"][at][:, None], b], 1)
    for i in range(c["t"]):
        h[:, i + 1] += a[:, i] * h[:, i]
    s["state"][at] = h[:, -1]
    return {"h": h[:, 1:].to(s["x"].dtype), "state": s["state"]}


def _plain_beam(s):
    """Each beam's best by (logit, lowest token), then the best of all by (total in 64 bits, lowest beam, beam's order)."""
    c = s["case"]
    x, beams = s["logits"].float() + 0.0, torch.arange(c["beams"], device=DEV)
    bits = x.view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()             # rises with the number
    key = (order << 32) - torch.arange(c["vocab"], device=DEV)      # of equal ones the lowest token's is largest
    best = key.topk(min(c["width"], c["vocab"]), dim=-1).indices
    top = x.amax(-1, keepdim=True)
    lse = top.double() + (x - top).exp().sum(-1, keepdim=True, dtype=torch.float64).log()
    total = s["scores"].double()[..., None] + (x.gather(-1, best).double() - lse)
    tokens = best.to(torch.int32)
    if s["ended"] is not None:  # a beam at its end offers itself once, as it is
        done, once = s["ended"].bool()[..., None], torch.arange(best.shape[-1], device=DEV) == 0
        total = torch.where(done, torch.where(once, s["scores"].double()[..., None], float("-inf")), total)
        tokens = torch.where(done, s["eos"], tokens)
    rows = (torch.arange(c["batch"], device=DEV)[:, None] * c["beams"] + beams)[..., None].expand_as(tokens).to(torch.int32)
    total, at = total.flatten(1).sort(dim=-1, descending=True, stable=True)
    at, score = at[:, :c["width"]], total[:, :c["width"]].float()
    none = score == float("-inf")
    pick = lambda t: torch.where(none, -1, t.flatten(1).gather(1, at))  # noqa: E731
    out = {"scores": score, "parents": pick(rows), "tokens": pick(tokens)}
    if s["ended"] is not None:
        was = s["ended"].flatten()[out["parents"].clamp(min=0).long()].bool()
        out["ended"] = ((was | (out["tokens"] == s["eos"])) & ~none).to(torch.uint8)
    return out


def _plain_reorder(s):
    """The first row that continues a row keeps its page; the others get, in order, the pages that nobody continues."""
    slots, parents = s["slots"], s["parents"].long()
    n = slots.numel()
    row = torch.arange(n, device=DEV)
    first = torch.full((n,), n, device=DEV).scatter_reduce(0, parents, row, "amin")
    keeps = first[parents] == row
    free = slots[first == n]
    to = torch.where(keeps, slots[parents], free[((~keeps).cumsum(0) - 1).clamp(min=0)] if free.numel() else slots)
    src, dst = slots[parents][~keeps].long(), to[~keeps].long()
    for pool in s["pools"]:
        pool[dst] = pool[src]
    return {"slots": to, "pools": s["pools"]}


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    kind = c["kind"]
    if not own:
        with torch.no_grad():
            return {"prompt": _plain_prompt, "train": _plain_train, "step": _plain_step, "beam": _plain_beam,
                    "reorder": _plain_reorder}[kind](s)
    from prefix_scan_gb300 import api
    if kind == "prompt":
        h, state = api.linear_recurrence(s["x"], s["g"], tied=c["tied"], cu_seqlens=s["cu"], initial_state=s["h0"],
                                         output_final_state=True)
        return {"h": h, "state": state}
    if kind == "train":
        h, _, saved = api.linear_recurrence_forward(s["x"], s["g"], tied=c["tied"], cu_seqlens=s["cu"], initial_state=s["h0"])
        dx, dg, dh0 = api.linear_recurrence_backward(saved, s["dh"], d_final_state=s["dht"])
        out = {"h": h, "dx": dx, "dg": dg}
        return dict(out, dh0=dh0) if s["h0"] is not None else out
    if kind == "step":
        h = api.linear_recurrence_step(s["x"], s["g"], s["state"], tied=c["tied"], slots=s["slots"])
        return {"h": h, "state": s["state"]}
    if kind == "beam":
        if s["ended"] is None:
            scores, parents, tokens, _ = api.beam_select(s["logits"], s["scores"], width=c["width"])
            return {"scores": scores, "parents": parents, "tokens": tokens}
        scores, parents, tokens, ended = api.beam_select(s["logits"], s["scores"], width=c["width"], ended=s["ended"],
                                                         eos_token=s["eos"])
        return {"scores": scores, "parents": parents, "tokens": tokens, "ended": ended}
    slots, _ = api.pages_reorder(s["slots"], s["parents"], s["pools"])
    return {"slots": slots, "pools": s["pools"]}


# ---- in 64 bits -------------------------------------------------------------------------------------------------------

def _exact_scan(a, b):
    """h_t = a_t h_{t-1} + b_t over [sequences, tokens, channels] from h = 0: token by token within stretches, then stretch
    by stretch."""
    n, t, d = b.shape
    size = max(1, int(t ** 0.5))
    pad = -t % size
    cut = lambda y, fill: torch.cat([y, y.new_full((n, pad, d), fill)], 1).view(n, -1, size, d)  # noqa: E731
    a, h = cut(a, 1.0), cut(b, 0.0)
    decay = a.clone()
    for i in range(1, size):
        h[:, :, i] += a[:, :, i] * h[:, :, i - 1]
        decay[:, :, i] *= decay[:, :, i - 1]
    for k in range(1, h.shape[1]):
        h[:, k] += decay[:, k] * h[:, k - 1, -1:]
    return h.reshape(n, -1, d)[:, :t]


def _exact_sequence(s):
    """Each sequence by itself (equal ones together); a start's state is a token before the first."""
    c = s["case"]
    x, g = s["x"].double(), s["g"].double()
    if s["cu"] is None:
        groups = [(x, g, s["dh"].double() if c["kind"] == "train" else None)]
    else:
        lens = (s["cu"][1:] - s["cu"][:-1]).tolist()
        dh = s["dh"].double().split(lens) if c["kind"] == "train" else [None] * c["n"]
        groups = [(y[None], z[None], e if e is None else e[None]) for y, z, e in zip(x.split(lens), g.split(lens), dh)]
    zero = torch.zeros(c["n"], c["d"], dtype=torch.float64, device=DEV)
    h0, dht = (zero if s.get(name) is None else s[name].double() for name in ("h0", "dht"))
    out, at = {"h": [], "state": [], "dx": [], "dg": [], "dh0": []}, 0
    for x, g, dh in groups:
        n = x.shape[0]
        start, end = h0[at:at + n, None], dht[at:at + n, None]
        at += n
        weight = -torch.expm1(g) if c["tied"] else 1.0
        decay = torch.cat([torch.zeros_like(start), g.exp()], 1)
        h = _exact_scan(decay, torch.cat([start, weight * x], 1))
        out["h"].append(h[:, 1:])
        out["state"].append(h[:, -1])
        if dh is not None:
            push = torch.cat([end, dh.flip(1)], 1)       # from behind: the end's gradient, then every token's
            pull = torch.cat([torch.zeros_like(end), torch.ones_like(end), decay[:, 1:].flip(1)], 1)[:, :-1]
            lam = _exact_scan(pull, push)[:, 1:].flip(1)
            back = decay[:, 1:] * lam
            out["dg"].append(back * (h[:, :-1] - x if c["tied"] else h[:, :-1]))
            out["dx"].append(lam * weight)
            out["dh0"].append(torch.cat([back, end], 1)[:, 0])
    whole = lambda name: torch.cat(out[name], 0) if s["cu"] is None else torch.cat(out[name], 1)[0]  # noqa: E731
    if c["kind"] == "prompt":
        return {"h": whole("h"), "state": torch.cat(out["state"])}
    result = {"h": whole("h"), "dx": whole("dx"), "dg": whole("dg")}
    return dict(result, dh0=torch.cat(out["dh0"])) if s["h0"] is not None else result


def _exact_step(s):
    c, state = s["case"], s["state"].double()
    h, out = state[s["slots"].long()], []
    for i in range(c["t"]):
        x, g = s["x"][:, i].double(), s["g"][:, i].double()
        h = h * g.exp() + (x * -torch.expm1(g) if c["tied"] else x)
        out.append(h)
    state[s["slots"].long()] = h
    return {"h": torch.stack(out, 1), "state": state}


def _exact_beam(s):
    """The chosen scores: the largest of each item's, over every token of every beam; which ones they are has no 64-bit value."""
    c, scores = s["case"], []
    for i in range(c["batch"]):
        total = s["scores"][i].double()[:, None] + torch.log_softmax(s["logits"][i].double(), -1)
        if s["ended"] is not None:
            done = s["ended"][i].bool()
            total[done] = float("-inf")
            total[done, 0] = s["scores"][i].double()[done]
        scores.append(total.flatten().topk(c["width"]).values)
    out = {"scores": torch.stack(scores), "parents": None, "tokens": None}
    return dict(out, ended=None) if s["ended"] is not None else out


def _exact_reorder(s):
    """Worked out row by row on the host."""
    slots, parents = s["slots"].tolist(), s["parents"].tolist()
    used = set(parents)
    free = iter([p for r, p in enumerate(slots) if r not in used])
    seen, moves = set(), []
    for p in parents:
        if p in seen:
            moves.append((slots[p], next(free)))
        seen.add(p)
    pools = []
    for pool in s["pools"]:
        now = pool.double()
        if moves:
            src, dst = (torch.tensor(x, device=DEV) for x in zip(*moves))
            now[dst] = pool.double()[src]
        pools.append(now)
    return {"slots": None, "pools": pools}


def exact(c, seed):
    s = prepare(c, seed)
    with torch.no_grad():
        return {"step": _exact_step, "prompt": _exact_sequence, "train": _exact_sequence, "beam": _exact_beam,
                "reorder": _exact_reorder}[c["kind"]](s)
