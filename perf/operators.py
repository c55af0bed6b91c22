"""Measured cases of the gated delta rule and of the paged caches that hold its states.

The gated delta rule is the recurrence, for each value head of a sequence, of a K x V state S:

    S <- exp(g) S;   u = beta (v - k^T S);   S <- S + k u^T;   o = scale q^T S

``step`` advances the states of many sequences by a token or a few, in place, in a pool of pages; ``prompt`` runs whole
sequences; ``train`` runs them forward and backward.  ``branch``, ``compact`` and ``copy`` manage pages of a cache: shared by
reference counts, forked with the last, part-filled page copied, grown, freed, moved to the front of their pool.

Each case's plain form is elementary torch operations in 32 bits; ``exact`` is the recurrence token by token in 64 bits.
"""
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one user's next token: 16 key heads shared by 32 value heads; 4 MiB of state move, so latency counts
        dict(name="step: one sequence", kind="step", n=1, t=1, hk=16, hv=32, k=128, v=128, dtype="bf16", spare=3),
        # the next token of a full serving batch: over 1 GB of state move
        dict(name="step: full batch", kind="step", n=256, t=1, hk=16, hv=32, k=128, v=128, dtype="bf16", spare=8),
        # prompts of very different lengths in one packed batch, as a server takes them in
        dict(name="prompt: ragged batch", kind="prompt", n=48, tokens=12345, spread=7, hk=16, hv=32, k=128, v=128,
             dtype="bf16", fused=True),
        # one long document and few heads: little to do at a time, a long way to go
        dict(name="prompt: one long", kind="prompt", n=1, tokens=32768, spread=0, hk=4, hv=8, k=128, v=128,
             dtype="bf16", fused=True),
        # a small model in 32 bits with odd head sizes, as in an experiment or a check
        dict(name="prompt: f32 odd sizes", kind="prompt", n=3, tokens=1111, spread=3, hk=3, hv=3, k=80, v=56,
             dtype="f32", fused=False),
        # an ordinary training batch
        dict(name="train: batch", kind="train", n=4, tokens=16384, spread=0, hk=16, hv=16, k=128, v=128, dtype="bf16",
             fused=True, h0=False),
        # a long training context with few heads and shared key heads
        dict(name="train: long", kind="train", n=1, tokens=16384, spread=0, hk=4, hv=8, k=128, v=128, dtype="bf16",
             fused=True, h0=False),
        # packed documents, states carried in and gradients carried out, small heads in 16-bit floats
        dict(name="train: ragged f16", kind="train", n=9, tokens=3001, spread=5, hk=4, hv=4, k=64, v=64, dtype="f16",
             fused=False, h0=True),
        # four candidates branch off one sequence's recurrent state and are dropped: latency
        dict(name="branch: four states", kind="branch", seqs=8, rows=4, pages=64, width=1, page_tokens=1 << 30,
             elems=32 * 64 * 64, pools=1, dtype="f32", draft=0),
        # a batch of candidates branches off key and value pages, grows by draft tokens and is dropped
        dict(name="branch: wide", kind="branch", seqs=128, rows=512, pages=16384, width=160, page_tokens=16,
             elems=16 * 8 * 128, pools=2, dtype="bf16", draft=5),
        # a cache of key and value pages after many sequences have ended: the rest moves to the front
        dict(name="compact: large cache", kind="compact", seqs=192, pages=16384, width=128, elems=16 * 8 * 128, pools=2,
             dtype="bf16", drop=3),
        # pages of a few sequences copied elsewhere in the cache, as before they are written to
        dict(name="copy: few pages", kind="copy", pages=2048, moves=37, elems=16 * 8 * 128, pools=2, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["step", "prompt", "train", "branch", "compact", "copy"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    hk = rng.choice([1, 2, 3, 4, 5, 8, 16])
    hv = hk * rng.choice([1, 1, 2, 3] if hk < 8 else [1, 2])
    k, v = rng.choice([64, 128, 128, rng.randrange(5, 17) * 8]), rng.choice([64, 128, 128, rng.randrange(5, 26) * 8])
    if kind == "step":
        t = rng.choice([1, 1, 1, 2, 3, 5, 8])
        return dict(kind=kind, n=_log(rng, 1, max(2, 8192 // hv // t)), t=t, hk=hk, hv=hv, k=k, v=v, dtype=dtype,
                    spare=rng.randrange(1, 10))
    if kind in ("prompt", "train"):
        tokens = _log(rng, 33, (262144 if kind == "prompt" else 131072) // hv // (1 if dtype == "bf16" else 8))
        tokens = min(tokens, 32768 if kind == "prompt" else 16384)
        n = _log(rng, 1, max(2, min(64, tokens // 16)))
        c = dict(kind=kind, n=n, tokens=tokens, spread=rng.randrange(1, 1000), hk=hk, hv=hv, k=k, v=v, dtype=dtype,
                 fused=rng.random() < 0.5)
        return dict(c, h0=rng.random() < 0.5) if kind == "train" else c
    elems, pools = rng.choice([1, 2, 3, 8, 16]) * 1024 * rng.choice([1, 2, 4]), rng.choice([1, 2, 3])
    pages = _log(rng, 200, 16384 * 32 * 1024 // (elems * BYTES[dtype] * pools))
    pages = min(pages, 65536)
    if kind == "copy":
        return dict(kind=kind, pages=pages, moves=_log(rng, 1, pages // 3), elems=elems, pools=pools, dtype=dtype)
    width = _log(rng, 2, max(3, min(256, pages // 16)))
    if kind == "compact":
        return dict(kind=kind, seqs=_log(rng, 2, max(3, pages // width)), pages=pages, width=width, elems=elems,
                    pools=pools, dtype=dtype, drop=rng.randrange(2, 7))
    seqs = _log(rng, 1, max(2, pages // (2 * width)))
    return dict(kind=kind, seqs=seqs, rows=_log(rng, 1, max(2, min(1024, pages // 12))), pages=pages, width=width,
                page_tokens=rng.choice([16, 32, 64, 1, 7]), elems=elems, pools=pools, dtype=dtype, draft=rng.choice([0, 1, 4, 6]))


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


def _sequence_pages(c):
    """For branch and compact: the sequences' lengths in pages, and which of the pool's pages each holds, in order."""
    r = random.Random(c["pages"] * 31 + c["seqs"])
    free = list(range(c["pages"]))
    r.shuffle(free)
    room = c["pages"] - (c["rows"] * (2 + c["draft"]) if c["kind"] == "branch" else 0)
    full = max(1, c["width"] - (1 + c["draft"] if c["kind"] == "branch" and c["width"] > 1 + c["draft"] else 0))
    rows = []
    for _ in range(c["seqs"]):
        n = min(r.randrange((full + 1) // 2, full + 1), room)
        room -= n
        rows.append([free.pop() for _ in range(n)])
    return rows, r


def work(c):
    kind = c["kind"]
    if kind in ("step", "prompt", "train"):
        hk, hv, k, v, b = c["hk"], c["hv"], c["k"], c["v"], BYTES[c["dtype"]]
        tokens = c["n"] * c["t"] if kind == "step" else sum(_lengths(c))
        io = tokens * (2 * hk * k * b + 2 * hv * v * b + hv * (4 + b))
        state = c["n"] * hv * k * v * 4
        flops = 7 * k * v * hv * tokens
        if kind == "step":
            return {"bytes": io + 2 * state, "flops": flops}
        if kind == "prompt":
            return {"bytes": io + 2 * state, "flops": flops}
        # forward and backward: inputs, the output and its gradient, the inputs' gradients
        io += tokens * (2 * hk * k * b + 2 * hv * v * b + hv * (4 + b))
        return {"bytes": io + (4 * state if c["h0"] else 0), "flops": 3 * flops}
    page = c["elems"] * BYTES[c["dtype"]] * c["pools"]
    if kind == "copy":
        return {"bytes": 2 * c["moves"] * page + 8 * c["moves"], "flops": 0}
    rows, r = _sequence_pages(c)
    if kind == "compact":
        kept = [p for i, s in enumerate(rows) if i % c["drop"] for p in s]
        moves = sum(p >= len(kept) for p in kept)
        return {"bytes": 2 * moves * page + 8 * (c["pages"] + c["seqs"] * c["width"]), "flops": 0}
    lens, parents = _branch(c, rows, r)
    copies = sum(lens[p] % c["page_tokens"] != 0 for p in parents)
    return {"bytes": 2 * copies * page + 8 * c["rows"] * c["width"] + 8 * c["pages"], "flops": 0}


def _branch(c, rows, r):
    pt = c["page_tokens"]
    lens = [len(s) * pt - (r.randrange(0, pt) if s and pt < 1 << 20 else pt // 2 if s else 0) for s in rows]
    return lens, [r.randrange(c["seqs"]) for _ in range(c["rows"])]


# ---- inputs -----------------------------------------------------------------------------------------------------------

def _qkvgb(c, shape, gen, fused):
    """Queries and keys of unit norm, normal values, log decays from long to short memory head by head, gates in (0, 1)."""
    hk, hv, k, v, dt = c["hk"], c["hv"], c["k"], c["v"], TYPES[c["dtype"]]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q = unit(torch.randn(*shape, hk, k, device=DEV, generator=gen)).to(dt)
    key = unit(torch.randn(*shape, hk, k, device=DEV, generator=gen)).to(dt)
    val = torch.randn(*shape, hv, v, device=DEV, generator=gen).to(dt)
    if fused:  # views of one projection's output, as a layer has them
        x = torch.cat([t.reshape(*shape, -1) for t in (q, key, val)], -1)
        q = x[..., :hk * k].unflatten(-1, (hk, k))
        key = x[..., hk * k:2 * hk * k].unflatten(-1, (hk, k))
        val = x[..., 2 * hk * k:].unflatten(-1, (hv, v))
    rate = torch.exp(-4.6 + 4.6 * torch.rand(hv, device=DEV, generator=gen))
    g = -rate * torch.nn.functional.softplus(torch.randn(*shape, hv, device=DEV, generator=gen))
    beta = torch.sigmoid(torch.randn(*shape, hv, device=DEV, generator=gen)).to(dt)
    return {"q": q, "k": key, "v": val, "g": g, "beta": beta}


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind = c["kind"]
    if kind == "step":
        s = _qkvgb(c, (c["n"], c["t"]), gen, False)
        pages = c["n"] + c["spare"]
        s["slots"] = torch.randperm(pages, device=DEV, generator=gen)[:c["n"]].to(torch.int32)
        s["state"] = 0.3 * torch.randn(pages, c["hv"], c["k"], c["v"], device=DEV, generator=gen)
        return dict(s, case=c)
    if kind in ("prompt", "train"):
        lens, uniform = _lengths(c), c["spread"] == 0
        s = _qkvgb(c, (c["n"], lens[0]) if uniform else (sum(lens),), gen, c["fused"])
        s["lens"], s["cu"] = lens, None
        if not uniform:
            s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        size = (c["n"], c["hv"], c["k"], c["v"])
        s["h0"] = 0.3 * torch.randn(size, device=DEV, generator=gen) if kind == "prompt" or c["h0"] else None
        if kind == "train":
            s["do"] = torch.randn(s["v"].shape, device=DEV, generator=gen).to(s["v"].dtype)
            s["dht"] = 0.3 * torch.randn(size, device=DEV, generator=gen) if c["h0"] else None
        return dict(s, case=c)
    pools = [torch.randn(c["pages"], c["elems"], device=DEV, generator=gen).to(TYPES[c["dtype"]]) for _ in range(c["pools"])]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    if kind == "copy":
        perm = torch.randperm(c["pages"], device=DEV, generator=gen).to(torch.int32)
        return {"case": c, "pools": pools, "src": perm[:c["moves"]].clone(), "dst": perm[c["moves"]:2 * c["moves"]].clone()}
    rows, r = _sequence_pages(c)
    turn = int(torch.randint(c["pages"], (1,), generator=torch.Generator().manual_seed(seed)))
    rows = [[(p + turn) % c["pages"] for p in s] for s in rows]
    table = ints([s + [-1] * (c["width"] - len(s)) for s in rows])
    refcount = torch.zeros(c["pages"], dtype=torch.int32, device=DEV)
    refcount[table[table >= 0].long()] = 1
    s = {"case": c, "pools": pools, "table": table, "refcount": refcount}
    if kind == "compact":
        s["flags"] = (torch.arange(c["seqs"], device=DEV) % c["drop"] == 0).to(torch.uint8)
        return s
    lens, parents = _branch(c, rows, r)
    return dict(s, lengths=ints(lens), parents=ints(parents))


# ---- the plain forms --------------------------------------------------------------------------------------------------

CHUNK = 64


def _padded(s, name, fill=0.0):
    """[sequences, heads, tokens padded to whole chunks, ...] in 32 bits, key heads repeated for the value heads that share them."""
    x, lens, hv = s[name].float(), s["lens"], s["case"]["hv"]
    top = max(CHUNK, -(-max(lens) // CHUNK) * CHUNK)
    if s["cu"] is None:
        x = torch.cat([x, x.new_zeros(x.shape[0], top - x.shape[1], *x.shape[2:])], 1)
    else:
        at = torch.arange(top, device=DEV)
        cu = s["cu"].long()
        inside = at < (cu[1:] - cu[:-1])[:, None]
        where = torch.where(inside, cu[:-1, None] + at, 0)
        x = x[where] * inside.view(*inside.shape, *[1] * (x.dim() - 1))
    return x.repeat_interleave(hv // x.shape[2], 2).transpose(1, 2)


def _unpadded(s, x):
    """The tokens of _padded()'s layout in the order of the inputs."""
    x = x.transpose(1, 2)
    if s["cu"] is None:
        return x[:, :s["lens"][0]]
    cu = s["cu"].long()
    at = torch.arange(x.shape[1], device=DEV)
    return x[at < (cu[1:] - cu[:-1])[:, None]]


def _chunked(q, k, v, g, beta, scale, s0):
    """The recurrence in chunks of tokens: within a chunk (I + L) U = beta (V - exp(G) K S), solved by the doubling product
    of the nilpotent L; all chunks' L, inverses and masked products at once, the states one chunk after another."""
    n, h, t = g.shape
    cut = lambda x: x.reshape(n, h, t // CHUNK, CHUNK, *x.shape[3:])  # noqa: E731
    q, k, v, g, beta = (cut(x) for x in (q, k, v, g, beta))
    G = g.cumsum(-1)
    below = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    decay = (G[..., :, None] - G[..., None, :]).masked_fill(~below, float("-inf")).exp()
    L = (k @ k.mT * decay * beta[..., None]).masked_fill(torch.eye(CHUNK, dtype=torch.bool, device=DEV), 0.0)
    P = q @ k.mT * decay * scale
    eye = torch.eye(CHUNK, device=DEV)
    X, power = eye - L, L
    for _ in range(5):
        power = power @ power
        X = X + X @ power
    eG = G.exp()[..., None]
    R0, RK = X @ (v * beta[..., None]), X @ (k * eG * beta[..., None])
    qs, kt, last = q * eG * scale, k * (G[..., -1:] - G).exp()[..., None], G[..., -1].exp()[..., None, None]
    S, out = s0, []
    for r0, rk, p, qc, kc, a in zip(*(x.unbind(2) for x in (R0, RK, P, qs, kt, last))):
        u = r0 - rk @ S
        out.append(qc @ S + p @ u)
        S = a * S + kc.mT @ u
    return torch.stack(out, 2).flatten(2, 3), S


def _plain_prompt(s, leaves=None):
    c = s["case"]
    q, k, v, g, beta = (_padded(s if leaves is None else {**s, **leaves}, x) for x in ("q", "k", "v", "g", "beta"))
    h0 = (leaves or s)["h0"]
    if h0 is None:
        h0 = torch.zeros(c["n"], c["hv"], c["k"], c["v"], device=DEV)
    o, last = _chunked(q, k, v, g, beta, c["k"] ** -0.5, h0)
    return _unpadded(s, o), last


def _plain_train(s):
    names = ["q", "k", "v", "g", "beta"] + (["h0"] if s["h0"] is not None else [])
    leaves = {x: s[x].float().detach().requires_grad_() for x in names}
    with torch.enable_grad():
        o, last = _plain_prompt(s, leaves if "h0" in leaves else {**leaves, "h0": None})
        outs, grads = [o], [s["do"].float()]
        if s["dht"] is not None:
            outs, grads = outs + [last], grads + [s["dht"]]
        d = torch.autograd.grad(outs, [leaves[x] for x in names], grads)
    result = {"d" + x: y.to(s[x].dtype) for x, y in zip(names, d)}
    return dict(result, o=o.detach().to(s["q"].dtype))


def _plain_step(s):
    c, at = s["case"], s["slots"].long()
    rep = c["hv"] // c["hk"]
    q, k = (s[x].float().repeat_interleave(rep, 2) for x in ("q", "k"))
    v, a, beta = s["v"].float(), s["g"].exp(), s["beta"].float()
    S, out = s["state"][at], []
    for i in range(c["t"]):
        S = S * a[:, i, :, None, None]
        u = beta[:, i, :, None] * (v[:, i] - (k[:, i, :, :, None] * S).sum(-2))
        S = S + k[:, i, :, :, None] * u[..., None, :]
        out.append((q[:, i, :, :, None] * S).sum(-2) * c["k"] ** -0.5)
    s["state"][at] = S
    return {"o": torch.stack(out, 1).to(s["q"].dtype), "state": s["state"]}


def _take_free(refcount, n):
    """The n lowest pages that nobody holds."""
    return torch.argsort((refcount > 0).to(torch.int8), stable=True)[:n]


def _plain_branch(s):
    c, pt = s["case"], s["case"]["page_tokens"]
    refcount, pools = s["refcount"], s["pools"]
    table, lengths = s["table"][s["parents"].long()], s["lengths"][s["parents"].long()]
    slot = torch.arange(c["width"], device=DEV)
    full, part = lengths // pt, lengths % pt != 0
    refcount.index_add_(0, table.clamp(min=0).flatten().long(), (slot < full[:, None]).flatten().to(torch.int32))
    new = _take_free(refcount, c["rows"])[(part.cumsum(0) - 1).clamp(min=0)]
    at = full.clamp(max=c["width"] - 1).long()[:, None]
    old = table.gather(1, at)[:, 0]
    table.scatter_(1, at, torch.where(part, new.to(torch.int32), old)[:, None])
    src, dst = old[part].long(), new[part]
    for pool in pools:
        pool[dst] = pool[src]
    refcount[dst] = 1
    grown = lengths + c["draft"]
    have, need = -(-lengths // pt), -(-grown // pt)
    want = (slot >= have[:, None]) & (slot < need[:, None])
    rank = want.flatten().cumsum(0).view_as(want) - 1
    free = _take_free(refcount, c["rows"] * (c["draft"] + 1))
    table = torch.where(want, free[rank.clamp(min=0)].to(torch.int32), table)
    refcount.index_add_(0, table.clamp(min=0).flatten().long(), want.flatten().to(torch.int32))
    held = refcount.clone()
    refcount.index_add_(0, table.clamp(min=0).flatten().long(), -(table >= 0).flatten().to(torch.int32))
    return {"table": table, "lengths": lengths, "held": held, "refcount": refcount, "pools": pools}


def _plain_compact(s):
    table, pools = s["table"], s["pools"]
    gone = (s["flags"] != 0)[:, None] & (table >= 0)
    refcount = s["refcount"].clone()
    refcount.index_add_(0, table.clamp(min=0).flatten().long(), -gone.flatten().to(torch.int32))
    table = torch.where(gone, -1, table)
    used = refcount > 0
    n = int(used.sum())
    holes, movers = (~used[:n]).nonzero()[:, 0], used[n:].nonzero()[:, 0] + n
    to = torch.arange(used.numel(), device=DEV)
    to[movers] = holes
    for pool in pools:
        pool[holes] = pool[movers]
    table = torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table)
    out = torch.zeros_like(refcount)
    out[to[used]] = refcount[used]
    return {"table": table, "refcount": out, "used": torch.full((1,), n, dtype=torch.int32, device=DEV), "pools": pools}


def _plain_copy(s):
    for pool in s["pools"]:
        pool[s["dst"].long()] = pool[s["src"].long()]
    return {"pools": s["pools"]}


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    kind = c["kind"]
    if not own:
        with torch.no_grad():
            if kind == "prompt":
                o, last = _plain_prompt(s)
                return {"o": o.to(s["q"].dtype), "state": last}
            return {"step": _plain_step, "train": _plain_train, "branch": _plain_branch, "compact": _plain_compact,
                    "copy": _plain_copy}[kind](s)
    from prefix_scan_gb300 import api
    if kind == "step":
        o = api.delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return {"o": o, "state": s["state"]}
    if kind == "prompt":
        o, last = api.delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"], initial_state=s["h0"],
                                 output_final_state=True)
        return {"o": o, "state": last}
    if kind == "train":
        o, _, saved = api.delta_rule_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"], initial_state=s["h0"])
        d = api.delta_rule_backward(saved, s["do"], d_final_state=s["dht"])
        out = dict(zip(("dq", "dk", "dv", "dg", "dbeta"), d), o=o)
        return dict(out, dh0=d[5]) if s["h0"] is not None else out
    if kind == "copy":
        api.pages_copy(s["pools"], s["src"], s["dst"])
        return {"pools": s["pools"]}
    if kind == "compact":
        refcount = s["refcount"].clone()
        table = s["table"].clone()
        api.pages_free(table, refcount, flags=s["flags"])
        used = api.pages_compact(table, refcount, s["pools"])
        return {"table": table, "refcount": refcount, "used": used, "pools": s["pools"]}
    pt = c["page_tokens"]
    table, lengths, _ = api.pages_fork(s["table"], s["lengths"], s["parents"], s["refcount"], s["pools"], page_tokens=pt)
    api.pages_grow(table, lengths, lengths + c["draft"], s["refcount"], page_tokens=pt)
    held = s["refcount"].clone()
    grown = table.clone()
    api.pages_free(table, s["refcount"])
    return {"table": grown, "lengths": lengths, "held": held, "refcount": s["refcount"], "pools": s["pools"]}


# ---- in 64 bits -------------------------------------------------------------------------------------------------------

def _by_token(s, name):
    """[tokens, sequences, heads, ...] in 64 bits, zero past each sequence's end."""
    x, c = s[name].double(), s["case"]
    if s["cu"] is not None:
        parts = x.split(s["lens"])
        x = torch.nn.utils.rnn.pad_sequence(parts, batch_first=True)
    return x.transpose(0, 1).repeat_interleave(c["hv"] // x.shape[2], 2)


def _back(s, x):
    """The inputs' order of what _by_token() laid out; groups of value heads stay apart."""
    x = x.transpose(0, 1)
    return x if s["cu"] is None else torch.cat([x[i, :n] for i, n in enumerate(s["lens"])])


def _advance(S, q, k, v, g, beta, scale):
    """One token of the recurrence: the decayed state, what was missing from it, the state after, the output."""
    D = S * g.exp()[..., None, None]
    miss = v - torch.einsum("...kv,...k->...v", D, k)
    N = D + k[..., :, None] * (beta[..., None] * miss)[..., None, :]
    return D, miss, N, scale * torch.einsum("...kv,...k->...v", N, q)


def _exact_sequence(s):
    c = s["case"]
    scale = c["k"] ** -0.5
    x = [_by_token(s, name) for name in ("q", "k", "v", "g", "beta")]
    T, every = x[0].shape[0], 128
    S = torch.zeros(c["n"], c["hv"], c["k"], c["v"], dtype=torch.float64, device=DEV) if s["h0"] is None else s["h0"].double()
    o, marks = torch.zeros_like(x[2]), []
    train = c["kind"] == "train"
    for t in range(T):
        if train and t % every == 0:
            marks.append(S)
        _, _, S, o[t] = _advance(S, *(y[t] for y in x), scale)
    result = {"o": _back(s, o)}
    if not train:
        return dict(result, state=S)
    q, k, v, g, beta = x
    do = _by_token(s, "do")
    dq, dk, dv, dg, db = (torch.zeros_like(y) for y in x)
    dS = torch.zeros_like(S) if s["dht"] is None else s["dht"].double()
    for m in range(len(marks) - 1, -1, -1):
        S, kept = marks[m], []
        for t in range(m * every, min(T, (m + 1) * every)):
            kept.append(S)
            S = _advance(S, *(y[t] for y in x), scale)[2]
        for t in range(min(T, (m + 1) * every) - 1, m * every - 1, -1):
            D, miss, N, _ = _advance(kept.pop(), *(y[t] for y in x), scale)
            dS = dS + scale * q[t][..., :, None] * do[t][..., None, :]
            dq[t] = scale * torch.einsum("...kv,...v->...k", N, do[t])
            du = torch.einsum("...kv,...k->...v", dS, k[t])
            db[t] = (du * miss).sum(-1)
            dv[t] = beta[t][..., None] * du
            dk[t] = torch.einsum("...kv,...v->...k", dS, beta[t][..., None] * miss) - torch.einsum("...kv,...v->...k", D, dv[t])
            dS = dS - k[t][..., :, None] * dv[t][..., None, :]
            dg[t] = (dS * D).sum((-2, -1))
            dS = dS * g[t].exp()[..., None, None]
    shared = lambda y: y.unflatten(-2, (c["hk"], c["hv"] // c["hk"])).sum(-2)  # noqa: E731
    result.update(dq=shared(_back(s, dq)), dk=shared(_back(s, dk)), dv=_back(s, dv), dg=_back(s, dg), dbeta=_back(s, db))
    return dict(result, dh0=dS) if s["h0"] is not None else result


def _exact_step(s):
    c, at = s["case"], s["slots"].long()
    state = s["state"].double()
    S, out = state[at], []
    rep = c["hv"] // c["hk"]
    q, k = (s[x].double().repeat_interleave(rep, 2) for x in ("q", "k"))
    for i in range(c["t"]):
        _, _, S, o = _advance(S, q[:, i], k[:, i], s["v"][:, i].double(), s["g"][:, i].double(), s["beta"][:, i].double(), c["k"] ** -0.5)
        out.append(o)
    state[at] = S
    return {"o": torch.stack(out, 1), "state": state}


def _exact_pages(s):
    """What the pages hold afterwards, worked out page by page on the host; the counts and tables have no 64-bit value."""
    c, moves = s["case"], []
    if c["kind"] == "copy":
        moves = list(zip(s["src"].tolist(), s["dst"].tolist()))
    elif c["kind"] == "compact":
        keep = {p for row, f in zip(s["table"].tolist(), s["flags"].tolist()) if not f for p in row if p >= 0}
        holes = [p for p in range(len(keep)) if p not in keep]
        moves = list(zip(sorted(p for p in keep if p >= len(keep)), holes))
    else:
        pt, table, lengths = c["page_tokens"], s["table"].tolist(), s["lengths"].tolist()
        free = iter([p for p, n in enumerate(s["refcount"].tolist()) if n == 0])
        for p in s["parents"].tolist():
            if lengths[p] % pt:
                moves.append((table[p][lengths[p] // pt], next(free)))
    pools = []
    for pool in s["pools"]:
        was = pool.double()
        now = was.clone()
        if moves:
            src, dst = (torch.tensor(x, device=DEV) for x in zip(*moves))
            now[dst] = was[src]
        pools.append(now)
    out = {"pools": pools}
    if c["kind"] != "copy":
        out.update({x: None for x in (("table", "refcount", "used") if c["kind"] == "compact" else
                                      ("table", "lengths", "held", "refcount"))})
    return out


def exact(c, seed):
    s = prepare(c, seed)
    with torch.no_grad():
        if c["kind"] == "step":
            return _exact_step(s)
        return _exact_sequence(s) if c["kind"] in ("prompt", "train") else _exact_pages(s)
