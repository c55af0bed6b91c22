"""The gated linear recurrence in 64 bits, token by token, and how far 32-bit results may be from it.

    h_t = a_t h_{t-1} + w_t x_t,  a = exp(g),  w = 1 or 1 - a
    lam_t = dh_t + mu_{t+1},  mu_t = a_t lam_t,  dx_t = w_t lam_t,  dg_t = mu_t (h_{t-1} - [tied] x_t),  dh0 = mu_1

Tolerance, with u = 2^-24 and M_t the same recurrence over absolute values, which bounds every term of h_t.
- Each token's product, sum with the state and w x are rounded: three roundings of at most u M_t, uniform and independent, with a
  deviation of at most u M_t together.  They decay with the state: R_t^2 = a_t^2 R_{t-1}^2 + u^2 M_t^2, taken six times.
- Each token's factor is off to one side by at most 2^-22.5 of 1 - a where -1/16 < g <= 0 (a series cut at 2^-22.9, and its
  rounding) and 2^-21.5 of a elsewhere (the hardware's 2^x within 2^-22, its argument within u of itself, of which
  |g| exp(g) <= 0.37 remains; 1 - a of tied inputs within as much): L_t = a_t L_{t-1} + that times (M_{t-1} + |x_t| if tied).
- What a run of up to 32 tokens and a tile of 16 runs hand on is multiplied by exp of the sum of their log decays.  A sum of n
  numbers is off by n roundings of at most u |s|, uniform and independent, with a deviation of (n / 3)^0.5 u |s|, and
  |s| exp(s) <= 0.37: 32 of a run, 1 of a pair of them, 8 of the pairs, 3.7 u |s|, six times and by 0.37 less than 9 u; exp itself
  2 u, two roundings 2 u; a token sees a run's and a tile's: 26 u M_t.
- Backward, what a run of up to 16 tokens adds is the sum of P_i dh_i, P_i the product of its factors so far: 16 additions and as
  many roundings of P, each of at most u M, with a deviation of (32 / 3)^0.5 u M, six times 20 u M.  It takes the place of the
  first point's roundings, which are 24 u M where the run decays little and 6 u M at least; where it decays much |s| exp(s) is
  near 0 and the sums' 18 u of the third point are free.
Outputs of fewer bits are off by half a step more, and f16 by half its smallest step."""
from __future__ import annotations

import torch

U = 2.0 ** -24


def _run(a, b, start, lin, sq):
    """The recurrence from `start` = (value, absolute sum, linear error, squared error), with every token's results."""
    h, m, el, er = start
    out = [[], [], [], []]
    for t in range(a.shape[0]):
        el = a[t] * el + lin[t] * (m + b[t].abs() * sq)
        h = a[t] * h + b[t]
        m = a[t] * m + b[t].abs()
        er = a[t] ** 2 * er + (U * m) ** 2
        for o, x in zip(out, (h, m, el, er)):
            o.append(x)
    return [torch.stack(o) if o else a.new_zeros(0, *a.shape[1:]) for o in out]


def _error(m, el, er):
    return el + 6 * er.sqrt() + 26 * U * m


def sequence(x, g, h0=None, tied=False, dh=None, dht=None):
    """One sequence's [tokens, channels] in 64 bits: {name: (value, tolerance of a 32-bit result)}."""
    x, g = x.double(), g.double()
    a = g.exp()
    w = -torch.expm1(g) if tied else torch.ones_like(g)
    zero = x.new_zeros(x.shape[1:])
    h0 = zero if h0 is None else h0.double()
    lin = torch.where((g > -1 / 16) & (g <= 0), (1 - a) * 2.0 ** -22.5, a * 2.0 ** -21.5)
    # tied: w x is off by as much, relative to x: |b| / w of it
    extra = torch.where(w > 0, 1 / w.clamp(min=1e-300), torch.ones_like(w)) if tied else torch.ones_like(w)
    b = w * x
    h, m, el, er = _run(a, b, (h0, h0.abs(), zero, zero), lin, 0.0)
    if tied:   # the inputs' own part, decayed like the rest
        el = el + _run(a, lin * (b.abs() * extra), (zero, zero, zero, zero), lin, 0.0)[0]
    state = h[-1] if len(h) else h0
    eh = _error(m, el, er)
    result = {"h": (h, eh), "state": (state, eh[-1] if len(h) else zero)}
    if dh is None:
        return result
    dh = dh.double()
    end = zero if dht is None else dht.double()
    # lam_t = dh_t + a_{t+1} lam_{t+1}; before the last token comes the end's gradient, whole
    af = torch.cat([a[1:], torch.ones_like(a[:1])]).flip(0)
    lf = torch.cat([lin[1:], torch.zeros_like(lin[:1])]).flip(0)
    lam, ml, ell, erl = (y.flip(0) for y in _run(af, dh.flip(0), (end, end.abs(), zero, zero), lf, 0.0))
    el_lam = _error(ml, ell, erl)
    mu, m_mu, e_mu = a * lam, a * ml, a * el_lam + (lin + 2 * U * a) * ml
    hp, mp, ep = (torch.cat([first[None], y[:-1]]) for first, y in ((h0, h), (h0.abs(), m), (zero, eh))) if len(h) else (h, h, h)
    if tied:
        hp, mp = hp - x, mp + x.abs()
    result["dx"] = (w * lam, w.abs() * el_lam + (lin + 2 * U) * ml if tied else el_lam)
    result["dg"] = (mu * hp, mp * e_mu + m_mu * (ep + U * mp) + 2 * U * mp * m_mu)
    result["dh0"] = (mu[0], e_mu[0]) if len(h) else (end, zero)
    return result


def packed(x, g, lens, first=0, h0=None, tied=False, dh=None, dht=None):
    """Sequences one after the other from token `first` on: values and tolerances laid out as the inputs, and which tokens are
    held."""
    names = ("h",) if dh is None else ("h", "dx", "dg")
    per = ("state",) if dh is None else ("state", "dh0")
    whole = {n: (torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)) for n in names}
    ends = {n: ([], []) for n in per}
    held = torch.zeros(x.shape[0], dtype=torch.bool)
    at = first
    for i, n in enumerate(lens):
        cut = lambda y: None if y is None else y[at:at + n]  # noqa: E731
        row = lambda y: None if y is None else y[i]  # noqa: E731
        r = sequence(x[at:at + n], g[at:at + n], row(h0), tied, cut(dh), row(dht))
        for name in names:
            for to, value in zip(whole[name], r[name]):
                to[at:at + n] = value
        for name in per:
            for to, value in zip(ends[name], r[name]):
                to.append(value)
        held[at:at + n] = True
        at += n
    whole.update({n: tuple(torch.stack(y) for y in v) for n, v in ends.items()})
    return whole, held


def check(got, want, name=""):
    """Whether `got` is within the tolerance of `want` = (value, tolerance), its own rounding included."""
    value, tol = want
    got = got.detach().cpu()
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    tol = tol * (1 + half) + half * value.abs() + (2.0 ** -25 if got.dtype == torch.float16 else 0.0) + 1e-37
    off = (got.double() - value).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
        f"{off[bad][0].item():.3e} > {tol[bad][0].item():.3e} of {value[bad][0].item():.3e}"
