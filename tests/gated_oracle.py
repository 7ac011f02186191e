"""The gated recurrent layer's operators in 64 bits, token by token, with the bounds that the kernels' fp32
arithmetic has.

u = 2^-24.  A gate is e / (1 + e), e = exp(-|z|), or 1 minus it.  The smaller of the two is off by
delta = (2 |z| + 16) u of itself at most: |z| log2(e) and its constant are each off by u of the exponent, ex2 by
2^-22 = 4u, the sum and the product by u each, the reciprocal by 2u (the fp32 path's expf and division
stay within it: 4u and 4u).  The larger one is off by that and by its own rounding, u.

States.  With m_t = a m_(t-1) + w |x| the recurrence of magnitudes, an error E_t obeys
E_t <= a E_(t-1) + (delta min(a, 1 - a) + 8 u a) m_(t-1) + (delta_w + 4 u) w |x|: the gates' errors and, for each token,
the roundings of a, of the product P, of the fused operation and of the joins of lanes, warps and
tiles.  Gates below 2^-126 count as zero; the tests' values stay above.
"""
import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}     # half a step, relative


def gates(f, i):
    f = f.double()
    a, c = torch.sigmoid(f), torch.sigmoid(-f)
    return (a, c, c, a) if i is None else (a, c, torch.sigmoid(i.double()), torch.sigmoid(-i.double()))


def delta(z):
    return (2 * z.double().abs() + 16) * U


def lengths(x, lens):
    B, T = x.shape[:2]
    return torch.full((B,), T) if lens is None else lens.clamp(0, T)


def _live(x, lens):
    return torch.arange(x.shape[1])[None, :] < lengths(x, lens)[:, None]


def scan(x, f, i=None, s0=None, lens=None):
    """out and final state in fp64, the states before every token, magnitudes, and errors of the states.
    Padding's values are not looked at."""
    live = _live(x, lens)[..., None]
    a, c, w, _ = gates(f, i)
    B, T, D = x.shape
    h = torch.zeros(B, D, dtype=torch.float64) if s0 is None else s0.double()
    m, E = h.abs(), torch.zeros_like(h)
    out, before, mags, errs = [], [], [m], [E]
    da = delta(f) * torch.minimum(a, c) + 8 * U * a
    dw = delta(f if i is None else i) + 4 * U
    for t in range(T):
        on, b = live[:, t], torch.where(live[:, t], w[:, t] * x[:, t].double(), 0.0)
        before.append(h)
        E = torch.where(on, a[:, t] * E + da[:, t] * m + dw[:, t] * b.abs(), E)
        h, m = torch.where(on, a[:, t] * h + b, h), torch.where(on, a[:, t] * m + b.abs(), m)
        out.append(torch.where(on, h, 0.0))
        mags.append(m)
        errs.append(E)
    st = lambda v: torch.stack(v, 1)  # noqa: E731
    return dict(out=st(out), final=h, before=st(before), mag=st(mags), err=st(errs))


def scan_back(x, f, d_out, i=None, s0=None, d_final=None, lens=None):
    """The gradients by their formulas, and a bound for the error of each before it is rounded."""
    s = scan(x, f, i, s0, lens)
    live = _live(x, lens)[..., None]
    a, c, w, v = gates(f, i)
    B, T, D = x.shape
    r = torch.zeros(B, D, dtype=torch.float64) if d_final is None else d_final.double()
    m, E = r.abs(), torch.zeros_like(r)
    da = delta(f) * torch.minimum(a, c) + 8 * U * a
    df_, di_ = delta(f), delta(f if i is None else i)
    got = {n: torch.zeros(B, T, D, dtype=torch.float64) for n in ("x", "forget", "input_gate")}
    bound = {n: torch.zeros_like(t) for n, t in got.items()}
    for t in reversed(range(T)):
        on = live[:, t]
        z = lambda y: torch.where(on, y, 0.0)  # noqa: E731
        xt, d = z(x[:, t].double()), z(d_out[:, t].double())
        G, mG = d + r, d.abs() + m
        EG = E + 2 * U * mG
        hb, mh, Eh = s["before"][:, t], s["mag"][:, t], s["err"][:, t]
        got["x"][:, t] = z(w[:, t] * G)
        bound["x"][:, t] = z(w[:, t] * (EG + (di_[:, t] + 4 * U) * mG))
        rest, mrest, Erest = (hb, mh, Eh) if i is not None else (hb - xt, mh + xt.abs(), Eh + 2 * U * (mh + xt.abs()))
        ac = a[:, t] * c[:, t]
        got["forget"][:, t] = z(ac * G * rest)
        bound["forget"][:, t] = z(ac * (EG * mrest + mG * Erest + (2 * df_[:, t] + 8 * U) * mG * mrest))
        wv = w[:, t] * v[:, t]
        got["input_gate"][:, t] = z(wv * G * xt)
        bound["input_gate"][:, t] = z(wv * xt.abs() * (EG + (2 * di_[:, t] + 8 * U) * mG))
        E = torch.where(on, a[:, t] * EG + da[:, t] * mG, E)
        r, m = torch.where(on, a[:, t] * G, r), torch.where(on, a[:, t] * mG, m)
    got["initial_state"], bound["initial_state"] = r, E + 4 * U * m
    if i is None:
        got["input_gate"] = None
    return got, bound


def layer_norm(x, w, b, eps, lens=None):
    """y in fp64 and the error before its rounding.  A sum of D values runs over at most 8 values of up to 8 pieces a
    thread, 5 shuffles and 32 warps: 104 roundings of partial sums of magnitudes, e = 104 u mean|x| for the mean.
    The squares after it are off by 2 e * (sum of centred values, 0) + e^2 and 104 u again."""
    live = _live(x, lens)[..., None]
    x = torch.where(live, x.double(), 0.0)
    mean = x.mean(-1, keepdim=True)
    e = 104 * U * x.abs().mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    n = (x - mean) * rstd
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    y = n * w + b
    rel = 64 * U + (e * rstd) ** 2
    bound = w.abs() * ((e * rstd) * (1 + rel) + n.abs() * rel) + 4 * U * ((n * w).abs() + b.abs())
    return torch.where(live, y, 0.0), torch.where(live, bound, 0.0)


def layer_norm_back(x, d_out, w, eps, lens=None):
    """dx, dw and db by their formulas, with bounds."""
    live = _live(x, lens)[..., None]
    x, d = torch.where(live, x.double(), 0.0), torch.where(live, d_out.double(), 0.0)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    mu = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    e = 104 * U * mu(x.abs())
    rstd = (mu((x - mu(x)).square()) + eps).rsqrt()
    n, g = (x - mu(x)) * rstd, d * w
    eta = e * rstd                                        # what n is off by, beside what is relative to it
    dx = rstd * (g - mu(g) - n * mu(g * n))
    rel = 300 * U + 2 * eta ** 2
    size = rstd * (g.abs() + mu(g.abs()) + n.abs() * mu((g * n).abs()))
    bx = rel * size + 2 * rstd * eta * (mu((g * n).abs()) + (n.abs() + eta) * mu(g.abs()))
    rows = int(lengths(x, lens).sum())
    many = (64 + rows) * U                                # a sum over the rows, in whatever grouping
    bw = (d.abs() * (n.abs() * (rel + many) + 2 * eta)).sum((0, 1))
    bb = many * d.abs().sum((0, 1))
    zero = lambda t: torch.where(live, t, 0.0)  # noqa: E731
    return ({"x": zero(dx), "weight": (d * n).sum((0, 1)), "bias": d.sum((0, 1))},
            {"x": zero(bx), "weight": bw, "bias": bb})


def assert_within(got, want, bound, what="", rounded=None):
    """|got - want| <= bound, plus half a step of type ``rounded`` where given (a relative one, or below the
    type's normal numbers the smallest normal's)."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if rounded is not None:
        bound = bound + ROUND[rounded] * (want.abs() + bound)
    off = (got - want).abs() - bound - 2.0 ** -126
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0.0, f"{what}: {(off > 0).sum().item()} of {off.numel()} beyond the bound, by up to {worst:.3e}"
