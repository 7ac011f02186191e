"""Layer norm and its gradient in 64 bits, on the tensors' own device, with bounds that count the roundings of the kernels'
sums, so that a row that is left out of the weights' sums is seen among tens of thousands.

u = 2^-24.  A row's sum: at most 4 pieces of 4 packed pairs a thread one after another, the pair (17 roundings), 5 shuffles, 16
warps: 38, and with 1 / D and the product 40 u of the mean's magnitude; e = 42 u mean|x|, eta = e rstd.
rstd: the squares' sum has 38 + the squares' own 2 u, D and eps 3 more, and e^2 from the mean (its linear part sums
to 0); half of that and 4 u of the root: rho = 32 u + eta^2.

A weight's sum over the rows: a thread adds its rows one after another, at most 4 or, where the grid of at least 152 groups
takes more than one tile, rows / 152 + 4; at most 64 groups or warps of a CTA; at most 456 CTAs in 32 warps, 15 each;
5 shuffles: rows / 152 + 88 roundings of partial sums of the terms' magnitudes.
"""
import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def mean(t):
    return t.mean(-1, keepdim=True)


def parts(x, eps):
    """n, rstd, and what they are off by: eta and rho."""
    x = x.double()
    m = mean(x)
    rstd = (mean((x - m).square()) + eps).rsqrt()
    eta = 42 * U * mean(x.abs()) * rstd
    return (x - m) * rstd, rstd, eta, 32 * U + eta ** 2


def forward(x, w, b, eps):
    n, _, eta, rho = parts(x, eps)
    w, b = w.double(), b.double()
    return n * w + b, w.abs() * (eta + n.abs() * (rho + 2 * U)) + 2 * U * ((n * w).abs() + b.abs())


def backward(x, d, w, eps):
    """dx, dw, db and their bounds; the rows are those that are there."""
    n, rstd, eta, rho = parts(x, eps)
    d, w = d.double(), w.double()
    g = d * w
    p, q = mean(g.abs()), mean((g * n).abs())
    dx = rstd * (g - mean(g) - n * mean(g * n))
    bx = rstd * (g.abs() * (rho + 4 * U) + p * (rho + 48 * U) + n.abs() * q * (3 * rho + 52 * U)
                 + eta * (q + (n.abs() + eta) * p)) * (1 + 2.0 ** -10)
    rows = x.numel() // x.shape[-1]
    adds = (rows / 152 + 88) * U
    over = tuple(range(x.dim() - 1))
    bw = (d.abs() * (n.abs() * (rho + 2 * U + adds) + eta)).sum(over) * (1 + 2.0 ** -10)
    return {"x": dx, "weight": (d * n).sum(over), "bias": d.sum(over)}, {"x": bx, "weight": bw, "bias": adds * d.abs().sum(over)}


def worst(got, want, bound, rounded=None):
    """By how much the worst value is beyond its bound (not above 0: none is)."""
    if rounded is not None:
        bound = bound + ROUND[rounded] * (want.abs() + bound)
    off = (got.double() - want).abs() - bound - 2.0 ** -126
    return float("inf") if not torch.isfinite(got).all() else off.max().item()
