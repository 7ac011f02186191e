"""The linear attention layer's operators from their definitions, in fp64 on the CPU, token by
token, and the error bounds that the GPU tests hold the kernels to.

Bounds.  ``magnitude`` runs a definition on absolute values, so every product and sum that a
kernel forms is at most its result M.  One rounding to fp32 is off by u = 2^-24 of the value at
most, one to bf16 (8 significant bits) by 2^-8:

* fp32 arithmetic over T tokens and D dims: n roundings in a row, n <= T + D + 256 (the last
  term for the decay powers, whose exponents are rounded too): |error| <= n u M;
* bf16 products: the scores, and the state that a chunk reads, are rounded once each, and the
  output once: |error| <= 2^-8 |o| + 1.1 2^-8 M;
* the bf16 path's fp32 states: the decayed key (or query) enters in two bf16 terms, which
  leaves 2^-16 of it at most: |error| <= (2^-16 + n u) M.
"""
import torch

U, BF16 = 2.0 ** -24, 2.0 ** -8


def linattn(q, k, v, log_decay, scale=1.0, initial_state=None, lens=None):
    """out [B,T,H,D], final_state [B,H,D,D]; tokens at or past ``lens`` are padding."""
    B, T, H, D = q.shape
    a = log_decay.exp()[None, :, None, None]
    S = torch.zeros(B, H, D, D, dtype=q.dtype) if initial_state is None else initial_state
    outs = []
    for t in range(T):
        on = torch.ones(B, dtype=torch.bool) if lens is None else t < lens
        kt, vt, qt = (torch.where(on[:, None, None], x[:, t], torch.zeros_like(x[:, t])) for x in (k, v, q))
        S = torch.where(on[:, None, None, None], a * S + vt[..., :, None] * kt[..., None, :], S)
        outs.append(scale * torch.einsum("bhvk,bhk->bhv", S, qt))
    return torch.stack(outs, 1), S


def linattn_backward(q, k, v, log_decay, d_out, scale=1.0, initial_state=None, d_state=None, lens=None):
    """dq, dk, dv, d_initial_state by the recurrences of the definition's gradient."""
    B, T, H, D = q.shape
    a = log_decay.exp()[None, :, None, None]
    S = torch.zeros(B, H, D, D, dtype=q.dtype) if initial_state is None else initial_state
    G = torch.zeros(B, H, D, D, dtype=q.dtype) if d_state is None else d_state
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))

    def at(x, t, on):
        return torch.where(on[:, None, None], x[:, t], torch.zeros_like(x[:, t]))

    for t in range(T):
        on = torch.ones(B, dtype=torch.bool) if lens is None else t < lens
        S = torch.where(on[:, None, None, None], a * S + at(v, t, on)[..., :, None] * at(k, t, on)[..., None, :], S)
        dq[:, t] = scale * torch.einsum("bhvk,bhv->bhk", S, at(d_out, t, on))
    for t in reversed(range(T)):
        on = torch.ones(B, dtype=torch.bool) if lens is None else t < lens
        here = G + scale * at(d_out, t, on)[..., :, None] * at(q, t, on)[..., None, :]
        dv[:, t] = torch.einsum("bhvk,bhk->bhv", here, at(k, t, on))
        dk[:, t] = torch.einsum("bhvk,bhv->bhk", here, at(v, t, on))
        G = torch.where(on[:, None, None, None], a * here, G)
    return dq, dk, dv, G


def rope(x, w, table, pos, scale=1.0, eps=1e-6, interleaved=False, live=None):
    """x [B,T,H,D] normed, weighted, scaled and turned; ``live`` [B,T]: the tokens that are there."""
    B, T, H, D = x.shape
    if live is not None:
        x = torch.where(live[:, :, None, None], x, torch.ones_like(x))
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * scale
    if w is not None:
        y = y * w
    if table is not None:
        r = table.shape[1]
        row = table[pos.clamp(0, table.shape[0] - 1)][:, :, None]
        c, s = row[..., :r // 2], row[..., r // 2:]
        i = torch.arange(r // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        z = y.clone()
        z[..., ia] = y[..., ia] * c - y[..., ib] * s
        z[..., ib] = y[..., ib] * c + y[..., ia] * s
        y = z
    if live is not None:
        y = torch.where(live[:, :, None, None], y, torch.zeros_like(y))
    return y


def rope_live(T, B, table, pos, lens):
    live = torch.ones(B, T, dtype=torch.bool)
    if lens is not None:
        live &= torch.arange(T)[None] < lens[:, None]
    if table is not None:
        live &= (pos >= 0) & (pos < table.shape[0])
    return live


def angles(rows, r, base=10000.0):
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], -1)


def out_bound(o, m, dtype, T, D):
    n = (T + D + 256) * U
    return n * m if dtype == torch.float32 else BF16 * o.abs() + 1.1 * BF16 * m


def state_bound(m, dtype, T, D):
    n = (T + D + 256) * U
    return n * m if dtype == torch.float32 else (2.0 ** -16 + n) * m


def assert_within(got, want, bound, what=""):
    got = got.detach().double().cpu()
    # below fp32's range the nearest value that an output can hold is 0
    want = torch.where(want.abs() < 2.0 ** -150, 0.0, want)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - want).abs() - bound
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0.0, f"{what}: {(off > 0).sum().item()} of {off.numel()} beyond the bound, by up to {worst:.3e}"
