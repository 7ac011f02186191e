"""The fp64 oracle of the linear attention layer against itself (CPU): its gradients against
autograd and differences, its chunked form against the recurrence, the norm's gradient."""
import pytest
import torch

from tests import linattn_oracle as lo


def draw(B, T, H, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return (n(B, T, H, D), n(B, T, H, D), n(B, T, H, D), -torch.rand(H, generator=g, dtype=torch.float64),
            n(B, T, H, D), n(B, H, D, D), n(B, H, D, D))


@pytest.mark.parametrize("T", [1, 2, 9])
@pytest.mark.parametrize("lens", [None, (0, 1), (3, 9)])
def test_gradient_is_autograds_and_the_differences(T, lens):
    q, k, v, ld, do, s0, ds = draw(2, T, 2, 4)
    lens = None if lens is None else torch.tensor(lens).clamp(max=T)
    ins = [x.clone().requires_grad_() for x in (q, k, v, s0)]
    o, s = lo.linattn(*ins[:3], ld, 0.7, ins[3], lens)
    loss = (o * do).sum() + (s * ds).sum()
    auto = torch.autograd.grad(loss, ins)
    mine = lo.linattn_backward(q, k, v, ld, do, 0.7, s0, ds, lens)
    for a, m in zip(auto, mine):
        assert torch.allclose(a, m, rtol=1e-11, atol=1e-12)
    g = torch.Generator().manual_seed(5)
    step = [torch.randn(x.shape, generator=g, dtype=torch.float64) for x in (q, k, v, s0)]

    def value(e):
        o, s = lo.linattn(q + e * step[0], k + e * step[1], v + e * step[2], ld, 0.7, s0 + e * step[3], lens)
        return ((o * do).sum() + (s * ds).sum()).item()

    slope = (value(1e-5) - value(-1e-5)) / 2e-5
    assert abs(slope - sum((m * d).sum().item() for m, d in zip(mine, step))) <= 1e-6 * max(1.0, abs(slope))


@pytest.mark.parametrize("C,T,rev", [(4, 11, False), (4, 12, False), (4, 11, True), (8, 8, True), (4, 3, True)])
def test_chunks_and_runs_give_the_recurrence(C, T, rev):
    """The pass of the kernels, in chunks and in runs of chunks joined through their own states."""
    x, y, z, ld, _, s0, _ = draw(1, T, 1, 5, seed=T)
    x, y, z, s0, lam = x[0, :, 0], y[0, :, 0], z[0, :, 0], s0[0, 0], ld.exp().item()
    su, so = 0.3, 1.3
    sp = so * su                  # as in every call of the library
    want = torch.zeros_like(x)
    chunks = -(-T // C)

    def chunk(c, S, out):
        t0, n = c * C, min(C, T - c * C)
        i = torch.arange(n, dtype=torch.float64)
        X, Y, Z = x[t0:t0 + n], y[t0:t0 + n], z[t0:t0 + n]
        apart = (i[None] - i[:, None]) if rev else (i[:, None] - i[None])
        P = torch.where(apart >= 0, sp * lam ** apart.clamp(min=0) * (X @ Y.T), torch.zeros((), dtype=torch.float64))
        e, f = ((n - 1 - i), (i + 1)) if rev else ((i + 1), (n - 1 - i))
        if out is not None:
            out[t0:t0 + n] = P @ Z + so * lam ** e[:, None] * (X @ S.T)
        return lam ** n * S + su * (Z.T * lam ** f) @ Y

    order = list(reversed(range(chunks))) if rev else list(range(chunks))
    one, S1 = torch.zeros_like(x), s0.clone()
    for c in order:
        S1 = chunk(c, S1, one)
    # token by token
    S = s0.clone()
    for t in (reversed(range(T)) if rev else range(T)):
        if rev:
            want[t] = sp * torch.outer(z[t], y[t]) @ x[t] + so * S @ x[t]
            S = lam * (S + su * torch.outer(z[t], y[t]))
        else:
            before = lam * S
            want[t] = sp * torch.outer(z[t], y[t]) @ x[t] + so * before @ x[t]
            S = before + su * torch.outer(z[t], y[t])
    assert torch.allclose(S1, S, rtol=1e-12, atol=1e-12)
    assert torch.allclose(one, want, rtol=1e-12, atol=1e-12)
    # two runs, the second from lambda^done S_0 + lambda^(done - done_1) D_0
    cut = len(order) // 2
    D0 = torch.zeros(5, 5, dtype=torch.float64)
    for c in order[:cut]:
        D0 = chunk(c, D0, None)
    done = sum(min(C, T - c * C) for c in order[:cut])
    S2 = lam ** done * s0 + D0
    two = one.clone()
    for c in order[cut:]:
        two[c * C:(c + 1) * C] = float("nan")
    for c in order[cut:]:
        S2 = chunk(c, S2, two)
    assert torch.allclose(S2, S1, rtol=1e-12, atol=1e-12) and torch.allclose(two, one, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("rev", [False, True])
def test_two_pieces_are_the_whole(rev):
    """A sequence in two pieces, the state (or its gradient) handed from one to the other."""
    x, y, z, ld, _, s0, _ = draw(1, 10, 1, 3, seed=1)
    q, k, v, do = x, y, z, x
    if not rev:
        o4, _ = lo.linattn(q, k, v, ld, 0.5, s0)
        o, S = lo.linattn(q[:, :4], k[:, :4], v[:, :4], ld, 0.5, s0)
        o2, _ = lo.linattn(q[:, 4:], k[:, 4:], v[:, 4:], ld, 0.5, S)
        assert torch.allclose(torch.cat([o, o2], 1), o4)
    else:
        whole = lo.linattn_backward(q, k, v, ld, do, 0.5, None, s0)
        tail = lo.linattn_backward(q[:, 4:], k[:, 4:], v[:, 4:], ld, do[:, 4:], 0.5, None, s0)
        head = lo.linattn_backward(q[:, :4], k[:, :4], v[:, :4], ld, do[:, :4], 0.5, None, tail[3])
        assert torch.allclose(whole[1], torch.cat([head[1], tail[1]], 1))
        assert torch.allclose(whole[3], head[3])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("r", [0, 8, 16])
def test_norm_and_rotation(interleaved, r):
    g = torch.Generator().manual_seed(r)
    x = torch.randn(2, 3, 2, 16, generator=g, dtype=torch.float64)
    table = lo.angles(5, r) if r else None
    pos = torch.tensor([[0, 1, 2], [4, 3, 0]])
    y = lo.rope(x, None, table, pos, 16 ** -0.5, 0.0, interleaved)
    assert torch.allclose(y.norm(dim=-1), torch.ones(2, 3, 2, dtype=torch.float64))     # unit vectors, turned
    if r:                                                          # position 0 turns nothing
        assert torch.allclose(y[0, 0], lo.rope(x, None, None, pos, 16 ** -0.5, 0.0)[0, 0])
        # products of a query and a key depend on their distance alone
        q, k = x[:1, :1].expand(1, 5, 2, 16), x[1:, 1:2].expand(1, 5, 2, 16)
        at = torch.arange(5)[None]
        a, b = (lo.rope(v, None, table, at, 1.0, 1e-6, interleaved)[0] for v in (q, k))
        dots = torch.einsum("thd,shd->hts", a, b)
        assert torch.allclose(dots[:, 1:, 1:], dots[:, :-1, :-1])


def test_the_roundings_of_the_bounds():
    """One rounding is off by 2^-8 of the value at most in bf16, 2^-24 in fp32, and comes close."""
    x = torch.linspace(1.0, 2.0, 100_001, dtype=torch.float64)
    for t, u in ((torch.bfloat16, lo.BF16), (torch.float32, lo.U)):
        off = ((x.to(t).double() - x).abs() / x).max().item()
        assert off <= u and (t == torch.float32 or off > 0.9 * u)
