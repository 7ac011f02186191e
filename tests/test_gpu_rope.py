"""The norm of query and key heads with the position rotation, and its gradient, against fp64.

Bounds, with u = 2^-24.  Forward: a dozen fp32 roundings of a normed value and of the two that
a rotation joins, at most the largest |scale w n| of the head vector each, then one
rounding of the result.  Backward: dx = rstd (u w - n mean(u w n)) with |n| <= sqrt(D), so its
roundings are at most rstd max|u w| (1 + sqrt(D)) each; dw sums N rows of at most |u n|."""
import math

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn
from tests import linattn_oracle as lo

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(B, T, Hq, Hk, D, r, dtype, seed=0, weights=True, rows=None):
    g = torch.Generator().manual_seed(seed + 31 * T + D)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = TYPES[dtype]
    x = n(B, T, Hq + 2 * Hk, D).to(dt)
    return dict(x=x, q=x[:, :, :Hq].contiguous(), k=x[:, :, Hq:Hq + Hk].contiguous(),
                qw=1 + 0.3 * n(D) if weights else None, kw=1 + 0.3 * n(D) if weights else None,
                table=lo.angles(rows or T, r).float() if r else None, dq=n(B, T, Hq, D).to(dt), dk=n(B, T, Hk, D).to(dt))


def check(x, c, *, scales=(0.5, 1.0), eps=1e-6, pos=None, lens=None, interleaved=False):
    B, T, Hq, D = x["q"].shape
    dev = lambda t: None if t is None else t.to(device="cuda", dtype=torch.int32)  # noqa: E731
    how = dict(q_weight=c["qw"], k_weight=c["kw"], q_scale=scales[0], k_scale=scales[1], eps=eps, positions=dev(pos),
               seq_lens=dev(lens), interleaved=interleaved)
    at = pos if pos is not None else torch.arange(T).expand(B, T)
    table = None if x["table"] is None else x["table"].double()
    live = lo.rope_live(T, B, table, at, lens)
    y = linattn.prism_qk_norm_rope(c["q"], c["k"], c["table"], **how)
    g = linattn.prism_qk_norm_rope_backward(c["q"], c["k"], c["table"], c["dq"], c["dk"], **how)
    for i, n in enumerate("qk"):
        dt = x[n].dtype
        rnd = lo.BF16 if dt == torch.bfloat16 else lo.U
        xs, w = x[n].double().requires_grad_(), x[n + "w"]
        ws = (torch.ones(D) if w is None else w).double().requires_grad_()
        want = lo.rope(xs, ws, table, at, scales[i], eps, interleaved, live)
        dy = torch.where(live[:, :, None, None], x["d" + n].double(), 0.0)
        dx, dw = torch.autograd.grad((want * dy).sum(), (xs, ws))
        want = want.detach()
        big = lo.rope(xs.detach(), ws.detach(), None, at, scales[i], eps, False, live).abs().amax(-1, keepdim=True)
        lo.assert_within(y[i], want, rnd * want.abs() + 24 * lo.U * big, n)
        assert y[i].dtype == dt and (y[i][~live.cuda()] == 0).all() and (g[n][~live.cuda()] == 0).all()
        rstd = torch.where(live[:, :, None, None], (xs.detach().square().mean(-1, keepdim=True) + eps).rsqrt(), 0.0)
        rstd = torch.nan_to_num(rstd, nan=0.0)
        u = abs(scales[i]) * dy.abs().amax(-1, keepdim=True) * 2
        size = rstd * u * ws.detach().abs().max() * (1 + math.sqrt(D))
        lo.assert_within(g[n], dx, rnd * dx.abs() + (24 + D) * lo.U * size, "d" + n)
        if w is None:
            assert g[n + "_weight"] is None
        else:
            rows = live.sum().item() * x[n].shape[2]
            nn = torch.where(live[:, :, None, None], xs.detach(), 0.0).abs() * rstd
            most = (u * nn).sum((0, 1, 2))
            lo.assert_within(g[n + "_weight"], dw, (24 + min(rows, 4096)) * lo.U * most, "dw")
    return y, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,D,r", [
    (1, 1, 1, 1, 16, 16), (2, 3, 5, 1, 32, 16), (1, 129, 4, 2, 64, 64), (3, 7, 9, 3, 128, 128), (2, 33, 8, 8, 128, 64),
    (4, 5, 3, 3, 64, 8), (1, 2, 6, 2, 32, 24), (2, 9, 4, 4, 16, 0), (1, 700, 16, 4, 128, 128)])
def test_norm_and_rotation(B, T, Hq, Hk, D, r, interleaved, dtype):
    x = make(B, T, Hq, Hk, D, r, dtype)
    check(x, {n: (None if t is None else t.cuda()) for n, t in x.items()}, interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unit_norm_without_weights(dtype):
    """What the mixer wants: unit vectors, no weights."""
    x = make(2, 40, 2, 2, 64, 0, dtype, weights=False)
    c = {n: (None if t is None else t.cuda()) for n, t in x.items()}
    (q, k), _ = check(x, c, scales=(64 ** -0.5, 64 ** -0.5), eps=1e-6 / 64)
    assert (q.float().norm(dim=-1) - 1).abs().max() < (2.0 ** -8 if dtype == "bf16" else 1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 128])
def test_padding(D, dtype):
    """Ragged and empty sequences, positions outside the table, NaN and infinities in padding."""
    B, T = 5, 11
    x = make(B, T, 3, 2, D, D, dtype, rows=50)
    lens = torch.tensor([0, 1, 11, 7, 11])
    pos = torch.arange(T)[None] + torch.tensor([0, 3, 39, 5, 20])[:, None]
    pos[2, 3], pos[4, 0], pos[4, 5] = -1, 50, -(2 ** 31)
    c = {n: (None if t is None else t.cuda()) for n, t in x.items()}
    live = lo.rope_live(T, B, x["table"], pos, lens).cuda()
    for i, n in enumerate(("q", "k", "dq", "dk")):
        c[n][~live] = float("nan") if i % 2 else float("-inf")
    check(x, c, pos=pos, lens=lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_a_fused_projection(dtype):
    x = make(3, 17, 6, 2, 64, 64, dtype)
    c = {n: (None if t is None else t.cuda()) for n, t in x.items()}
    y1, g1 = check(x, c)
    c["q"], c["k"] = c["x"][:, :, :6], c["x"][:, :, 6:8]
    wide = torch.zeros(3, 20, 9, 64, device="cuda", dtype=TYPES[dtype])
    wide[:, 2:19, :6], wide[:, 2:19, 6:8] = c["dq"], c["dk"]
    c["dq"], c["dk"] = wide[:, 2:19, :6], wide[:, 2:19, 6:8]
    y2, g2 = check(x, c)
    assert all(torch.equal(a, b) for a, b in zip(y1, y2)) and all(torch.equal(g1[n], g2[n]) for n in g1)


def test_zero_vectors_and_large_ones():
    x = make(1, 6, 2, 2, 64, 64, "f32")
    x["q"][0, 0] = 0.0
    x["q"][0, 1] *= 2.0 ** 40
    x["q"][0, 2] *= 2.0 ** -40
    check(x, {n: t.cuda() for n, t in x.items()})


def test_differences():
    """The weights' and the inputs' gradients of the kernels' own forward pass, in fp32."""
    x = make(2, 9, 3, 2, 32, 32, "f32")
    c = {n: t.cuda() for n, t in x.items()}
    g = linattn.prism_qk_norm_rope_backward(c["q"], c["k"], c["table"], c["dq"], c["dk"], q_weight=c["qw"], k_weight=c["kw"])
    gen = torch.Generator(device="cuda").manual_seed(1)
    for n, m in (("q", "q"), ("k", "k"), ("qw", "q_weight"), ("kw", "k_weight")):
        d = torch.randn(c[n].shape, generator=gen, device="cuda")
        e = 2.0 ** -8

        def value(f):
            y = dict(c)
            y[n] = c[n] + f * e * d
            a, b = linattn.prism_qk_norm_rope(y["q"], y["k"], y["table"], q_weight=y["qw"], k_weight=y["kw"])
            return (a.double() * c["dq"].double()).sum() + (b.double() * c["dk"].double()).sum()

        slope = ((value(1.0) - value(-1.0)) / (2 * e)).item()
        want = (g[m].double() * d.double()).sum().item()
        size = (g[m].double().norm() * d.double().norm()).item()
        # truncation e^2 / 6 of third derivatives (a few dozen times the size), rounding u / e
        assert abs(slope - want) <= (64 * e * e + 64 * lo.U / e) * size, (n, slope, want)


def test_streams_and_graphs():
    x = make(2, 200, 4, 4, 128, 128, "bf16")
    c = {n: t.cuda() for n, t in x.items()}
    how = dict(q_weight=c["qw"], k_weight=c["kw"])
    a = linattn.prism_qk_norm_rope_backward(c["q"], c["k"], c["table"], c["dq"], c["dk"], **how)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = linattn.prism_qk_norm_rope_backward(c["q"], c["k"], c["table"], c["dq"], c["dk"], **how)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d = linattn.prism_qk_norm_rope_backward(c["q"], c["k"], c["table"], c["dq"], c["dk"], **how)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) and torch.equal(a[n], d[n]) for n in a)
