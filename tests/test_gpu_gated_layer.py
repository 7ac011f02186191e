"""A gated recurrent layer out of the library's operators, as it is used: layer norm, one projection of values and
gates, the recurrence, a projection back; trained, then served by prompt and single tokens."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated
from tests import gated_oracle as go

pytestmark = pytest.mark.gpu


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, lens):
        ctx.save_for_backward(x, w, b, lens)
        return gated.prism_layer_norm(x, weight=w, bias=b, seq_lens=lens)

    @staticmethod
    def backward(ctx, dy):
        x, w, b, lens = ctx.saved_tensors
        g = gated.prism_layer_norm_backward(x, dy.contiguous(), weight=w, bias=b, seq_lens=lens)
        return g["x"], g["weight"], g["bias"], None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, f, i, s0, lens):
        states = gated.gated_scan_states(x)
        out, final = gated.prism_gated_scan_forward(x, f, input_gate=i, initial_state=s0, states=states, seq_lens=lens)
        ctx.save_for_backward(x, f, i, states, lens)
        return out, final

    @staticmethod
    def backward(ctx, d_out, d_final):
        x, f, i, states, lens = ctx.saved_tensors
        g = gated.prism_gated_scan_backward(x, f, states, d_out.contiguous(), input_gate=i, d_final_state=d_final.contiguous(),
                                            seq_lens=lens, want_initial_state=True)
        return g["x"], g["forget"], g["input_gate"], g["initial_state"], None


def make(B, T, width, D):
    g = torch.Generator().manual_seed(T)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = dict(x=n(B, T, width), w=1 + 0.2 * n(width), b=0.2 * n(width), up=n(3 * D, width) / width ** 0.5,
             down=n(width, D) / D ** 0.5, s0=n(B, D))
    return p, n(B, T, width), n(B, D)


def layer(p, lens=None):
    B, T, _ = p["x"].shape
    D = p["down"].shape[1]
    y = Norm.apply(p["x"], p["w"], p["b"], lens)
    u = (y @ p["up"].T).view(B, T, 3, D)
    h, final = Scan.apply(u[:, :, 0], u[:, :, 1], u[:, :, 2], p["s0"], lens)
    return p["x"] + h @ p["down"].T, final


def exact(p, lens):
    """The same in fp64 out of torch operations, differentiable."""
    B, T, _ = p["x"].shape
    D = p["down"].shape[1]
    y, _ = go.layer_norm(p["x"], p["w"], p["b"], 1e-5, lens)
    u = (y @ p["up"].T).view(B, T, 3, D)
    s = go.scan(u[:, :, 0], u[:, :, 1], u[:, :, 2], p["s0"], lens)
    return p["x"] + s["out"] @ p["down"].T, s["final"]


@pytest.mark.parametrize("B,T,width,D", [(3, 150, 72, 40), (1, 300, 264, 64)])
def test_gradients_of_a_layer(B, T, width, D):
    """In fp32, where each operator is off by a few 1e-6 of its magnitudes at most; a layer multiplies that by the norms
    of its two projections, about 4 each way: 1e-4 of the largest gradient is beyond what roundings give."""
    p, d, ds = make(B, T, width, D)
    lens = torch.tensor([T, T // 3, 0][:B])
    live = (torch.arange(T)[None] < lens[:, None])[..., None]
    want = {n: t.double().requires_grad_() for n, t in p.items()}
    out, final = exact(want, lens)
    (torch.where(live, out * d, 0.0).sum() + (final * ds).sum()).backward()
    got = {n: t.cuda().requires_grad_() for n, t in p.items()}
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        o, f = layer(got, lens.cuda().int())
        (torch.where(live.cuda(), o * d.cuda(), 0.0).sum() + (f * ds.cuda()).sum()).backward()
    finally:
        torch.backends.cuda.matmul.allow_tf32 = before
    assert (torch.where(live, o.detach().cpu() - out.detach(), 0.0).abs().max() <= 1e-4 * out.abs().max()).item()
    assert ((f.detach().cpu() - final.detach()).abs().max() <= 1e-4 * final.abs().max()).item()
    for n in p:
        a, b = got[n].grad.double().cpu(), want[n].grad
        assert (a - b).abs().max() <= 1e-4 * b.abs().max(), n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_then_single_tokens(dtype):
    """The same bits as the whole sequence at once for the norm, and for the recurrence in one tile."""
    p, _, _ = make(4, 40, 136, 64)
    c = {n: (t.cuda() if n in ("w", "b", "s0") else t.cuda().to(dtype)) for n, t in p.items()}

    def up(x):
        y = gated.prism_layer_norm(x, weight=c["w"], bias=c["b"])
        return y, (y.double() @ c["up"].double().T).to(dtype).unflatten(-1, (3, 64))

    y, u = up(c["x"])
    whole, last = gated.prism_gated_scan_forward(u[:, :, 0], u[:, :, 1], input_gate=u[:, :, 2], initial_state=c["s0"])
    y0, u0 = up(c["x"][:, :30])
    assert torch.equal(y0, y[:, :30])
    _, state = gated.prism_gated_scan_forward(u0[:, :, 0], u0[:, :, 1], input_gate=u0[:, :, 2], initial_state=c["s0"])
    for t in range(30, 40):
        y1, u1 = up(c["x"][:, t:t + 1])
        assert torch.equal(y1[:, 0], y[:, t])
        out = gated.prism_gated_scan_decode_step(u1[:, 0, 0], u1[:, 0, 1], state, input_gate=u1[:, 0, 2])
        tol = 2 * go.ROUND[dtype] * whole[:, t].abs().double() + 64 * go.U * (1 + whole.abs().max().double())
        assert ((out.double() - whole[:, t].double()).abs() <= tol).all()
    assert ((state - last).abs() <= 64 * go.U * (1 + last.abs())).all()
    assert gated.gated_status() == 0


def test_training_step_in_a_graph():
    """Forward and backward captured together and replayed."""
    p, d, ds = make(2, 200, 72, 64)
    c = {n: t.cuda() for n, t in p.items()}
    dc, sc = d.cuda(), ds.cuda()

    def step():
        y = gated.prism_layer_norm(c["x"], weight=c["w"], bias=c["b"])
        u = (y @ c["up"].T).view(2, 200, 3, 64)
        st = gated.gated_scan_states(u[:, :, 0])
        h, f = gated.prism_gated_scan_forward(u[:, :, 0], u[:, :, 1], input_gate=u[:, :, 2], initial_state=c["s0"], states=st)
        g = gated.prism_gated_scan_backward(u[:, :, 0], u[:, :, 1], st, (dc @ c["down"]), input_gate=u[:, :, 2], d_final_state=sc)
        du = torch.stack([g["x"], g["forget"], g["input_gate"]], 2).flatten(2)
        n = gated.prism_layer_norm_backward(c["x"], du @ c["up"], weight=c["w"], bias=c["b"])
        return h, f, n["x"], n["weight"], n["bias"]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(3):
        c["x"].add_(0.25 * k)
        want = step()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
