"""The linear attention layer's calls captured in CUDA graphs and replayed, as a serving loop does: the
same bits as the calls themselves, on new inputs in the same places."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn

pytestmark = pytest.mark.gpu


def capture(f):
    """f's outputs in a graph, warmed up before."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


def draw(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("slotted", [False, True])
def test_single_tokens(slotted, dtype):
    B, H, D, N = 8, 4, 64, 11
    q, k, v = (draw((B, H, D), dtype, i) for i in range(3))
    ld, pool = -torch.rand(H, device="cuda"), draw((N, H, D, D), torch.float32, 4)
    slots = torch.randperm(N, device="cuda")[:B].to(torch.int32) if slotted else None
    g, out = capture(lambda: linattn.prism_linattn_decode_step(q, k, v, ld, pool, slots=slots))
    for step in range(3):
        for i, t in enumerate((q, k, v)):
            t.copy_(draw(t.shape, dtype, 10 * step + i))
        other = pool.clone()
        want = linattn.prism_linattn_decode_step(q, k, v, ld, other, slots=slots)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, other)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_and_rotation(dtype):
    q, k = draw((8, 1, 16, 128), dtype, 0), draw((8, 1, 4, 128), dtype, 1)
    w, table = draw((128,), torch.float32, 2), draw((64, 128), torch.float32, 3)
    pos = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    g, out = capture(lambda: linattn.prism_qk_norm_rope(q, k, table, q_weight=w, positions=pos))
    for step in range(3):
        q.copy_(draw(q.shape, dtype, 5 + step))
        pos.fill_(step * 7)
        want = linattn.prism_qk_norm_rope(q, k, table, q_weight=w, positions=pos)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_sequence_in_runs(dtype):
    """Two launches, the second one's set-up beside the first."""
    q, k, v, do = (draw((1, 2000, 2, 64), dtype, i) for i in range(4))
    ld, s0 = torch.tensor([-1e-3, -0.1], device="cuda"), draw((1, 2, 64, 64), torch.float32, 4)
    k.div_(8)
    f = capture(lambda: linattn.prism_linattn_forward(q, k, v, ld, initial_state=s0))
    b = capture(lambda: linattn.prism_linattn_backward(q, k, v, ld, do, initial_state=s0))
    for step in range(3):
        v.copy_(draw(v.shape, dtype, 9 + step))
        want = linattn.prism_linattn_forward(q, k, v, ld, initial_state=s0)
        grads = linattn.prism_linattn_backward(q, k, v, ld, do, initial_state=s0)
        f[0].replay()
        b[0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(f[1], want)) and all(torch.equal(b[1][n], grads[n]) for n in grads)
    assert linattn.linattn_status() == 0
