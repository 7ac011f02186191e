"""The gated layer's calls on two streams, captured in graphs, and on workspaces that are used again."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated

pytestmark = pytest.mark.gpu


def make(seed, B, T, D, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = {m: n(B, T, D).to(dtype) for m in ("x", "i", "do")}
    x.update(f=(2 + n(B, T, D)).to(dtype), s=n(B, D), ds=n(B, D), w=n(D), b=n(D))
    x["st"] = gated.gated_scan_states(x["x"])
    gated.prism_gated_scan_forward(x["x"], x["f"], input_gate=x["i"], initial_state=x["s"], states=x["st"])
    return x


def forward(x, **k):
    return gated.prism_gated_scan_forward(x["x"], x["f"], input_gate=x["i"], initial_state=x["s"], **k)


def backward(x, **k):
    g = gated.prism_gated_scan_backward(x["x"], x["f"], x["st"], x["do"], input_gate=x["i"], d_final_state=x["ds"],
                                        want_initial_state=True, **k)
    return tuple(g[n] for n in ("x", "forget", "input_gate", "initial_state"))


def norm(x, **k):
    return (gated.prism_layer_norm(x["x"], weight=x["w"], bias=x["b"], **k),)


def norm_backward(x, **k):
    g = gated.prism_layer_norm_backward(x["x"], x["do"], weight=x["w"], bias=x["b"], **k)
    return tuple(g[n] for n in ("x", "weight", "bias"))


CALLS = [forward, backward, norm, norm_backward]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("call", CALLS)
def test_calls_on_two_streams(call, dtype):
    """Side by side, tiles that wait for tiles among them; memory that is freed meanwhile is not theirs."""
    sets = [make(i, 2, 1500, 520, dtype) for i in range(4)]
    want = [tuple(t.clone() for t in call(x)) for x in sets]
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []
    for i in range(12):
        got.append((i % 4, call(sets[i % 4])))
        torch.full((1 << 21,), float("nan"), device="cuda")            # what the call freed, written again
        got.append(((i + 1) % 4, call(sets[(i + 1) % 4], stream=side)))
        for n in (1 << 17, 1 << 19, 1 << 21):
            torch.full((n,), float("nan"), device="cuda")
        if i % 3 == 2:
            torch.cuda.current_stream().wait_stream(side)
            assert all(same(outs, want[j]) for j, outs in got)
            got.clear()
    torch.cuda.synchronize()
    assert gated.gated_status() == 0


def capture(f):
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("call", CALLS)
def test_captured_and_replayed(call, dtype):
    """Again and again on new inputs in the same places: nothing is left from the replay before."""
    x, other = make(1, 2, 700, 264, dtype), make(2, 2, 700, 264, dtype)
    g, out = capture(lambda: call(x))
    for step in range(4):
        y = make(5 + step, 2, 700, 264, dtype)
        for n in x:
            x[n].copy_(y[n])
        want = call(y)
        for _ in range(2):
            g.replay()
            call(other)                                                # eager calls in between
            torch.cuda.synchronize()
            assert same(out, want)
    assert gated.gated_status() == 0


@pytest.mark.parametrize("slotted", [False, True])
def test_single_tokens_captured(slotted):
    x, N = make(3, 8, 1, 264), 11
    pool = torch.randn(N, 264, device="cuda")
    slots = torch.randperm(N, device="cuda")[:8].to(torch.int32) if slotted else None
    a = [x[n][:, 0] for n in ("x", "f", "i")]
    g, out = capture(lambda: gated.prism_gated_scan_decode_step(a[0], a[1], pool, input_gate=a[2], slots=slots))
    for step in range(3):
        a[0].copy_(torch.randn(8, 264, device="cuda"))
        other = pool.clone()
        want = gated.prism_gated_scan_decode_step(a[0], a[1], other, input_gate=a[2], slots=slots)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, other)


def test_two_graphs_on_one_workspace():
    """One after the other: each call clears what it needs."""
    x, y = make(1, 2, 900, 136), make(2, 3, 500, 72)
    room = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    a, b = capture(lambda: forward(x, workspace=room)), capture(lambda: backward(y, workspace=room))
    wa, wb = forward(x), backward(y)
    for _ in range(3):
        for t in (*a[1], *b[1]):
            t.fill_(float("nan"))
        a[0].replay()
        b[0].replay()
        torch.cuda.synchronize()
        assert same(a[1], wa) and same(b[1], wb)
        room.fill_(7)
    assert gated.gated_status() == 0


def test_inputs_dropped_at_once():
    x = make(5, 1, 3000, 64)
    want = forward(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(8):
        y = {n: t.clone() for n, t in x.items()}
        side.wait_stream(torch.cuda.current_stream())
        got = forward(y, stream=side)
        y.clear()
        for n in ("x", "f", "i"):
            torch.full_like(x[n], float("nan"))
        torch.cuda.current_stream().wait_stream(side)
        assert same(got, want)
