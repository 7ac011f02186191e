"""Calls of the linear attention layer on a stream beside the current one, with nothing waiting in between:
memory that is freed and allocated again meanwhile is not theirs.  Bit for bit against the same
calls one after another."""
import ctypes

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn

pytestmark = pytest.mark.gpu


def make(seed, B, T, H, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = {m: n(B, T, H, D).to(dtype) for m in ("v", "do")}
    x.update({m: torch.nn.functional.normalize(n(B, T, H, D), dim=-1).to(dtype) for m in ("q", "k")})
    x.update(ld=-torch.exp(-2 - 4 * torch.rand(H, generator=g, device="cuda")), s=n(B, H, D, D), ds=n(B, H, D, D),
             w=n(D), table=n(T, D))
    return x


def forward(x, **k):
    return linattn.prism_linattn_forward(x["q"], x["k"], x["v"], x["ld"], initial_state=x["s"], **k)


def backward(x, **k):
    g = linattn.prism_linattn_backward(x["q"], x["k"], x["v"], x["ld"], x["do"], initial_state=x["s"],
                                       d_final_state=x["ds"], **k)
    return tuple(g[n] for n in ("q", "k", "v", "initial_state"))


def norm_backward(x, **k):
    g = linattn.prism_qk_norm_rope_backward(x["q"], x["k"], x["table"], x["do"], x["v"], q_weight=x["w"], k_weight=x["w"], **k)
    return tuple(g[n] for n in ("q", "k", "q_weight", "k_weight"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("call", [forward, backward, norm_backward])
def test_calls_on_two_streams(call, dtype):
    sets = [make(i, 1, 3000, 2, 64, dtype) for i in range(4)]
    x = sets[0]
    if call is not norm_backward:                    # the sequence is cut, so the call needs its workspace
        _, dims, nbytes = linattn._linattn_dims(x["q"].shape, dtype, 1.0, *[x[n].stride() for n in "qkv"], None)
        assert nbytes > 0 and nbytes == linattn.load().prism_linattn_workspace_bytes(ctypes.c_void_p(dims))
    want = [tuple(t.clone() for t in call(x)) for x in sets]
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []
    for i in range(12):
        got.append((i % 4, call(sets[i % 4])))
        torch.full((1 << 21,), float("nan"), device="cuda")            # what the call freed, written again
        got.append(((i + 1) % 4, call(sets[(i + 1) % 4], stream=side)))
        for n in (1 << 17, 1 << 19, 1 << 21):
            torch.full((n,), float("nan"), device="cuda")
        if i % 3 == 2:                               # outputs of both streams go back to the allocator
            torch.cuda.current_stream().wait_stream(side)
            for j, outs in got:
                assert all(torch.equal(a, b) for a, b in zip(outs, want[j]))
            got.clear()
    torch.cuda.synchronize()
    assert linattn.linattn_status() == 0


def test_inputs_dropped_at_once():
    """An input that only the call holds stays until its kernels are done."""
    x = make(5, 1, 3000, 2, 64, torch.bfloat16)
    want = forward(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(8):
        y = {n: t.clone() for n, t in x.items()}
        side.wait_stream(torch.cuda.current_stream())
        out, state = forward(y, stream=side)
        y.clear()
        for n in ("q", "k", "v"):
            torch.full_like(x[n], float("nan"))
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want[0]) and torch.equal(state, want[1])
