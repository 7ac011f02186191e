"""The mixer binding's memory on streams (CPU), with the noted tensors of test_linattn_streams: what a call on
a stream beside the current one allocates comes from that stream, and what it uses is recorded
where it is used, so that the caching allocator hands none of it out while kernels use it."""
import contextlib
import types

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import prism
from tests.test_linattn_streams import Stream, gpu

B, T, H, D, L, W = 2, 64, 2, 32, 2, 4


class World:
    def __init__(self, monkeypatch):
        self.now, self.made, self.calls = Stream(0), [], []
        names = ("float32", "bfloat16", "uint8", "dtype", "Tensor")
        fake = types.SimpleNamespace(**{n: getattr(torch, n) for n in names}, empty=self.empty,
                                     empty_like=lambda t: self.empty(t.shape, dtype=t.dtype, device=t.device))
        fake._C = types.SimpleNamespace(_cuda_getDevice=lambda: 0)
        fake.cuda = types.SimpleNamespace(stream=self.on, current_stream=lambda d=None: self.now)
        monkeypatch.setattr(prism, "torch", fake)
        monkeypatch.setattr(prism, "load", lambda: self)

    @contextlib.contextmanager
    def on(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    def empty(self, shape, dtype, device):
        t = gpu(torch.empty(shape, dtype=dtype), self.now.cuda_stream, device.index)
        self.made.append(t)
        return t

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda dims: 4096
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def operands():
    bf = lambda *s: gpu(torch.zeros(s, dtype=torch.bfloat16))  # noqa: E731
    f = lambda *s: gpu(torch.zeros(s))  # noqa: E731
    x = dict(q=bf(B, T, H, D), k=bf(B, T, H, D), v=bf(B, T, H, D), la=f(B, T, H), be=f(B, T, H), cw=f(H, W, D), Wk=f(H, L, D, D),
             Wp=f(H, L, D, D), wb=f(H, L, D), s=f(B, H, D, D), ds=f(B, H, D, D), do=f(B, T, H, D), vh=bf(B, H, W, D),
             lens=gpu(torch.zeros(B, dtype=torch.int32)), ws=gpu(torch.zeros(4096, dtype=torch.uint8)), q1=bf(B, H, D),
             la1=f(B, H), be1=f(B, H))
    return types.SimpleNamespace(**x)


def mixer(x):
    return x.q, x.k, x.v, x.la, x.be, x.cw, x.Wk, x.Wp, x.wb, L


CALLS = {
    "forward": lambda x, **k: prism.prism_forward(*mixer(x), 64, seq_lens=x.lens, **k),
    "forward_from": lambda x, **k: prism.prism_forward_from(*mixer(x), 64, initial_state=x.s, v_hist=x.vh, seq_lens=x.lens, **k),
    "forward_static": lambda x, **k: prism.prism_forward_static(*mixer(x), 64, seq_lens=x.lens, **k),
    "backward": lambda x, **k: prism.prism_backward(*mixer(x), x.do, d_final_state=x.ds, seq_lens=x.lens, **k),
    "decode": lambda x, **k: prism.prism_decode_step(x.q1, x.q1, x.q1, x.la1, x.be1, x.cw, x.Wk, x.Wp, x.wb, L, x.s, x.vh, **k),
    "prepare": lambda x, **k: prism.prism_prepare(*mixer(x), 64, x.ws, seq_lens=x.lens, **k),
    "scan": lambda x, **k: prism.prism_scan(x.q, x.k, x.v, x.la, x.be, L, 64, W, x.ws, seq_lens=x.lens, **k),
    "activation": lambda x, **k: prism.debug_activation(x.s, **k),
}


@pytest.mark.parametrize("call", CALLS)
def test_nothing_is_handed_out_while_its_kernels_run(world, call):
    x, side = operands(), Stream(0x51de)
    got = CALLS[call](x, stream=side)
    (_, args), = world.calls
    assert args[-1] == side.cuda_stream
    known = {a for a in args if isinstance(a, int) and a > 1 << 16}
    used = [t for t in (*world.made, *vars(x).values()) if t.data_ptr() in known]
    assert len(used) >= 2 and all(t.data_ptr() in known for t in world.made)
    for t in used:
        assert t.home == side.cuda_stream or side.cuda_stream in t.noted, "memory that another stream may get"
    outs = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    for t in outs:
        assert t is None or t.home == 0 or 0 in t.noted, "an output that its caller's stream may lose"


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [None, Stream(0)])
def test_the_current_stream(world, call, stream):
    x = operands()
    CALLS[call](x, stream=stream)
    assert world.calls[0][1][-1] == 0
    assert all(t.noted == () and t.home == 0 for t in (*world.made, *vars(x).values()))


@pytest.mark.parametrize("call", CALLS)
def test_the_current_device(world, call):
    """The library launches on the current device: a tensor of another one is refused before that."""
    for n in ("q", "q1", "s", "cw", "lens", "ws"):
        x = operands()
        getattr(x, n).index = 1
        before = len(world.calls)
        try:
            CALLS[call](x)
        except prism.PrismError:
            assert len(world.calls) == before
        else:
            known = {a for a in world.calls[-1][1] if isinstance(a, int) and a > 1 << 16}
            assert getattr(x, n).data_ptr() not in known, "launched with another device's memory"
