"""The linear attention binding's memory on streams (CPU): an allocator and a library that only take notes.

A caching allocator hands freed memory out again to work on the stream that it came from, and
waits for no other stream unless the tensor was recorded on it.  So whatever a call's kernels
use must come from the call's stream or be recorded there, and an output that comes from the
call's stream must be recorded on the one that its caller reads it on."""
import contextlib
import types

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn, prism


class Stream:
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", device)


class OnGpu(torch.Tensor):
    """A CPU tensor that says that it lies on a GPU, and on which streams it was noted."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = property(lambda t: True)
    device = property(lambda t: torch.device("cuda", t.index))
    index, home, noted = 0, 0, ()

    def get_device(self):
        return self.index

    def record_stream(self, s):
        self.noted = (*self.noted, s.cuda_stream)


def gpu(t, home=0, index=0):
    t = t.as_subclass(OnGpu)
    t.home, t.index, t.noted = home, index, ()
    return t


class World:
    """Torch's streams and allocations, and the library, as the binding sees them."""

    def __init__(self, monkeypatch, handle=0):
        self.now, self.made, self.calls, self.devices = Stream(handle), [], [], []
        linattn_torch = types.SimpleNamespace(**{n: getattr(torch, n) for n in (
            "Size", "float32", "bfloat16", "uint8", "int32")})
        linattn_torch.empty = self.empty
        linattn_torch.empty_like = lambda t: self.empty(t.shape, dtype=t.dtype, device=t.device)
        linattn_torch._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: self.now.cuda_stream,
                                                 _cuda_getDevice=lambda: self.devices[-1] if self.devices else 0)
        linattn_torch.cuda = types.SimpleNamespace(stream=self.on, current_stream=lambda d=None: self.now, device=self.at)
        monkeypatch.setattr(linattn, "torch", linattn_torch)
        monkeypatch.setattr(linattn, "load", lambda: self)
        for c in (linattn._rope_dims, linattn._linattn_dims, linattn._decode_dims):
            c.cache_clear()

    @contextlib.contextmanager
    def on(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    @contextlib.contextmanager
    def at(self, d):
        self.devices.append(d if isinstance(d, int) else d.index)
        yield
        self.devices.pop()

    def empty(self, shape, dtype, device):
        t = gpu(torch.empty(shape, dtype=dtype), self.now.cuda_stream, device.index)
        self.made.append(t)
        return t

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda dims: 4096
        return lambda *a: self.calls.append((name, a, self.devices[-1] if self.devices else 0)) or 0


@pytest.fixture
def world(monkeypatch):
    yield World(monkeypatch)
    for c in (linattn._rope_dims, linattn._linattn_dims, linattn._decode_dims):
        c.cache_clear()


def operands():
    bf = lambda *s: gpu(torch.zeros(s, dtype=torch.bfloat16))  # noqa: E731
    f = lambda *s: gpu(torch.zeros(s))  # noqa: E731
    i = lambda *s: gpu(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    x = dict(q=bf(2, 8, 2, 16), k=bf(2, 8, 2, 16), v=bf(2, 8, 2, 16), ld=f(2), do=bf(2, 8, 2, 16), s=f(2, 2, 16, 16),
             ds=f(2, 2, 16, 16), lens=i(2), table=f(8, 16), w=f(16), pos=i(2, 8), q1=bf(2, 2, 16), slots=i(2))
    return types.SimpleNamespace(**x)


CALLS = {
    "rope": lambda x, **k: linattn.prism_qk_norm_rope(x.q, x.k, x.table, q_weight=x.w, k_weight=x.w, positions=x.pos,
                                                      seq_lens=x.lens, **k),
    "rope_backward": lambda x, **k: linattn.prism_qk_norm_rope_backward(
        x.q, x.k, x.table, x.do, x.do, q_weight=x.w, k_weight=x.w, positions=x.pos, seq_lens=x.lens, **k),
    "forward": lambda x, **k: linattn.prism_linattn_forward(x.q, x.k, x.v, x.ld, initial_state=x.s, seq_lens=x.lens, **k),
    "backward": lambda x, **k: linattn.prism_linattn_backward(x.q, x.k, x.v, x.ld, x.do, initial_state=x.s,
                                                              d_final_state=x.ds, seq_lens=x.lens, **k),
    "decode": lambda x, **k: linattn.prism_linattn_decode_step(x.q1, x.q1, x.q1, x.ld, x.s, slots=x.slots, **k),
}


def pointers(args):
    return {a for a in args if isinstance(a, int) and a > 1 << 16}


@pytest.mark.parametrize("call", CALLS)
def test_nothing_is_handed_out_while_its_kernels_run(world, call):
    x, side = operands(), Stream(0x51de)
    got = CALLS[call](x, stream=side)
    (_, args, _), = world.calls
    assert args[-1] == side.cuda_stream
    used = [t for t in (*world.made, *vars(x).values()) if t.data_ptr() in pointers(args)]
    assert len(used) >= 5 and all(t.data_ptr() in pointers(args) for t in world.made)
    for t in used:
        assert t.home == side.cuda_stream or side.cuda_stream in t.noted, "memory that another stream may get"
    outs = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    for t in outs:
        assert t.home == 0 or 0 in t.noted, "an output that its caller's stream may lose"


@pytest.mark.parametrize("call", CALLS)
def test_memory_that_is_passed_in(world, call):
    """Preallocated outputs and workspaces belong to the caller's stream: they are recorded too."""
    x, side = operands(), Stream(0x51de)
    first = CALLS[call](x)
    mine = [*world.made]
    assert all(t.noted == () for t in (*mine, *vars(x).values())), "on the current stream there is nothing to record"
    world.made.clear()
    more = {"rope": lambda: dict(q_out=first[0], k_out=first[1]), "rope_backward": lambda: dict(grads=first, workspace=mine[-1]),
            "forward": lambda: dict(out=first[0], final_state=first[1], workspace=mine[-1]),
            "backward": lambda: dict(grads=first, workspace=mine[-1]), "decode": lambda: dict(out=first)}[call]()
    CALLS[call](x, stream=side, **more)
    assert not world.made and all(side.cuda_stream in t.noted for t in mine)


@pytest.mark.parametrize("call", CALLS)
def test_the_current_stream_by_name(world, call):
    x = operands()
    CALLS[call](x, stream=Stream(0))
    assert world.calls[0][1][-1] == 0 and all(t.noted == () and t.home == 0 for t in world.made)


OPERANDS = {"rope": ("k", "table", "w", "pos", "lens"), "rope_backward": ("k", "table", "w", "pos", "lens", "do"),
            "forward": ("k", "v", "ld", "s", "lens"), "backward": ("k", "v", "ld", "do", "s", "ds", "lens"),
            "decode": ("ld", "s", "slots")}


@pytest.mark.parametrize("call", CALLS)
def test_one_device(world, call):
    """An operand on another device, or on none, is refused before anything is launched."""
    for n in OPERANDS[call]:
        for wrong in (lambda t: gpu(t, index=1), lambda t: t.as_subclass(torch.Tensor)):
            x = operands()
            setattr(x, n, wrong(getattr(x, n)))
            for side in (None, Stream(0x51de)):
                with pytest.raises(prism.PrismError):
                    CALLS[call](x, stream=side)
    with pytest.raises(prism.PrismError):
        CALLS[call](operands(), stream=Stream(0x51de, device=1))
    assert not world.calls


@pytest.mark.parametrize("call", CALLS)
def test_the_tensors_device_is_made_current(world, call):
    """With all tensors on device 1 while device 0 is current, the library is called with 1 current."""
    x = operands()
    for n, t in vars(x).items():
        t.index = 1
    CALLS[call](x)
    (_, _, device), = world.calls
    assert device == 1 and not world.devices


@pytest.mark.parametrize("call", ["rope_backward", "forward", "backward"])
def test_workspaces(world, call):
    """A workspace that is elsewhere, or smaller than its element count says, is refused; its size is in bytes."""
    plain = torch.zeros(8192, dtype=torch.uint8)
    for wrong in (plain, gpu(plain.clone(), index=1), gpu(plain.clone()[::2]), gpu(plain[:1].clone().expand(8192))):
        with pytest.raises(prism.PrismError):
            CALLS[call](operands(), workspace=wrong)
    assert not world.calls
    CALLS[call](operands(), workspace=gpu(torch.zeros(1024)))
    assert 4096 in world.calls[0][1]
