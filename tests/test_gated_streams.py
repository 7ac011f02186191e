"""The gated layer's binding (CPU): which stream's memory a call uses, devices, workspaces and settings, with the
allocator and library of test_linattn_streams that only take notes."""
import types

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated, linattn, prism
from tests.test_linattn_streams import Stream, World, gpu, pointers

CACHES = (gated._norm_dims, gated._gated_dims, gated._decode_dims)


@pytest.fixture
def world(monkeypatch):
    w = World(monkeypatch)
    monkeypatch.setattr(gated, "torch", linattn.torch)
    monkeypatch.setattr(gated, "load", lambda: w)
    for c in CACHES:
        c.cache_clear()
    yield w
    for c in CACHES:
        c.cache_clear()


def operands():
    bf = lambda *s: gpu(torch.zeros(s, dtype=torch.bfloat16))  # noqa: E731
    f = lambda *s: gpu(torch.zeros(s))  # noqa: E731
    i = lambda *s: gpu(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    return types.SimpleNamespace(x=bf(2, 200, 16), f=bf(2, 200, 16), i=bf(2, 200, 16), do=bf(2, 200, 16), s=f(2, 16), ds=f(2, 16),
                                 st=f(2, 4, 16), lens=i(2), w=f(16), b=f(16), x1=bf(2, 16), f1=bf(2, 16), i1=bf(2, 16),
                                 slots=i(2))


CALLS = {
    "norm": lambda x, **k: gated.prism_layer_norm(x.x, weight=x.w, bias=x.b, seq_lens=x.lens, **k),
    "norm_backward": lambda x, **k: gated.prism_layer_norm_backward(x.x, x.do, weight=x.w, bias=x.b, seq_lens=x.lens, **k),
    "forward": lambda x, **k: gated.prism_gated_scan_forward(x.x, x.f, input_gate=x.i, initial_state=x.s, states=x.st,
                                                             seq_lens=x.lens, **k),
    "backward": lambda x, **k: gated.prism_gated_scan_backward(x.x, x.f, x.st, x.do, input_gate=x.i, d_final_state=x.ds,
                                                               seq_lens=x.lens, want_initial_state=True, **k),
    "decode": lambda x, **k: gated.prism_gated_scan_decode_step(x.x1, x.f1, x.s, input_gate=x.i1, slots=x.slots, **k),
}


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
    # the norm's bias is only checked on the way back
    outs = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    for t in outs:
        assert t.home == 0 or 0 in t.noted, "an output that its caller's stream may lose"


@pytest.mark.parametrize("call", CALLS)
def test_memory_that_is_passed_in(world, call):
    x, side = operands(), Stream(0x51de)
    first = CALLS[call](x)
    mine = [*world.made]
    assert all(t.noted == () for t in (*mine, *vars(x).values())), "on the current stream there is nothing to record"
    world.made.clear()
    more = {"norm": lambda: dict(out=first), "norm_backward": lambda: dict(grads=first, workspace=mine[-1]),
            "forward": lambda: dict(out=first[0], final_state=first[1], workspace=mine[-1]),
            "backward": lambda: dict(grads=first, workspace=mine[-1]), "decode": lambda: dict(out=first)}[call]()
    CALLS[call](x, stream=side, **more)
    assert not world.made and all(side.cuda_stream in t.noted for t in mine)


@pytest.mark.parametrize("call", CALLS)
def test_the_current_stream_by_name(world, call):
    CALLS[call](operands(), stream=Stream(0))
    assert world.calls[0][1][-1] == 0 and all(t.noted == () and t.home == 0 for t in world.made)


OPERANDS = {"norm": ("w", "b", "lens"), "norm_backward": ("w", "b", "lens", "do"), "forward": ("f", "i", "s", "st", "lens"),
            "backward": ("f", "i", "st", "do", "ds", "lens"), "decode": ("f1", "i1", "s", "slots")}


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
    assert not world.calls


@pytest.mark.parametrize("call", CALLS)
def test_another_device(world, call):
    """All of them on a device that is not the current one: it is made current for the call."""
    x = types.SimpleNamespace(**{n: gpu(t, index=1) for n, t in vars(operands()).items()})
    CALLS[call](x)
    assert world.calls[0][2] == 1 and all(t.device.index == 1 for t in world.made)
    with pytest.raises(prism.PrismError):
        CALLS[call](x, stream=Stream(0x51de, 0))


@pytest.mark.parametrize("call", ["norm_backward", "forward", "backward"])
def test_workspaces(world, call):
    x = operands()
    for bad in (gpu(torch.zeros(64, dtype=torch.uint8), index=1), torch.zeros(64, dtype=torch.uint8),
                gpu(torch.zeros(64, 2, dtype=torch.uint8)[:, 0])):
        with pytest.raises(prism.PrismError):
            CALLS[call](x, workspace=bad)
    room = gpu(torch.zeros(4096, dtype=torch.uint8))
    CALLS[call](x, workspace=room)
    assert room.data_ptr() in world.calls[-1][1] and 4096 in world.calls[-1][1]


@pytest.mark.parametrize("holder", [lambda v: torch.tensor(v), float])
def test_settings_count_by_their_value_at_the_call(world, holder):
    x, eps = operands(), holder(0.5)
    for value in (0.5, 2.0):
        if isinstance(eps, torch.Tensor):
            eps.fill_(value)
        else:
            eps = value
        gated.prism_layer_norm(x.x, eps=eps)
        assert gated.LayerNormDims.from_address(world.calls[-1][1][0]).eps == value
        gated.prism_layer_norm_backward(x.x, x.do, eps=eps)
        assert gated.LayerNormDims.from_address(world.calls[-1][1][0]).eps == value


def test_what_is_not_wanted_is_not_made(world):
    x = operands()
    out, state = gated.prism_gated_scan_forward(x.x, x.f, want_state=False)
    assert state is None and len(world.made) == 2                    # out and the workspace
    g = gated.prism_gated_scan_backward(x.x, x.f, x.st, x.do)
    assert g["input_gate"] is None and g["initial_state"] is None
    g = gated.prism_layer_norm_backward(x.x, x.do)
    assert g["weight"] is None and g["bias"] is None and world.calls[-1][1][-3] is None     # no workspace either
