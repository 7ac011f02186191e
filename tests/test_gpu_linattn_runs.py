"""Linear attention where the state matters: heads that hardly forget or do not forget at all, over
sequences cut into runs and over many chunks of one run, and states given apart.

Bounds of linattn_oracle; test_linattn_bounds shows on the CPU that they see a run or a state that is lost.
"""
import ctypes

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn
from tests import linattn_oracle as lo
from tests.test_gpu_linattn import TYPES, check_backward, check_forward, gpu, make

pytestmark = pytest.mark.gpu
SLOW = torch.tensor([0.0, -1e-4, -2e-3])


def runs(x):
    """Runs that a sequence of these inputs is cut into, forward and backward."""
    B, T, H, D = x["q"].shape
    d = linattn.LinattnDims(B=B, T=T, H=H, d=D, dtype=1 if x["q"].dtype == torch.bfloat16 else 0, scale=1.0)
    lib, a = linattn.load(), ctypes.addressof(d)
    return (lib.prism_linattn_workspace_bytes(a) // (B * H * D * D * 4) + 1,
            lib.prism_linattn_backward_workspace_bytes(a) // (3 * B * H * D * D * 4) + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
def test_slow_decays_in_runs(D, dtype):
    """A sequence that fills all runs, and one that ends inside a middle one."""
    x = make(2, 1300, 3, D, dtype, state=True)
    x["ld"] = SLOW
    assert min(runs(x)) >= 4
    lens = torch.tensor([1300, 777])
    check_forward(x, gpu(x), scale=0.5, lens=lens)
    check_backward(x, gpu(x), scale=0.5, lens=lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 128])
def test_a_longer_sequence(D, dtype):
    x = make(1, 2049, 3, D, dtype, state=True)
    x["ld"] = SLOW
    assert min(runs(x)) >= 8
    check_forward(x, gpu(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_slow_decays_in_one_run(D, dtype):
    """Enough sequences that none is cut: a state is carried over all chunks.  Some of them are compared."""
    B, T = 640, 700
    g = torch.Generator(device="cuda").manual_seed(D)
    dt = TYPES[dtype]
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    c = {m: torch.nn.functional.normalize(n(B, T, 1, D), dim=-1).to(dt) for m in ("q", "k")}
    c.update(v=n(B, T, 1, D).to(dt), do=n(B, T, 1, D).to(dt), s0=n(B, 1, D, D), ds=n(B, 1, D, D))
    assert runs(c) == (1, 1)
    some = [0, 301, B - 1]
    w = {m: t[some].double().cpu() for m, t in c.items()}
    a = {m: t.abs() for m, t in w.items()}
    for ld in (0.0, -1e-4):
        cl, wl = torch.tensor([ld], device="cuda"), torch.tensor([ld]).double()
        out, fs = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], cl, initial_state=c["s0"])
        o, s = lo.linattn(w["q"], w["k"], w["v"], wl, 1.0, w["s0"])
        mo, ms = lo.linattn(a["q"], a["k"], a["v"], wl, 1.0, a["s0"])
        lo.assert_within(out[some], o, lo.out_bound(o, mo, dt, T, D), "out")
        lo.assert_within(fs[some], s, lo.state_bound(ms, dt, T, D), "state")
        got = linattn.prism_linattn_backward(c["q"], c["k"], c["v"], cl, c["do"], initial_state=c["s0"], d_final_state=c["ds"])
        want = lo.linattn_backward(w["q"], w["k"], w["v"], wl, w["do"], 1.0, w["s0"], w["ds"])
        most = lo.linattn_backward(a["q"], a["k"], a["v"], wl, a["do"], 1.0, a["s0"], a["ds"])
        for m, d, b in zip("qkv", want, most):
            lo.assert_within(got[m][some], d, lo.out_bound(d, b, dt, T, D), "d" + m)
        lo.assert_within(got["initial_state"][some], want[3], lo.state_bound(most[3], dt, T, D), "d_initial_state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [90, 900])
@pytest.mark.parametrize("D", [32, 128])
def test_states_apart(D, T, dtype):
    """A state that comes in without a gradient of the one that goes out, and the other way round."""
    lens = torch.tensor([T, T - 31])
    x = make(2, T, 3, D, dtype, state=True)
    x["ld"] = SLOW
    first = dict(x, ds=None)
    check_forward(first, gpu(first), lens=lens)
    check_backward(first, gpu(first), lens=lens)
    last = dict(x, s0=None)
    c = gpu(last)
    check_backward(last, c, lens=lens)
    # the gradient of an initial state of zeros, asked for
    g = linattn.prism_linattn_backward(c["q"], c["k"], c["v"], c["ld"], c["do"], d_final_state=c["ds"],
                                       seq_lens=lens.to(device="cuda", dtype=torch.int32),
                                       grads={"initial_state": torch.full((2, 3, D, D), float("nan"), device="cuda")})
    w = {n: (None if t is None else t.double()) for n, t in last.items()}
    a = {n: (None if t is None else t.abs()) for n, t in w.items()}
    want = lo.linattn_backward(w["q"], w["k"], w["v"], w["ld"], w["do"], 1.0, None, w["ds"], lens)[3]
    most = lo.linattn_backward(a["q"], a["k"], a["v"], w["ld"], a["do"], 1.0, None, a["ds"], lens)[3]
    lo.assert_within(g["initial_state"], want, lo.state_bound(most, x["q"].dtype, T, D), "d_initial_state")
