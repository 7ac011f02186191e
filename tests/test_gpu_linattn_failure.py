"""The failure path of the linear attention kernel's bounded waits, without a fault or a hang.

With PRISM_FLAG_CHECK_WAIT_TIMEOUT the warp that copies first waits, for a millisecond or so, for what
never comes, and gives up; the roles that wait for its tiles give up after their second, everything
in flight is waited for, the TMEM goes back, and the call returns with the word set.  A call
after it gets its TMEM and is right, bit for bit."""
import time

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn, prism

pytestmark = pytest.mark.gpu
CHECK = prism.PRISM_FLAG_CHECK_WAIT_TIMEOUT


def make(B, T, H, D, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = [torch.nn.functional.normalize(n(B, T, H, D), dim=-1).to(dtype) for _ in range(2)]
    return (*x, n(B, T, H, D).to(dtype), -0.01 - torch.rand(H, generator=g, device="cuda")), n(B, T, H, D).to(dtype), n(B, H, D, D)


@pytest.mark.parametrize("B,T,H,D", [(2, 100, 2, 16), (2, 100, 2, 32), (2, 100, 2, 64), (1, 3000, 2, 128), (80, 300, 2, 128)])
def test_waits_that_run_out(B, T, H, D):
    """One chunk; a sequence in runs, so both launches fail; more CTAs than are resident."""
    args, do, s0 = make(B, T, H, D)
    assert linattn.linattn_status() == 0
    want = linattn.prism_linattn_forward(*args, initial_state=s0)
    wg = linattn.prism_linattn_backward(*args, do, initial_state=s0)
    assert linattn.linattn_status() == 0
    begin = time.monotonic()
    linattn.prism_linattn_forward(*args, initial_state=s0, flags=CHECK)
    assert linattn.linattn_status(clear=False) != 0
    assert linattn.linattn_status(clear=True) != 0          # the word stays until it is cleared
    assert linattn.linattn_status() == 0
    linattn.prism_linattn_backward(*args, do, initial_state=s0, flags=CHECK)
    assert linattn.linattn_status() != 0
    assert time.monotonic() - begin < 30.0                  # a second or so a turn of the SMs
    got = linattn.prism_linattn_forward(*args, initial_state=s0)
    g = linattn.prism_linattn_backward(*args, do, initial_state=s0)
    assert linattn.linattn_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(g[n], wg[n]) for n in wg)


def test_calls_without_waits():
    """Empty sequences wait for nothing, and the fp32 path has no such waits: the flag changes nothing."""
    args, _, s0 = make(2, 100, 2, 64)
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, fs = linattn.prism_linattn_forward(*args, initial_state=s0, seq_lens=none, flags=CHECK)
    assert linattn.linattn_status() == 0 and (out == 0).all() and torch.equal(fs, s0)
    args, _, s0 = make(2, 100, 2, 64, torch.float32)
    want = linattn.prism_linattn_forward(*args, initial_state=s0)
    got = linattn.prism_linattn_forward(*args, initial_state=s0, flags=CHECK)
    assert linattn.linattn_status() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
