"""Non-finite values in linear attention: as in the recurrence, token by token, they reach what comes
after them and nothing before, inside a chunk of the kernels as well.

The fp64 oracle runs on the same inputs, NaN and infinities included.  Where it is finite the
kernel is held to the usual bounds, where it is not the kernel is not either."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn
from tests import linattn_oracle as lo

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(B, T, H, D, dtype, seed):
    g = torch.Generator().manual_seed(7 * T + D + seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = TYPES[dtype]
    x = {m: n(B, T, H, D) for m in ("q", "k", "v", "do")}
    for m in ("q", "k"):
        x[m] /= x[m].norm(dim=-1, keepdim=True)
    x = {m: t.to(dt) for m, t in x.items()}
    x.update(ld=-0.02 * torch.rand(H, generator=g) - 1e-3, s0=n(B, H, D, D), ds=n(B, H, D, D))
    return x


def agree(got, want, bound, what):
    got, ok = got.detach().double().cpu(), torch.isfinite(want)
    assert torch.isfinite(got[ok]).all(), f"{what}: a non-finite value where the recurrence has none"
    assert not torch.isfinite(got[~ok]).any(), f"{what}: a finite value where the recurrence has none"
    lo.assert_within(got[ok], want[ok], bound[ok], what)


def at_tokens(lens, *tensors):
    """Outputs of the oracle with the zeros of padding (which its products make of a state that is NaN)."""
    if lens is None:
        return tensors
    gone = torch.arange(tensors[0].shape[1])[None] >= lens[:, None]
    return tuple(t.masked_fill(gone[:, :, None, None], 0.0) for t in tensors)


def check(x, scale=0.5, lens=None):
    w = {n: t.double() for n, t in x.items()}
    a = {n: t.abs() for n, t in w.items()}
    c = {n: t.cuda() for n, t in x.items()}
    B, T, H, D = x["q"].shape
    dt = x["q"].dtype
    dl = None if lens is None else lens.to(device="cuda", dtype=torch.int32)
    out, fs = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], scale=scale, initial_state=c["s0"], seq_lens=dl)
    o, s = lo.linattn(w["q"], w["k"], w["v"], w["ld"], scale, w["s0"], lens)
    mo, ms = lo.linattn(a["q"], a["k"], a["v"], w["ld"], scale, a["s0"], lens)
    o, mo = at_tokens(lens, o, mo)
    agree(out, o, lo.out_bound(o, mo, dt, T, D), "out")
    agree(fs, s, lo.state_bound(ms, dt, T, D), "state")
    g = linattn.prism_linattn_backward(c["q"], c["k"], c["v"], c["ld"], c["do"], scale=scale, initial_state=c["s0"],
                                       d_final_state=c["ds"], seq_lens=dl)
    want = lo.linattn_backward(w["q"], w["k"], w["v"], w["ld"], w["do"], scale, w["s0"], w["ds"], lens)
    most = lo.linattn_backward(a["q"], a["k"], a["v"], w["ld"], a["do"], scale, a["s0"], a["ds"], lens)
    for n, d, m in zip("qkv", at_tokens(lens, *want[:3]), at_tokens(lens, *most[:3])):
        agree(g[n], d, lo.out_bound(d, m, dt, T, D), "d" + n)
    agree(g["initial_state"], want[3], lo.state_bound(most[3], dt, T, D), "d_initial_state")
    assert linattn.linattn_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_one_value(name, D, dtype):
    """One element of one token in each head, early and late in a chunk, in the last token, in a short chunk."""
    x = make(1, 150, 5, D, dtype, ord(name[0]))
    for h, (t, v) in enumerate(((0, "nan"), (37, "inf"), (127, "-inf"), (149, "nan"), (100, "nan"))):
        x[name][0, t, h, (3 * t) % D] = float(v)
    check(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_whole_tokens(D, dtype):
    """Tokens that hold nothing but NaN, in sequences of other lengths, and a head that is all NaN."""
    x = make(3, 300, 2, D, dtype, 1)
    for n in ("q", "k", "v", "do"):
        x[n][0, 200, 0] = float("nan")
        x[n][1, 129:, 1] = float("nan")
        x[n][2, :, 0] = float("nan")
    check(x, lens=torch.tensor([300, 170, 255]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 128])
def test_runs(D, dtype):
    """In a sequence that is cut into runs, in the first, a middle and the last one, and in the states."""
    x = make(1, 1300, 4, D, dtype, 2)
    x["ld"] = torch.tensor([-1e-3, -2e-3, -5e-3, 0.0])
    for h, t in enumerate((70, 600, 1290)):
        for n in ("q", "k", "v", "do"):
            x[n][0, t + 3 * (n == "do"), h, 5] = float("nan")
    x["s0"][0, 3, 4, 9] = x["ds"][0, 3, 1, 2] = float("inf")
    check(x)


def test_prompt_and_single_tokens_agree():
    """The outputs of a prompt are finite where those of its tokens one by one are."""
    x = make(2, 60, 2, 64, "bf16", 3)
    x["v"][0, 41, 1, 7] = float("nan")
    x["k"][1, 20, 0, 3] = float("inf")
    c = {n: t.cuda() for n, t in x.items()}
    out, fs = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], initial_state=c["s0"])
    state = c["s0"].clone()
    for t in range(60):
        o = linattn.prism_linattn_decode_step(c["q"][:, t], c["k"][:, t], c["v"][:, t], c["ld"], state)
        assert torch.equal(torch.isfinite(o), torch.isfinite(out[:, t]))
    assert torch.equal(torch.isfinite(state), torch.isfinite(fs))
