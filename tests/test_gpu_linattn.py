"""Linear attention with a decay per head against the fp64 recurrence: prompts, gradients and
single tokens, over types, head dims, lengths, ragged and empty sequences, strides, states,
decays, streams and large offsets.  The bounds are those of linattn_oracle."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn
from tests import linattn_oracle as lo

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(B, T, H, D, dtype, seed=0, state=False, fused=False, slow=1.0):
    g = torch.Generator().manual_seed(1000 * T + 10 * D + seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = TYPES[dtype]
    qkv = n(B, T, 3, H, D)
    qkv[:, :, :2] /= qkv[:, :, :2].norm(dim=-1, keepdim=True)
    qkv = qkv.to(dt)
    q, k, v = (qkv[:, :, i] for i in range(3))
    if not fused:
        q, k, v = (x.contiguous() for x in (q, k, v))
    ld = -slow * torch.exp(-3.0 * torch.rand(H, generator=g))
    return dict(q=q, k=k, v=v, ld=ld, do=n(B, T, H, D).to(dt), s0=n(B, H, D, D) if state else None,
                ds=n(B, H, D, D) if state else None, whole=qkv)


def gpu(x, fused=False):
    c = {n: (None if t is None else t.cuda()) for n, t in x.items()}
    if fused:
        c["q"], c["k"], c["v"] = (c["whole"][:, :, i] for i in range(3))
    return c


def wide(x):
    return {n: (None if t is None else t.double()) for n, t in x.items()}


def check_forward(x, c, scale=1.0, lens=None, what=""):
    w = wide(x)
    B, T, H, D = x["q"].shape
    dl = None if lens is None else lens.to(device="cuda", dtype=torch.int32)
    out, fs = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], scale=scale, initial_state=c["s0"],
                                            seq_lens=dl)
    assert out.dtype == x["q"].dtype and fs.dtype == torch.float32
    o, s = lo.linattn(w["q"], w["k"], w["v"], w["ld"], scale, w["s0"], lens)
    mo, ms = lo.linattn(*(w[n].abs() for n in ("q", "k", "v")), w["ld"], abs(scale), None if w["s0"] is None else w["s0"].abs(),
                        lens)
    lo.assert_within(out, o, lo.out_bound(o, mo, out.dtype, T, D), what + " out")
    lo.assert_within(fs, s, lo.state_bound(ms, out.dtype, T, D), what + " state")
    if lens is not None:
        for b, n in enumerate(lens.tolist()):
            assert (out[b, n:] == 0).all(), "padding is not zero"
    assert linattn.linattn_status() == 0
    return out, fs


def check_backward(x, c, scale=1.0, lens=None):
    w = wide(x)
    B, T, H, D = x["q"].shape
    dl = None if lens is None else lens.to(device="cuda", dtype=torch.int32)
    g = linattn.prism_linattn_backward(c["q"], c["k"], c["v"], c["ld"], c["do"], scale=scale, initial_state=c["s0"],
                                       d_final_state=c["ds"], seq_lens=dl)
    a = {n: (None if t is None else t.abs()) for n, t in w.items() if n != "ld"}
    want = lo.linattn_backward(w["q"], w["k"], w["v"], w["ld"], w["do"], scale, w["s0"], w["ds"], lens)
    most = lo.linattn_backward(a["q"], a["k"], a["v"], w["ld"], a["do"], abs(scale), a["s0"], a["ds"], lens)
    for n, o, m in zip("qkv", want, most):
        assert g[n].dtype == x["q"].dtype
        lo.assert_within(g[n], o, lo.out_bound(o, m, g[n].dtype, T, D), "d" + n)
        if lens is not None:
            for b, k in enumerate(lens.tolist()):
                assert (g[n][b, k:] == 0).all(), "padding is not zero"
    if x["s0"] is None:
        assert g["initial_state"] is None
    else:
        lo.assert_within(g["initial_state"], want[3], lo.state_bound(most[3], x["q"].dtype, T, D), "d_initial_state")
    assert linattn.linattn_status() == 0
    return g


SHAPES = [(1, 1, 1, 16), (2, 2, 3, 128), (3, 31, 2, 64), (1, 127, 2, 32), (2, 128, 1, 128), (1, 129, 2, 64),
          (2, 257, 3, 16), (1, 700, 1, 128), (1, 1300, 1, 64), (5, 200, 2, 32), (1, 2049, 1, 16), (1, 1025, 2, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,D", SHAPES)
def test_prompt(B, T, H, D, dtype):
    x = make(B, T, H, D, dtype, state=T % 2 == 1)
    check_forward(x, gpu(x), scale=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,D", SHAPES)
def test_gradient(B, T, H, D, dtype):
    x = make(B, T, H, D, dtype, state=T % 2 == 1)
    check_backward(x, gpu(x), scale=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [150, 900])
def test_ragged_and_empty(D, T, dtype):
    """Lengths 0, 1, odd ones and full ones; NaN and infinities in the padding reach nothing."""
    lens = torch.tensor([0, 1, T - 1, T, 77, 128, 129])
    x = make(len(lens), T, 2, D, dtype, state=True)
    c = gpu(x)
    for n in ("q", "k", "v", "do"):
        for b, k in enumerate(lens.tolist()):
            c[n][b, k:] = float("nan") if b % 2 else float("inf")
    check_forward(x, c, lens=lens)
    check_backward(x, c, lens=lens)


@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
def test_more_sequences_than_are_resident(D, ragged):
    """Many short sequences, in several turns of the SMs: shared memory and TMEM still hold what the
    last CTA left there, and nothing of it reaches a short chunk or an empty sequence."""
    B, T = (100, 140) if D == 128 else (160, 140)
    x = make(B, T, 2, D, "bf16", state=True, seed=ragged)
    c = gpu(x)
    lens = None
    if ragged:
        g = torch.Generator().manual_seed(D)
        lens = torch.where(torch.rand(B, generator=g) < 0.2, torch.zeros(B), torch.rand(B, generator=g) * (T + 1)).long()
        for n in ("q", "k", "v", "do"):
            for b, k in enumerate(lens.tolist()):
                c[n][b, k:] = float("nan")
    check_forward(x, c, lens=lens)
    check_backward(x, c, lens=lens)


def test_lengths_are_clamped():
    x = make(2, 40, 1, 32, "bf16")
    c = gpu(x)
    lens = torch.tensor([-3, 99], dtype=torch.int32, device="cuda")
    out, fs = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], seq_lens=lens)
    want, ws = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"],
                                             seq_lens=torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, want) and torch.equal(fs, ws) and (out[0] == 0).all() and (fs[0] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
def test_slices_of_a_fused_projection(D, dtype):
    x = make(2, 140, 3, D, dtype, fused=True)
    c = gpu(x, fused=True)
    assert not c["q"].is_contiguous()
    o1, s1 = check_forward(x, c)
    g1 = check_backward(x, c)
    o2, s2 = linattn.prism_linattn_forward(*(c[n].contiguous() for n in "qkv"), c["ld"])
    g2 = linattn.prism_linattn_backward(*(c[n].contiguous() for n in "qkv"), c["ld"], c["do"])
    assert torch.equal(o1, o2) and torch.equal(s1, s2)
    assert all(torch.equal(g1[n], g2[n]) for n in "qkv")


def test_a_window_of_longer_sequences():
    """Sequence strides that are not T token strides."""
    x = make(3, 90, 2, 32, "bf16")
    c = gpu(x)
    big = {n: torch.randn(3, 150, 2, 32, device="cuda").to(torch.bfloat16) for n in ("q", "k", "v", "do")}
    for n in big:
        big[n][:, 20:110] = c[n]
        c[n] = big[n][:, 20:110]
    check_forward(x, c)
    check_backward(x, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ld", [0.0, -1e-4, -20.0, -200.0, float("-inf")])
def test_decays(ld, dtype):
    """No decay, slow and fast ones, and no memory at all."""
    x = make(1, 300, 2, 64, dtype, state=True)
    x["ld"] = torch.tensor([ld, -0.1])
    check_forward(x, gpu(x))
    check_backward(x, gpu(x))


@pytest.mark.parametrize("scale", [0.0, -2.0])
def test_scales(scale):
    x = make(1, 70, 2, 64, "bf16", state=True)
    check_forward(x, gpu(x), scale=scale)
    check_backward(x, gpu(x), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_tiny_values(dtype):
    """Values beyond fp16's range, and ones below it."""
    x = make(1, 200, 2, 64, dtype, state=True)
    x["v"][:, ::3] *= 2.0 ** 30
    x["v"][:, 1::3] *= 2.0 ** -30
    x["do"] *= 2.0 ** 20
    check_forward(x, gpu(x))
    check_backward(x, gpu(x))


def test_differences():
    """The gradient of the kernels' own fp32 forward pass, along random directions."""
    x = make(2, 90, 2, 32, "f32", state=True)
    c = gpu(x)
    g = linattn.prism_linattn_backward(c["q"], c["k"], c["v"], c["ld"], c["do"], initial_state=c["s0"],
                                       d_final_state=c["ds"])
    gen = torch.Generator(device="cuda").manual_seed(3)
    names = (("q", "q"), ("k", "k"), ("v", "v"), ("s0", "initial_state"))
    for n, m in names:
        d = torch.randn(c[n].shape, generator=gen, device="cuda")
        e = 2.0 ** -3 * c[n].norm() / d.norm()       # the loss is linear in each input: no truncation error

        def value(f):
            y = dict(c)
            y[n] = c[n] + f * e * d
            o, s = linattn.prism_linattn_forward(y["q"], y["k"], y["v"], y["ld"], initial_state=y["s0"])
            return (o.double() * c["do"].double()).sum() + (s.double() * c["ds"].double()).sum(), o, s

        (a, o, s), (b, _, _) = value(1.0), value(-1.0)
        slope = ((a - b) / (2 * e.double())).item()
        want = (g[m].double() * d.double()).sum().item()
        # the values' own rounding: fp32 sums of (90 + 32 + 256) terms, random signs over the elements
        noise = 378 * lo.U * ((o.double() * c["do"].double()).norm() + (s.double() * c["ds"].double()).norm()).item() / e.item()
        assert abs(slope - want) <= 4 * noise + 1e-5 * abs(want), (n, slope, want, noise)


def test_pieces_and_tokens_continue_each_other():
    """A prompt, then single tokens from its state: the outputs of the whole prompt."""
    x = make(2, 150, 2, 64, "bf16")
    c = gpu(x)
    w = wide(x)
    o, s = lo.linattn(w["q"], w["k"], w["v"], w["ld"])
    mo, ms = lo.linattn(*(w[n].abs() for n in "qkv"), w["ld"])
    a, state = linattn.prism_linattn_forward(c["q"][:, :140], c["k"][:, :140], c["v"][:, :140], c["ld"])
    outs = [a]
    for t in range(140, 150):
        outs.append(linattn.prism_linattn_decode_step(c["q"][:, t], c["k"][:, t], c["v"][:, t], c["ld"], state)[:, None])
    got = torch.cat(outs, 1)
    lo.assert_within(got, o, lo.out_bound(o, mo, torch.bfloat16, 150, 64), "out")
    lo.assert_within(state, s, lo.state_bound(ms, torch.bfloat16, 150, 64), "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (33, 2)])
def test_decode(B, H, D, dtype):
    x = make(B, 1, H, D, dtype, state=True, fused=True)
    c = gpu(x, fused=True)
    w = wide(x)
    state = c["s0"].clone()
    out = linattn.prism_linattn_decode_step(c["q"][:, 0], c["k"][:, 0], c["v"][:, 0], c["ld"], state, scale=0.3)
    o, s = lo.linattn(w["q"], w["k"], w["v"], w["ld"], 0.3, w["s0"])
    mo, ms = lo.linattn(*(w[n].abs() for n in "qkv"), w["ld"], 0.3, w["s0"].abs())
    n = (D + 8) * lo.U                            # fp32 arithmetic, then one rounding of the output
    lo.assert_within(state, s, n * ms, "state")
    lo.assert_within(out, o[:, 0], n * mo[:, 0] + (lo.BF16 * o[:, 0].abs() if dtype == "bf16" else 0.0), "out")


def test_decode_slots():
    """States in a pool: any order, and sequences that are not there."""
    B, H, D, N = 5, 2, 64, 9
    x = make(B, 1, H, D, "bf16")
    c = gpu(x)
    pool = torch.randn(N, H, D, D, device="cuda")
    before = pool.clone()
    slots = torch.tensor([7, -1, 0, 9, 3], dtype=torch.int32, device="cuda")
    c["v"][1] = float("nan")
    out = linattn.prism_linattn_decode_step(c["q"][:, 0], c["k"][:, 0], c["v"][:, 0], c["ld"], pool, slots=slots)
    at = [0, 2, 4]
    mine = before[slots[at].long()].clone()
    want = linattn.prism_linattn_decode_step(c["q"][at, 0], c["k"][at, 0], c["v"][at, 0], c["ld"], mine)
    assert torch.equal(out[at], want) and torch.equal(pool[slots[at].long()], mine)
    assert (out[[1, 3]] == 0).all()
    rest = [i for i in range(N) if i not in (7, 0, 3)]
    assert torch.equal(pool[rest], before[rest])


def test_another_stream_and_reruns():
    """Work on a stream of its own; the same inputs give the same bits."""
    x = make(1, 1500, 2, 64, "bf16", state=True)
    c = gpu(x)
    first = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], initial_state=c["s0"])
    g1 = linattn.prism_linattn_backward(c["q"], c["k"], c["v"], c["ld"], c["do"], initial_state=c["s0"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], initial_state=c["s0"])
        g2 = linattn.prism_linattn_backward(c["q"], c["k"], c["v"], c["ld"], c["do"], initial_state=c["s0"])
    side.synchronize()
    third = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], initial_state=c["s0"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(first, second, third))
    assert all(torch.equal(g1[n], g2[n]) for n in ("q", "k", "v", "initial_state"))


def test_captured_in_a_graph():
    x = make(2, 300, 2, 64, "bf16", state=True)
    c = gpu(x)
    want, ws = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], initial_state=c["s0"])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, fs = linattn.prism_linattn_forward(c["q"], c["k"], c["v"], c["ld"], initial_state=c["s0"])
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(fs, ws)


def test_offsets_past_32_bits():
    """Over 2^31 elements of q, and a state pool of over 2^31 values."""
    H, D = 16, 128
    T = (1 << 31) // (H * D) + 300
    q = torch.full((1, T, H, D), 0.0, dtype=torch.bfloat16, device="cuda")
    x = make(1, 200, H, D, "bf16", slow=2.0)
    c = gpu(x)
    q[:, -200:] = c["q"]
    ld = torch.full((H,), -1.0, device="cuda")
    out, fs = linattn.prism_linattn_forward(q, q, q, ld)
    w = x["q"].double()
    o, s = lo.linattn(w, w, w, ld.double().cpu())
    mo, ms = lo.linattn(w.abs(), w.abs(), w.abs(), ld.double().cpu())
    lo.assert_within(out[:, -200:], o, lo.out_bound(o, mo, torch.bfloat16, 200, D), "out")
    lo.assert_within(fs, s, lo.state_bound(ms, torch.bfloat16, 200, D), "state")
    assert (out[:, :T - 200] == 0).all()
    del q, out
    N = (1 << 31) // (D * D) + 2
    pool = torch.empty(N, 1, D, D, device="cuda")
    pool[-1] = 1.0
    slots = torch.tensor([N - 1], dtype=torch.int32, device="cuda")
    one = torch.ones(1, 1, D, device="cuda")
    out = linattn.prism_linattn_decode_step(one, one, one, torch.zeros(1, device="cuda"), pool, slots=slots)
    assert (pool[-1] == 2.0).all() and (out == 2.0 * D).all()
