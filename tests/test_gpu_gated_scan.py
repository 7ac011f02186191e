"""The gated recurrence, its gradient and its single-token step against the 64-bit oracle, within the bounds of
tests/gated_oracle.py."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated, prism
from tests import gated_oracle as go

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(B, T, D, dtype, gate=True, seed=0, fused=False, spread=7.0):
    g = torch.Generator().manual_seed(seed + 131 * T + D)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = TYPES[dtype]
    p = n(B, T, 3, D)
    p[:, :, 1] += spread * torch.rand(D, generator=g)      # memories of a few tokens to a thousand
    p = p.to(dt)
    x, f, i = (p[:, :, k] if fused else p[:, :, k].contiguous() for k in range(3))
    return dict(x=x, f=f, i=i if gate else None, s0=n(B, D), do=n(B, T, D).to(dt), ds=n(B, D), p=p)


def dev(z, fused=False):
    """On the GPU, the gates still slices of one tensor where they were."""
    c = {n: None if t is None else t.cuda() for n, t in z.items()}
    if fused:
        c["x"], c["f"] = c["p"][:, :, 0], c["p"][:, :, 1]
        c["i"] = None if z["i"] is None else c["p"][:, :, 2]
    return c


def check(z, c, *, resumed=True, lens=None):
    lc = None if lens is None else lens.to(device="cuda", dtype=torch.int32)
    s0, ds = (z["s0"], z["ds"]) if resumed else (None, None)
    s0c, dsc = (c["s0"], c["ds"]) if resumed else (None, None)
    dt = z["x"].dtype
    states = gated.gated_scan_states(c["x"]).fill_(float("nan"))
    out, final = gated.prism_gated_scan_forward(c["x"], c["f"], input_gate=c["i"], initial_state=s0c, seq_lens=lc,
                                                states=states)
    want = go.scan(z["x"], z["f"], z["i"], s0, lens)
    assert out.dtype == dt and out.is_contiguous()
    go.assert_within(out, want["out"], want["err"][:, 1:], "out", dt)
    go.assert_within(final, want["final"], want["err"][:, -1] + 2 * go.U * want["mag"][:, -1], "final state")
    n = go.lengths(z["x"], lens)
    for b in range(len(n)):
        rows = -(-int(n[b]) // 64)
        go.assert_within(states[b, :rows], want["before"][b, :n[b]][::64],
                         want["err"][b, :n[b]][::64] + 2 * go.U * want["mag"][b, :n[b]][::64], "states")
        assert torch.isnan(states[b, rows:]).all(), "rows behind a sequence's end are left as they are"
        assert (out[b, n[b]:] == 0).all()
    g = gated.prism_gated_scan_backward(c["x"], c["f"], states, c["do"], input_gate=c["i"], d_final_state=dsc,
                                        seq_lens=lc, want_initial_state=True)
    wg, bound = go.scan_back(z["x"], z["f"], z["do"], z["i"], s0, ds, lens)
    for m in ("x", "forget", "input_gate"):
        if wg[m] is None:
            assert g[m] is None
        else:
            assert g[m].dtype == dt
            go.assert_within(g[m], wg[m], bound[m], "d" + m, dt)
    go.assert_within(g["initial_state"], wg["initial_state"], bound["initial_state"], "d initial state")
    assert gated.gated_status() == 0
    return out, final, states, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (2, 1, 64), (3, 7, 72), (1, 63, 40), (2, 64, 128), (1, 65, 8), (2, 129, 200),
                                   (1, 700, 64), (3, 257, 136), (1, 4100, 16), (2, 8, 72), (2, 9, 72), (3, 16, 136), (3, 17, 72), (2, 32, 200),
                                   (2, 33, 72)])
def test_scan(B, T, D, gate, dtype):
    z = make(B, T, D, dtype, gate)
    check(z, dev(z))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
def test_slices_of_a_projection(gate, dtype):
    z = make(3, 150, 72, dtype, gate, fused=True)
    check(z, dev(z, True), resumed=False)
    whole = dev(make(3, 150, 72, dtype, gate))
    c = dev(z, True)
    for a, b in zip(gated.prism_gated_scan_forward(c["x"], c["f"], input_gate=c["i"]),
                    gated.prism_gated_scan_forward(whole["x"], whole["f"], input_gate=whole["i"])):
        assert torch.equal(a, b)


def time_major(t):
    return t.transpose(0, 1).contiguous().transpose(0, 1)


def windows(t):
    """Sequences that begin a token apart in one recording."""
    B, T, D = t.shape
    return torch.cat((t[0], t[1:, 0])).as_strided((B, T, D), (D, D, 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("lay", [time_major, windows])
@pytest.mark.parametrize("B,T,D", [(3, 5, 72), (500, 7, 264), (4, 14, 72), (5, 30, 40), (5, 70, 72), (2, 300, 8), (2, 2500, 136)])
def test_other_orders(B, T, D, lay, gate, dtype):
    """Tokens further apart than sequences, and sequences that share tokens: the bits of contiguous inputs."""
    c = dev(make(B, T, D, dtype, gate))
    ways = []
    for there in (True, False):
        x, f, i, do = (None if c[n] is None else lay(c[n]) for n in ("x", "f", "i", "do"))
        if there:
            x, f, i, do = (None if t is None else t.contiguous() for t in (x, f, i, do))
        states = gated.gated_scan_states(x)
        out, final = gated.prism_gated_scan_forward(x, f, input_gate=i, initial_state=c["s0"], states=states)
        g = gated.prism_gated_scan_backward(x, f, states, do, input_gate=i, d_final_state=c["ds"], want_initial_state=True)
        ways.append((out, final, states, *(t for t in g.values() if t is not None)))
    assert all(torch.equal(a, b) for a, b in zip(*ways)) and all(t.is_contiguous() for t in ways[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("T", [1, 7, 16, 30, 64, 300])
def test_ragged(T, gate, dtype):
    """Lengths of none, one, a tile's border and past the end; padding is NaN and reaches nothing."""
    lens = torch.tensor([0, 1, min(T, 64), min(T, 65), T, T + 9, -3, T // 2])
    z = make(8, T, 72, dtype, gate)
    gone = (torch.arange(T)[None] >= lens[:, None])[..., None]
    for n in ("x", "f", "i", "do"):
        if z[n] is not None:
            z[n] = torch.where(gone, torch.tensor(float("nan"), dtype=z[n].dtype), z[n])
    for resumed in (True, False):
        c = dev(z)
        out, final, _, g = check(z, c, resumed=resumed, lens=lens)
        if resumed:
            for b in (0, 6):                               # no tokens: the state and its gradient go through
                assert torch.equal(final[b], c["s0"][b]) and torch.equal(g["initial_state"][b], c["ds"][b])
        for n in ("x", "forget", "input_gate"):
            assert g[n] is None or (g[n][gone.expand_as(g[n])] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tiles_and_sequences(dtype):
    """More tiles than are resident at once; the same bits in every call, whoever comes first."""
    z = make(16, 1500, 520, dtype)
    c = dev(z)
    lens = torch.randint(0, 1501, (16,), generator=torch.Generator().manual_seed(2))
    first = check(z, c, lens=lens)
    for _ in range(3):
        again = gated.prism_gated_scan_forward(c["x"], c["f"], input_gate=c["i"], initial_state=c["s0"],
                                               seq_lens=lens.cuda().int())
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
        g = gated.prism_gated_scan_backward(c["x"], c["f"], first[2], c["do"], input_gate=c["i"], d_final_state=c["ds"],
                                            seq_lens=lens.cuda().int(), want_initial_state=True)
        assert all(torch.equal(g[n], first[3][n]) for n in g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("B,T,D", [(2000, 4, 40), (1100, 20, 40), (1300, 130, 24), (300, 64, 136), (300, 65, 136), (40, 400, 520), (4, 1000, 256), (1, 2048, 136),
                                   (2, 900, 40), (8, 1024, 64), (620, 200, 40), (60, 200, 704),
                                   (1, 1024, 72), (1, 1025, 72), (2, 520, 64), (1, 3000, 72), (2, 512, 136), (2, 513, 24), (3, 2000, 72),
                                   (200, 100, 264), (30, 128, 136), (30, 129, 136), (130, 250, 72), (300, 150, 64), (20, 256, 264),
                                   (460, 192, 40), (460, 193, 40), (700, 16, 72), (500, 32, 72), (600, 8, 264), (700, 20, 264),
                                   (900, 50, 72), (350, 100, 72)])
def test_every_way(B, T, D, gate, dtype):
    """Token by token, a cluster a chain, looking back in tiles of each length: the rules' borders."""
    lens = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(B))
    z = make(B, T, D, dtype, gate)
    check(z, dev(z), lens=lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_sequence(dtype):
    """A chain of 400 tiles, with channels that hardly forget."""
    z = make(1, 25600, 8, dtype, spread=12.0)
    check(z, dev(z))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
def test_gates_at_their_ends(gate, dtype):
    """Gates that are 0 or 1 to the last bit, infinite ones among them."""
    z = make(2, 140, 16, dtype, gate)
    for n in ("f", "i"):
        if z[n] is not None:
            for k, v in enumerate((80.0, -80.0, 30.0, -30.0, float("inf"), -float("inf"), 0.0)):
                z[n][:, k::9, k:k + 8] = v
    c = dev(z)
    states = gated.gated_scan_states(c["x"])
    out, final = gated.prism_gated_scan_forward(c["x"], c["f"], input_gate=c["i"], initial_state=c["s0"], states=states)
    y = {n: None if t is None else t.float().clamp(-1e4, 1e4) if n in "fi" else t for n, t in z.items()}
    want = go.scan(y["x"], y["f"], y["i"], y["s0"])
    # delta of the largest |z| that is not lost: behind 88 a gate is below 2^-126
    y2 = {n: None if t is None else t.clamp(-88, 88) if n in "fi" else t for n, t in y.items()}
    err = go.scan(y2["x"], y2["f"], y2["i"], y2["s0"])["err"] + 2.0 ** -100
    go.assert_within(out, want["out"], err[:, 1:], "out", z["x"].dtype)
    g = gated.prism_gated_scan_backward(c["x"], c["f"], states, c["do"], input_gate=c["i"], d_final_state=c["ds"],
                                        want_initial_state=True)
    wg, _ = go.scan_back(y["x"], y["f"], y["do"], y["i"], y["s0"], y["ds"])
    _, bound = go.scan_back(y2["x"], y2["f"], y2["do"], y2["i"], y2["s0"], y2["ds"])
    for m in ("x", "forget", "input_gate"):
        if wg[m] is not None:
            go.assert_within(g[m], wg[m], bound[m] + 2.0 ** -100, "d" + m, z["x"].dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_reach_nothing_before_them(bad, dtype):
    """In its own channel alone, and what comes after it alone; in the gradients what comes before."""
    z = make(2, 300, 24, dtype)
    c = dev(z)
    run = lambda: gated.prism_gated_scan_forward(c["x"], c["f"], input_gate=c["i"], states=states)[0]  # noqa: E731
    states = gated.gated_scan_states(c["x"])
    want = run()
    grads = lambda: gated.prism_gated_scan_backward(c["x"], c["f"], states, c["do"], input_gate=c["i"])  # noqa: E731
    wg = grads()
    c["x"][1, 130, 5] = bad
    out = run()
    there = torch.zeros_like(out, dtype=torch.bool)
    there[1, 130:, 5] = True
    assert torch.equal(out[~there], want[~there]) and not torch.isfinite(out[1, 130, 5])
    c["x"][1, 130, 5] = z["x"][1, 130, 5].cuda()
    run()
    c["do"][0, 150, 7] = bad
    g = grads()
    there = torch.zeros_like(out, dtype=torch.bool)
    there[0, :151, 7] = True
    for n in ("x", "forget", "input_gate"):
        assert torch.equal(g[n][~there], wg[n][~there]) and not torch.isfinite(g[n][0, 150, 7])


@pytest.mark.parametrize("T", [64, 1000])
def test_state_in_place(T):
    """The final state over the initial one, and its gradient over the one that came in."""
    z = make(3, T, 72, "bf16")
    c = dev(z)
    lens = torch.tensor([T, 0, T // 3], device="cuda", dtype=torch.int32)
    out, final, states, g = check(z, c, lens=lens.cpu())
    s = c["s0"].clone()
    out2, same = gated.prism_gated_scan_forward(c["x"], c["f"], input_gate=c["i"], initial_state=s, final_state=s,
                                                seq_lens=lens)
    assert same is s and torch.equal(s, final) and torch.equal(out, out2)
    d = c["ds"].clone()
    g2 = gated.prism_gated_scan_backward(c["x"], c["f"], states, c["do"], input_gate=c["i"], d_final_state=d,
                                         seq_lens=lens, grads={"initial_state": d})
    assert all(torch.equal(g[n], g2[n]) for n in g) and g2["initial_state"] is d


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_by_differences(gate, dtype):
    """The kernel's gradient along a random direction against central differences of the 64-bit forward pass.
    L has a third derivative along v of at most a few times |v|^3 sums, so the step 1e-4 leaves a relative 1e-6; what
    remains is the gradients' own error, bounded elementwise."""
    z = make(2, 100, 16, dtype, gate, spread=3.0)
    c = dev(z)
    states = gated.gated_scan_states(c["x"])
    gated.prism_gated_scan_forward(c["x"], c["f"], input_gate=c["i"], initial_state=c["s0"], states=states)
    g = gated.prism_gated_scan_backward(c["x"], c["f"], states, c["do"], input_gate=c["i"], d_final_state=c["ds"],
                                        want_initial_state=True)
    _, bound = go.scan_back(z["x"], z["f"], z["do"], z["i"], z["s0"], z["ds"])
    names = {"x": "x", "f": "forget", "i": "input_gate", "s0": "initial_state"}
    for n, m in names.items():
        if z[n] is None:
            continue
        v = torch.randn(z[n].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)

        def loss(h):
            y = {k: None if z[k] is None else z[k].double() for k in names}
            y[n] = y[n] + h * v
            s = go.scan(y["x"], y["f"], y["i"], y["s0"])
            return (s["out"] * z["do"].double()).sum().item() + (s["final"] * z["ds"].double()).sum().item()

        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        mine = g[m].double().cpu()
        rnd = 0 if n == "s0" else go.ROUND[z["x"].dtype]
        tol = ((bound[m] + rnd * (mine.abs() + bound[m])) * v.abs()).sum().item()
        assert abs((mine * v).sum().item() - slope) <= tol + 1e-6 * (1 + (mine * v).abs().sum().item()), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("B,D", [(1, 8), (3, 72), (8, 2048), (130, 256)])
def test_single_tokens(B, D, gate, dtype):
    z = make(B, 1, D, dtype, gate, fused=True)
    c = dev(z, True)
    N = B + 5
    pool = torch.randn(N, D, generator=torch.Generator().manual_seed(B))
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(D))[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, N                         # not there
    mine = pool.cuda()
    sq = lambda t: None if t is None else t[:, 0]  # noqa: E731
    out = gated.prism_gated_scan_decode_step(sq(c["x"]), sq(c["f"]), mine, input_gate=sq(c["i"]), slots=slots.cuda())
    there = (slots >= 0) & (slots < N)
    at = slots.clamp(0, N - 1).long()
    want = go.scan(z["x"], z["f"], z["i"], pool[at])
    assert out.dtype == z["x"].dtype and (out[~there.cuda()] == 0).all()
    go.assert_within(out[there.cuda()], want["out"][there, 0], want["err"][there, 1], "out", out.dtype)
    expect, bound = pool.double(), torch.zeros(N, D, dtype=torch.float64)
    expect[at[there]], bound[at[there]] = want["final"][there], want["err"][there, 1]
    go.assert_within(mine, expect, bound, "pool")
    own = c["s0"].clone()
    out2 = gated.prism_gated_scan_decode_step(sq(c["x"]), sq(c["f"]), own, input_gate=sq(c["i"]))
    a, b = gated.prism_gated_scan_forward(c["x"], c["f"], input_gate=c["i"], initial_state=c["s0"])
    assert torch.equal(out2, a[:, 0]) and torch.equal(own, b)


@pytest.mark.parametrize("T", [2100, 3000])
def test_waits_that_run_out(T):
    """The failure path's check sets the word and leaves the outputs as they are; short sequences wait for nothing."""
    z = make(2, T, 72, "bf16")
    c = dev(z)
    assert gated.gated_status() == 0
    out, final, states, g = check(z, c)
    how = dict(input_gate=c["i"], flags=prism.PRISM_FLAG_CHECK_WAIT_TIMEOUT)
    got = gated.prism_gated_scan_forward(c["x"], c["f"], initial_state=c["s0"], **how)
    assert gated.gated_status(clear=False) != 0 and gated.gated_status() != 0 and gated.gated_status() == 0
    assert torch.equal(got[0], out) and torch.equal(got[1], final)
    g2 = gated.prism_gated_scan_backward(c["x"], c["f"], states, c["do"], d_final_state=c["ds"], want_initial_state=True,
                                         **how)
    assert gated.gated_status() != 0 and all(torch.equal(g[n], g2[n]) for n in g)
    x, f, i = (c[n][:, :32].contiguous() for n in ("x", "f", "i"))
    gated.prism_gated_scan_forward(x, f, input_gate=i, flags=prism.PRISM_FLAG_CHECK_WAIT_TIMEOUT)
    assert gated.gated_status() == 0


def test_offsets_past_32_bits():
    """2.2e9 elements a tensor: the last sequence as by itself, in the same way (bit for bit), gradient and all."""
    B, T, D = 4, 35000, 16384
    x = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda")
    f, d = torch.empty_like(x), torch.empty_like(x)
    for t, s in ((x, 1), (f, 2), (d, 3)):
        g = torch.Generator(device="cuda").manual_seed(s)
        for b in range(B):
            t[b].normal_(generator=g)
    states = gated.gated_scan_states(x)
    out, final = gated.prism_gated_scan_forward(x, f, states=states)
    g = gated.prism_gated_scan_backward(x, f, states, d)
    st = gated.gated_scan_states(x[3:])
    o3, f3 = gated.prism_gated_scan_forward(x[3:], f[3:], states=st)
    g3 = gated.prism_gated_scan_backward(x[3:], f[3:], st, d[3:])
    assert torch.equal(out[3:], o3) and torch.equal(final[3:], f3) and torch.equal(states[3:], st)
    assert torch.equal(g["x"][3:], g3["x"]) and torch.equal(g["forget"][3:], g3["forget"])
    y = gated.prism_layer_norm(x)
    n = gated.prism_layer_norm_backward(x, d)
    assert torch.equal(y[3:], gated.prism_layer_norm(x[3:]))
    assert torch.equal(n["x"][3:], gated.prism_layer_norm_backward(x[3:], d[3:])["x"])
    assert gated.gated_status() == 0
