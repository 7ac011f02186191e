"""Layer norm and its gradient against the 64-bit oracle, within the bounds of tests/gated_oracle.py."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated
from tests import gated_oracle as go

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(B, T, D, dtype, seed=0, shift=0.5, weights=True):
    g = torch.Generator().manual_seed(seed + 17 * T + D)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=(n(B, T, D) * (1 + n(D).abs()) + shift).to(TYPES[dtype]), d=n(B, T, D).to(TYPES[dtype]),
                w=1 + 0.3 * n(D) if weights else None, b=n(D) if weights else None)


def check(z, c=None, lens=None, eps=1e-5):
    c = c or {n: None if t is None else t.cuda() for n, t in z.items()}
    lc = None if lens is None else lens.to(device="cuda", dtype=torch.int32)
    dt = z["x"].dtype
    y = gated.prism_layer_norm(c["x"], weight=c["w"], bias=c["b"], eps=eps, seq_lens=lc)
    want, bound = go.layer_norm(z["x"], z["w"], z["b"], eps, lens)
    assert y.dtype == dt and y.is_contiguous()
    go.assert_within(y, want, bound, "y", dt)
    g = gated.prism_layer_norm_backward(c["x"], c["d"], weight=c["w"], bias=c["b"], eps=eps, seq_lens=lc)
    want, bound = go.layer_norm_back(z["x"], z["d"], z["w"], eps, lens)
    go.assert_within(g["x"], want["x"], bound["x"], "dx", dt)
    for n, t in (("weight", z["w"]), ("bias", z["b"])):
        if t is None:
            assert g[n] is None
        else:
            assert g[n].dtype == torch.float32
            go.assert_within(g[n], want[n], bound[n], "d" + n)
    gone = ~go._live(z["x"], lens)
    assert (y.cpu()[gone] == 0).all() and (g["x"].cpu()[gone] == 0).all()
    return y, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 16, 32, 40, 64, 72, 96, 104, 128, 136, 160, 168, 192, 200, 256, 264, 304, 312, 384, 392, 512, 520, 640, 648, 768,
                               776, 832, 840, 1000, 1024, 1032, 1280, 1288, 1536, 1544, 2048, 2056, 2560, 2568, 4096, 4104, 5000,
                               6144, 6152, 8192, 8200, 16384])
def test_widths(D, dtype):
    """Every variant's largest width and the one behind it."""
    check(make(3, 7, D, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (1, 1, 2048), (40, 500, 64), (5, 700, 1000), (1, 3001, 520), (700, 3, 24),
                                   (1, 20000, 32), (3, 6001, 64), (1, 9000, 96), (1, 9000, 128), (2, 4001, 160), (1, 8000, 192), (1, 6000, 256),
                                   (1, 4000, 288), (1, 4000, 384), (5, 800, 512), (3, 901, 768), (1, 2000, 800), (1, 1500, 1280), (1, 1100, 2560),
                                   (1, 700, 6144)])
def test_rows(B, T, D, dtype):
    check(make(B, T, D, dtype))
    check(make(B, T, D, dtype, weights=False))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [24, 64, 96, 160, 320, 768, 1000, 1280, 2320, 4096])
def test_ragged_and_strided(D, dtype):
    z = make(5, 9, D, dtype)
    lens = torch.tensor([0, 9, 1, 12, 4])
    gone = (torch.arange(9)[None] >= lens[:, None])[..., None]
    for n in ("x", "d"):
        z[n] = torch.where(gone, torch.tensor(float("nan"), dtype=z[n].dtype), z[n])
    y, g = check(z, lens=lens)
    c = {n: t.cuda() for n, t in z.items()}
    wide = torch.full((5, 9, 2, D), float("inf"), dtype=z["x"].dtype, device="cuda")
    wide[:, :, 0], wide[:, :, 1] = c["x"], c["d"]
    c["x"], c["d"] = wide[:, :, 0], wide[:, :, 1]
    y2, g2 = check(z, c, lens=lens)
    assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)
    none = torch.zeros(5, dtype=torch.int64)
    y, g = check(z, lens=none)
    assert (g["weight"] == 0).all() and (g["bias"] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 96, 128, 152, 192, 256, 288, 384, 512, 640, 1024])
def test_many_ragged_rows(D, dtype):
    """Every warp of a CTA goes over rows of its own, padding among them."""
    lens = torch.randint(0, 71, (60,), generator=torch.Generator().manual_seed(D))
    check(make(60, 70, D, dtype), lens=lens)


@pytest.mark.parametrize("D", [64, 2048, 4096])
def test_a_mean_far_from_zero(D):
    """The variance keeps its bits: 300 away from 0, and rows that are constant."""
    z = make(2, 5, D, "f32", shift=300.0)
    z["x"][1, 2] = 7.25
    check(z)
    z["x"][1, 3] = 0
    check(z, eps=1e-3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 264, 2048, 4096])
def test_other_orders(D, dtype):
    """Tokens further apart than sequences, and sequences that share tokens: the bits of contiguous inputs."""
    g = torch.Generator().manual_seed(D)
    line = torch.randn(2, 90, D, generator=g).to("cuda", dtype)
    w, b = (torch.randn(D, generator=g).cuda() for _ in range(2))
    for step in ((D, 3 * D, 1), (D, D, 1)):
        x, do = (t.as_strided((3, 29, D), step, t.storage_offset()) for t in line)
        lens = torch.tensor([29, 0, 11], device="cuda", dtype=torch.int32)
        for n in (None, lens):
            a = gated.prism_layer_norm(x, weight=w, bias=b, seq_lens=n)
            assert torch.equal(a, gated.prism_layer_norm(x.contiguous(), weight=w, bias=b, seq_lens=n))
            a = gated.prism_layer_norm_backward(x, do, weight=w, bias=b, seq_lens=n)
            c = gated.prism_layer_norm_backward(x.contiguous(), do.contiguous(), weight=w, bias=b, seq_lens=n)
            assert all(torch.equal(a[m], c[m]) for m in c)


def test_rows_apart():
    """A row that is not finite leaves the others alone, and the sums of the weights are not finite."""
    z = make(1, 40, 64, "f32")
    c = {n: t.cuda() for n, t in z.items()}
    run = lambda: (gated.prism_layer_norm(c["x"], weight=c["w"], bias=c["b"]),  # noqa: E731
                   gated.prism_layer_norm_backward(c["x"], c["d"], weight=c["w"], bias=c["b"]))
    y, g = run()
    c["x"][0, 11, 3] = float("inf")
    y2, g2 = run()
    keep = torch.arange(40, device="cuda") != 11
    assert torch.equal(y[:, keep], y2[:, keep]) and torch.equal(g["x"][:, keep], g2["x"][:, keep])
    assert not torch.isfinite(y2[0, 11]).all() and not torch.isfinite(g2["weight"]).any()
    assert torch.equal(g["bias"], g2["bias"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [72, 2048])
def test_the_same_bits_twice(D, dtype):
    z = make(4, 999, D, dtype)
    a, b = check(z), check(z)
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[1][n], b[1][n]) for n in a[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_only_what_is_asked_for(dtype):
    """Weight or bias alone: the same values as with both."""
    z = make(2, 30, 264, dtype)
    c = {n: t.cuda() for n, t in z.items()}
    both = gated.prism_layer_norm_backward(c["x"], c["d"], weight=c["w"], bias=c["b"])
    one = gated.prism_layer_norm_backward(c["x"], c["d"], weight=c["w"])
    assert one["bias"] is None and torch.equal(one["weight"], both["weight"]) and torch.equal(one["x"], both["x"])
    ones = torch.ones(264, device="cuda")
    plain = gated.prism_layer_norm_backward(c["x"], c["d"], weight=ones, bias=c["b"])
    one = gated.prism_layer_norm_backward(c["x"], c["d"], bias=c["b"])
    assert one["weight"] is None and torch.equal(one["bias"], plain["bias"]) and torch.equal(one["x"], plain["x"])
    y = gated.prism_layer_norm(c["x"], bias=c["b"])
    assert torch.equal(y, gated.prism_layer_norm(c["x"], weight=ones, bias=c["b"]))


def test_gradient_by_differences():
    z = make(2, 6, 40, "f32")
    _, g = check(z)
    _, bound = go.layer_norm_back(z["x"], z["d"], z["w"], 1e-5)
    for n, m in (("x", "x"), ("w", "weight"), ("b", "bias")):
        v = torch.randn(z[n].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)

        def loss(h):
            y = {k: z[k].double() for k in "xwb"}
            y[n] = y[n] + h * v
            return (go.layer_norm(y["x"], y["w"], y["b"], 1e-5)[0] * z["d"].double()).sum().item()

        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        mine = g[m].double().cpu()
        tol = ((bound[m] + go.U * mine.abs()) * v.abs()).sum().item()
        assert abs((mine * v).sum().item() - slope) <= tol + 1e-6 * (1 + (mine * v).abs().sum().item()), n
