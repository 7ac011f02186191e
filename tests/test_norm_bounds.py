"""The bounds of tests/norm_bounds.py (CPU): they hold for sums in 32 bits, and they see one row that is left out."""
import pytest
import torch

from tests import gated_oracle as go
from tests import norm_bounds as nb

ROWS = [(20000, 32), (20000, 64), (2100, 2000), (3500, 1000), (3001, 520), (2100, 24), (18003, 64), (9000, 96), (9000, 128), (8002, 160),
        (8000, 192), (6000, 256), (4000, 288), (4000, 384), (2000, 800), (1500, 1280), (1100, 2560), (700, 6144)]


def make(rows, D):
    g = torch.Generator().manual_seed(rows + D)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return n(rows, D) * (1 + n(D).abs()) + 0.5, n(rows, D), 1 + 0.3 * n(D), n(D)


@pytest.mark.parametrize("rows,D", ROWS)
def test_a_row_that_is_left_out_is_seen(rows, D):
    x, d, w, _ = make(rows, D)
    n, _, _, _ = nb.parts(x, 1e-5)
    want, bound = nb.backward(x, d, w, 1e-5)
    terms = {"weight": d.double() * n, "bias": d.double()}
    for m, t in terms.items():
        for row in (0, rows // 2, rows - 1):
            assert (t[row].abs() > 2 * bound[m]).any(), (m, row)


@pytest.mark.parametrize("rows,D", [(4000, 64), (700, 520)])
def test_the_same_as_the_other_oracle(rows, D):
    x, d, w, b = make(rows, D)
    y, bound = nb.forward(x, w, b, 1e-5)
    other, loose = go.layer_norm(x[None], w, b, 1e-5)
    assert torch.allclose(y, other[0], rtol=1e-13, atol=1e-13) and (bound <= loose[0]).all()
    got, bounds = nb.backward(x, d, w, 1e-5)
    other, loose = go.layer_norm_back(x[None], d[None], w, 1e-5)
    for m in got:
        a, c = (other[m][0], loose[m][0]) if m == "x" else (other[m], loose[m])
        assert torch.allclose(got[m], a, rtol=1e-11, atol=1e-11) and (bounds[m] <= c).all()


def test_32_bits_stay_within():
    x, d, w, b = make(3000, 136)
    m = x.mean(-1, keepdim=True)
    r = ((x - m).square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    n, g = (x - m) * r, d * w
    y, bound = nb.forward(x, w, b, 1e-5)
    assert nb.worst(n * w + b, y, bound, torch.float32) <= 0
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    want, bound = nb.backward(x, d, w, 1e-5)
    assert nb.worst(dx, want["x"], bound["x"], torch.float32) <= 0
    assert nb.worst((d * n).sum(0), want["weight"], bound["weight"]) <= 0 and nb.worst(d.sum(0), want["bias"], bound["bias"]) <= 0
    assert nb.worst(d[:-1].sum(0), want["bias"], bound["bias"]) > 0
