"""Layer norm with several tiles of rows for every CTA, in each class of widths: stages that are filled again, parities
that turn twice, and the weights' sums over all rows, within the bounds of tests/norm_bounds.py (which see a row that is left out)."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated
from tests import norm_bounds as nb
from tests.test_norm_bounds import ROWS

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Widths, and the rows of 2 S + 1 tiles for every CTA of the direction that takes more: rows of a tile x CTAs x (2 S + 1).
MANY = {"bf16": [(24, 32 * 8 * 304 * 7), (56, 16 * 12 * 152 * 7), (96, 16 * 2432 * 7), (128, 8 * 2432 * 7), (192, 8 * 2432 * 7),
                 (256, 8 * 1824 * 7), (384, 4 * 2432 * 7), (512, 4 * 1824 * 7), (768, 2 * 2432 * 7), (1024, 2 * 1824 * 7), (1528, 2 * 1216 * 7),
                 (2048, 4 * 456 * 9), (2552, 4 * 456 * 7), (4096, 4 * 304 * 7), (6136, 4 * 152 * 5), (8192, 4 * 152 * 5),
                 (16384, 2 * 152 * 5)],
        "f32": [(24, 128 * 304 * 3), (64, 64 * 304 * 3), (128, 32 * 304 * 3), (160, 64 * 152 * 5), (256, 16 * 304 * 3), (304, 32 * 152 * 5),
                (384, 16 * 152 * 7), (512, 8 * 304 * 3), (640, 16 * 152 * 5), (832, 2 * 608 * 7), (1024, 4 * 304 * 3), (1272, 2 * 456 * 7),
                (2048, 2 * 304 * 7), (2552, 2 * 304 * 5), (4096, 304 * 7), (8192, 152 * 7), (16384, 152 * 3)]}


def check(rows, D, dtype, ragged, T=37):
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    B = rows // T + 1                                     # a remainder that no tile divides
    x = (n(B, T, D) * (1 + n(D).abs()) + 0.5).to(TYPES[dtype])
    d, w, b = n(B, T, D).to(TYPES[dtype]), 1 + 0.3 * n(D), n(D)
    lens = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    there = torch.arange(T, device="cuda") < (T if lens is None else lens[:, None])
    there = there.expand(B, T)
    y = gated.prism_layer_norm(x, weight=w, bias=b, seq_lens=lens)
    got = gated.prism_layer_norm_backward(x, d, weight=w, bias=b, seq_lens=lens)
    want, bound = nb.forward(x[there], w, b, 1e-5)
    assert nb.worst(y[there], want, bound, x.dtype) <= 0, "y"
    want, bounds = nb.backward(x[there], d[there], w, 1e-5)
    assert nb.worst(got["x"][there], want["x"], bounds["x"], x.dtype) <= 0, "dx"
    for m in ("weight", "bias"):
        assert nb.worst(got[m], want[m], bounds[m]) <= 0, m
    assert (y[~there] == 0).all() and (got["x"][~there] == 0).all()
    assert gated.gated_status() == 0


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dtype,D,rows", [(t, *c) for t, cs in MANY.items() for c in cs])
def test_many_tiles(dtype, D, rows, ragged):
    check(rows, D, dtype, ragged)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", ROWS)
def test_rows(rows, D, dtype):
    check(rows, D, dtype, False, T=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [24, 96, 160, 512, 2048, 4096])
def test_tiles_without_a_row(dtype, D):
    """Sequences that are not there, between those that are: a tile that copies nothing is done at once, and its rows are 0."""
    g = torch.Generator(device="cuda").manual_seed(D)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    B, T = 400, 70
    x, d, w, b = n(B, T, D).to(TYPES[dtype]), n(B, T, D).to(TYPES[dtype]), n(D), n(D)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[::3] = T
    x[1::3] = float("nan")
    y = gated.prism_layer_norm(x, weight=w, bias=b, seq_lens=lens)
    got = gated.prism_layer_norm_backward(x, d, weight=w, bias=b, seq_lens=lens)
    alone = gated.prism_layer_norm(x[::3].contiguous(), weight=w, bias=b)
    assert torch.equal(y[::3], alone) and (y[1::3] == 0).all() and (y[2::3] == 0).all()
    want, bounds = nb.backward(x[::3], d[::3], w, 1e-5)
    assert nb.worst(got["x"][::3], want["x"], bounds["x"], x.dtype) <= 0 and (got["x"][1::3] == 0).all()
    assert nb.worst(got["weight"], want["weight"], bounds["weight"]) <= 0 and nb.worst(got["bias"], want["bias"], bounds["bias"]) <= 0
