"""What the bf16 terms of a decayed key leave of it (CPU)."""
import torch

from tests import linattn_oracle as lo


def split(x, terms):
    """The sum of `terms` bf16 terms of fp32 x."""
    got, left = torch.zeros_like(x), x
    for _ in range(terms):
        t = left.bfloat16().float()
        got, left = got + t, left - t
    return got


def test_a_lost_third_term_is_seen():
    """59 u hold for three terms of a decayed key, and not for two."""
    g = torch.Generator().manual_seed(1)
    k = torch.nn.functional.normalize(torch.randn(200, 64, generator=g), dim=-1).bfloat16().float()
    w = torch.exp(-1e-3 * torch.arange(200, dtype=torch.float64))[:, None].float()
    x = w * k
    off = {n: ((split(x, n).double() - x.double()).abs() / x.double().abs()).max().item() / lo.U for n in (2, 3)}
    assert off[3] <= 1.0 and off[2] > 2 * 59
