"""What the bounds of the linear attention tests can tell apart (CPU): mistakes planted in the oracle."""
import pytest
import torch

from tests import linattn_oracle as lo

SLOW = torch.tensor([0.0, -1e-4, -2e-3], dtype=torch.float64)


def draw(T, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = [torch.nn.functional.normalize(n(1, T, 3, D), dim=-1) for _ in range(2)] + [n(1, T, 3, D)]
    return [t.bfloat16().double() for t in x] + [n(1, 3, D, D).double()]


@pytest.mark.parametrize("D", [16, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_lost_run_or_state_is_seen(D, dtype):
    """Runs of 256 tokens whose start leaves out one earlier run, or the initial state: seen in the
    final state and in the outputs, for every head."""
    T, run = 1300, 256
    q, k, v, s0 = draw(T, D)
    o, s = lo.linattn(q, k, v, SLOW, 1.0, s0)
    mo, ms = lo.linattn(q.abs(), k.abs(), v.abs(), SLOW, 1.0, s0.abs())
    bo, bs = lo.out_bound(o, mo, dtype, T, D), lo.state_bound(ms, dtype, T, D)
    lost = [(v * (torch.arange(T) // run != 1)[None, :, None, None], s0), (v, torch.zeros_like(s0))]
    for value, start in lost:
        o1, s1 = lo.linattn(q, k, value, SLOW, 1.0, start)
        for h in range(3):
            assert ((s1 - s).abs() > bs)[0, h].double().mean() > 0.5
            after = slice(2 * run, T) if dtype == torch.float32 else slice(2 * run, 3 * run)
            assert ((o1 - o).abs() > bo)[0, after, h].any()
