"""The 64-bit oracle of the gated recurrent layer (CPU): its gradients against differences of its own forward
pass and against automatic differentiation, and the joins of runs that the kernels use."""
import pytest
import torch

from tests import gated_oracle as go


def make(B, T, D, gated, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(x=n(B, T, D), f=n(B, T, D) + 2, i=n(B, T, D) if gated else None, s0=n(B, D), do=n(B, T, D), ds=n(B, D),
                lens=torch.tensor([T, T // 2, 0][:B]))


@pytest.mark.parametrize("gated", [True, False])
def test_scan_gradients(gated):
    """Of L = sum(out do) + sum(final ds), by autograd and by central differences along a random direction."""
    z = make(3, 9, 4, gated)
    names = [n for n in ("x", "f", "i", "s0") if z[n] is not None]
    leaves = {n: z[n].clone().requires_grad_() for n in names}

    def loss(v):
        s = go.scan(v["x"], v["f"], v.get("i"), v["s0"], z["lens"])
        return (s["out"] * z["do"]).sum() + (s["final"] * z["ds"]).sum()

    auto = dict(zip(names, torch.autograd.grad(loss(leaves), [leaves[n] for n in names])))
    got, _ = go.scan_back(z["x"], z["f"], z["do"], z["i"], z["s0"], z["ds"], z["lens"])
    for n, m in (("x", "x"), ("f", "forget"), ("i", "input_gate"), ("s0", "initial_state")):
        if n in auto:
            assert torch.allclose(got[m], auto[n], rtol=1e-12, atol=1e-13)
            v = torch.randn_like(z[n])
            at = lambda h: loss({**{k: z[k] for k in names}, n: z[n] + h * v}).item()  # noqa: E731, B023
            slope = (at(1e-5) - at(-1e-5)) / 2e-5
            assert abs(slope - (got[m] * v).sum().item()) <= 1e-7 * (1 + abs(slope))
    assert (got["input_gate"] is None) == (not gated)


def test_layer_norm_gradients():
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, d, lens = 3 + n(2, 5, 16), n(16), n(16), n(2, 5, 16), torch.tensor([5, 2])
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y, _ = go.layer_norm(*leaves, 1e-5, lens)
    auto = torch.autograd.grad((y * d).sum(), leaves)
    got, _ = go.layer_norm_back(x, d, w, 1e-5, lens)
    for a, m in zip(auto, ("x", "weight", "bias")):
        assert torch.allclose(a, got[m], rtol=1e-11, atol=1e-12)
    live = torch.nn.functional.layer_norm(x, (16,), w, b, 1e-5) * (torch.arange(5) < lens[:, None])[..., None]
    assert torch.allclose(y.detach(), live, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("backward", [False, True])
def test_runs_joined(backward):
    """A run of tokens maps h to P h + L; run after run gives the recurrence, from either end."""
    z = make(1, 37, 3, True)
    a, _, w, _ = go.gates(z["f"], z["i"])
    if backward:                                          # r_t = a_t r_(t+1) + a_t dout_t
        a, u = a.flip(1), (a * z["do"]).flip(1)
    else:
        u = w * z["x"]
    h = z["s0"].clone()
    want = []
    for t in range(37):
        h = a[:, t] * h + u[:, t]
        want.append(h)
    h = z["s0"].clone()
    for first in range(0, 37, 8):
        P, L = torch.ones_like(h), torch.zeros_like(h)
        for t in range(first, min(first + 8, 37)):
            P, L = a[:, t] * P, a[:, t] * L + u[:, t]
        h = P * h + L
        assert torch.allclose(h, want[min(first + 8, 37) - 1], rtol=1e-12, atol=1e-13)


def test_bounds_are_tight_enough():
    """The bounds see a gate rounded to bf16 and a token that is left out."""
    z = make(1, 200, 8, True, seed=5)
    s = go.scan(z["x"], z["f"], z["i"], z["s0"])
    off = go.scan(z["x"], z["f"] * (1 + 2.0 ** -9), z["i"], z["s0"])["out"] - s["out"]
    assert (off.abs() > s["err"][:, 1:]).float().mean() > 0.9
    x = z["x"].clone()
    x[:, 100] = 0
    off = go.scan(x, z["f"], z["i"], z["s0"])["out"] - s["out"]
    assert (off.abs() > s["err"][:, 1:])[:, 100:110].all()
