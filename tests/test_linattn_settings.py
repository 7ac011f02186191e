"""Settings of the linear attention calls (CPU): their values count at the time of the call, whatever
object holds them."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn
from tests.test_linattn_streams import World, operands


@pytest.fixture
def world(monkeypatch):
    yield World(monkeypatch)
    for c in (linattn._rope_dims, linattn._linattn_dims, linattn._decode_dims):
        c.cache_clear()


def dims(world, kind):
    """The dims that the last call passed."""
    return kind.from_address(world.calls[-1][1][0])


@pytest.mark.parametrize("holder", [lambda v: torch.tensor(v), lambda v: torch.tensor([v])[0], float])
def test_a_setting_that_changes_between_calls(world, holder):
    """A scale held in a tensor that is changed in place: each call takes the value that it has then."""
    x, c = operands(), holder(0.5)
    for value in (0.5, 2.0):
        if isinstance(c, torch.Tensor):
            c.fill_(value)
        else:
            c = value
        linattn.prism_linattn_forward(x.q, x.k, x.v, x.ld, scale=c)
        assert dims(world, linattn.LinattnDims).scale == value
        linattn.prism_linattn_backward(x.q, x.k, x.v, x.ld, x.do, scale=c)
        assert dims(world, linattn.LinattnDims).scale == value
        linattn.prism_linattn_decode_step(x.q1, x.q1, x.q1, x.ld, x.s, scale=c)
        assert dims(world, linattn.LinattnDims).scale == value
        linattn.prism_qk_norm_rope(x.q, x.k, x.table, q_scale=c, k_scale=c, eps=c)
        d = dims(world, linattn.RopeDims)
        assert d.q_scale == d.k_scale == d.eps == value
        linattn.prism_qk_norm_rope_backward(x.q, x.k, x.table, x.do, x.do, q_scale=c, k_scale=c, eps=c)
        d = dims(world, linattn.RopeDims)
        assert d.q_scale == d.k_scale == d.eps == value


def test_a_flag_held_in_a_tensor(world):
    x, on = operands(), torch.tensor(True)
    for value in (True, False):
        on.fill_(value)
        linattn.prism_qk_norm_rope(x.q, x.k, x.table, interleaved=on)
        assert dims(world, linattn.RopeDims).flags == (linattn.PRISM_ROPE_INTERLEAVED if value else 0)
