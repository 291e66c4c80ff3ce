"""States that go on: the final state of one call is the initial state of the next, in two buffers that change places."""
import numpy as np
import pytest

from helpers import from_dev
from oracle import glr as O
from test_glr_gpu import E, NAMES, args, make, near, oracle_args, put

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [40, 3000, 9000])
def test_pieces_of_a_sequence_go_on_from_state_to_state(L, dev):
    """Three pieces against the oracle's whole sequence; each state written into the buffer of the one before last."""
    import torch
    import selective_state_space_75_amd as m
    B, D = 1, 3
    x = make(B, D, 3 * L, "f32", 130 + L, False, True, True, True)
    t = put(x, dev, NAMES)
    yr, hr = O.glr(*oracle_args(x), initial_state=x["initial_state"])
    states = [t["initial_state"].clone(), torch.empty_like(t["initial_state"])]
    for k in range(3):
        part = {n: t[n][:, :, k * L:(k + 1) * L].contiguous() for n in ("x", "r", "i", "z")}
        with pytest.raises(ValueError, match="overlap"):
            m.glr_fwd(*args({**t, **part}), initial_state=states[0], return_final_state=True, final_state=states[0])
        y, h = m.glr_fwd(*args({**t, **part}), initial_state=states[0], return_final_state=True, final_state=states[1])
        assert h is states[1]
        near(y, yr[:, :, k * L:(k + 1) * L], E, "piece %d" % k)
        states.reverse()
    near(states[0], hr, E, "final state")


def test_a_token_is_refused_over_its_own_states(dev):
    import torch
    import selective_state_space_75_amd as m
    pool = torch.zeros(3, 4, device=dev)
    x, A = torch.ones(2, 4, device=dev), -torch.ones(4, device=dev)
    with pytest.raises(ValueError, match="y must not overlap"):
        m.glr_update(pool, x, x.clone(), None, A, y=pool[:2])
    with pytest.raises(ValueError, match="state must not overlap"):
        m.glr_update(pool, pool[1:], x, None, A)
    assert not from_dev(pool).any()
