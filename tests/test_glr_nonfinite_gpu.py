"""NaN among the inputs of the gated linear recurrence, both rules, on every way that a row is laid out (short rows,
the last lane's overlap, waves, segments, one token): where the definition gives NaN, so do the outputs, the states and the
gradients, and what it does not reach keeps the bits that it has without it."""
import numpy as np
import pytest

from helpers import f64, from_dev, log
from oracle import glr as O
from test_glr_gpu import NAMES, args, gradients, make, oracle_args, put

pytestmark = pytest.mark.gpu

B, D, ROW, CH = 2, 5, 1, 2
NAN = float("nan")
#       L    waves segments: a short row; of bf16, a last lane that overlaps; one wave; segments
LAYOUTS = [(1, 0, 0), (7, 0, 0), (100, 0, 0), (255, 0, 0), (1500, 0, 0), (1503, 0, 0), (1503, 1, 0), (1100, 2, 3)]


def nan_where(ref, got, what):
    """Where the definition gives NaN, the GPU does."""
    bad = np.isnan(ref) & ~np.isnan(from_dev(got))
    assert not bad.any(), "%s: %d numbers are not NaN" % (what, bad.sum())


def planted(x, t, name, at):
    """The inputs with a NaN at one token of one channel (or in the channel's bias)."""
    q, v = {**t, name: t[name].clone()}, dict(x)
    v[name] = x[name].copy()
    where = (CH,) if name.endswith("bias") else (ROW, CH, at)
    q[name][where] = NAN
    v[name][where] = 0x7fc0 if v[name].dtype == np.uint16 else NAN
    return v, q


@pytest.mark.parametrize("L,waves,segments", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("blend", [True, False])
@pytest.mark.parametrize("name", ["x", "r", "i", "z", "r_bias", "i_bias"])
def test_nan_is_not_lost(name, blend, dtype, L, waves, segments, dev):
    import torch
    import selective_state_space_75_amd as m
    log("[glr nan] %s" % ((name, blend, dtype, L, waves, segments),))
    x = make(B, D, L, dtype, 30 + L, blend, True, True, True)
    t = put(x, dev, NAMES)
    v, q = planted(x, t, name, L // 2)
    kw = dict(blend=blend, return_final_state=True)
    with m.glr_test_knobs(waves=waves, segments=segments):
        clean = m.glr_fwd(*args(t), initial_state=t["initial_state"], **kw)
        y, h = m.glr_fwd(*args(q), initial_state=q["initial_state"], **kw)
        gc, g = gradients(t, t["dy"], blend, None), gradients(q, q["dy"], blend, None)
        torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        yr, hr = O.glr(*oracle_args(v), blend=blend, initial_state=x["initial_state"])
        ref = O.glr_bwd(*oracle_args(v), f64(x["dy"]), blend=blend, initial_state=x["initial_state"],
                        dfinal_state=x["dfinal_state"])
    assert np.isnan(yr).any()
    for a, r, n in ((y, yr, "y"), (h, hr, "final state")):
        nan_where(r, a, n)
        assert not (np.isnan(from_dev(a)) & ~np.isnan(r)).any(), n
    assert torch.equal(y[torch.from_numpy(~np.isnan(yr)).to(dev)], clean[0][torch.from_numpy(~np.isnan(yr)).to(dev)])
    assert torch.equal(h[torch.from_numpy(~np.isnan(hr)).to(dev)], clean[1][torch.from_numpy(~np.isnan(hr)).to(dev)])
    own = torch.zeros((B, D), dtype=torch.bool, device=dev)
    own[slice(None) if name.endswith("bias") else ROW, CH] = True
    for n in g:
        if g[n] is None:
            continue
        nan_where(ref[n], g[n], n)
        keep = ~(own.any(0) if g[n].dim() == 1 else own)
        assert torch.equal(g[n][keep], gc[n][keep]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("blend", [True, False])
@pytest.mark.parametrize("name", ["x", "r", "i", "z", "r_bias", "i_bias"])
def test_nan_in_one_token(name, blend, dtype, dev):
    import torch
    import selective_state_space_75_amd as m
    x = make(B, D, 1, dtype, 60, blend, True, True, True)
    t = put(x, dev, NAMES)
    v, q = planted(x, t, name, 0)
    got = []
    for s in (t, q):
        pool = s["initial_state"].clone()
        one = {k: s[k].squeeze(2) for k in ("x", "r", "i", "z")}
        got.append((m.glr_update(pool, *args({**s, **one}), blend=blend), pool))
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        ref = O.glr(*oracle_args(v), blend=blend, initial_state=x["initial_state"])
    for clean, a, r, n in zip(got[0], got[1], (ref[0][..., 0], ref[1]), ("y", "state")):
        assert np.array_equal(np.isnan(from_dev(a)), np.isnan(r)), n
        keep = torch.from_numpy(~np.isnan(r)).to(dev)
        assert torch.equal(a[keep], clean[keep]), n


@pytest.mark.parametrize("L,waves,segments", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_growing_decay_gives_nan(dtype, L, waves, segments, dev):
    """A above zero: sqrt(1 - a^2) has no value.  A row without tokens keeps its state all the same."""
    import torch
    import selective_state_space_75_amd as m
    x = make(3, D, L, dtype, 70 + L, False, True, True, True)
    t = put(x, dev, NAMES)
    lengths = [L, L - L // 3, 0]
    ln = torch.tensor(lengths, dtype=torch.int32, device=dev)
    up = np.float32([0.0, 0.01, 0.5, 3.0, 90.0])                 # added in: channel 0 stays as it is
    q = {**t, "A": t["A"].clone()}
    q["A"][1:] = torch.from_numpy(up[1:]).to(dev)
    with m.glr_test_knobs(waves=waves, segments=segments):
        kw = dict(lengths=ln, return_final_state=True)
        clean = m.glr_fwd(*args(t), initial_state=t["initial_state"], **kw)
        y, h = m.glr_fwd(*args(q), initial_state=q["initial_state"], **kw)
        gc, g = gradients(t, t["dy"], False, ln), gradients(q, q["dy"], False, ln)
        torch.cuda.synchronize()
    for b, n in enumerate(lengths):
        assert torch.isnan(y[b, 1:, :n]).all() and not y[b, :, n:].any()
        assert torch.isnan(h[b, 1:]).all() if n else torch.equal(h[b], t["initial_state"][b])
    assert torch.equal(y[:, 0], clean[0][:, 0]) and torch.equal(h[:, 0], clean[1][:, 0])
    for n in g:
        assert torch.equal(g[n][..., 0] if g[n].dim() < 3 else g[n][:, 0], gc[n][..., 0] if g[n].dim() < 3 else gc[n][:, 0]), n
    live = torch.arange(L, device=dev) < ln[:, None]
    for n in ("dx", "dr", "di", "dz"):
        assert torch.isnan(g[n][:, 1:].transpose(1, 2)[live]).all(), n
    for n in ("dA", "dr_bias", "di_bias"):
        assert torch.isnan(g[n][1:]).all(), n
    assert torch.equal(g["dinitial_state"][2], t["dfinal_state"][2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_growing_decay_gives_nan_in_one_token(dtype, dev):
    import torch
    import selective_state_space_75_amd as m
    x = make(B, D, 1, dtype, 71, False, True, True, True)
    t = put(x, dev, NAMES)
    t["A"][1:] = torch.tensor([0.01, 0.5, 3.0, 90.0], device=dev)
    pool = t["initial_state"].clone()
    y = m.glr_update(pool, *args({**t, **{k: t[k].squeeze(2) for k in ("x", "r", "i", "z")}}))
    torch.cuda.synchronize()
    assert torch.isnan(y[:, 1:]).all() and torch.isnan(pool[:, 1:]).all()
    assert torch.isfinite(y[:, 0]).all() and torch.isfinite(pool[:, 0]).all()


@pytest.mark.parametrize("L,waves,segments", LAYOUTS)
@pytest.mark.parametrize("name,value,blend", [(n, v, blend) for n in ("r_bias", "i_bias") for v in (np.inf, -np.inf)
                                              for blend in (True, False)] + [("A", -np.inf, False), ("A", -3.4e38, False)])
def test_infinite_parameters_are_gates_held_open_or_closed(name, value, blend, L, waves, segments, dev):
    """Absent tokens, behind a length or behind L in a wave's last lanes, are absent for such a channel too.  The bars are
    those of the finite gates.  (dr of A = -inf is 0 * inf.)"""
    import torch
    import selective_state_space_75_amd as m
    from test_glr_gpu import E, near
    x = make(3, D, L, "f32", 90 + L, blend, True, True, True)
    x[name][CH] = value
    t = put(x, dev, NAMES)
    for lengths in (None, [L, L - L // 3, 0]):
        ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)
        with m.glr_test_knobs(waves=waves, segments=segments):
            y, h = m.glr_fwd(*args(t), blend=blend, initial_state=t["initial_state"], lengths=ln, return_final_state=True)
            g = gradients(t, t["dy"], blend, ln)
            torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            yr, hr = O.glr(*oracle_args(x), blend=blend, initial_state=x["initial_state"], lengths=lengths)
            ref = O.glr_bwd(*oracle_args(x), f64(x["dy"]), blend=blend, initial_state=x["initial_state"],
                            dfinal_state=x["dfinal_state"], lengths=lengths)
        near(y, yr, E, "y")
        near(h, hr, E, "final state")
        for n in ("dx", "dr", "di", "dz", "dA", "dr_bias", "di_bias", "dinitial_state"):
            if g[n] is None or name == "A" and n in ("dr", "dr_bias"):
                continue
            near(g[n], ref[n], 2 * E, n, ref["scale"].get(n))


@pytest.mark.parametrize("L,waves,segments", LAYOUTS)
@pytest.mark.parametrize("name,blend", [("r_bias", True), ("r_bias", False), ("i_bias", True), ("i_bias", False), ("A", False)])
def test_a_row_without_tokens_looks_at_no_parameter(name, blend, L, waves, segments, dev):
    import torch
    import selective_state_space_75_amd as m
    x = make(2, D, L, "bf16", 110 + L, blend, True, True, True)
    t = put(x, dev, NAMES)
    t[name][CH] = NAN
    ln = torch.tensor([0, 0], dtype=torch.int32, device=dev)
    with m.glr_test_knobs(waves=waves, segments=segments):
        y, h = m.glr_fwd(*args(t), blend=blend, initial_state=t["initial_state"], lengths=ln, return_final_state=True)
        g = gradients(t, t["dy"], blend, ln)
        torch.cuda.synchronize()
    assert torch.equal(h, t["initial_state"]) and torch.equal(g["dinitial_state"], t["dfinal_state"])
    assert not y.any()
    for n in ("dx", "dr", "di", "dz", "dA", "dr_bias", "di_bias"):
        assert g[n] is None or not g[n].any(), n              # NaN is not zero either


@pytest.mark.parametrize("L,waves,segments", LAYOUTS)
@pytest.mark.parametrize("blend", [True, False])
def test_absent_tokens_leave_nothing_in_the_sums(blend, L, waves, segments, dev):
    """Channels whose tokens add nothing (no gradient but the final state's, behind rows' ends or of closed gates): zeros, not
    very small numbers."""
    import torch
    import selective_state_space_75_amd as m
    x = make(2, D, L, "f32", 140 + L, blend, True, True, True)
    t = put(x, dev, NAMES)
    zero = torch.zeros_like(t["dy"])
    for r, lengths in ((t["r"], [0, 0]), (torch.full_like(t["r"], -np.inf), None)):
        ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)
        q = {**t, "r": r}
        with m.glr_test_knobs(waves=waves, segments=segments):
            g = gradients(q, zero, blend, ln)
            torch.cuda.synchronize()
        assert torch.equal(g["dinitial_state"], t["dfinal_state"])
        for n in ("dr", "dA", "dr_bias"):
            assert g[n] is None or not g[n].any(), n


@pytest.mark.parametrize("name,value,blend", [(n, v, blend) for n in ("r_bias", "i_bias") for v in (np.inf, -np.inf)
                                              for blend in (True, False)] + [("A", -np.inf, False), ("A", -3.4e38, False)])
def test_infinite_parameters_in_one_token(name, value, blend, dev):
    """As in a sequence of one token, also where r closes the gate to its last bit."""
    import torch
    import selective_state_space_75_amd as m
    from test_glr_gpu import E, near
    x = make(4, D, 1, "f32", 150, blend, True, True, True)
    x[name][CH] = value
    x["r"][2] = -200.0
    t = put(x, dev, NAMES)
    y, h = m.glr_fwd(*args(t), blend=blend, initial_state=t["initial_state"], return_final_state=True)
    pool = t["initial_state"].clone()
    y1 = m.glr_update(pool, *args({**t, **{k: t[k].squeeze(2) for k in ("x", "r", "i", "z")}}), blend=blend)
    torch.cuda.synchronize()
    near(y1, from_dev(y)[..., 0], E, "y")
    near(pool, from_dev(h), E, "state")
