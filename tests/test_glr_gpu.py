"""The gated linear recurrence on the GPU against the fp64 oracle: lengths from one token to several
segments, every cut of a row over waves and segments, all types, options, padded batches, channel
ranges, NaN and infinities, alignments, pools of states.

Bars.  fp32 outputs: a state sums about M = 1 / (|A| s) inputs; every step multiplies it by a decay that
is off by about two units of 2^-24 (the hardware's exp2 and its rounded argument) and rounds once, with
either sign, so that it is off by about sqrt(M) 1.8e-7 of itself: 4e-6 for the slowest channels here
(|A| = 0.008, s = 1/4), less for all others; the bar is 1e-5 relative L2 (the framework's fp32 bar).
Gradients are products of an adjoint and a state of that kind, 2e-5, relative to the magnitudes that they
are differences of (the oracle's "scale").  bf16 outputs add one rounding, 2^-8 of each number at most."""
import numpy as np
import pytest

from helpers import f64, from_dev, log, rel_l2, to_dev
from oracle import glr as O
from selective_state_space_75_amd import workloads as W

pytestmark = pytest.mark.gpu

E = 1e-5


def bar(t, e=E):
    import torch
    return 2.0 ** -8 * (1 + e) + e if t.dtype == torch.bfloat16 else e


def near(t, ref, e, what, scale=None):
    """||t - ref|| within e ||scale||, and one bf16 rounding of the result where there is one."""
    import torch
    got = from_dev(t)
    assert np.isfinite(got).all(), what
    err = np.linalg.norm(got - ref)
    size = np.linalg.norm(ref if scale is None else scale)
    bound = e * size + (2.0 ** -8 * (np.linalg.norm(ref) + e * size) if t.dtype == torch.bfloat16 else 0.0)
    log("  %s: off by %.3e of %.3e allowed" % (what, err, bound))
    assert err <= bound or size == 0.0 and err == 0.0, what


def put(x, dev, names, ranges=False):
    """Inputs on the GPU; with ranges, as channel ranges of one wider tensor."""
    import torch
    t = {n: to_dev(x[n], dev) for n in names if x.get(n) is not None}
    if ranges:
        big = [n for n in ("x", "r", "i", "z") if n in t]
        wide = torch.cat([t[n] for n in big] + [torch.full_like(t["x"][:, :3], float("nan"))], 1)
        D = t["x"].shape[1]
        for k, n in enumerate(big):
            t[n] = wide[:, k * D:(k + 1) * D]
    return t


def make(B, D, L, dtype, seed, blend, with_i, with_z, init):
    x = W.glr_inputs(B, D, L, dtype, seed)
    if blend:
        x["A"] = None
    if not with_i:
        x["i"] = x["i_bias"] = None
    if not with_z:
        x["z"] = None
    if not init:
        x["initial_state"] = x["dfinal_state"] = None
    return x


NAMES = ("x", "r", "i", "z", "A", "r_bias", "i_bias", "initial_state", "dfinal_state", "dy")


def args(t):
    return [t.get(n) for n in ("x", "r", "i", "A", "r_bias", "i_bias", "z")]


def oracle_args(x):
    big = ("x", "r", "i", "z")
    return [None if x[n] is None else f64(x[n]) if n in big else x[n].astype(np.float64)
            for n in ("x", "r", "i", "A", "r_bias", "i_bias", "z")]


#        B  D   L     dtype   out    blend  i     z     init  lengths          ranges waves segments
CASES = [(1, 1, 1, "f32", "f32", False, True, True, True, None, False, 0, 0),
         (2, 3, 2, "bf16", "f32", True, True, True, True, None, False, 0, 0),
         (3, 5, 7, "f32", "bf16", False, False, True, False, [7, 0, 3], False, 0, 0),
         (1, 70, 8, "bf16", "bf16", False, True, False, True, None, True, 0, 0),
         (2, 33, 9, "f32", "f32", False, True, True, True, [9, 8], True, 0, 0),
         (1, 16, 256, "f32", "f32", True, False, True, False, None, False, 0, 0),
         (2, 6, 511, "bf16", "f32", False, True, True, True, [511, 505], True, 0, 0),
         (1, 6, 512, "f32", "f32", False, True, True, True, None, False, 1, 0),
         (2, 6, 513, "bf16", "f32", False, True, True, True, [513, 512], False, 1, 0),
         (2, 6, 1003, "bf16", "bf16", True, True, True, True, [1003, 600], True, 2, 0),
         (1, 4, 2048, "bf16", "f32", False, True, True, True, None, False, 4, 0),
         (1, 4, 2049, "f32", "f32", False, True, True, True, [2048], False, 3, 0),
         (2, 3, 2050, "f32", "f32", False, True, False, True, [17, 2050], False, 16, 2),
         (1, 3, 4100, "bf16", "f32", False, True, True, True, [4099], True, 1, 5),
         (1, 2, 1100, "f32", "f32", True, True, True, True, [1001], False, 1, 130),
         (2, 2, 8192, "bf16", "f32", False, False, True, True, None, False, 0, 0),
         (1, 3, 8193, "bf16", "f32", False, True, True, True, [8192], True, 0, 0),
         (1, 2, 17001, "f32", "f32", False, True, True, True, None, False, 0, 0),
         (2, 1, 40000, "bf16", "f32", False, True, True, False, [40000, 12345], False, 0, 0),
         (2, 300, 1100, "bf16", "f32", False, True, True, True, [1100, 801], True, 0, 3),     # rows enough to walk a row's tiles
         (1, 600, 700, "f32", "f32", True, True, False, True, None, False, 1, 0),
         (1, 515, 9000, "bf16", "f32", False, True, True, True, [8500], False, 0, 0),
         (8, 520, 600, "bf16", "f32", False, False, True, False, None, False, 0, 0)]


@pytest.mark.parametrize("B,D,L,dtype,out,blend,with_i,with_z,init,lengths,ranges,waves,segments", CASES)
def test_forward(B, D, L, dtype, out, blend, with_i, with_z, init, lengths, ranges, waves, segments, dev):
    import torch
    import selective_state_space_75_amd as m
    log("[glr fwd] %s" % ((B, D, L, dtype, out, blend, with_i, with_z, lengths, ranges, waves, segments),))
    x = make(B, D, L, dtype, 100 + L, blend, with_i, with_z, init)
    t = put(x, dev, NAMES, ranges)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)
    with m.glr_test_knobs(waves=waves, segments=segments):
        y, h = m.glr_fwd(*args(t), blend=blend, initial_state=t.get("initial_state"), lengths=ln,
                         return_final_state=True, out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
        torch.cuda.synchronize()
    yr, hr = O.glr(*oracle_args(x), blend=blend, initial_state=x["initial_state"], lengths=lengths)
    near(y, yr, E, "y")
    near(h, hr, E, "final state")
    if lengths is not None:
        for b in range(B):
            assert not from_dev(y)[b, :, max(0, lengths[b]):].any()


def gradients(t, dy, blend, ln, **kw):
    import selective_state_space_75_amd as m
    return m.glr_bwd(*args(t), dy, blend=blend, initial_state=t.get("initial_state"),
                     dfinal_state=t.get("dfinal_state"), lengths=ln, **kw)


def check_gradients(g, ref, x, what=""):
    for n in ("dx", "dr", "di", "dz", "dA", "dr_bias", "di_bias", "dinitial_state"):
        if g[n] is None:
            assert ref[n] is None or n == "dinitial_state" and x["initial_state"] is None
            continue
        near(g[n], ref[n], 2 * E, what + n, ref["scale"].get(n))


@pytest.mark.parametrize("B,D,L,dtype,out,blend,with_i,with_z,init,lengths,ranges,waves,segments", CASES)
def test_backward(B, D, L, dtype, out, blend, with_i, with_z, init, lengths, ranges, waves, segments, dev):
    import torch
    import selective_state_space_75_amd as m
    log("[glr bwd] %s" % ((B, D, L, dtype, out, blend, with_i, with_z, lengths, ranges, waves, segments),))
    x = make(B, D, L, dtype, 200 + L, blend, with_i, with_z, init)
    t = put(x, dev, NAMES, ranges)
    dy = t["dy"].to(torch.float32 if out == "f32" else torch.bfloat16)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)
    with m.glr_test_knobs(waves=waves, segments=segments):
        g = gradients(t, dy, blend, ln)
        torch.cuda.synchronize()
    ref = O.glr_bwd(*oracle_args(x), f64(from_dev(dy)), blend=blend, initial_state=x["initial_state"],
                    dfinal_state=x["dfinal_state"], lengths=lengths)
    check_gradients(g, ref, x)
    if lengths is not None:
        for n in ("dx", "dr", "di", "dz"):
            for b in range(B):
                assert g[n] is None or not from_dev(g[n])[b, :, max(0, lengths[b]):].any(), n


@pytest.mark.parametrize("with_i,with_z", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("blend", [False, True])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_every_split_of_every_type(dtype, out, blend, with_i, with_z, dev):
    """A wave, 16 waves, segments of few rows, and segments that one workgroup goes through."""
    for B, D, L, waves in ((2, 3, 301, 0), (1, 2, 8192, 0), (2, 2, 9001, 0), (1, 516, 1203, 1)):
        for test in (test_forward, test_backward):
            test(B, D, L, dtype, out, blend, with_i, with_z, True, [L - 5 * b for b in range(B)], False, waves, 0, dev)


@pytest.mark.parametrize("L", [1, 3, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 100, 127, 129, 250, 255, 256, 257, 511, 519])
def test_short_rows_and_their_last_lanes(L, dev):
    """Rows share waves; a row's last lane has the tokens of the one before it too; lengths that end in either, before
    both, or at once."""
    lengths = [L, max(0, L - 3), max(0, L - 9), 0, L // 2]
    for dtype, out, blend, ranges in (("bf16", "bf16", False, False), ("f32", "f32", False, True), ("bf16", "f32", True, True)):
        for ln in (None, lengths):
            for test in (test_forward, test_backward):
                test(5, 37, L, dtype, out, blend, True, True, True, ln, ranges, 0, 0, dev)


@pytest.mark.parametrize("with_init,with_final", [(True, False), (False, True)])
@pytest.mark.parametrize("waves,segments", [(0, 0), (1, 3)])
def test_one_of_the_two_states(with_init, with_final, waves, segments, dev):
    """A given state without a gradient of the last one, and the other way round."""
    import selective_state_space_75_amd as m
    x = make(2, 7, 900, "f32", 14, False, True, True, True)
    x["initial_state"] = x["initial_state"] if with_init else None
    x["dfinal_state"] = x["dfinal_state"] if with_final else None
    t = put(x, dev, NAMES)
    with m.glr_test_knobs(waves=waves, segments=segments):
        g = gradients(t, t["dy"], False, None)
    ref = O.glr_bwd(*oracle_args(x), f64(x["dy"]), initial_state=x["initial_state"], dfinal_state=x["dfinal_state"])
    assert (g["dinitial_state"] is None) == (not with_init)
    check_gradients(g, ref, x)


def test_gradients_are_differences_of_the_forward(dev):
    """Along random directions, the change of sum(y dy) over a step of 2^-6 both ways against the gradients.
    The change is a difference of sums of fp32 outputs (taken in fp64): numbers off by 1e-6 with either
    sign, over 2^-5, leave 3e-5 sqrt(n), three times that at most.  The third derivatives add the step
    squared over six, 4e-5, times themselves: through sigmoid, exp and the state's memory they are held
    to 120 times the gradient's size for directions of unit numbers, 4.8e-3 in all."""
    import torch
    import selective_state_space_75_amd as m
    B, D, L = 2, 8, 300
    x = make(B, D, L, "f32", 5, False, True, True, True)
    t = put(x, dev, NAMES)
    g = gradients(t, t["dy"], False, None)
    rng = np.random.default_rng(0)
    for n, gn in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("A", "dA"), ("r_bias", "dr_bias"),
                  ("i_bias", "di_bias"), ("initial_state", "dinitial_state")):
        v = torch.from_numpy(rng.standard_normal(tuple(t[n].shape)).astype(np.float32)).to(dev)
        if n == "A":
            v = v * t["A"].abs() * 0.1
        step, vals = 2.0 ** -6, []
        for s in (step, -step):
            q = {**t, n: t[n] + s * v}
            y, h = m.glr_fwd(*args(q), initial_state=q["initial_state"], return_final_state=True)
            vals.append(float((y.double() * t["dy"].double()).sum() + (h.double() * t["dfinal_state"].double()).sum()))
        num = (vals[0] - vals[1]) / (2 * step)
        want = float((g[gn].double() * v.double()).sum())
        size = float((g[gn].double() * v.double()).norm())
        log("  %s: %.6e against %.6e" % (n, num, want))
        assert abs(num - want) <= 4.8e-3 * size + 9e-5 * (B * D * L) ** 0.5, n


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["x", "r", "i", "z"])
def test_what_is_not_finite_goes_forward_only(name, bad, dev):
    import torch
    import selective_state_space_75_amd as m
    B, D, L, at = 2, 4, 1500, 777
    x = make(B, D, L, "f32", 8, False, True, True, True)
    t = put(x, dev, NAMES)
    for waves, segments in ((0, 0), (1, 0), (2, 3)):
        with m.glr_test_knobs(waves=waves, segments=segments):
            clean = m.glr_fwd(*args(t), initial_state=t["initial_state"])
            q = {**t, name: t[name].clone()}
            q[name][1, 2, at] = bad
            y = m.glr_fwd(*args(q), initial_state=q["initial_state"])
            torch.cuda.synchronize()
        same = torch.ones_like(y, dtype=torch.bool)
        same[1, 2, at:] = False
        assert torch.equal(y[same], clean[same])
        if name != "z" and not (name in ("r", "i") and bad > 0 and bad == float("inf")):   # an open gate is finite
            assert not torch.isfinite(y[1, 2, at:]).any() or name == "x"
            assert not torch.isfinite(y[1, 2, at])


def test_behind_a_rows_end_nothing_is_looked_at_or_lost(dev):
    """NaN behind the ends, and what lies around the outputs stays."""
    import torch
    import selective_state_space_75_amd as m
    B, D, L, ln = 3, 5, 1030, [1030, 0, 517]
    x = make(B, D, L, "bf16", 9, False, True, True, True)
    t = put(x, dev, NAMES)
    lens = torch.tensor(ln, dtype=torch.int32, device=dev)
    q = {**t}
    for n in ("x", "r", "i", "z", "dy"):
        q[n] = t[n].clone()
        for b in range(B):
            q[n][b, :, ln[b]:] = float("nan")
    for waves, segments in ((0, 0), (1, 4)):
        with m.glr_test_knobs(waves=waves, segments=segments):
            a = m.glr_fwd(*args(t), initial_state=t["initial_state"], lengths=lens, return_final_state=True)
            b = m.glr_fwd(*args(q), initial_state=q["initial_state"], lengths=lens, return_final_state=True)
            ga, gb = gradients(t, t["dy"], False, lens), gradients(q, q["dy"], False, lens)
            # lengths beyond both ends are held to 0 .. L
            wild = torch.tensor([1 << 30, -5, 517], dtype=torch.int32, device=dev)
            c = m.glr_fwd(*args(t), initial_state=t["initial_state"], lengths=wild, return_final_state=True)
            torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert torch.equal(a[1][1], t["initial_state"][1])                   # a row without tokens keeps its state
        assert torch.equal(ga["dinitial_state"][1], t["dfinal_state"][1])
        for n in ga:
            assert torch.equal(ga[n], gb[n]), n
        assert torch.equal(c[0], a[0]) and torch.equal(c[1], a[1])


@pytest.mark.parametrize("L", [4, 12, 100, 255, 511, 1207])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nothing_comes_from_behind_a_rows_length(L, bad, dev):
    import torch
    import selective_state_space_75_amd as m
    ends = [L - 1, L // 2, 0]
    x = make(3, 9, L, "bf16", 12, False, True, True, True)
    t = put(x, dev, NAMES)
    ln = torch.tensor(ends, dtype=torch.int32, device=dev)
    q = {k: v.clone() for k, v in t.items()}
    for k in ("x", "r", "i", "z", "dy"):
        for b, n in enumerate(ends):
            q[k][b, :, n:] = bad
    call = lambda v: m.glr_fwd(*args(v), initial_state=v["initial_state"], lengths=ln, return_final_state=True)  # noqa: E731
    a, b = call(t), call(q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = gradients(t, t["dy"], False, ln), gradients(q, q["dy"], False, ln)
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n


@pytest.mark.parametrize("L", [5, 99, 603, 1999])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alignment_and_neighbours(dtype, L, dev):
    """Arrays that begin at any element: the same bits, and nothing written around the outputs."""
    import torch
    import selective_state_space_75_amd as m
    B, D = 2, 3
    n = B * D * L
    x = make(B, D, L, dtype, 10, False, True, True, True)
    t = put(x, dev, NAMES)
    ref = m.glr_fwd(*args(t), initial_state=t["initial_state"])
    gref = gradients(t, t["dy"], False, None)
    for off in (1, 3, 7):
        q = {**t}
        for k in ("x", "r", "i", "z", "dy"):
            buf = torch.empty(n + 16, dtype=t[k].dtype, device=dev)
            q[k] = buf[off:off + n].view(B, D, L).copy_(t[k])
        out = torch.full((n + 32,), 5.0, dtype=ref.dtype, device=dev)
        m.glr_fwd(*args(q), initial_state=q["initial_state"], y=out[8 + off:8 + off + n].view(B, D, L))
        torch.cuda.synchronize()
        assert torch.equal(out[8 + off:8 + off + n].view(B, D, L), ref)
        assert (out[:8 + off] == 5.0).all() and (out[8 + off + n:] == 5.0).all()
        g = gradients(q, q["dy"], False, None)
        for k in gref:
            assert torch.equal(g[k], gref[k]), k


def test_the_same_call_gives_the_same_bits(dev):
    import torch
    import selective_state_space_75_amd as m
    x = make(3, 40, 9000, "bf16", 11, False, True, True, True)
    t = put(x, dev, NAMES)
    a = gradients(t, t["dy"], False, None)
    ya = m.glr_fwd(*args(t), return_final_state=True)
    for _ in range(3):
        b = gradients(t, t["dy"], False, None)
        yb = m.glr_fwd(*args(t), return_final_state=True)
        assert all(torch.equal(a[n], b[n]) for n in a)
        assert all(torch.equal(u, v) for u, v in zip(ya, yb))


def test_extreme_gates(dev):
    """Gates at both ends of their range: s from 1e-18 to 1, decays from 1 - 1e-19 to e^-60."""
    import torch
    B, D, L = 1, 6, 64
    x = make(B, D, L, "f32", 12, False, True, True, True)
    rng = np.random.default_rng(1)
    x["r"] = rng.choice(np.float32([-40, -20, -10, 0, 10, 40]), size=(B, D, L)).astype(np.float32)
    x["A"] = -np.float32([60, 20, 5, 1, 0.1, 0.001])
    for blend in (False, True):
        if blend:
            x["A"] = None
        t = put(x, dev, NAMES)
        t["A"] = t.get("A")
        import selective_state_space_75_amd as m
        y, h = m.glr_fwd(*args(t), blend=blend, initial_state=t["initial_state"], return_final_state=True)
        yr, hr = O.glr(*oracle_args(x), blend=blend, initial_state=x["initial_state"])
        near(y, yr, E, "y")
        near(h, hr, E, "h")
        ref = O.glr_bwd(*oracle_args(x), f64(x["dy"]), blend=blend, initial_state=x["initial_state"],
                        dfinal_state=x["dfinal_state"])
        check_gradients(gradients(t, t["dy"], blend, None), ref, x)


@pytest.mark.parametrize("B,D,dtype,out,blend,with_i,with_z,slots,ranges", [
    (1, 1, "f32", "f32", False, True, True, False, False), (1, 4096, "bf16", "bf16", False, True, True, False, False),
    (5, 257, "bf16", "f32", True, True, False, True, True), (128, 300, "f32", "bf16", False, False, True, True, False),
    (7, 1023, "f32", "f32", False, True, True, True, True), (64, 5120, "bf16", "bf16", False, True, True, True, True)])
def test_update(B, D, dtype, out, blend, with_i, with_z, slots, ranges, dev):
    import torch
    import selective_state_space_75_amd as m
    log("[glr update] %s" % ((B, D, dtype, out, blend, with_i, with_z, slots, ranges),))
    x = make(B, D, 1, dtype, 300 + D, blend, with_i, with_z, True)
    t = put(x, dev, NAMES, ranges)
    for n in ("x", "r", "i", "z"):
        if n in t:
            t[n] = t[n].squeeze(2)
    rng = np.random.default_rng(B)
    S = B + 3 if slots else B
    pool = rng.standard_normal((S, D)).astype(np.float32)
    idx = rng.permutation(S)[:B].astype(np.int32) if slots else np.arange(B, dtype=np.int32)
    if slots and B > 2:
        idx[1], idx[2] = -1, S                                    # two rows without a state
    state = to_dev(pool, dev)
    y = m.glr_update(state, *args(t), blend=blend, slots=torch.from_numpy(idx).to(dev) if slots else None,
                     out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    torch.cuda.synchronize()
    on = (idx >= 0) & (idx < S)
    h0 = np.zeros((B, D))
    h0[on] = pool[idx[on]]
    yr, hr = O.glr(*oracle_args(x), blend=blend, initial_state=h0)
    yr = np.where(on[:, None], yr[..., 0], 0.0)
    near(y, yr, E, "y")
    want = pool.astype(np.float64)
    want[idx[on]] = hr[on]
    near(state, want, E, "state")
    rest = np.setdiff1d(np.arange(S), idx[on])
    assert np.array_equal(from_dev(state)[rest], pool[rest].astype(np.float64))
    assert not from_dev(y)[~on].any()


def test_update_goes_on_where_the_sequence_ended(dev):
    """Tokens one by one from the prompt's state equal the whole sequence, to fp32 rounding."""
    import torch
    import selective_state_space_75_amd as m
    B, D, L, T = 2, 100, 40, 9
    x = make(B, D, L + T, "f32", 13, False, True, True, False)
    t = put(x, dev, NAMES)
    whole = m.glr_fwd(*args(t))
    cut = {n: t[n][:, :, :L].contiguous() for n in ("x", "r", "i", "z")}
    _, h = m.glr_fwd(*args({**t, **cut}), return_final_state=True)
    for k in range(L, L + T):
        one = {n: t[n][:, :, k].contiguous() for n in ("x", "r", "i", "z")}
        y = m.glr_update(h, *args({**t, **one}))
        assert rel_l2(from_dev(y), from_dev(whole)[:, :, k]) <= E
    torch.cuda.synchronize()


def test_refusals_on_the_gpu(dev):
    import torch
    import selective_state_space_75_amd as m
    x = torch.zeros(2, 4, 8, device=dev)
    A = -torch.ones(4, device=dev)
    with pytest.raises(ValueError, match="A is needed"):
        m.glr_fwd(x, x)
    with pytest.raises(ValueError, match="A is not used"):
        m.glr_fwd(x, x, None, A, blend=True)
    with pytest.raises(ValueError, match="i_bias without i"):
        m.glr_fwd(x, x, None, A, None, A)
    with pytest.raises(TypeError, match="r must be"):
        m.glr_fwd(x, None, None, A)
    with pytest.raises(TypeError, match="i has dtype"):
        m.glr_fwd(x, x, x.bfloat16(), A)
    with pytest.raises(ValueError, match="dense within"):
        m.glr_fwd(x, x.transpose(1, 2).contiguous().transpose(1, 2), None, A)
    with pytest.raises(ValueError, match="dense within"):
        m.glr_fwd(x[:1].expand(2, 4, 8), x, None, A)
    with pytest.raises(ValueError, match="lengths has shape"):
        m.glr_fwd(x, x, None, A, lengths=torch.zeros(3, dtype=torch.int32, device=dev))
    with pytest.raises(TypeError, match="lengths has dtype"):
        m.glr_fwd(x, x, None, A, lengths=torch.zeros(2, dtype=torch.int64, device=dev))
    with pytest.raises(TypeError, match="unsupported dtype"):
        m.glr_fwd(x.half(), x.half(), None, A)
    with pytest.raises(ValueError, match="dy has shape"):
        m.glr_bwd(x, x, None, A, None, None, None, x[:, :2].contiguous())
    with pytest.raises(TypeError, match="dy must be"):
        m.glr_bwd(x, x, None, A, None, None, None, None)
    with pytest.raises(m.MambaError):
        m.glr_bwd(x, x, None, A, None, None, None, x, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError, match="state must be"):
        m.glr_update(x, x[:, :, 0].contiguous(), x[:, :, 0].contiguous(), None, A)
    with pytest.raises(m.MambaError):
        m.glr_update(torch.zeros(1, 4, device=dev), x[:, :, 0].contiguous(), x[:, :, 0].contiguous(), None, A)
    with pytest.raises(ValueError, match="must be contiguous|dense"):
        m.glr_update(torch.zeros(2, 4, device=dev), x[:, :, 0], x[:, :, 0], None, A)
    with pytest.raises(ValueError, match="overlap"):
        m.glr_fwd(x, x.clone(), None, A, y=x)
    with pytest.raises(ValueError, match="overlap"):
        q = torch.zeros(2, 4, device=dev)
        m.glr_update(torch.zeros(2, 4, device=dev), q.clone(), q, None, A, y=q)
