"""The layer norm over channels on the GPU against the fp64 oracle: both layouts, groups, gates, types,
sizes around every boundary, offsets and alignments.

Bars.  x - mean is off by the mean's rounding (2^-24 of its size; inputs here are offset by half their
scale) and one rounding, the root by about one unit: 1e-6 relative L2 leaves a factor of five.  Gradients
of x relative to the size of the terms that they are differences of (the oracle's "scale"), weight sums
relative to the sums of magnitudes, summed in fp32 over fixed trees, 2e-6.  bf16 results add one rounding."""
import numpy as np
import pytest

from helpers import f64, from_dev, log, to_dev
from oracle import glr as O
from selective_state_space_75_amd import workloads as W
from test_glr_gpu import near

pytestmark = pytest.mark.gpu

E = 1e-6

#        shape            groups dtype  out    gated  rms   affine ranges
CASES = [((1, 1, 1), 1, "f32", "f32", False, False, True, False),
         ((2, 7, 3), 1, "f32", "f32", True, False, True, False),
         ((2, 16, 9), 4, "bf16", "f32", False, True, True, True),
         ((3, 60, 65), 3, "f32", "bf16", True, True, False, False),
         ((1, 96, 64), 1, "bf16", "bf16", False, False, True, False),
         ((2, 80, 63), 1, "bf16", "f32", True, False, True, True),
         ((2, 384, 129), 3, "f32", "f32", True, True, True, True),
         ((1, 1000, 130), 1, "bf16", "f32", False, False, True, False),
         ((1, 2047, 40), 1, "f32", "f32", False, False, True, False),
         ((1, 2500, 17), 1, "bf16", "f32", True, False, True, False),
         ((1, 5120, 72), 1, "bf16", "f32", False, False, True, False),
         ((1, 5000, 33), 1, "f32", "f32", True, False, True, True),
         ((1, 10007, 10), 1, "bf16", "f32", False, False, True, False),
         ((1, 9000, 21), 1, "f32", "f32", True, True, True, False),
         ((70, 24, 5), 2, "bf16", "f32", False, False, True, False),
         ((3, 20, 8), 1, "bf16", "f32", True, False, True, False),
         ((1, 3000, 8), 1, "f32", "f32", True, True, True, False),
         ((2, 200, 70), 1, "bf16", "f32", True, False, True, True),
         ((2, 400, 50), 2, "f32", "bf16", True, False, True, False),
         ((1, 400, 50), 1, "bf16", "bf16", True, True, True, False),
         ((1, 512, 33), 1, "f32", "f32", False, False, True, False),
         ((1, 1500, 70), 1, "bf16", "f32", True, False, False, True),
         ((1, 600, 300), 1, "bf16", "f32", True, False, True, True),
         ((2, 2600, 515), 1, "f32", "f32", False, False, True, False),
         ((1, 5200, 1030), 2, "bf16", "f32", True, True, True, False),
         ((9, 24, 2), 1, "f32", "f32", True, True, True, False),
         ((1, 1), 1, "f32", "f32", False, False, True, False),
         ((5, 7), 7, "f32", "f32", True, True, True, False),
         ((3, 8), 1, "bf16", "f32", False, False, True, False),
         ((4, 100), 4, "bf16", "bf16", True, False, True, True),
         ((130, 768), 6, "f32", "f32", True, True, True, True),
         ((9, 513), 1, "bf16", "f32", False, False, False, False),
         ((600, 1000), 1, "bf16", "f32", True, False, True, False),
         ((33, 5120), 1, "bf16", "f32", False, False, True, True),
         ((5, 4097), 1, "f32", "f32", True, False, True, False),
         ((3, 8193), 1, "bf16", "f32", False, False, True, False),
         ((300, 8200), 1, "f32", "f32", True, False, True, True),
         ((5, 9003), 1, "f32", "bf16", False, True, False, False),
         ((4, 20480), 2, "bf16", "bf16", True, False, True, True),
         ((3, 16383), 1, "bf16", "f32", True, True, False, False),
         ((2, 16384), 1, "f32", "f32", True, False, True, False),
         ((3, 16385), 1, "f32", "f32", True, False, True, False),
         ((3, 20001), 1, "bf16", "f32", False, False, True, False),
         ((2, 70001), 1, "f32", "f32", True, True, True, False)]


def tensors(shape, dtype, seed, gated, affine, ranges, dev, offset=0.5):
    import torch
    x = W.norm_inputs(shape, dtype, seed, offset)
    t = {n: to_dev(x[n], dev) for n in x}
    if not gated:
        x["z"] = t["z"] = None
    if not affine:
        x["weight"] = x["bias"] = t["weight"] = t["bias"] = None
    if ranges:                                         # channel ranges of a wider tensor
        D = shape[1]
        wide = torch.cat([t["x"], t["dy"] if t["z"] is None else t["z"], t["x"][:, :1]], 1)
        t["x"] = wide[:, :D]
        if gated:
            t["z"] = wide[:, D:2 * D]
    return x, t


def opt(x):
    return None if x is None else f64(x)


@pytest.mark.parametrize("shape,groups,dtype,out,gated,rms,affine,ranges", CASES)
def test_forward_and_backward(shape, groups, dtype, out, gated, rms, affine, ranges, dev):
    import torch
    import selective_state_space_75_amd as m
    log("[norm] %s" % ((shape, groups, dtype, out, gated, rms, affine, ranges),))
    x, t = tensors(shape, dtype, 400 + shape[1], gated, affine, ranges, dev)
    kw = dict(groups=groups, rms=rms)
    odt = torch.float32 if out == "f32" else torch.bfloat16
    y = m.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"], out_dtype=odt, **kw)
    ins = (f64(x["x"]), opt(x["weight"]), opt(x["bias"]), opt(x["z"]))
    yr = O.layer_norm(*ins, **kw)
    near(y, yr, E, "y", np.maximum(np.abs(yr), 1e-3 if shape[1] // groups == 1 else 0.0))
    dy = t["dy"].to(odt)
    g = m.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], dy, **kw)
    torch.cuda.synchronize()
    ref = O.layer_norm_bwd(*ins, f64(from_dev(dy)), **kw)
    near(g["dx"], ref["dx"], E, "dx", ref["scale"]["dx"])
    if gated:
        near(g["dz"], ref["dz"], E, "dz")
    else:
        assert g["dz"] is None
    for n in ("dweight", "dbias"):
        near(g[n], ref[n], 2 * E, n, np.maximum(ref["scale"][n], 1e-30))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_every_layout_of_every_type(dtype, out, gated, rms, dev):
    """One shape for each way that a group is laid out over lanes, waves and launches, the last lanes' tokens and channels
    their neighbours' too."""
    for shape in ((2, 100, 41), (1, 200, 70), (1, 400, 37), (1, 900, 33), (1, 1800, 40), (1, 2600, 45), (1, 2600, 300),
                  (1, 2601, 523), (4, 50, 5), (70, 96), (70, 99), (20, 520), (20, 515), (9, 5000), (5, 7001), (7, 9000),
                  (5, 9003), (3, 16500), (5, 6)):
        test_forward_and_backward(shape, 1, dtype, out, gated, rms, True, False, dev)


@pytest.mark.parametrize("shape", [(2, 300, 50), (20, 1500), (1, 6000, 20), (3, 12000), (2, 40000)])
def test_a_large_mean_is_taken_off(shape, dev):
    """Offsets a thousand times the spread: x - mean loses 2^-24 of the offset, 1e3 * 6e-8 = 6e-5 of the
    spread per number, to the inputs' own rounding none (they are given); the variance around the mean is
    unhurt, where a difference of squares would lose all of it."""
    import selective_state_space_75_amd as m
    x, t = tensors(shape, "f32", 77, False, True, False, dev)
    t["x"] = t["x"] * 0.5 + 1000.0
    xs = from_dev(t["x"])
    y = m.layer_norm_fwd(t["x"], t["weight"], t["bias"])
    near(y, O.layer_norm(xs, x["weight"], x["bias"]), 1.2e-4, "y")
    g = m.layer_norm_bwd(t["x"], t["weight"], t["bias"], None, t["dy"])
    ref = O.layer_norm_bwd(xs, x["weight"], x["bias"], None, f64(x["dy"]))
    near(g["dx"], ref["dx"], 2.4e-4, "dx", ref["scale"]["dx"])


@pytest.mark.parametrize("shape,groups", [((2, 24, 70), 2), ((1, 3000, 30), 1), ((9, 640), 4), ((3, 9001), 1), ((3, 30000), 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_token_and_group(shape, groups, bad, dev):
    import torch
    import selective_state_space_75_amd as m
    x, t = tensors(shape, "f32", 78, True, True, False, dev)
    kw = dict(groups=groups)
    at = (shape[0] - 1, 5) + ((17,) if len(shape) == 3 else ())
    a = m.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"], **kw)
    ga = m.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], t["dy"], **kw)
    q = t["x"].clone()
    q[at] = bad
    b = m.layer_norm_fwd(q, t["weight"], t["bias"], t["z"], **kw)
    gb = m.layer_norm_bwd(q, t["weight"], t["bias"], t["z"], t["dy"], **kw)
    torch.cuda.synchronize()
    own = torch.zeros(shape, dtype=torch.bool, device=dev)
    own[(at[0], slice(0, shape[1] // groups)) + at[2:]] = True
    for u, v in ((a, b), (ga["dx"], gb["dx"]), (ga["dz"], gb["dz"])):
        assert torch.equal(u[~own], v[~own])
    assert torch.isnan(b[own]).all()


@pytest.mark.parametrize("shape,groups", [((2, 30, 67), 3), ((1, 2100, 19), 1), ((7, 1030), 2), ((3, 10007), 1), ((3, 9), 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alignment_and_neighbours(shape, groups, dtype, dev):
    import torch
    import selective_state_space_75_amd as m
    x, t = tensors(shape, dtype, 79, True, True, False, dev)
    n = t["x"].numel()
    kw = dict(groups=groups)
    ref = m.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"], **kw)
    gref = m.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], t["dy"], **kw)
    for off in (1, 5):
        q = {k: torch.empty(n + 16, dtype=t[k].dtype, device=dev)[off:off + n].view(shape).copy_(t[k]) for k in ("x", "z", "dy")}
        out = torch.full((n + 32,), 5.0, dtype=ref.dtype, device=dev)
        m.layer_norm_fwd(q["x"], t["weight"], t["bias"], q["z"], y=out[8 + off:8 + off + n].view(shape), **kw)
        g = m.layer_norm_bwd(q["x"], t["weight"], t["bias"], q["z"], q["dy"], **kw)
        torch.cuda.synchronize()
        assert torch.equal(out[8 + off:8 + off + n].view(shape), ref)
        assert (out[:8 + off] == 5.0).all() and (out[8 + off + n:] == 5.0).all()
        for k in gref:
            assert torch.equal(g[k], gref[k]), k


def test_a_tokens_bits_do_not_depend_on_the_batch(dev):
    import torch
    import selective_state_space_75_amd as m
    for shape, groups in (((6, 700, 40), 4), ((6, 250, 300), 1), ((900, 700), 1), ((300, 9000), 1), ((40, 96), 3)):
        x, t = tensors(shape, "bf16", 80, True, True, False, dev)
        kw = dict(groups=groups)
        y = m.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"], **kw)
        g = m.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], t["dy"], **kw)
        one = slice(3, 4)
        z1 = t["z"][one]
        assert torch.equal(m.layer_norm_fwd(t["x"][one], t["weight"], t["bias"], z1, **kw), y[one])
        g1 = m.layer_norm_bwd(t["x"][one], t["weight"], t["bias"], z1, t["dy"][one], **kw)
        assert torch.equal(g1["dx"], g["dx"][one]) and torch.equal(g1["dz"], g["dz"][one])


@pytest.mark.parametrize("shape,groups", [((3, 700, 333), 1), ((2, 240, 700), 3), ((700, 900), 1), ((3000, 96), 3), ((600, 9000), 1),
                                          ((5, 60, 6), 2)])
def test_the_same_call_gives_the_same_bits(shape, groups, dev):
    import torch
    import selective_state_space_75_amd as m
    x, t = tensors(shape, "bf16", 81, True, True, False, dev)
    call = lambda: m.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], t["dy"], groups=groups)  # noqa: E731
    a = call()
    for _ in range(3):
        b = call()
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_gradients_are_differences_of_the_forward(dev):
    """Along random directions over a step of 2^-6 both ways: sums of fp32 outputs off by 1e-6 of their
    numbers with either sign, over 2^-5, leave 3e-5 sqrt(n), three times that at most; the third derivatives add the
    step squared over six, 4e-5, times themselves, held to 120 times the gradient's size."""
    import torch
    import selective_state_space_75_amd as m
    for shape, groups, rms in (((2, 24, 40), 2, False), ((1, 700, 20), 1, True), ((6, 640), 1, False)):
        x, t = tensors(shape, "f32", 82, True, True, False, dev)
        kw = dict(groups=groups, rms=rms)
        g = m.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], t["dy"], **kw)
        rng = np.random.default_rng(1)
        for n, gn in (("x", "dx"), ("z", "dz"), ("weight", "dweight"), ("bias", "dbias")):
            v = torch.from_numpy(rng.standard_normal(tuple(t[n].shape)).astype(np.float32)).to(dev)
            vals = []
            for s in (2.0 ** -6, -2.0 ** -6):
                q = {**t, n: t[n] + s * v}
                vals.append(float((m.layer_norm_fwd(q["x"], q["weight"], q["bias"], q["z"], **kw).double() * t["dy"].double()).sum()))
            num, want = (vals[0] - vals[1]) * 32, float((g[gn].double() * v.double()).sum())
            size, count = float((g[gn].double() * v.double()).norm()), t["x"].numel() ** 0.5
            log("  %s: %.6e against %.6e" % (n, num, want))
            assert abs(num - want) <= 4.8e-3 * size + 9e-5 * count, n


def test_zero_variance_and_eps(dev):
    import torch
    import selective_state_space_75_amd as m
    for shape in ((1, 64, 16), (4, 64)):
        x = torch.full(shape, 3.0, device=dev)
        assert not from_dev(m.layer_norm_fwd(x)).any()                            # x - mean = 0
        y = m.layer_norm_fwd(x, rms=True, eps=7.0)
        assert np.allclose(from_dev(y), 3.0 / 4.0, rtol=1e-6)


def test_refusals_on_the_gpu(dev):
    import torch
    import selective_state_space_75_amd as m
    x = torch.zeros(2, 6, 8, device=dev)
    with pytest.raises(ValueError, match="do not divide"):
        m.layer_norm_fwd(x, groups=4)
    with pytest.raises(ValueError, match="do not divide"):
        m.layer_norm_fwd(x, groups=0)
    with pytest.raises(TypeError, match="weight has dtype"):
        m.layer_norm_fwd(x, torch.ones(6, device=dev).bfloat16())
    with pytest.raises(ValueError, match="z has shape"):
        m.layer_norm_fwd(x, None, None, x[:, :3])
    with pytest.raises(ValueError, match="dense within"):
        m.layer_norm_fwd(x.transpose(1, 2))
    with pytest.raises(m.MambaError):
        m.layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(TypeError, match="dy must be"):
        m.layer_norm_bwd(x, None, None, None, None)
    with pytest.raises(m.MambaError):
        m.layer_norm_bwd(x, None, None, None, x, workspace=torch.empty(8, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError, match="y has shape"):
        m.layer_norm_fwd(x, y=torch.zeros(2, 6, 9, device=dev))
    with pytest.raises(ValueError, match="overlap"):
        m.layer_norm_fwd(x, y=x)
    with pytest.raises(ValueError, match="overlap"):
        wide = torch.zeros(2, 12, 8, device=dev)
        m.layer_norm_fwd(wide[:, :6], y=wide.view(-1)[96:].view(2, 6, 8))
    wide = torch.zeros(1, 12, 8, device=dev)
    m.layer_norm_fwd(wide[:, :6], y=wide[:, 6:])                # one row: beside it
