"""Pins of the fp64 oracle of the gated linear recurrence and of the layer norm: closed forms,
torch's own norm in 64 bits, and central differences of every gradient."""
import numpy as np
import pytest

from oracle import glr as O


def _draw(B, D, L, seed):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    return {"x": n(B, D, L), "r": n(B, D, L), "i": n(B, D, L), "z": n(B, D, L), "A": -np.exp(n(D)) - 0.05,
            "r_bias": n(D), "i_bias": n(D), "h0": n(B, D), "dy": n(B, D, L), "df": n(B, D)}


def test_constant_gates_sum_a_geometric_series():
    B, D, L = 2, 3, 40
    v = _draw(B, D, L, 0)
    one = np.ones((B, D, L))
    y, h = O.glr(one, 0.3 * one, None, v["A"], initial_state=v["h0"])
    a = np.exp(v["A"] / (1.0 + np.exp(-0.3)))
    t = np.arange(1, L + 1)
    want = a[None, :, None] ** t * v["h0"][:, :, None] + (np.sqrt(1 - a * a) / (1 - a))[:, None] * (1 - a[:, None] ** t)
    assert np.allclose(y, want, rtol=1e-12, atol=1e-13)
    assert np.allclose(h, want[:, :, -1], rtol=1e-12, atol=1e-13)


def test_blend_is_theorem_one():
    """h <- (1 - g) h + g x, one number per channel."""
    v = _draw(2, 3, 25, 1)
    y, _ = O.glr(v["x"], v["r"], blend=True, initial_state=v["h0"])
    h = v["h0"].copy()
    for t in range(25):
        g = 1.0 / (1.0 + np.exp(-v["r"][:, :, t]))
        h = (1 - g) * h + g * v["x"][:, :, t]
        assert np.allclose(y[:, :, t], h, rtol=1e-13, atol=1e-14)


def test_limits_of_the_decay():
    v = _draw(1, 2, 9, 2)
    y, _ = O.glr(v["x"], np.full((1, 2, 9), 40.0), None, np.full(2, -80.0), initial_state=v["h0"])
    assert np.allclose(y, v["x"], rtol=0, atol=1e-30)                 # everything forgotten, n = 1
    y, h = O.glr(v["x"], np.full((1, 2, 9), -800.0), None, v["A"], initial_state=v["h0"])
    assert np.array_equal(h, v["h0"])                                 # everything kept, n = 0


def test_stationary_variance_is_that_of_the_inputs():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 400, 300))
    y, _ = O.glr(x, np.zeros_like(x), None, np.full(400, -0.2))
    # squares of a chain with decay a = e^-0.1 decorrelate as a^2: 400 x 150 of them count as 400 x 150 / 10, whose
    # mean has a deviation of sqrt(2 / 6000) = 0.018
    assert abs(np.mean(y[:, :, 150:] ** 2) - 1.0) < 4 * 0.018


@pytest.mark.parametrize("blend,with_i,with_z,lengths", [(False, True, True, None), (False, False, False, [3, 0, 7]),
                                                         (True, True, False, None), (True, False, True, [7, 2, 9])])
def test_gradients_are_differences(blend, with_i, with_z, lengths):
    B, D, L = 3, 2, 7
    v = _draw(B, D, L, 4)
    args = {k: v[k] for k in ("x", "r", "i", "z", "A", "r_bias", "i_bias", "h0")}
    if not with_i:
        args["i"] = args["i_bias"] = None
    if not with_z:
        args["z"] = None
    if blend:
        args["A"] = None

    def loss(q):
        y, h = O.glr(q["x"], q["r"], q["i"], q["A"], q["r_bias"], q["i_bias"], q["z"], blend=blend,
                     initial_state=q["h0"], lengths=lengths)
        return (y * v["dy"]).sum() + (h * v["df"]).sum()

    g = O.glr_bwd(args["x"], args["r"], args["i"], args["A"], args["r_bias"], args["i_bias"], args["z"], v["dy"],
                  blend=blend, initial_state=args["h0"], dfinal_state=v["df"], lengths=lengths)
    eps = 1e-5
    for k, name in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("A", "dA"), ("r_bias", "dr_bias"),
                    ("i_bias", "di_bias"), ("h0", "dinitial_state")):
        if args[k] is None:
            assert g[name] is None
            continue
        num = np.zeros_like(args[k])
        for at in np.ndindex(*num.shape):
            up, dn = ({**args, k: args[k].copy()} for _ in range(2))
            up[k][at] += eps
            dn[k][at] -= eps
            num[at] = (loss(up) - loss(dn)) / (2 * eps)
        assert np.allclose(num, g[name], rtol=1e-7, atol=1e-8), name


def test_what_stands_behind_a_row_is_not_looked_at():
    v = _draw(2, 3, 8, 5)
    ln = [5, 0]
    bad = {k: v[k].copy() for k in ("x", "r", "i", "z")}
    for k in bad:
        for b in range(2):
            bad[k][b, :, ln[b]:] = np.nan
    call = lambda q: O.glr(q["x"], q["r"], q["i"], v["A"], v["r_bias"], v["i_bias"], q["z"], initial_state=v["h0"],  # noqa: E731
                           lengths=ln)
    for p, q in zip(call(v), call(bad)):
        assert np.array_equal(p, q)
    assert not call(v)[0][0, :, 5:].any() and np.array_equal(call(v)[1][1], v["h0"][1])


@pytest.mark.parametrize("shape,groups", [((3, 12, 5), 1), ((2, 12, 4), 3), ((5, 8), 2), ((4, 7), 1)])
def test_norm_is_torchs_in_64_bits(shape, groups):
    import torch
    rng = np.random.default_rng(6)
    x, w, b, z = rng.standard_normal(shape) * 3 + 1, rng.standard_normal(shape[1]), rng.standard_normal(shape[1]), \
        rng.standard_normal(shape)
    t = torch.from_numpy(x)
    for rms in (False, True):
        rows = t.movedim(1, -1).reshape(-1, groups, shape[1] // groups)
        n = (torch.nn.functional.rms_norm if rms else torch.nn.functional.layer_norm)(rows, rows.shape[-1:], eps=1e-5)
        n = n.reshape(t.movedim(1, -1).shape) * torch.from_numpy(w) + torch.from_numpy(b)
        n = n.movedim(-1, 1) * torch.nn.functional.silu(torch.from_numpy(z))
        assert np.allclose(O.layer_norm(x, w, b, z, groups=groups, rms=rms), n.numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("rms,gated,affine", [(False, True, True), (True, False, True), (False, False, False),
                                              (True, True, False)])
def test_norm_gradients_are_differences(rms, gated, affine):
    rng = np.random.default_rng(7)
    shape = (2, 6, 3)
    a = {"x": rng.standard_normal(shape), "w": rng.standard_normal(6) if affine else None,
         "b": rng.standard_normal(6) if affine else None, "z": rng.standard_normal(shape) if gated else None}
    dy = rng.standard_normal(shape)
    kw = dict(groups=2, eps=1e-3, rms=rms)
    g = O.layer_norm_bwd(a["x"], a["w"], a["b"], a["z"], dy, **kw)
    loss = lambda q: (O.layer_norm(q["x"], q["w"], q["b"], q["z"], **kw) * dy).sum()  # noqa: E731
    if not affine:                                   # ones and zeros stand in
        a["w"], a["b"] = np.ones(6), np.zeros(6)
    for k, name in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("z", "dz")):
        if a[k] is None:
            assert g[name] is None
            continue
        num = np.zeros_like(a[k])
        for at in np.ndindex(*num.shape):
            up, dn = ({**a, k: a[k].copy()} for _ in range(2))
            up[k][at] += 1e-5
            dn[k][at] -= 1e-5
            num[at] = (loss(up) - loss(dn)) / 2e-5
        assert np.allclose(num, g[name], rtol=1e-7, atol=1e-8), name
