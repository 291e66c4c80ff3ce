"""fp64 numpy oracle of the gated linear recurrence and of the layer norm over channels.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  The recurrence is followed token by
token from its definition (include/mamba_glr.h) and differentiated by the chain rule of each
step; the norm is differentiated through its mean and its deviation.  Nothing is shared with the
HIP path.  Pinned by closed forms and finite differences in tests/test_glr_oracle.py.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def _tokens(x, live):
    """(B, D, L) -> (L, B, D); what stands behind a row's end is not looked at."""
    return None if x is None else np.where(live, _f64(x).transpose(2, 0, 1), 0.0)


def _prepare(x, r, i, z, A, r_bias, i_bias, blend, lengths):
    B, D, L = np.shape(x)
    live = np.ones((L, B, 1), dtype=bool)
    if lengths is not None:
        live = (np.arange(L)[:, None] < np.clip(np.asarray(lengths), 0, L)[None, :])[:, :, None]
    v = {"live": live, "x": _tokens(x, live), "z": _tokens(z, live), "L": L}
    pre = _tokens(r, live) + (0.0 if r_bias is None else _f64(r_bias))
    v["s"], v["not_s"] = sigmoid(pre), sigmoid(-pre)          # 1 - s, also where s is 1 to the last bit
    if blend:
        v["a"], v["n"] = v["not_s"], v["s"]
    else:
        l = _f64(A) * v["s"]
        v["a"], v["n"] = np.exp(l), np.sqrt(-np.expm1(2.0 * l))
    v["g"], v["not_g"] = np.ones_like(v["x"]), np.zeros_like(v["x"])
    if i is not None:
        pre = _tokens(i, live) + (0.0 if i_bias is None else _f64(i_bias))
        v["g"], v["not_g"] = sigmoid(pre), sigmoid(-pre)
    return v


def _states(v, h0):
    h, out = h0, []
    for t in range(v["L"]):
        h = np.where(v["live"][t], v["a"][t] * h + v["n"][t] * v["g"][t] * v["x"][t], h)
        out.append(h)
    return np.stack(out)


def _rows(t):
    return np.ascontiguousarray(t.transpose(1, 2, 0))


def glr(x, r, i=None, A=None, r_bias=None, i_bias=None, z=None, *, blend=False, initial_state=None, lengths=None):
    """(y (B, D, L), final state (B, D))"""
    B, D, _ = np.shape(x)
    v = _prepare(x, r, i, z, A, r_bias, i_bias, blend, lengths)
    h = _states(v, np.zeros((B, D)) if initial_state is None else _f64(initial_state))
    y = h if z is None else h * v["z"] * sigmoid(v["z"])
    return _rows(np.where(v["live"], y, 0.0)), h[-1]


def glr_bwd(x, r, i, A, r_bias, i_bias, z, dy, *, blend=False, initial_state=None, dfinal_state=None, lengths=None):
    """Gradients as the binding names them, and under "scale" the sums of magnitudes that dr (per
    token), dA and the biases' gradients are differences of."""
    B, D, L = np.shape(x)
    v = _prepare(x, r, i, z, A, r_bias, i_bias, blend, lengths)
    h0 = np.zeros((B, D)) if initial_state is None else _f64(initial_state)
    h = _states(v, h0)
    live, a, n, s, not_s, g, xs = (v[k] for k in ("live", "a", "n", "s", "not_s", "g", "x"))
    dys = _tokens(dy, live)
    e = dys
    dz = None
    if z is not None:
        sz = sigmoid(v["z"])
        e = dys * v["z"] * sz
        dz = dys * h * (sz + v["z"] * sz * (1.0 - sz))
    c = np.zeros((B, D)) if dfinal_state is None else _f64(dfinal_state)
    q = np.zeros((L, B, D))
    for t in reversed(range(L)):
        q[t] = e[t] + c
        c = np.where(live[t], a[t] * q[t], c)
    q = np.where(live, q, 0.0)
    hp = np.concatenate([h0[None], h[:-1]])
    dx = q * n * g
    di = q * n * xs * g * v["not_g"]
    out, scale = {}, {}
    if blend:
        dr = q * (g * xs - hp) * s * not_s
        scale["dr"] = np.abs(q) * (np.abs(g * xs) + np.abs(hp)) * s * not_s
        out["dA"] = None
    else:
        with np.errstate(divide="ignore", invalid="ignore"):
            ra = np.where(n > 0, a * a / n, 0.0)
        dl, sl = q * (a * hp - g * xs * ra), np.abs(q) * (np.abs(a * hp) + np.abs(g * xs * ra))
        f = _f64(A) * s * not_s
        dr, scale["dr"] = dl * f, sl * np.abs(f)
        out["dA"], scale["dA"] = (dl * s).sum((0, 1)), (sl * s).sum((0, 1))
    out["dr_bias"], scale["dr_bias"] = dr.sum((0, 1)), scale["dr"].sum((0, 1))
    out["dx"], out["dr"], scale["dr"] = _rows(dx), _rows(dr), _rows(scale["dr"])
    out["di"] = None if i is None else _rows(di)
    out["di_bias"] = None if i is None else di.sum((0, 1))
    scale["di_bias"] = np.abs(di).sum((0, 1))
    out["dz"] = None if z is None else _rows(dz)
    out["dinitial_state"] = c
    out["scale"] = scale
    return out


# ----------------------------------------------------------------------------- layer norm over channels
def _normed(x, groups, eps, rms):
    x = _f64(x)
    B, D = x.shape[:2]
    L = x.shape[2] if x.ndim == 3 else 1
    x = x.reshape(B, groups, D // groups, L)
    c = x if rms else x - x.mean(2, keepdims=True)
    sd = np.sqrt((c * c).mean(2, keepdims=True) + eps)
    return c, sd, (B, D, L)


def _param(p, B, groups, fill):
    return fill if p is None else _f64(p).reshape(1, groups, -1, 1)


def layer_norm(x, weight=None, bias=None, z=None, *, groups=1, eps=1e-5, rms=False):
    c, sd, (B, D, L) = _normed(x, groups, eps, rms)
    y = c / sd * _param(weight, B, groups, 1.0) + _param(bias, B, groups, 0.0)
    if z is not None:
        zz = _f64(z).reshape(y.shape)
        y = y * zz * sigmoid(zz)
    return y.reshape(np.shape(x))


def layer_norm_bwd(x, weight, bias, z, dy, *, groups=1, eps=1e-5, rms=False):
    """dx, dz, dweight, dbias, and under "scale" the sums of magnitudes behind dweight and dbias and
    the size of the terms of dx."""
    c, sd, (B, D, L) = _normed(x, groups, eps, rms)
    Dg = D // groups
    xh = c / sd
    w, b = _param(weight, B, groups, 1.0), _param(bias, B, groups, 0.0)
    dm = _f64(dy).reshape(c.shape)
    out = {"dz": None}
    if z is not None:
        zz = _f64(z).reshape(c.shape)
        sz = sigmoid(zz)
        out["dz"] = (dm * (xh * w + b) * (sz + zz * sz * (1.0 - sz))).reshape(np.shape(x))
        dm = dm * zz * sz
    dxh = dm * w
    dsd = -(dxh * c).sum(2, keepdims=True) / (sd * sd)
    dc = dxh / sd + dsd * c / (sd * Dg)
    dx = dc if rms else dc - dc.mean(2, keepdims=True)
    out["dx"] = dx.reshape(np.shape(x))
    out["dweight"], out["dbias"] = (dm * xh).sum((0, 3)).reshape(D), dm.sum((0, 3)).reshape(D)
    out["scale"] = {"dweight": np.abs(dm * xh).sum((0, 3)).reshape(D), "dbias": np.abs(dm).sum((0, 3)).reshape(D),
                    "dx": ((np.abs(dxh) + np.abs(xh) * np.abs(dxh * xh).mean(2, keepdims=True)
                            + np.abs(dxh).mean(2, keepdims=True)) / sd).reshape(np.shape(x))}
    return out
