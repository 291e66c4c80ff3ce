"""fp64 numpy oracle of the gated delta rule and of the 8-bit state cache.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  The rule is followed
token by token from its definition (include/mamba_gdr.h) and differentiated by
the chain rule of each step; nothing here is chunked and nothing is shared with
the HIP path.  Pinned by closed forms and finite differences in
tests/test_gdr_oracle.py.
"""
from __future__ import annotations

import numpy as np

NORM_EPS = 1e-6


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def _tokens(x, heads, width):
    """(B, heads * width, L) -> (L, B, heads, width)"""
    B, C, L = x.shape
    return np.ascontiguousarray(_f64(x).reshape(B, heads, width, L).transpose(3, 0, 1, 2))


def _rows(x):
    """(L, B, heads, width) -> (B, heads * width, L)"""
    L, B, H, W = x.shape
    return np.ascontiguousarray(x.transpose(1, 2, 3, 0)).reshape(B, H * W, L)


def _prepare(q, k, v, delta, beta, A, bias, groups, lengths, scale, norm):
    B, H, L = delta.shape
    G = H if groups is None else groups
    P, N = v.shape[1] // H, q.shape[1] // G
    live = np.ones((L, B), dtype=bool)
    if lengths is not None:
        live = np.arange(L)[:, None] < np.clip(np.asarray(lengths), 0, L)[None, :]
    d = {"B": B, "H": H, "G": G, "P": P, "N": N, "L": L, "live": live,
         "scale": N ** -0.5 if scale is None else scale}
    mask = live[:, :, None, None]

    def tok(x, heads, width):        # what stands behind a row's end is not looked at
        return np.where(mask, _tokens(x, heads, width), 0.0)

    for n, x in (("q", q), ("k", k)):
        raw = tok(x, G, N)
        r = np.sqrt((raw * raw).sum(-1, keepdims=True) + NORM_EPS) if norm else np.ones_like(raw[..., :1])
        d["raw_" + n], d["len_" + n] = raw, r
        d[n] = np.repeat(raw / r, H // G, axis=2)
    d["v"] = tok(v, H, P)
    x = tok(delta, H, 1)[..., 0] + (0.0 if bias is None else _f64(bias))
    d["x"] = x
    d["step"] = np.logaddexp(0.0, x)
    d["a"] = np.exp(_f64(A) * d["step"])
    with np.errstate(over="ignore"):
        d["b"] = 1.0 / (1.0 + np.exp(-tok(beta, H, 1)[..., 0]))
    return d


def _token(S, d, t):
    Sd = d["a"][t][..., None, None] * S
    p = np.einsum("bhpn,bhn->bhp", Sd, d["k"][t])
    u = d["b"][t][..., None] * (d["v"][t] - p)
    Sn = Sd + u[..., None] * d["k"][t][:, :, None, :]
    return Sd, p, u, np.where(d["live"][t][:, None, None, None], Sn, S)


def _start(initial_state, d):
    shape = (d["B"], d["H"], d["P"], d["N"])
    return np.zeros(shape) if initial_state is None else _f64(initial_state).reshape(shape).copy()


def gdr(q, k, v, delta, beta, A, delta_bias=None, groups=None, initial_state=None, lengths=None, scale=None,
        norm=False):
    """Returns (y (B, H*P, L), final_state (B, H*P, N)), float64."""
    d = _prepare(q, k, v, delta, beta, A, delta_bias, groups, lengths, scale, norm)
    S = _start(initial_state, d)
    y = np.zeros((d["L"], d["B"], d["H"], d["P"]))
    for t in range(d["L"]):
        S = _token(S, d, t)[3]
        o = d["scale"] * np.einsum("bhpn,bhn->bhp", S, d["q"][t])
        y[t] = np.where(d["live"][t][:, None, None], o, 0.0)
    return _rows(y), S.reshape(d["B"], -1, d["N"])


def gdr_update(state, q, k, v, delta, beta, A, delta_bias=None, groups=None, slots=None, scale=None, norm=False):
    """One token; returns (y (B, H*P), new pool of states)."""
    pool = _f64(state).copy()
    B = q.shape[0]
    idx = np.arange(B) if slots is None else np.asarray(slots)
    y = np.zeros((B, v.shape[1]))
    for r in range(B):
        if not 0 <= idx[r] < pool.shape[0]:
            continue
        yr, sr = gdr(*(np.asarray(x)[r:r + 1, :, None] for x in (q, k, v, delta, beta)), A, delta_bias,
                     groups=groups, initial_state=pool[idx[r]][None], scale=scale, norm=norm)
        y[r], pool[idx[r]] = yr[0, :, 0], sr[0]
    return y, pool


def gdr_bwd(q, k, v, delta, beta, A, delta_bias, dy, groups=None, initial_state=None, dfinal_state=None,
            lengths=None, scale=None, norm=False):
    """Gradients of every input for the gradients dy of y and dfinal_state of the final state."""
    d = _prepare(q, k, v, delta, beta, A, delta_bias, groups, lengths, scale, norm)
    B, H, G, P, N, L = (d[n] for n in "BHGPNL")
    S, kept = _start(initial_state, d), []
    for t in range(L):
        kept.append(_token(S, d, t))
        S = kept[-1][3]
    dS = np.zeros((B, H, P, N)) if dfinal_state is None else _f64(dfinal_state).reshape(B, H, P, N).copy()
    do = np.where(d["live"][:, :, None, None], _tokens(dy, H, P), 0.0) * d["scale"]
    dq, dk = np.zeros((L, B, H, N)), np.zeros((L, B, H, N))
    dv, db, dg = np.zeros((L, B, H, P)), np.zeros((L, B, H)), np.zeros((L, B, H))
    for t in reversed(range(L)):
        Sd, p, u, Sn = kept[t]
        qt, kt, b = d["q"][t], d["k"][t], d["b"][t][..., None]
        dq[t] = np.einsum("bhpn,bhp->bhn", Sn, do[t])
        full = dS + do[t][..., None] * qt[:, :, None, :]
        du = np.einsum("bhpn,bhn->bhp", full, kt)
        dp = -b * du
        dk[t] = np.einsum("bhpn,bhp->bhn", full, u) + np.einsum("bhpn,bhp->bhn", Sd, dp)
        dv[t] = b * du
        db[t] = (du * (d["v"][t] - p)).sum(-1)
        dSd = full + dp[..., None] * kt[:, :, None, :]
        dg[t] = (dSd * Sd).sum((-1, -2))                 # of the log decay A * step
        dS = np.where(d["live"][t][:, None, None, None], d["a"][t][..., None, None] * dSd, dS)
    on = d["live"][:, :, None]
    dg, db = np.where(on, dg, 0.0), np.where(on, db, 0.0)
    sig = 1.0 / (1.0 + np.exp(-d["x"]))
    out = {"dv": _rows(np.where(on[..., None], dv, 0.0))}
    for n, gr in (("q", dq), ("k", dk)):
        gr = np.where(on[..., None], gr, 0.0).reshape(L, B, G, H // G, N).sum(3)
        if norm:
            raw, r = d["raw_" + n], d["len_" + n]
            gr = gr / r - raw * (gr * raw).sum(-1, keepdims=True) / r ** 3
        out["d" + n] = _rows(gr)
    ddelta = dg * _f64(A) * sig
    out["ddelta"] = np.ascontiguousarray(ddelta.transpose(1, 2, 0))
    out["dbeta"] = np.ascontiguousarray((db * d["b"] * (1.0 - d["b"])).transpose(1, 2, 0))
    out["dA"] = (dg * d["step"]).sum((0, 1))
    out["ddelta_bias"] = ddelta.sum((0, 1))
    out["dinitial_state"] = dS.reshape(B, H * P, N)
    return out


# ----------------------------------------------------------------------------- 8-bit state cache
def cache_write(x):
    """One row x (n): (codes int8 (n), exponent bytes (ceil(n / 32)))."""
    x = _f64(x)
    codes = np.zeros(x.size, dtype=np.int8)
    exps = np.zeros((x.size + 31) // 32, dtype=np.uint8)
    for g in range(exps.size):
        part = x[32 * g:32 * g + 32]
        if not np.all(np.isfinite(part)):
            exps[g] = 255
            continue
        e8 = 1
        while e8 < 248 and 127.0 * 2.0 ** (e8 - 127) < np.abs(part).max():
            e8 += 1
        exps[g] = e8
        codes[32 * g:32 * g + 32] = np.clip(np.rint(part / 2.0 ** (e8 - 127)), -127, 127).astype(np.int8)
    return codes, exps


def cache_read(codes, exps):
    step = np.repeat(np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127.0)), 32)[:codes.size]
    return np.where(np.repeat(exps == 0, 32)[:codes.size], 0.0, codes.astype(np.float64) * step)
