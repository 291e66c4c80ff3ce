"""NaN and infinities among a token's inputs of the gated delta rule: the tokens before it keep
the bits that they have without it, on every path; from it on, what it reaches is not finite
(and the same outputs are on every path); rows of the batch, heads and channels that it does
not reach keep their bits; tokens behind a row's end stay zero, also in the gradients."""
import numpy as np
import pytest

from helpers import log, to_dev
from oracle import gdr as O
from selective_state_space_75_amd import workloads as W

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "delta_raw", "beta_raw")
B, H, G, P, L = 2, 4, 2, 24, 75
LENGTHS = [75, 70]
ROW, HEAD, CHANNEL, NUMBER = 1, 2, 5, 7          # where the value is put: head 2 is served by key head 1

# input, value, heads of the row whose outputs it reaches, all later tokens or only its own
POISON = [
    ("v", np.inf, (HEAD,), True), ("v", np.nan, (HEAD,), True), ("v", -np.inf, (HEAD,), True),
    ("k", np.nan, (2, 3), True), ("k", np.inf, (2, 3), True),
    ("q", np.nan, (2, 3), False), ("q", -np.inf, (2, 3), False),
    ("delta_raw", np.nan, (HEAD,), True), ("beta_raw", np.nan, (HEAD,), True),
]


def _channel(name, N):
    return {"v": HEAD * P + CHANNEL, "k": 1 * N + NUMBER, "q": 1 * N + NUMBER}.get(name, HEAD)


def _run(t, kernel, segments, out, dev, lengths):
    import torch
    import selective_state_space_75_amd as m
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)
    with m.gdr_test_knobs(kernel=kernel, segments=segments):
        y, S = m.gdr_fwd(*[t[n] for n in NAMES], t["A"], t["delta_bias"], groups=G, initial_state=t["initial_state"],
                         lengths=ln, qk_norm=True, return_final_state=True, out_dtype=out)
    torch.cuda.synchronize()
    return y, S


@pytest.mark.parametrize("kernel,segments", [("token", 0), ("chunk", 0), ("chunk", 3)])
@pytest.mark.parametrize("token", [0, 5, 31, 50, 69])
@pytest.mark.parametrize("dtype,N", [("f32", 40), ("bf16", 40), ("f32", 128), ("bf16", 100)])
def test_tokens_before_keep_their_bits(dtype, N, token, kernel, segments, dev):
    import torch
    x = W.gdr_inputs(B, H, G, P, N, L, dtype, 8400)
    clean = {n: to_dev(a, dev) for n, a in x.items()}
    for out in (torch.float32, torch.bfloat16):
        y0, S0 = _run(clean, kernel, segments, out, dev, LENGTHS)
        assert torch.isfinite(y0).all() and torch.isfinite(S0).all()
        for name, value, heads, later in POISON:
            log("[gdr nonfinite] %s=%s at %d, %s, %s %d, %s" % (name, value, token, dtype, kernel, segments, out))
            t = dict(clean)
            t[name] = clean[name].clone()
            t[name][ROW, _channel(name, N), token] = value
            y, S = _run(t, kernel, segments, out, dev, LENGTHS)
            hit = torch.zeros((B, H, P, L), dtype=torch.bool, device=dev)
            state = torch.zeros((B, H, P, N), dtype=torch.bool, device=dev)
            for h in heads:
                ch = slice(CHANNEL, CHANNEL + 1) if name == "v" else slice(None)
                hit[ROW, h, ch, token:LENGTHS[ROW] if later else token + 1] = True
                state[ROW, h, ch] = later
            hit, state = hit.view(y.shape), state.view(S.shape)
            assert torch.equal(torch.isfinite(y), ~hit), name
            assert torch.equal(y[~hit], y0[~hit]), name
            assert not torch.isfinite(S[state]).any(), name
            assert torch.equal(S[~state], S0[~state]), name
            assert not y[ROW, :, LENGTHS[ROW]:].any(), name


@pytest.mark.parametrize("kernel,segments", [("token", 0), ("chunk", 0), ("chunk", 3)])
def test_infinite_gates_are_resets(kernel, segments, dev):
    """delta = +inf forgets the state (A < 0), -inf keeps it, beta = +-inf is 1 or 0: finite, and the
    oracle's (whose gates take the same limits).  fp32 bar of test_gdr_variants_gpu.py."""
    import torch
    from helpers import f64, from_dev, rel_l2
    N = 40
    x = W.gdr_inputs(B, H, G, P, N, L, "f32", 8450)
    for i, (n, v) in enumerate([("delta_raw", np.inf), ("delta_raw", -np.inf), ("beta_raw", np.inf), ("beta_raw", -np.inf)]):
        x[n][:, :, 9 + 14 * i] = v
    t = {n: to_dev(a, dev) for n, a in x.items()}
    y, S = _run(t, kernel, segments, torch.float32, dev, None)
    yr, Sr = O.gdr(*[f64(x[n]) for n in NAMES], f64(x["A"]), f64(x["delta_bias"]), groups=G,
                   initial_state=f64(x["initial_state"]), norm=True)
    assert rel_l2(from_dev(y), yr) <= 20 * 2.0 ** -24 and rel_l2(from_dev(S), Sr) <= 20 * 2.0 ** -24


def test_gradients_of_infinite_gates(dev):
    """The gradients' limits: those of a step of 1e5 for delta = +inf (A < -1: exp(-1e5) is 0), of delta =
    -1e5 for -inf, of |beta| = 800.  Bars of test_gdr_variants_gpu.py."""
    import selective_state_space_75_amd as m
    from helpers import f64, from_dev, rel_l2
    N = 40
    x = W.gdr_inputs(B, H, G, P, N, L, "f32", 8480)
    ref = {n: f64(a) for n, a in x.items()}
    for i, (n, v, far) in enumerate([("delta_raw", np.inf, 1e5), ("delta_raw", -np.inf, -1e5), ("beta_raw", np.inf, 800.0),
                                     ("beta_raw", -np.inf, -800.0)]):
        x[n][:, :, 9 + 14 * i], ref[n][:, :, 9 + 14 * i] = v, far
    t = {n: to_dev(a, dev) for n, a in x.items()}
    g = m.gdr_bwd(*[t[n] for n in NAMES], t["A"], t["delta_bias"], t["dy"], groups=G, initial_state=t["initial_state"],
                  dfinal_state=t["dfinal_state"], qk_norm=True)
    with np.errstate(over="ignore"):
        want = O.gdr_bwd(*[ref[n] for n in NAMES], ref["A"], ref["delta_bias"], ref["dy"], groups=G, norm=True,
                         initial_state=ref["initial_state"], dfinal_state=ref["dfinal_state"])
    for n, a in g.items():
        e = rel_l2(from_dev(a), want[n])
        log("  %s: rel_l2=%.3e" % (n, e))
        assert e <= (4e-5 if n in ("dA", "ddelta_bias") else 20 * 2.0 ** -24), n


@pytest.mark.parametrize("kernel,segments", [("token", 0), ("chunk", 0), ("chunk", 3)])
def test_a_row_without_tokens_keeps_its_state(kernel, segments, dev):
    import torch
    N = 40
    t = {n: to_dev(a, dev) for n, a in W.gdr_inputs(B, H, G, P, N, L, "f32", 8470).items()}
    t["initial_state"][ROW, 7, 3] = float("inf")
    t["initial_state"][ROW, 9, 38] = float("nan")
    y, S = _run(t, kernel, segments, torch.float32, dev, [L, 0])
    assert torch.equal(S[ROW].view(torch.int32), t["initial_state"][ROW].view(torch.int32))
    assert not y[ROW].any() and torch.isfinite(y[0]).all() and torch.isfinite(S[0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_behind_the_end_stay_zero(dtype, dev):
    import torch
    import selective_state_space_75_amd as m
    N = 40
    x = W.gdr_inputs(B, H, G, P, N, L, dtype, 8460)
    t = {n: to_dev(a, dev) for n, a in x.items()}
    t["v"][ROW, _channel("v", N), 66] = float("nan")
    t["dy"][0, 3, 2] = float("inf")
    lengths = [41, 70]
    g = m.gdr_bwd(*[t[n] for n in NAMES], t["A"], t["delta_bias"], t["dy"], groups=G, initial_state=t["initial_state"],
                  dfinal_state=t["dfinal_state"], qk_norm=True,
                  lengths=torch.tensor(lengths, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv", "ddelta", "dbeta"):
        for b, ln in enumerate(lengths):
            assert not g[n][b, :, ln:].any(), n
    # dv is linear in dy and holds no v; dk has the updates u, which hold v
    assert torch.isfinite(g["dv"][ROW]).all() and torch.isnan(g["dk"][ROW]).any() and torch.isnan(g["dv"][0]).any()
