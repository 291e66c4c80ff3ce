"""dbeta of the gated delta rule where the gate b = sigmoid(beta) is small: dbeta = b (1 - b) du . (v - p)
is a number down to b = 2^-126, though the kernels hold b du and b (v - p), whose product is not.

Bars.  b's own error: the exponent beta log2(e) is a product of two rounded numbers, off by at
most 2 * 2^-24 of itself, so b is off by |beta| 2 * 2^-24, and the update carries b once more:
4 |beta| 2^-24 + 20 * 2^-24 (test_gdr_variants_gpu.py) of the numbers, relative L2 over the tokens of
one gate."""
import numpy as np
import pytest

from helpers import f64, from_dev, log, rel_l2, to_dev
from oracle import gdr as O
from selective_state_space_75_amd import workloads as W

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "delta_raw", "beta_raw", "A", "delta_bias")
GATES = (-20.0, -26.0, -29.0, -36.0, -44.5, -52.0, -60.0, -69.0)      # 2^-40 = sigmoid(-27.7), 2^-63 = sigmoid(-43.7)


@pytest.mark.parametrize("B,H,G,P,N,L,dtype", [(2, 4, 2, 40, 64, 75, "f32"), (1, 2, 1, 200, 128, 96, "bf16")])
def test_dbeta_of_small_gates(B, H, G, P, N, L, dtype, dev):
    import torch
    import selective_state_space_75_amd as m
    x = W.gdr_inputs(B, H, G, P, N, L, dtype, 8600)
    t = {n: to_dev(a, dev) for n, a in x.items()}
    for i, b in enumerate(GATES):
        t["beta_raw"][:, :, 3 + i::len(GATES) + 5] = b
    g = m.gdr_bwd(*[t[n] for n in NAMES], t["dy"].float(), groups=G, initial_state=t["initial_state"], qk_norm=True)
    torch.cuda.synchronize()
    ref = O.gdr_bwd(*[f64(from_dev(t[n])) for n in NAMES], f64(from_dev(t["dy"])), groups=G, norm=True,
                    initial_state=f64(x["initial_state"]))
    got, raw = from_dev(g["dbeta"]), f64(from_dev(t["beta_raw"]))
    for b in GATES:
        at = raw == b
        assert at.any() and np.abs(ref["dbeta"][at]).max() > 0
        scale = np.exp(-b)                     # (squares of the numbers themselves would underflow)
        e = rel_l2(got[at] * scale, ref["dbeta"][at] * scale)
        log("  beta %.1f: rel_l2=%.3e" % (b, e))
        assert e <= (4 * abs(b) + 20) * 2.0 ** -24, b
    rest = ~np.isin(raw, GATES)
    assert rel_l2(got[rest], ref["dbeta"][rest]) <= 20 * 2.0 ** -24


def test_closed_gates(dev):
    """b = 0 (beta = -inf, or so low that b is no number): dbeta is zero, nothing is NaN."""
    import torch
    import selective_state_space_75_amd as m
    B, H, G, P, N, L = 1, 2, 1, 24, 40, 40
    t = {n: to_dev(a, dev) for n, a in W.gdr_inputs(B, H, G, P, N, L, "f32", 8610).items()}
    t["beta_raw"][:, 0, ::2] = -float("inf")
    t["beta_raw"][:, 1, ::2] = -200.0
    g = m.gdr_bwd(*[t[n] for n in NAMES], t["dy"], groups=G, qk_norm=True)
    assert not g["dbeta"][:, :, ::2].any() and (g["dbeta"][:, :, 1::2] != 0).all()
    assert all(torch.isfinite(a).all() for a in g.values() if a is not None)
