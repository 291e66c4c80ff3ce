"""The gradient that the adjoint chain of the gated delta rule carries from chunk to chunk is rounded once
per chunk at its own size.

Without decay (A = 0: all factors are exactly 1) and with small gates (b = sigmoid(-4) = 0.018) a chunk of 32
tokens changes dS by about 0.018 * 32 / N = 0.5% of itself and by q dy of a tenth of it, so that what the
products round is far below the rounding of their sum with dS: half a unit in the last place at most, 2^-24 *
0.41 of the number in the root mean square (uniform over a binade).  Over 32 chunks sqrt(32) * 0.41 * 2^-24 =
1.4e-7 at the initial state; the bar is 1.6 times that.  Four to seven roundings per chunk (the decay's, and
one for each part of each product) would be 2.8e-7 to 3.7e-7."""
import pytest

from helpers import f64, from_dev, log, rel_l2, to_dev
from oracle import gdr as O
from selective_state_space_75_amd import workloads as W

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "delta_raw", "beta_raw", "A", "delta_bias")
BAR = 1.6 * 32 ** 0.5 * 0.41 * 2.0 ** -24


@pytest.mark.parametrize("dtype,N", [("bf16", 128), ("f32", 128), ("bf16", 64)])
def test_one_rounding_per_chunk(dtype, N, dev):
    import selective_state_space_75_amd as m
    B, H, G, P, L = 1, 2, 1, 32, 1024
    x = W.gdr_inputs(B, H, G, P, N, L, dtype, 9600)
    x["A"][:] = 0.0
    x["dfinal_state"] *= 10.0                         # N(0, 1)
    t = {n: to_dev(a, dev) for n, a in x.items()}
    t["beta_raw"][:] = -4.0
    dy = t["dy"].float()
    g = m.gdr_bwd(*[t[n] for n in NAMES], dy, groups=G, initial_state=t["initial_state"],
                  dfinal_state=t["dfinal_state"], qk_norm=True)
    want = O.gdr_bwd(*[f64(from_dev(t[n])) for n in NAMES], f64(from_dev(dy)), groups=G, norm=True,
                     initial_state=f64(x["initial_state"]), dfinal_state=f64(x["dfinal_state"]))
    e = rel_l2(from_dev(g["dinitial_state"]), want["dinitial_state"])
    log("  dinitial_state: rel_l2=%.3e, bar %.3e" % (e, BAR))
    assert e <= BAR
