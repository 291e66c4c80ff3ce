"""Gradients of the gated delta rule against differences of the GPU's own forward pass, along the
gradient itself: with d = g / |g| the slope of J = <dy, y> + <dfinal, S> is |g|, so a relative bar
says something (along a random direction the slope is |g| / sqrt(numbers), less than a bar that
rounding needs).

Bar.  The difference is (4 D(h/2) - D(h)) / 3 of central differences at h = 2^-6, whose error is of
fourth order: h^4 times the fourth power of what bends J, at most about 16 (decays exp(A step), |A| <= 16), over 480:
8e-6 of the slope.  Rounding: y and S are off by 4e-7 in the root mean square, so J is
off by 4e-7 of its terms' root sum of squares, and the difference by that / h * (4 + 1) / 3.
The bar is 2e-2 |g|; the test holds the rounding to a quarter of it, and a gradient that is a tenth
too small, or zero, is outside it."""
import pytest

from helpers import log, to_dev
from selective_state_space_75_amd import workloads as W

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "delta_raw", "beta_raw", "A", "delta_bias")
GRADS = dict(zip(NAMES + ("initial_state",), ("dq", "dk", "dv", "ddelta", "dbeta", "dA", "ddelta_bias", "dinitial_state")))
BAR = 2e-2


@pytest.mark.parametrize("B,H,G,P,N,L", [(2, 2, 1, 32, 64, 150), (1, 3, 3, 72, 100, 70)])
def test_slope_along_the_gradient(B, H, G, P, N, L, dev):
    import selective_state_space_75_amd as m
    t = {n: to_dev(a, dev) for n, a in W.gdr_inputs(B, H, G, P, N, L, "f32", 9970).items()}
    g = m.gdr_bwd(*[t[n] for n in NAMES], t["dy"], groups=G, initial_state=t["initial_state"],
                  dfinal_state=t["dfinal_state"], qk_norm=True)

    def terms(z):
        y, S = m.gdr_fwd(*[z[n] for n in NAMES], groups=G, initial_state=z["initial_state"], qk_norm=True,
                         return_final_state=True)
        return t["dy"].double() * y.double(), t["dfinal_state"].double() * S.double()

    def J(z):
        return float(sum(a.sum() for a in terms(z)))

    def slope(n, d, h):
        up, down = dict(t), dict(t)
        up[n], down[n] = t[n] + h * d, t[n] - h * d
        moved = float(((up[n].double() - down[n].double()) * d.double()).sum())       # the step that was really taken
        return (J(up) - J(down)) / moved

    h = 2.0 ** -6
    rounding = 4e-7 * float(sum((a * a).sum() for a in terms(t))) ** 0.5 / h * 5 / 3
    for n, gn in GRADS.items():
        size = float(g[gn].double().norm())
        d = g[gn] / size
        got = (4 * slope(n, d, h / 2) - slope(n, d, h)) / 3
        log("  %s: difference %.5f, gradient %.5f" % (n, got, size))
        assert rounding <= BAR * size / 4, n
        assert abs(got - size) <= BAR * size, n
        for wrong in (0.9, 0.0):
            assert abs(got - wrong * size) > BAR * size, n
