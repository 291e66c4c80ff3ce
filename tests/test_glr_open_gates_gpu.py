"""Gradients of gates that are nearly open or nearly closed.  dr holds the factor 1 - s and di the factor 1 - g: taken as
differences they are right to 2^-24 of 1, not of themselves (5e-4 of them at r = 10, all of them from r = 17 on).

Bars.  A gate's exponential e^-v is off by 2^-24 of its rounded argument v log2(e) and by as much for the constant's own
rounding, times ln 2: 2 * 2^-24 * |v| relative, 4.8e-6 at v = 40; the factor is two roundings and a reciprocal further.  With
the adjoint and the state beside it (2e-5, of the magnitudes that they are differences of) that is within 3e-5, for each gate value by
itself.  The gates of a channel are alike in all tokens here, and so are the roundings of their decays, which therefore add
up: a is off by a reciprocal's unit (2^-23) and a rounding (2^-24), 1.8e-7, for each of the tokens that a state or an adjoint
remembers, at most L and about 1 / (1 - a) of them, and a gradient holds one of each: 3.6e-7 min(L, 1 / (1 - a)) more.  bf16 results add
their rounding."""
import numpy as np
import pytest

from helpers import f64, from_dev, log
from oracle import glr as O
from test_glr_gpu import NAMES, gradients, make, near, oracle_args, put

pytestmark = pytest.mark.gpu

VALUES = np.float32([-40, -20, -14, -6, 0, 3, 6, 10, 12, 14, 17, 20, 30, 40])
BAR = 3e-5


#                                          a short row; a last lane that overlaps; one wave; tiles of one workgroup; tiles of their own
@pytest.mark.parametrize("L,waves,segments", [(64, 0, 0), (101, 0, 0), (1500, 0, 0), (1500, 1, 3), (1100, 1, 0)])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("blend", [False, True])
@pytest.mark.parametrize("name", ["r", "i"])
def test_every_gate_value_by_itself(name, blend, dtype, out, L, waves, segments, dev):
    import torch
    import selective_state_space_75_amd as m
    D = len(VALUES)
    rows = 40 if waves == 1 and not segments else 2              # 560 rows: a workgroup walks its row's tiles
    x = make(rows, D, L, dtype, 120 + L, blend, True, True, True)
    x[name + "_bias"] = VALUES                                   # a channel for each value, the gates around it
    x[name] = np.zeros_like(x[name])
    other = "i" if name == "r" else "r"
    x[other + "_bias"] = np.zeros(D, dtype=np.float32)
    t = put(x, dev, NAMES)
    dy = t["dy"].to(torch.float32 if out == "f32" else torch.bfloat16)
    with m.glr_test_knobs(waves=waves, segments=segments):
        g = gradients(t, dy, blend, None)
        torch.cuda.synchronize()
    ref = O.glr_bwd(*oracle_args(x), f64(from_dev(dy)), blend=blend, initial_state=x["initial_state"],
                    dfinal_state=x["dfinal_state"])
    grad, bias = "d" + name, "d%s_bias" % name
    s = O.sigmoid(x["r_bias"].astype(np.float64))
    rest = s if blend else -np.expm1(x["A"].astype(np.float64) * s)              # 1 - a
    e = BAR + 3.6e-7 * np.minimum(L, 1.0 / rest)
    for c, v in enumerate(VALUES):
        log("[open gates] %s = %g" % (name, v))
        size = ref["scale"].get(grad, np.abs(ref[grad]))
        near(g[grad][:, c], ref[grad][:, c], e[c], "%s at %g" % (grad, v), size[:, c])
        near(g[bias][c:c + 1], ref[bias][c:c + 1], e[c], "%s at %g" % (bias, v), ref["scale"][bias][c:c + 1])
