"""Rows of a batch of the gated delta rule: their bits do not depend on what the other rows hold;
in the update and in the backward pass not on the number of rows either; in the forward pass the
number of rows selects the kernel and the segments, whose results agree to fp32 rounding: each
is within 1.2e-6 of the exact result (test_gdr_variants_gpu.py), so two are within 2.4e-6 of
each other."""
import pytest

from helpers import from_dev, log, rel_l2, to_dev
from selective_state_space_75_amd import workloads as W

pytestmark = pytest.mark.gpu

SEQ = ("q", "k", "v", "delta_raw", "beta_raw")
TWO_BARS = 2 * 20 * 2.0 ** -24


def _inputs(B, H, G, P, N, L, seed, dev):
    return {n: to_dev(a, dev) for n, a in W.gdr_inputs(B, H, G, P, N, L, "bf16", seed).items()}


def _rows(t, rows):
    return {n: a if a.dim() == 1 else a[rows].contiguous() for n, a in t.items()}


def _fwd(t, G):
    import torch
    import selective_state_space_75_amd as m
    return m.gdr_fwd(*[t[n] for n in SEQ], t["A"], t["delta_bias"], groups=G, initial_state=t["initial_state"],
                     qk_norm=True, return_final_state=True, out_dtype=torch.float32)


# one batch size on either side of where the planner changes over
@pytest.mark.parametrize("H,G,P,N,L,few,many", [
    (32, 16, 128, 128, 8, 1, 2),             # token by token, chunks
    (16, 16, 128, 128, 2048, 1, 4),          # segments, none
])
def test_forward_over_batch_sizes(H, G, P, N, L, few, many, dev):
    import torch
    import selective_state_space_75_amd as m
    ws = [m.gdr_workspace_size(B, H, G, P, N, L) / B for B in (few, many)]
    assert ws[0] != ws[1]                    # the plans differ
    t = _inputs(many, H, G, P, N, L, 8500, dev)
    y, S = _fwd(t, G)
    y1, S1 = _fwd(_rows(t, slice(0, few)), G)
    for n, a, b in (("y", y1, y[:few]), ("state", S1, S[:few])):
        e = rel_l2(from_dev(a), from_dev(b))
        log("  %s: rel_l2=%.3e" % (n, e))
        assert e <= TWO_BARS, n
    # other contents of the other rows
    o = _inputs(many, H, G, P, N, L, 8501, dev)
    for n in t:
        if t[n].dim() > 1:
            o[n][0] = t[n][0]
        else:
            o[n] = t[n]
    y2, S2 = _fwd(o, G)
    assert torch.equal(y[0], y2[0]) and torch.equal(S[0], S2[0]) and not torch.equal(y[1], y2[1])


@pytest.mark.parametrize("H,G,P,N,B", [(8, 4, 128, 128, 70), (8, 8, 128, 64, 70), (3, 1, 40, 96, 5)])
def test_update_over_batch_sizes(H, G, P, N, B, dev):
    import torch
    import selective_state_space_75_amd as m
    t = _inputs(B, H, G, P, N, 1, 8510, dev)
    tok = [t[n][:, :, 0].contiguous() for n in SEQ]
    s, s1 = t["initial_state"].clone(), t["initial_state"][2:3].clone()
    y = m.gdr_update(s, *tok, t["A"], t["delta_bias"], groups=G, qk_norm=True)
    y1 = m.gdr_update(s1, *[a[2:3].contiguous() for a in tok], t["A"], t["delta_bias"], groups=G, qk_norm=True)
    assert torch.equal(y[2:3], y1) and torch.equal(s[2:3], s1)


def test_backward_over_batch_sizes(dev):
    import torch
    import selective_state_space_75_amd as m
    B, H, G, P, N, L = 9, 4, 2, 64, 128, 70
    t = _inputs(B, H, G, P, N, L, 8520, dev)

    def grads(x):
        return m.gdr_bwd(*[x[n] for n in SEQ], x["A"], x["delta_bias"], x["dy"], groups=G,
                         initial_state=x["initial_state"], dfinal_state=x["dfinal_state"], qk_norm=True)

    g, g1 = grads(t), grads(_rows(t, slice(4, 5)))
    for n in ("dq", "dk", "dv", "ddelta", "dbeta", "dinitial_state"):
        assert torch.equal(g[n][4:5], g1[n]), n


def test_the_same_call_gives_the_same_bits(dev):
    import torch
    for H, G, P, N, L in ((16, 16, 128, 128, 2048), (12, 4, 80, 96, 203), (4, 4, 64, 64, 19)):
        t = _inputs(2, H, G, P, N, L, 8530, dev)
        a = _fwd(t, G)
        for _ in range(3):
            b = _fwd(t, G)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
